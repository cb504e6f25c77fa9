"""Cases for timing and checking the layer norm, the 8-bit quantiser and the 8-bit matrix product.

  layer_norm, layer_norm_bwd   layer norm of the rows of x [T, C], with one weight and bias, or one row
                               of them for each sequence of tokens (adaptive norm); its gradient, with
                               the sums of dweight and dbias over the tokens of each sequence
  quantize_fp8                 rows to 8-bit floating point with a power-of-two scale for each block of
                               1 x 128 or 128 x 128 elements, and the transposed copy that a gradient
                               product reads
  matmul_fp8                   [M, K] x [N, K]^T of such operands: the projections of a block and their
                               gradients

`run` computes them with elementary torch operations in fp32, or, with `own` set, through the calls of this
package.  `exact` is the same in fp64, written separately.
"""
import math

import torch

own = False      # False: the plain torch form; True: the package's kernels

EPS = 1e-6
BLOCK = 128
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _norm(name, op, lens, C, per_seq, x="bf16"):
    """lens: tokens of each sequence; per_seq: a row of weight and bias for each of them."""
    return {"name": name, "op": op, "lens": lens, "C": C, "per_seq": per_seq, "x": x}


def _quant(name, R, C, rows, transpose, x="bf16", to="e4m3"):
    return {"name": name, "op": "quantize_fp8", "R": R, "C": C, "rows": rows, "transpose": transpose, "x": x, "to": to}


def _mm(name, M, N, K, b_rows, out, a_to="e4m3"):
    """a: a scale for each row and 128 of K; b: for each b_rows rows and 128 of K."""
    return {"name": name, "op": "matmul_fp8", "M": M, "N": N, "K": K, "b_rows": b_rows, "out": out, "a_to": a_to}


def listed():
    return [
        # the residual stream of the tiny workload (two heads of 64): one short launch
        _norm("norm_tiny", "layer_norm", "256", 128, False),
        # two clips of the stress workload, 16 heads of 128, scale and shift from each clip's conditioning
        _norm("norm_stress61k", "layer_norm", "61440,61440", 2048, True),
        # training on one small clip
        _norm("norm_bwd_tiny", "layer_norm_bwd", "256", 128, False),
        # training on clips of different lengths, fp32 residual stream of an odd width, a gradient row for each clip
        _norm("norm_bwd_packed", "layer_norm_bwd", "8191,5000,2049,1111,640,129,33,1", 1160, True, "fp32"),
        # training on a 16384-token clip, wide model
        _norm("norm_bwd_16k", "layer_norm_bwd", "16384", 5120, True),
        # activations of two clips for the product and for the weight's gradient
        _quant("quant_rows_61k", 61440, 2048, 1, True),
        # a projection's master weight after an optimiser step, both orders
        _quant("quant_weight", 6144, 2048, 128, True, "fp32"),
        # scale and shift of one conditioning vector: six rows of the model's width
        _mm("mm_one_token", 1, 12288, 2048, 128, "bf16"),
        # Q, K and V of two clips of the stress workload
        _mm("mm_qkv_61k", 61440, 6144, 2048, 128, "bf16"),
        # odd sizes: packed clips, ends inside every tile
        _mm("mm_ragged", 5003, 1001, 1160, 128, "bf16"),
        # gradient of those clips' tokens, in the wider-range type
        _mm("mm_dgrad_16k", 16384, 2048, 6144, 128, "bf16", "e5m2"),
        # gradient of the weight: sums over a packed batch's tokens, a scale for each row on both sides
        _mm("mm_wgrad_17k", 6144, 2048, 17154, 1, "fp32", "e5m2"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A width: any, a multiple of 8, or one of 128."""
    step = rng.choice([1, 8, 8, 128, 128])
    return max(step, _log_int(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice(["layer_norm", "layer_norm_bwd", "quantize_fp8", "matmul_fp8", "matmul_fp8"])
    if op.startswith("layer_norm"):
        C = _width(rng, 16, 8192)
        S = rng.randrange(1, 9)
        lens = [_log_int(rng, 1, 60000) for _ in range(S)]
        while sum(lens) * C > 61440 * 2048:
            lens = [max(1, n // 2) for n in lens]
        return {"op": op, "lens": ",".join(map(str, lens)), "C": C, "per_seq": rng.random() < 0.6,
                "x": rng.choice(["bf16", "bf16", "fp32"])}
    if op == "quantize_fp8":
        C, R = _width(rng, 16, 8192), _log_int(rng, 1, 61440)
        while R * C > 61440 * 2048:
            R //= 2
        return {"op": op, "R": R, "C": C, "rows": rng.choice([1, 1, 128]), "transpose": rng.random() < 0.5,
                "x": rng.choice(["bf16", "bf16", "fp32"]), "to": rng.choice(["e4m3", "e4m3", "e5m2"])}
    M, N, K = _log_int(rng, 1, 61440), _width(rng, 64, 8192), _width(rng, 64, 8192)
    if rng.random() < 0.25:                       # a weight's gradient: the tokens are summed over
        M, N, K = N, _width(rng, 64, 4096), _log_int(rng, 200, 40000)
    while M * N * K > 61440 * 6144 * 2048:
        M, K = (max(1, M // 2), K) if M >= K else (M, K // 2)
    return {"op": op, "M": M, "N": N, "K": K, "b_rows": rng.choice([128, 128, 1]), "out": rng.choice(["bf16", "bf16", "fp32"]),
            "a_to": rng.choice(["e4m3", "e4m3", "e5m2"])}


def _ints(text):
    return [int(v) for v in text.split(",")]


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    op = case["op"]
    if op.startswith("layer_norm"):
        lens, C = _ints(case["lens"]), case["C"]
        T, S, xb = sum(lens), len(lens) if case["per_seq"] else 1, 2 if case["x"] == "bf16" else 4
        if op == "layer_norm":
            return {"bytes": T * (C * (xb + 2) + 8) + 8 * S * C, "flops": 8 * T * C}
        return {"bytes": T * (C * (2 * xb + 2) + 8) + 12 * S * C, "flops": 16 * T * C}
    if op == "quantize_fp8":
        R, C, xb = case["R"], case["C"], 2 if case["x"] == "bf16" else 4
        scales = _blocks(C) * (R if case["rows"] == 1 else _blocks(R))
        scales_t = _blocks(R) * (C if case["rows"] == 1 else _blocks(C))
        two = case["transpose"]
        return {"bytes": R * C * (xb + (2 if two else 1)) + 4 * (scales + (scales_t if two else 0)), "flops": 4 * R * C}
    M, N, K = case["M"], case["N"], case["K"]
    scales = _blocks(K) * (M + (N if case["b_rows"] == 1 else _blocks(N)))
    return {"bytes": M * K + N * K + 4 * scales + M * N * (2 if case["out"] == "bf16" else 4), "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _randn(seed, tag, *shape):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + tag)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(seed, tag, rows, cols):
    """Channels of different sizes and offsets, as a residual stream has them, a few of them large."""
    size = torch.exp(0.7 * _randn(seed, tag + 1, cols))
    return _randn(seed, tag, rows, cols).mul_(size).add_(0.3 * _randn(seed, tag + 2, cols))


def prepare(case, seed):
    op = case["op"]
    if op.startswith("layer_norm"):
        lens, C = _ints(case["lens"]), case["C"]
        T, S = sum(lens), len(lens)
        rows = (S, C) if case["per_seq"] else (C,)
        ends = torch.tensor([0] + lens, device="cuda").cumsum(0)
        st = {"case": case, "x": _activations(seed, 1, T, C).to(TYPE[case["x"]]), "T": T, "S": S,
              "weight": 1.0 + 0.2 * _randn(seed, 4, *rows), "bias": 0.2 * _randn(seed, 5, *rows),
              "seq_ptr": ends.to(torch.int32) if case["per_seq"] else None}
        if op == "layer_norm_bwd":
            st["dy"] = _randn(seed, 6, T, C).to(torch.bfloat16)
            _, mean, rstd = _plain_norm(st)
            st["stats"] = torch.stack((mean, rstd))        # what the forward pass left behind
        return st
    if op == "quantize_fp8":
        return {"case": case, "x": _activations(seed, 1, case["R"], case["C"]).to(TYPE[case["x"]])}
    M, N, K = case["M"], case["N"], case["K"]
    a, sa = _plain_quant(_activations(seed, 1, M, K), 1, case["a_to"])
    b, sb = _plain_quant(_randn(seed, 4, N, K).mul_(1.0 / math.sqrt(K)), case["b_rows"], "e4m3")
    return {"case": case, "a": _padded(a), "a_scale": sa, "b": _padded(b), "b_scale": sb}


def _padded(q):
    """The rows of q a multiple of 16 bytes apart, as the quantiser writes them."""
    out = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16, dtype=torch.uint8, device=q.device)
    out[:, :q.shape[1]] = q.view(torch.uint8)
    return out.view(q.dtype)[:, :q.shape[1]]


# ---------------------------------------------------------------------------
# The operators: plain form, or the package's calls
# ---------------------------------------------------------------------------

def _row_of(st):
    """The sequence of each token."""
    return torch.searchsorted(st["seq_ptr"][1:], torch.arange(st["T"], device="cuda", dtype=torch.int32), right=True)


def _weights(st, v):
    return v if st["seq_ptr"] is None else v[_row_of(st)]


def _plain_norm(st):
    x = st["x"].float()
    mean = x.mean(-1, keepdim=True)
    x = x - mean
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    y = x * rstd * _weights(st, st["weight"]) + _weights(st, st["bias"])
    return y.to(torch.bfloat16), mean.squeeze(-1), rstd.squeeze(-1)


def _plain_norm_bwd(st):
    mean, rstd = st["stats"][0][:, None], st["stats"][1][:, None]
    dy, xhat = st["dy"].float(), (st["x"].float() - mean) * rstd
    g = dy * _weights(st, st["weight"])
    dx = rstd * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    if st["seq_ptr"] is None:
        dw, db = (dy * xhat).sum(0, dtype=torch.float64), dy.sum(0, dtype=torch.float64)
    else:
        pick = (torch.arange(st["S"], device="cuda")[:, None] == _row_of(st)[None]).double()
        dw, db = pick @ (dy * xhat).double(), pick @ dy.double()
    return dx.to(st["x"].dtype), dw.float(), db.float()


def _plain_quant(x, rows, to):
    """Blocks of rows x 128 of x: the values over the block's power of two, and that power [blocks of columns, blocks of rows]."""
    R, C = x.shape
    pad = torch.zeros(-(-R // rows) * rows, _blocks(C) * BLOCK, dtype=torch.float32, device=x.device)
    pad[:R, :C] = x
    tiles = pad.view(-1, rows, _blocks(C), BLOCK)
    amax = tiles.abs().amax((1, 3))
    half, e = torch.frexp(amax)                            # amax = half 2^e with half in [1/2, 1)
    top, e_top = math.frexp(LARGEST[to])
    e = e - e_top + (half > top).to(e.dtype)
    e = torch.where(amax > 0, e.clamp_min(-126), torch.zeros_like(e))
    scale = torch.ldexp(torch.ones_like(amax), e)
    q = torch.ldexp(tiles, -e[:, None, :, None]).to(FP8[to])
    return q.view(pad.shape)[:R, :C].contiguous(), scale.t().contiguous()


def _plain_quantize(st):
    c, x = st["case"], st["x"].float()
    q = _plain_quant(x, c["rows"], c["to"])
    return q + _plain_quant(x.t(), c["rows"], c["to"]) if c["transpose"] else q


def _values(q, scale):
    """The numbers that q and its scales stand for, fp32 (exact)."""
    R, C = q.shape
    rows = scale.t().repeat_interleave(-(-R // scale.shape[1]) if scale.shape[1] == R else BLOCK, 0)[:R]
    return q.float() * rows.repeat_interleave(BLOCK, 1)[:, :C]


def _plain_matmul(st):
    a, b = _values(st["a"], st["a_scale"]), _values(st["b"], st["b_scale"])
    return torch.matmul(a, b.t()).to(TYPE[st["case"]["out"]])


def run(state):
    c = state["case"]
    op = c["op"]
    if own:
        from dynamic_block_sparse_projection_gb300 import binding as dsv
        if op == "layer_norm":
            y, stats = dsv.layer_norm(state["x"], state["weight"], state["bias"], state["seq_ptr"], eps=EPS)
            return y, stats[0], stats[1]
        if op == "layer_norm_bwd":
            return dsv.layer_norm_bwd(state["dy"], state["x"], state["stats"], state["weight"], state["seq_ptr"])
        if op == "quantize_fp8":
            return dsv.quantize_fp8(state["x"], rows=c["rows"], transpose=c["transpose"], dtype=FP8[c["to"]])
        return dsv.matmul_fp8(state["a"], state["a_scale"], state["b"], state["b_scale"], out_dtype=TYPE[c["out"]])
    return {"layer_norm": _plain_norm, "layer_norm_bwd": _plain_norm_bwd, "quantize_fp8": _plain_quantize,
            "matmul_fp8": _plain_matmul}[op](state)


# ---------------------------------------------------------------------------
# The same in fp64, from the definitions
# ---------------------------------------------------------------------------

def _exact_norm(st, back):
    lens = _ints(st["case"]["lens"])
    x, C = st["x"].to(torch.float64), st["case"]["C"]
    rows = lens if st["seq_ptr"] is not None else [sum(lens)]
    w, b = (st[k].to(torch.float64).reshape(-1, C) for k in ("weight", "bias"))
    out, mean, rstd = torch.empty_like(x), x.new_empty(x.shape[0]), x.new_empty(x.shape[0])
    dw, db = torch.zeros_like(w), torch.zeros_like(w)
    at = 0
    for s, n in enumerate(rows):
        for i in range(at, at + n, 8192):
            j = min(at + n, i + 8192)
            xs = x[i:j]
            if not back:
                var, m = torch.var_mean(xs, -1, correction=0)
                mean[i:j], rstd[i:j] = m, (var + EPS) ** -0.5
                out[i:j] = torch.addcmul(b[s], (xs - m[:, None]) / torch.sqrt(var + EPS)[:, None], w[s])
                continue
            m, r = st["stats"][0, i:j].to(torch.float64), st["stats"][1, i:j].to(torch.float64)
            h = torch.einsum("ij,i->ij", xs - m[:, None], r)
            dy = st["dy"][i:j].to(torch.float64)
            dw[s] += torch.einsum("ij,ij->j", dy, h)
            db[s] += torch.einsum("ij->j", dy)
            along = torch.stack((dy @ w[s], torch.einsum("ij,ij,j->i", dy, h, w[s]))) / C
            out[i:j] = (dy * w[s] - along[0][:, None] - h * along[1][:, None]) / (1.0 / r)[:, None]
        at += n
    if not back:
        return out, mean, rstd
    return out, dw.reshape(st["weight"].shape), db.reshape(st["weight"].shape)


def _exact_quant(x, rows, to):
    """One block of columns at a time: the power from logarithms, checked against the largest value that fits."""
    R, C = x.shape
    q = torch.empty(R, C, dtype=torch.float64, device=x.device)
    scale = torch.empty(_blocks(C), -(-R // rows), dtype=torch.float64, device=x.device)
    digits, least = (3, -6) if to == "e4m3" else (2, -14)
    for j in range(_blocks(C)):
        part = x[:, j * BLOCK:(j + 1) * BLOCK].to(torch.float64)
        top = part.abs().amax(1)
        if rows > 1:
            top = torch.nn.functional.pad(top, (0, -R % rows)).view(-1, rows).amax(1)
        k = torch.floor(torch.log2(top.clamp_min(1e-300) / LARGEST[to])) - 1.0
        k = k + (top > LARGEST[to] * torch.exp2(k))
        k = k + (top > LARGEST[to] * torch.exp2(k))
        k = torch.where(top > 0, k.clamp_min(-126.0), torch.zeros_like(k))
        scale[j] = torch.exp2(k)
        v = part / scale[j].repeat_interleave(rows)[:R, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** least))).clamp_min(least) - digits)
        q[:, j * BLOCK:(j + 1) * BLOCK] = torch.round(v / step) * step      # halves to even
    return q, scale


def _exact_matmul(st):
    """One block of 128 at a time, each scaled behind its product."""
    M, N, K = (st["case"][k] for k in ("M", "N", "K"))
    out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
    row_m = torch.arange(M, device="cuda") // (1 if st["a_scale"].shape[1] == M else BLOCK)
    row_n = torch.arange(N, device="cuda") // (1 if st["b_scale"].shape[1] == N else BLOCK)
    for j in range(_blocks(K)):
        a, b = (st[k][:, j * BLOCK:(j + 1) * BLOCK].to(torch.float64) for k in ("a", "b"))
        out.addmm_(a * st["a_scale"][j].to(torch.float64)[row_m, None],
                   (b * st["b_scale"][j].to(torch.float64)[row_n, None]).T)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"].startswith("layer_norm"):
        return _exact_norm(st, case["op"] == "layer_norm_bwd")
    if case["op"] == "quantize_fp8":
        q = _exact_quant(st["x"], case["rows"], case["to"])
        return q + _exact_quant(st["x"].T, case["rows"], case["to"]) if case["transpose"] else q
    return _exact_matmul(st)
