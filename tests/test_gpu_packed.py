"""GPU parity of the packed-sequence attention, forward and backward, against
the fp64 oracle (needs a GB300).

Tolerances, element by element, from the arithmetic (u = 2^-8, half a step of
bf16; e = 2^-12, the fp32 part: an accumulated score of these sizes and its
exponential are good to that, relative to P):
  O    P is rounded to bf16 for the product, O to bf16:
       (u + e) sum_j P |v| + u |O|
  lse  e + 2^-20 |lse|
  D    dO . O with the bf16 O:            sum_c |dO| tol(O)
       (where a tile of queries sees at most 128 keys, sum_j P dP in fp32:
       2e sum_j P |dO| |v|; only `_bounds(exact_d=True)` counts on it)
  dV   (u + 2e) sum_i P |dO| + u |dV|
  dS   (u + 2e) |dS| + P (tol(D) + e sum_c |dO v|)
  dQ   scale sum_j tol(dS) |k| + u |dQ|;  dK likewise with q."""
import numpy as np
import pytest
import torch

import oracle
from parity_util import to64

pytestmark = pytest.mark.gpu
U, E = 2.0 ** -8, 2.0 ** -12


@pytest.fixture(scope="module")
def dsv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_block_sparse_projection_gb300 import binding
    binding.clear_device_error()
    yield binding
    st, info = binding.device_error()
    assert st == 0, (st, info)


def _ptr(lens, start=0):
    return np.concatenate([[start], start + np.cumsum(lens)]).astype(np.int32)


def _rand(seed, *shape, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (gain * torch.randn(*shape, generator=g, device="cuda")).to(torch.bfloat16)


def _heads(seed, heads, tokens, d, layout, gain=1.0):
    if layout == "htd":
        return _rand(seed, heads, tokens, d, gain=gain)
    if layout == "thd":
        return _rand(seed, tokens, heads, d, gain=gain).transpose(0, 1)
    return _rand(seed, tokens, heads + 3, d + 64, gain=gain).transpose(0, 1)[2:2 + heads, :, 64:]


class Case:
    def __init__(self, H, Hkv, d, ql, kl, layout="thd", seed=3, gain=1.0, pad=0):
        self.qp, self.kp = _ptr(ql, pad), _ptr(kl, pad)
        Tq, Tk = int(self.qp[-1]) + pad, int(self.kp[-1]) + pad
        self.Q = _heads(seed, H, Tq, d, layout, gain)
        self.K, self.V = (_heads(seed + i, Hkv, Tk, d, layout) for i in (1, 2))
        self.dO = _heads(seed + 3, H, Tq, d, layout)
        self.q_ptr, self.k_ptr = (torch.tensor(p, device="cuda") for p in (self.qp, self.kp))

    def fwd(self, dsv, causal, scale=0.0, **kw):
        return dsv.packed_attn_fwd(self.Q, self.K, self.V, self.q_ptr, self.k_ptr, scale, causal=causal, **kw)

    def bwd(self, dsv, O, lse, causal, scale=0.0, **kw):
        return dsv.packed_attn_bwd(self.Q, self.K, self.V, O, self.dO, lse, self.q_ptr, self.k_ptr, scale,
                                   causal=causal, **kw)

    def np(self):
        return tuple(to64(t) for t in (self.Q, self.K, self.V, self.dO))


def _bounds(Q, K, V, dO, qp, kp, causal, scale, exact_d=False):
    """Reference values and tolerances of every output."""
    scale = scale or 1 / np.sqrt(Q.shape[-1])
    O, lse = oracle.packed_attn_fwd(Q, K, V, qp, kp, causal, scale)
    dQ, dK, dV = oracle.packed_attn_bwd(Q, K, V, dO, qp, kp, causal, scale)
    tO, tdQ, tdK, tdV = (U * np.abs(t) + 1e-30 for t in (O, dQ, dK, dV))
    group = Q.shape[0] // K.shape[0]
    for s in range(len(qp) - 1):
        qs, ks = slice(qp[s], qp[s + 1]), slice(kp[s], kp[s + 1])
        lq, lk = qs.stop - qs.start, ks.stop - ks.start
        if lq == 0 or lk == 0:
            continue
        mask = np.ones((lq, lk), bool)
        if causal:
            mask = np.arange(lk)[None] <= np.arange(lq)[:, None] + lk - lq
        for h in range(Q.shape[0]):
            j = h // group
            sc = scale * (Q[h, qs] @ K[j, ks].T)
            with np.errstate(invalid="ignore"):
                P = np.where(mask, np.exp(sc - np.where(np.isfinite(lse[h, qs]), lse[h, qs], 0)[:, None]), 0.0)
            g, v, k, q = dO[h, qs], V[j, ks], K[j, ks], Q[h, qs]
            tO[h, qs] += (U + E) * (P @ np.abs(v))
            tD = np.sum(np.abs(g) * tO[h, qs], -1, keepdims=True)
            if exact_d:
                assert lk <= 128
                tD = 2 * E * np.sum(P * (np.abs(g) @ np.abs(v).T), -1, keepdims=True)
            dP = g @ v.T
            dS = P * (dP - np.sum(P * dP, -1, keepdims=True))
            tS = (U + 2 * E) * np.abs(dS) + P * (tD + E * (np.abs(g) @ np.abs(v).T))
            tdV[j, ks] += (U + 2 * E) * (P.T @ np.abs(g))
            tdQ[h, qs] += scale * (tS @ np.abs(k))
            tdK[j, ks] += scale * (tS.T @ np.abs(q))
    return (O, tO), (lse, E + 2.0 ** -20 * np.abs(np.where(np.isfinite(lse), lse, 0))), (dQ, tdQ), (dK, tdK), (dV, tdV)


def _near(got, ref_tol, rows, what):
    ref, tol = ref_tol
    got, ref, tol = to64(got)[:, rows], ref[:, rows], tol[:, rows]
    fin = np.isfinite(ref)
    assert np.array_equal(fin, np.isfinite(got)) and np.array_equal(got[~fin], ref[~fin]), what
    err = np.abs(got[fin] - ref[fin])
    assert np.all(err <= tol[fin]), f"{what}: {np.max(err / tol[fin]):.3f} of the tolerance"


def _check(dsv, c, causal, scale=0.0, backward=True):
    O, lse = c.fwd(dsv, causal, scale)
    Q, K, V, dO = c.np()
    b = _bounds(Q, K, V, dO, c.qp, c.kp, causal, scale)
    rq, rk = slice(c.qp[0], c.qp[-1]), slice(c.kp[0], c.kp[-1])
    _near(O, b[0], rq, "O")
    _near(lse, b[1], rq, "lse")
    if backward:
        for got, ref, rows, what in zip(c.bwd(dsv, O, lse, causal, scale), b[2:], (rq, rk, rk), ("dQ", "dK", "dV")):
            _near(got, ref, rows, what)
    st, info = dsv.device_error()
    assert st == 0, (st, info)
    return O, lse


SHAPES = [  # H, Hkv, d, query lengths, key lengths
    (1, 1, 64, (1,), (1,)),
    (2, 2, 128, (128,), (128,)),
    (2, 2, 64, (256, 1, 0, 77, 130), (256, 1, 0, 77, 130)),
    (3, 1, 128, (200, 129, 33), (200, 129, 33)),              # 42 tokens x 3 heads a tile
    (4, 2, 64, (127, 128, 129), (127, 128, 129)),
    (2, 1, 128, (5, 300), (700, 301)),                        # fewer queries than keys
    (2, 2, 64, (300, 40, 7), (10, 0, 7)),                     # fewer keys than queries; none
    (5, 1, 64, (26, 51), (26, 400)),                          # 25 tokens x 5 heads: rows 125..127 unused
    (1, 1, 128, (700,), (640,)),
]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [False, True])
def test_packed_parity(dsv, shape, causal):
    _check(dsv, Case(*shape), causal)


@pytest.mark.parametrize("H, Hkv", [(24, 1), (64, 1), (128, 1), (65, 1), (48, 2)])
def test_packed_many_shared_heads(dsv, H, Hkv):
    _check(dsv, Case(H, Hkv, 64, (3, 1, 9), (3, 150, 40)), True)


@pytest.mark.parametrize("layout", ["htd", "thd", "slice"])
def test_packed_layouts(dsv, layout):
    c = Case(4, 2, 64, (100, 61), (100, 90), layout)
    O, lse = _check(dsv, c, True)
    # the caller's buffers, in another order than the inputs', rows outside the sequences untouched
    c = Case(4, 2, 64, (100, 61), (100, 90), layout, pad=9)
    out = torch.full((c.Q.shape[1], 4, 64), 7.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    ls = torch.full((4, c.Q.shape[1]), 7.0, device="cuda")
    assert c.fwd(dsv, True, out=out, lse=ls)[0] is out
    outs = tuple(torch.full(tuple(t.shape), 7.0, dtype=torch.bfloat16, device="cuda") for t in (c.Q, c.K, c.V))
    c.bwd(dsv, out, ls, True, outs=outs)
    for t in (out, *outs):
        assert (t[:, :9] == 7).all() and (t[:, -9:] == 7).all()
    assert (ls[:, :9] == 7).all() and (ls[:, -9:] == 7).all()
    b = _bounds(*c.np(), c.qp, c.kp, True, 0.0)
    for got, ref, what in zip((out, ls, *outs), b, ("O", "lse", "dQ", "dK", "dV")):
        _near(got, ref, slice(9, -9), what)


@pytest.mark.parametrize("ql, kl, causal", [
    ((1,), (5000,), True), ((1, 1, 1), (1300, 1, 4000), True), ((1,), (513,), False), ((40,), (3000,), True),
    ((300,), (2900,), True), ((2, 0, 1), (700, 900, 0), False), ((700,), (600,), True)])
@pytest.mark.parametrize("H, Hkv, d", [(6, 2, 128), (1, 1, 64), (8, 1, 64)])
def test_packed_split_over_keys(dsv, ql, kl, causal, H, Hkv, d):
    """Few query tiles: the keys are split and joined (one new token included)."""
    group = H // Hkv
    least = 4 if group * min(sum(ql), 128 // group) < 32 else 8           # key tiles of a part: rows make a part dear
    split = dsv.packed_attn_fwd_workspace_bytes(len(ql), H, Hkv, sum(ql), sum(kl), d) > 0
    assert split == (-(-sum(kl) // 128) > least)
    _check(dsv, Case(H, Hkv, d, ql, kl), causal)


@pytest.mark.parametrize("ql, kl, causal", [
    ((2900,), (100,), False), ((1300, 2000, 5), (77, 300, 200), False), ((2500, 0, 600), (513, 40, 0), True),
    ((1700,), (1700,), True), ((3000,), (130,), True)])
@pytest.mark.parametrize("H, Hkv, d", [(2, 2, 128), (6, 2, 64)])
def test_packed_gradient_split_over_queries(dsv, ql, kl, causal, H, Hkv, d):
    """Few key tiles against many queries (text): the query tiles of a key tile
    are split and the parts of dK and dV joined."""
    S, Tq, Tk = len(ql), sum(ql), sum(kl)
    whole = 2 * Hkv * (Tq // (128 // (H // Hkv)) + S) * 128 * 4
    assert dsv.packed_attn_bwd_workspace_bytes(S, H, Hkv, Tq, Tk, d) > whole
    c = Case(H, Hkv, d, ql, kl)
    O, lse = _check(dsv, c, causal)
    g, g2 = c.bwd(dsv, O, lse, causal), c.bwd(dsv, O, lse, causal)
    assert all(torch.equal(a, b) for a, b in zip(g, g2))


def test_packed_enough_tiles_are_not_split(dsv):
    c = Case(20, 20, 64, (1000, 30), (1000, 600))
    assert dsv.packed_attn_fwd_workspace_bytes(2, 20, 20, 1030, 1600, 64) == 0
    _check(dsv, c, True)
    _check(dsv, c, False)


@pytest.mark.parametrize("kl", [(900,), (20000,)])
def test_packed_scores_that_grow_along_the_keys(dsv, kl):
    """Later tiles hold scores hundreds above the first tile's maximum (the
    running reference is replaced and O rescaled), and the parts of a split
    differ by as much."""
    c = Case(2, 2, 64, (150,), kl)
    ramp = torch.linspace(0.01, 30.0, kl[0], device="cuda")[None, :, None]
    K = (c.K.float() * 0.05 + c.Q[:, :1].float()) * ramp
    c.K = K.to(torch.bfloat16)
    c.Q = (c.Q[:, :1].float() * (1 + 0.01 * c.Q.float())).to(torch.bfloat16)
    O, lse = c.fwd(dsv, False)
    ref, lref = oracle.packed_attn_fwd(*c.np()[:3], c.qp, c.kp)
    # scores up to |s| ~ 250: an fp32 score is good to 64 2^-23 sum |q k| ~ 2^-17 * 250 * 3, so P to ~ 2^-7
    assert np.max(lref) > 100
    assert np.max(np.abs(to64(lse) - lref)) <= 2.0 ** -7
    assert np.max(np.abs(to64(O) - ref)) <= (2 * U + 2.0 ** -7) * np.max(np.abs(to64(c.V)))
    assert dsv.device_error()[0] == 0


@pytest.mark.parametrize("H,Hkv,d", [(2, 2, 128), (3, 1, 64), (5, 1, 128)])
@pytest.mark.parametrize("causal", [False, True])
def test_packed_gradient_over_a_handful_of_keys(dsv, H, Hkv, d, causal):
    """Few keys: O is as large as V, and D from the bf16 O would be too coarse
    beside dS (0 for a row that sees one key)."""
    for ql, kl in (((1, 2, 3, 300, 7, 20, 500), (1, 2, 3, 1, 0, 20, 128)), ((40, 9) * 40, (3, 11) * 40)):
        c = Case(H, Hkv, d, ql, kl, pad=5)
        O, lse = c.fwd(dsv, causal)
        Q, K, V, dO = c.np()
        b = _bounds(Q, K, V, dO, c.qp, c.kp, causal, 0.0, exact_d=True)
        rq, rk = slice(c.qp[0], c.qp[-1]), slice(c.kp[0], c.kp[-1])
        for got, ref, rows, what in zip(c.bwd(dsv, O, lse, causal), b[2:], (rq, rk, rk), ("dQ", "dK", "dV")):
            _near(got, ref, rows, what)


def test_packed_not_a_number_stays_in_its_sequence(dsv):
    """NaN and infinities in one sequence, and in the rows of no sequence, reach
    no other one: tiles that reach past a sequence's end read its neighbour."""
    for H, Hkv, d, ql, kl in ((2, 2, 64, (70, 50, 90), (70, 50, 90)), (3, 1, 128, (50, 9, 131), (150, 30, 131)),
                              (2, 1, 64, (1, 2, 1), (900, 70, 1300))):
        for causal in (False, True):
            c = Case(H, Hkv, d, ql, kl, pad=20)
            O, lse = c.fwd(dsv, causal)
            grads = c.bwd(dsv, O, lse, causal)
            clean = [t.clone() for t in (O, lse, *grads)]
            for i, t in enumerate((c.Q, c.K, c.V, c.dO)):
                p = c.qp if i in (0, 3) else c.kp
                bad = float("nan") if i % 2 else float("inf")
                t[:, :p[0]] = bad
                t[:, p[-1]:] = bad
                t[:, p[1]:p[2]] = bad
            O2, lse2 = c.fwd(dsv, causal)
            g2 = c.bwd(dsv, O2, lse2, causal)
            for a, b, p, what in zip((O2, lse2, *g2), clean, (c.qp, c.qp, c.qp, c.kp, c.kp),
                                     ("O", "lse", "dQ", "dK", "dV")):
                for s in (0, 2):
                    assert torch.equal(a[:, p[s]:p[s + 1]], b[:, p[s]:p[s + 1]]), (what, s, causal, H)


def test_packed_is_repeatable_and_scale_is_used(dsv):
    c = Case(6, 2, 128, (400, 77), (400, 900))
    O, lse = _check(dsv, c, True, 0.21)
    O2, lse2 = c.fwd(dsv, True, 0.21)
    g, g2 = c.bwd(dsv, O, lse, True, 0.21), c.bwd(dsv, O, lse, True, 0.21)
    assert torch.equal(O, O2) and torch.equal(lse, lse2) and all(torch.equal(a, b) for a, b in zip(g, g2))


def test_packed_gradient_against_differences(dsv):
    c = Case(3, 1, 64, (40, 21), (40, 60))
    O, lse = c.fwd(dsv, True)
    grads = c.bwd(dsv, O, lse, True)
    Q, K, V, dO = c.np()
    b = _bounds(Q, K, V, dO, c.qp, c.kp, True, 0.0)[2:]
    f = lambda t: (oracle.packed_attn_fwd(*t, c.qp, c.kp, True)[0] * dO).sum()   # noqa: E731
    h = 1e-5
    for i in range(3):
        u = np.random.default_rng(i).standard_normal(b[i][0].shape)
        hi, lo = [[t + (s * h * u if n == i else 0) for n, t in enumerate((Q, K, V))] for s in (1, -1)]
        num = (f(hi) - f(lo)) / (2 * h)
        assert abs(num - (to64(grads[i]) * u).sum()) <= np.sum(b[i][1] * np.abs(u)) + 1e-5 * abs(num)


def test_packed_bad_pointers_are_reported(dsv):
    """A sequence whose pointers fall or leave the tensor is skipped and
    reported; the others are computed."""
    c = Case(2, 2, 64, (60, 50, 70), (60, 50, 70))
    good = c.fwd(dsv, False)[0].clone()
    for which, ptr in (("q_ptr", [0, 60, 110, 181]), ("k_ptr", [0, 60, 110, 100]), ("q_ptr", [0, 60, 110, 90]),
                       ("k_ptr", [0, 60, 110, 1 << 30]), ("q_ptr", [0, 60, 110, -5])):
        kw = {"q_ptr": c.q_ptr, "k_ptr": c.k_ptr, which: torch.tensor(ptr, dtype=torch.int32, device="cuda")}
        out = torch.zeros_like(good)
        O, lse = dsv.packed_attn_fwd(c.Q, c.K, c.V, **kw, out=out)
        st, info = dsv.device_error()
        dsv.clear_device_error()
        assert st == dsv.DSV_ERR_BAD_INDEX and info == 2
        assert torch.equal(O[:, :110], good[:, :110])
        dsv.packed_attn_bwd(c.Q, c.K, c.V, O, c.dO, lse, **kw)
        assert dsv.device_error()[0] == dsv.DSV_ERR_BAD_INDEX
        dsv.clear_device_error()
    _check(dsv, c, False)


def test_packed_empty(dsv):
    e = lambda h, t: torch.empty(h, t, 64, dtype=torch.bfloat16, device="cuda")   # noqa: E731
    p = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")               # noqa: E731
    # no sequences; no queries; no keys
    dsv.packed_attn_fwd(e(2, 5), e(2, 5), e(2, 5), p(0), p(0))
    K = _rand(1, 2, 5, 64)
    O, lse = dsv.packed_attn_fwd(e(2, 0), K, K.clone(), p(0, 0), p(0, 5))
    assert O.numel() == 0
    dQ, dK, dV = dsv.packed_attn_bwd(e(2, 0), K, K.clone(), O, e(2, 0), lse, p(0, 0), p(0, 5))
    torch.cuda.synchronize()
    assert not dK.any() and not dV.any()
    Q = _rand(2, 2, 5, 64)
    O, lse = dsv.packed_attn_fwd(Q, e(2, 0), e(2, 0), p(0, 5), p(0, 0))
    dQ, dK, dV = dsv.packed_attn_bwd(Q, e(2, 0), e(2, 0), O, Q.clone(), lse, p(0, 5), p(0, 0))
    torch.cuda.synchronize()
    assert not O.any() and torch.isneginf(lse).all() and not dQ.any()
    assert dsv.device_error()[0] == 0


def test_packed_offsets_beyond_32_bits(dsv):
    """Keys whose element offset passes 2^31: one head-major key tensor of 4.6 GB,
    the last head's last sequence read by a few queries."""
    Hkv, Tk, d = 3, 6_000_000, 128
    kl = (Tk - 1500, 1500)
    K = torch.empty(Hkv, Tk, d, dtype=torch.bfloat16, device="cuda")
    V = torch.empty_like(K)
    K[:, -1500:] = _rand(1, Hkv, 1500, d)
    V[:, -1500:] = _rand(2, Hkv, 1500, d)
    Q, dO = _rand(3, Hkv, 5, d), _rand(4, Hkv, 5, d)
    qp, kp = torch.tensor([0, 0, 5], dtype=torch.int32, device="cuda"), torch.tensor(_ptr(kl), device="cuda")
    O, lse = dsv.packed_attn_fwd(Q, K, V, qp, kp, causal=True)
    dQ, dK, dV = dsv.packed_attn_bwd(Q, K, V, O, dO, lse, qp, kp, causal=True)
    b = _bounds(to64(Q), to64(K[:, -1500:]), to64(V[:, -1500:]), to64(dO), np.array([0, 5]), np.array([0, 1500]), True,
                0.0)
    al = slice(None)
    for got, ref, what in zip((O, lse, dQ, dK[:, -1500:], dV[:, -1500:]), b, ("O", "lse", "dQ", "dK", "dV")):
        _near(got, ref, al, what)
    assert not dK[:, :-1500:4097].any() and not dV[:, :-1500:4097].any()       # keys that nobody saw
    assert dsv.device_error()[0] == 0


def test_packed_on_streams_and_in_graphs(dsv):
    """Two captured graphs, each with a workspace of its own, replayed on two
    streams at once; pointers changed between replays."""
    cs = [Case(4, 2, 64, (3, 1), (900, 300), seed=s) for s in (1, 50)]
    refs = []
    for c in cs:
        O, lse = c.fwd(dsv, True)
        refs.append((O, lse, *c.bwd(dsv, O, lse, True)))
    torch.cuda.synchronize()
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in cs]
    for c, st in zip(cs, streams):
        n = max(dsv.packed_attn_fwd_workspace_bytes(2, 4, 2, 4, 1200, 64),
                dsv.packed_attn_bwd_workspace_bytes(2, 4, 2, 4, 1200, 64))
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        o = [torch.zeros_like(t) for t in (c.Q, c.K, c.V)]
        O, lse = torch.zeros_like(c.Q), torch.zeros(4, 4, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            c.fwd(dsv, True, out=O, lse=lse, workspace=ws, stream=st)
            c.bwd(dsv, O, lse, True, outs=o, workspace=ws, stream=st)
        graphs.append((g, ws))
        outs.append((O, lse, *o))
    for _ in range(3):
        for (g, _ws), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for got, ref in zip(outs, refs):
        for a, b in zip(got, ref):
            assert torch.equal(a, b)
    # other lengths of the same totals, read by the same graph
    c = cs[0]
    c.q_ptr.copy_(torch.tensor([0, 1, 4], dtype=torch.int32))
    c.k_ptr.copy_(torch.tensor([0, 200, 1200], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    O, lse = c.fwd(dsv, True)
    assert torch.equal(outs[0][0], O) and torch.equal(outs[0][1], lse)


def test_norm_rotation_and_attention_together(dsv):
    """A layer as it would be trained: norm and rotate q and k, attend over
    packed clips with shared heads, and back to the projections' gradients and
    the norm weights'."""
    H, Hkv, d, grids = 6, 2, 64, ((2, 5, 6), (1, 4, 9), (3, 7, 7))
    lens = [a * b * c for a, b, c in grids]
    T = sum(lens)
    pos = torch.cat([torch.stack(torch.meshgrid(*[torch.arange(v) for v in g], indexing="ij"), -1).reshape(-1, 3)
                     for g in grids]).to("cuda", torch.int32)
    qkv = _rand(1, 1, T, H + 2 * Hkv, d)
    q, k, v = (t.transpose(1, 2) for t in qkv.split((H, Hkv, Hkv), 2))
    wq, wk = (1 + 0.2 * _rand(s, d).float() for s in (2, 3))
    dO = _rand(4, H, T, d)
    sec, ptr = (16, 24, 24), torch.tensor(_ptr(lens), device="cuda")
    qr, kr = dsv.rope_axes(q, pos, sec, weight=wq), dsv.rope_axes(k, pos, sec, weight=wk)
    O, lse = dsv.packed_attn_fwd(qr[0], kr[0], v[0], ptr, ptr, causal=True)
    dqr, dkr, dv = dsv.packed_attn_bwd(qr[0], kr[0], v[0], O, dO, lse, ptr, ptr, causal=True)
    dq, dwq = dsv.rope_axes_bwd(dqr[None], pos, sec, x=q, weight=wq)
    dk, dwk = dsv.rope_axes_bwd(dkr[None], pos, sec, x=k, weight=wk)
    torch.cuda.synchronize()
    assert dsv.device_error()[0] == 0
    p, pn = _ptr(lens), pos.cpu().numpy()
    q64, k64, v64, w1, w2 = to64(q), to64(k), to64(v), to64(wq), to64(wk)
    Q, K = oracle.rope_axes(q64, pn, sec, weight=w1)[0], oracle.rope_axes(k64, pn, sec, weight=w2)[0]
    Or, lr = oracle.packed_attn_fwd(Q, K, v64[0], p, p, True)
    gQ, gK, gV = oracle.packed_attn_bwd(Q, K, v64[0], to64(dO), p, p, True)
    gq, gwq = oracle.rope_axes_bwd(gQ[None], pn, sec, x=q64, weight=w1)
    gk, gwk = oracle.rope_axes_bwd(gK[None], pn, sec, x=k64, weight=w2)
    # five bf16 roundings in a chain (q/k, P, O, dS, gradient), each at most 2^-8 of its value's size: 2e-2 in norm
    rel = lambda a, b: np.linalg.norm(to64(a) - b) / np.linalg.norm(b)   # noqa: E731
    for got, ref, what in ((O, Or, "O"), (dv, gV, "dv"), (dq, gq, "dq"), (dk, gk, "dk"), (dwq, gwq, "dwq"),
                           (dwk, gwk, "dwk")):
        assert rel(got, ref) <= 2e-2, (what, rel(got, ref))
    assert np.max(np.abs(to64(lse) - lr)) <= 2 * 8 * U       # |ds| <= 2 2^-8 |s|, |s| <= 8


def test_packed_equals_the_dense_sparse_call(dsv):
    """On one clip of whole blocks with every block selected the block-sparse
    call computes the same thing."""
    B, H, N, d, blk = 1, 2, 512, 128, 128
    c = Case(H, H, d, (N,), (N,), "htd")
    G = N // blk
    fp = torch.arange(0, B * H * G * G + 1, G, dtype=torch.int32, device="cuda")
    fc = torch.arange(G, dtype=torch.int32, device="cuda").repeat(B * H * G)
    O, lse = c.fwd(dsv, False)
    O2, lse2 = dsv.sparse_attn_fwd(c.Q[None], c.K[None], c.V[None], fp, fc, blk)
    assert torch.equal(O, O2[0]) or (O.float() - O2[0].float()).abs().max() <= 2 * U * c.V.float().abs().max()
    assert (lse - lse2[0]).abs().max() <= 2 * E



@pytest.mark.parametrize("H, Hkv, ql, kl, split", [(2, 2, (1, 3), (1300, 700), True), (6, 2, (40,), (3000,), True),
                                                   (20, 20, (1000, 30), (1000, 600), False)])
@pytest.mark.parametrize("causal", [False, True])
def test_packed_a_query_that_is_not_a_number_gives_none(dsv, H, Hkv, ql, kl, split, causal):
    """O and lse of a NaN query, and of one whose scores overflow, are NaN
    whether its keys are split or not (0 and -inf are for rows without keys);
    so is its gradient.  The other rows stay right."""
    assert (dsv.packed_attn_fwd_workspace_bytes(len(ql), H, Hkv, sum(ql), sum(kl), 64) > 0) == split
    c = Case(H, Hkv, 64, ql, kl)
    b = _bounds(*c.np(), c.qp, c.kp, causal, 0.0)
    bad = torch.zeros(H, sum(ql), dtype=torch.bool, device="cuda")
    bad[0, 0] = bad[1, -1] = True
    c.Q[0, 0, 5], c.Q[1, -1, 3] = float("nan"), float("inf")
    O, lse = c.fwd(dsv, causal)
    assert O[bad].isnan().all() and lse[bad].isnan().all()
    dQ = c.bwd(dsv, O, lse, causal)[0]
    assert dQ[bad].isnan().all()
    ok = ~bad.cpu().numpy()
    for got, (ref, tol), what in ((O, b[0], "O"), (lse, b[1], "lse")):
        assert np.all(np.abs(to64(got)[ok] - ref[ok]) <= tol[ok]), what



@pytest.mark.parametrize("H, ql, split", [(2, (150,), True), (20, (1000,), False)])
def test_packed_first_keys_that_weigh_nothing(dsv, H, ql, split):
    """Every score of the first key tile is -inf and the others lie far below
    zero: the row's reference is the first finite maximum, not 0, against which
    every exponential would be 0."""
    N = 1500
    assert (dsv.packed_attn_fwd_workspace_bytes(1, H, H, ql[0], N, 64) > 0) == split
    c = Case(H, H, 64, ql, (N,))
    c.Q = (c.Q.float().abs() + 0.5).clamp(max=3.0).to(torch.bfloat16)
    c.K = -(14.0 + c.K.float().abs().clamp(max=4.0)).to(torch.bfloat16)
    c.K[:, :200] = float("-inf")
    O, lse = c.fwd(dsv, False)
    ref, lref = oracle.packed_attn_fwd(*c.np()[:3], c.qp, c.kp)
    # scores of one sign: an fp32 sum of 64 products is good to 64 2^-24 |s|, |s| <= 64 * 3 * 18 / 8 = 432 < 2^9
    assert np.max(lref) < -104 and np.min(lref) > -432        # exp(-104) is 0 in fp32
    s = 64 * 2.0 ** -24 * 2.0 ** 9
    assert np.max(np.abs(to64(lse) - lref)) <= s + E + 2.0 ** -20 * 432
    assert np.max(np.abs(to64(O) - ref)) <= (2 * U + E + 2 * s) * np.max(np.abs(to64(c.V)))
    assert dsv.device_error()[0] == 0



def test_packed_gradient_without_queries_checks_its_pointers(dsv):
    K = _rand(1, 2, 300, 64)
    none = torch.empty(2, 0, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 0, device="cuda")
    p = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")               # noqa: E731
    for kp, bad in (((0, 130, 290), None), ((0, 130, 301), 1), ((0, 130, 120), 1), ((-1, 130, 290), 0)):
        outs = (none.clone(), *(torch.full_like(K, 7.0) for _ in range(2)))
        dsv.packed_attn_bwd(K[:, :0], K, K.clone(), none, none.clone(), lse, p(0, 0, 0), p(*kp), outs=outs)
        st, info = dsv.device_error()
        dsv.clear_device_error()
        assert (st, info) == ((0, 0) if bad is None else (dsv.DSV_ERR_BAD_INDEX, bad))
        for t in outs[1:]:
            for s in (0, 1):
                rows = t[:, max(kp[s], 0):kp[s + 1]]
                assert (rows == (7 if s == bad else 0)).all() or kp[s + 1] < kp[s]
            assert (t[:, 290:] == 7).all()



def test_packed_split_over_the_keys_of_many_sequences(dsv):
    """More split sequences than a warp has lanes: their items are counted 32 at a time."""
    g = np.random.default_rng(17)
    for S, H, Hkv in ((33, 4, 4), (70, 6, 2), (140, 3, 1)):
        ql, kl = tuple(g.integers(0, 4, S)), tuple(g.choice([0, 1, 63, 128, 129, 700, 1500], S))
        assert Hkv * S < 152 and dsv.packed_attn_fwd_workspace_bytes(S, H, Hkv, sum(ql), sum(kl), 64) > 0
        for causal in (False, True):
            _check(dsv, Case(H, Hkv, 64, ql, kl), causal)



def test_packed_overlapping_sequences_are_reported_and_stay_in_range(dsv):
    """Pointers that fall and rise again make later sequences overlap earlier
    ones: the call is reported, and writes rows of its own tensors only."""
    T, H, Hkv, d = 1000, 4, 2, 64

    def frame(heads, value):
        big = torch.full((T + 64, heads + 2, d), value, dtype=torch.bfloat16, device="cuda")
        return big, big[32:-32, 1:-1].transpose(0, 1)

    for qp, kp in (((0, 1000, 50, 200, 300), (0, 300, 600, 800, 1000)),
                   ((0, 300, 600, 800, 1000), (0, 1000, 50, 200, 300)),
                   ((0, 900, 100, 1000), (0, 900, 100, 1000))):
        for tq in (1000, 3):                           # 3: the keys are split
            q_ptr = torch.tensor([v * tq // 1000 for v in qp], dtype=torch.int32, device="cuda")
            k_ptr = torch.tensor(kp, dtype=torch.int32, device="cuda")
            Q, K, V, dO = _rand(1, H, tq, d), _rand(2, Hkv, T, d), _rand(3, Hkv, T, d), _rand(4, H, tq, d)
            frames = [frame(n, 7.0) for n in (H, H, Hkv, Hkv)]
            O, dQ, dK, dV = (f[1][:, :(tq if i < 2 else T)] for i, f in enumerate(frames))
            lse = torch.zeros(H, tq, device="cuda")
            dsv.packed_attn_fwd(Q, K, V, q_ptr, k_ptr, causal=True, out=O, lse=lse)
            assert dsv.device_error()[0] == dsv.DSV_ERR_BAD_INDEX
            dsv.clear_device_error()
            dsv.packed_attn_bwd(Q, K, V, O, dO, lse, q_ptr, k_ptr, causal=True, outs=(dQ, dK, dV))
            assert dsv.device_error()[0] == dsv.DSV_ERR_BAD_INDEX
            dsv.clear_device_error()
            for (big, own), t in zip(frames, (O, dQ, dK, dV)):
                inside = torch.zeros(big.shape[:2], dtype=torch.bool, device="cuda")
                inside[32:32 + t.shape[1], 1:1 + t.shape[0]] = True
                assert (big[~inside] == 7).all()
