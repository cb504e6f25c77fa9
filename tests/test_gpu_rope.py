"""GPU parity of the rotary positions (with and without the RMS norm) against
the fp64 oracle, forward and backward (needs a GB300).

Tolerances.  y is rounded once to bf16 (half a step: 2^-8 of the value) after
fp32 arithmetic; angle, sine, cosine, norm and the two products of a pair cost
at most a few 2^-24 of the pair's size each, taken together as 2^-20 (|a| + |b|).
dweight is an fp32 sum of R terms, each good to 2^-20: at most
(2^-20 + R 2^-24) sum |term|."""
import numpy as np
import pytest
import torch

import oracle
from parity_util import to64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dsv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_block_sparse_projection_gb300 import binding
    return binding


def _grid_pos(T, Hl, Wl, start=0):
    n = torch.arange(T * Hl * Wl, device="cuda")
    return torch.stack([start + n // (Hl * Wl), (n // Wl) % Hl, n % Wl], 1).to(torch.int32)


def _rand(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def _pair_size(z):
    s = np.abs(z[..., 0::2]) + np.abs(z[..., 1::2])
    return np.repeat(s, 2, -1)


def _close(got, ref, scale, what):
    tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * scale + 1e-30
    err = np.abs(to64(got) - ref)
    assert np.all(err <= tol), f"{what}: {np.max(err / tol):.3f} of the tolerance"


CASES = [  # B, H, grid, d, sections, start, layout
    (1, 2, (4, 8, 8), 64, (20, 20, 20), 0, "bhnd"),          # the tiny workload's queries
    (2, 3, (3, 5, 7), 128, (42, 42, 42), 0, "bnhd"),         # odd token count, projection layout
    (1, 24, (2, 6, 10), 128, (16, 56, 56), 1000003, "qkv"),  # far positions, a slice of a fused projection
    (3, 5, (1, 1, 1), 64, (16, 24, 24), 7, "bhnd"),          # one token
    (1, 1, (1, 17, 61), 128, (128,), -5, "bnhd"),            # one axis, negative positions
    (2, 2, (1, 9, 11), 64, (32, 16), 1 << 30, "bhnd"),       # two axes, very far
    (1, 7, (2, 5, 5), 128, (2, 4, 6, 8), 0, "bnhd"),         # four axes, most channels unrotated
]


def _case(seed, B, H, grid, d, sections, start, layout):
    N = grid[0] * grid[1] * grid[2]

    def t(k):
        if layout == "bhnd":
            return _rand(seed + k, B, H, N, d)
        if layout == "bnhd":
            return _rand(seed + k, B, N, H, d).transpose(1, 2)
        return _rand(seed + k, B, N, 3 * H, d).transpose(1, 2)[:, H:2 * H]

    pos = _grid_pos(*grid, start)
    A = len(sections)
    pos = torch.cat([pos, pos[:, 1:2] * 3 - 4], 1)[:, :A].contiguous()
    w = 1 + 0.25 * torch.randn(d, generator=torch.Generator(device="cuda").manual_seed(seed + 9), device="cuda")
    return t(0), t(1), pos, w


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("norm", [False, True])
def test_rope_forward(dsv, case, norm):
    sec = case[4]
    x, _, pos, w = _case(11, *case)
    w = w if norm else None
    y = dsv.rope_axes(x, pos, sec, weight=w, eps=1e-5)
    x64, p = to64(x), pos.cpu().numpy()
    ref = oracle.rope_axes(x64, p, sec, weight=None if w is None else to64(w), eps=1e-5)
    _close(y, ref, _pair_size(ref), "y")
    assert torch.equal(y, dsv.rope_axes(x, pos, sec, weight=w, eps=1e-5))
    if not norm:
        k = sum(sec)
        assert torch.equal(y[..., k:], x[..., k:])           # channels behind the bands: the same bits
    z = x.clone()
    assert dsv.rope_axes(z, pos, sec, weight=w, eps=1e-5, out=z) is z and torch.equal(z, y)   # in place


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("norm", [False, True])
def test_rope_backward(dsv, case, norm):
    sec = case[4]
    x, dy, pos, w = _case(23, *case)
    w = w if norm else None
    x64, g64, p = to64(x), to64(dy), pos.cpu().numpy()
    if not norm:
        ref = oracle.rope_axes_bwd(g64, p, sec)
        dx = dsv.rope_axes_bwd(dy, pos, sec)
        _close(dx, ref, _pair_size(ref), "dx")
        return
    dx, dw = dsv.rope_axes_bwd(dy, pos, sec, x=x, weight=w, eps=1e-5)
    w64 = to64(w)
    ref, dwr = oracle.rope_axes_bwd(g64, p, sec, x=x64, weight=w64, eps=1e-5)
    g = oracle.rope_axes_bwd(g64, p, sec)
    r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-5)
    xh = x64 * r
    # dx is a difference of two terms: its fp32 error goes by their sizes
    size = r * (_pair_size(g * w64) + np.abs(xh) * np.mean(np.abs(g * w64 * xh), -1, keepdims=True))
    _close(dx, ref, size, "dx")
    R = x64[..., 0].size
    tol = (2.0 ** -20 + R * 2.0 ** -24) * np.sum(_pair_size(g) * np.abs(xh), axis=(0, 1, 2))
    assert np.all(np.abs(to64(dw) - dwr) <= tol), np.max(np.abs(to64(dw) - dwr) / tol)
    # the gradient is that of the kernel's own forward: <dx, u> against differences of the fp64 forward
    u = np.random.default_rng(5).standard_normal(x64.shape)
    h = 1e-5
    f = lambda t: (oracle.rope_axes(t, p, sec, weight=w64, eps=1e-5) * g64).sum()   # noqa: E731
    num = (f(x64 + h * u) - f(x64 - h * u)) / (2 * h)
    bound = np.sum((2.0 ** -8 * np.abs(ref) + 2.0 ** -20 * size) * np.abs(u)) + 1e-6 * np.sum(size * np.abs(u))
    assert abs(num - (to64(dx) * u).sum()) <= bound
    # the same again, in place over dy, with the caller's workspace
    ws = torch.empty(dsv.rope_axes_bwd_workspace_bytes(case[3]), dtype=torch.uint8, device="cuda")
    z = dy.clone()
    dx2, dw2 = dsv.rope_axes_bwd(z, pos, sec, x=x, weight=w, eps=1e-5, dx=z, workspace=ws)
    assert dx2 is z and torch.equal(z, dx) and torch.equal(dw, dw2)


def test_rope_many_tokens_and_heads(dsv):
    """More token tiles and heads than CTAs hold at once; per-batch positions; rows sampled."""
    B, H, N, d, sec = 2, 9, 40961, 64, (20, 20, 20)
    x, dy = _rand(1, B, N, H, d).transpose(1, 2), _rand(2, B, H, N, d)
    g = torch.Generator(device="cuda").manual_seed(3)
    pos = torch.randint(-1000, 100000, (B, N, 3), generator=g, device="cuda", dtype=torch.int32)
    w = 1 + 0.25 * torch.randn(d, generator=g, device="cuda")
    y = dsv.rope_axes(x, pos, sec, weight=w)
    dx, dw = dsv.rope_axes_bwd(dy, pos, sec, x=x, weight=w)
    ref = oracle.rope_axes(to64(x), pos.cpu().numpy(), sec, weight=to64(w))
    _close(y, ref, _pair_size(ref), "y")
    _, dwr = oracle.rope_axes_bwd(to64(dy), pos.cpu().numpy(), sec, x=to64(x), weight=to64(w))
    # the error of a sum goes by its longest chain of additions: a thread's rows (at most twice the mean of
    # 608 CTAs x 32 rows), a CTA's 32 rows, and in the join 608 / 128 parts and 7 pairwise steps
    chain = 32 + 5 + 7 + 2 * (B * H * N) // (608 * 32)
    gg = oracle.rope_axes_bwd(to64(dy), pos.cpu().numpy(), sec)
    xh = to64(x) / np.sqrt((to64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
    tol = (2.0 ** -20 + chain * 2.0 ** -24) * np.sum(_pair_size(gg) * np.abs(xh), axis=(0, 1, 2))
    assert np.all(np.abs(to64(dw) - dwr) <= tol)


def test_rope_values_that_are_not_numbers_stay_in_their_row(dsv):
    x = _rand(4, 1, 2, 40, 64)
    pos = _grid_pos(1, 5, 8)
    clean = dsv.rope_axes(x, pos, (16, 16, 16), weight=torch.ones(64, device="cuda"))
    x[0, 1, 7, 3] = float("nan")
    x[0, 0, 9, 60] = float("inf")
    y = dsv.rope_axes(x, pos, (16, 16, 16), weight=torch.ones(64, device="cuda"))
    keep = torch.ones(2, 40, dtype=torch.bool, device="cuda")
    keep[1, 7] = keep[0, 9] = False
    assert torch.equal(y[0][keep], clean[0][keep]) and y[0, 1, 7].isnan().all()
    z = dsv.rope_axes(x, pos, (16, 16, 16))
    # without the norm a pair keeps to itself, and unrotated channels pass as they are
    assert z[0, 1, 7, 2:4].isnan().all() and z[0, 1, 7].isnan().sum() == 2
    assert torch.equal(z[0, 0, 9], dsv.rope_axes(x, pos, (16, 16, 16))[0, 0, 9]) and z[0, 0, 9, 60].isinf()


def test_rope_empty(dsv):
    x = torch.empty(0, 2, 5, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(5, 1, dtype=torch.int32, device="cuda")
    assert dsv.rope_axes(x, pos, (64,)).shape == x.shape
    dx, dw = dsv.rope_axes_bwd(x, pos, (64,), x=x, weight=torch.ones(64, device="cuda"),
                               dweight=torch.full((64,), 7.0, device="cuda"))
    torch.cuda.synchronize()
    assert not dw.any()


def test_rope_offsets_beyond_32_bits(dsv):
    """Rows whose element offset passes 2^31 (a strided view of a 4.4 GB buffer)."""
    big = torch.empty(2, 1 << 23, 2, 64, dtype=torch.bfloat16, device="cuda")    # [B, N, H, d], 2^31 elements
    x = big.transpose(1, 2)[:, :, -70:]
    x.copy_(_rand(6, 2, 2, 70, 64))
    pos = _grid_pos(1, 7, 10, 5)
    y = dsv.rope_axes(x, pos, (20, 20, 20), out=x.new_empty(2, 2, 70, 64))
    ref = oracle.rope_axes(to64(x), pos.cpu().numpy(), (20, 20, 20))
    _close(y, ref, _pair_size(ref), "y")


def test_rope_on_a_stream_and_in_a_graph(dsv):
    x, pos = _rand(8, 1, 4, 300, 128), _grid_pos(3, 10, 10)
    w = torch.full((128,), 1.5, device="cuda")
    ref = dsv.rope_axes(x, pos, (42, 42, 42), weight=w)
    dxr, dwr = dsv.rope_axes_bwd(ref, pos, (42, 42, 42), x=x, weight=w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(128, device="cuda")
    ws = torch.empty(dsv.rope_axes_bwd_workspace_bytes(128), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        dsv.rope_axes(x, pos, (42, 42, 42), weight=w, out=y, stream=st)
        dsv.rope_axes_bwd(y, pos, (42, 42, 42), x=x, weight=w, dx=dx, dweight=dw, workspace=ws, stream=st)
    for _ in range(2):
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref) and torch.equal(dx, dxr) and torch.equal(dw, dwr)


def test_sparse_path_on_normalised_and_rotated_queries(dsv):
    """The benchmark's step with norm and rotation: Q and K as the oracle's,
    the sparse path on them, and dQ, dK and the weights' gradients back through
    rotation and norm."""
    import bench
    from dynamic_block_sparse_projection_gb300 import workloads as wl
    from parity_util import O_REL_L2, SMALL, rel_l2
    w = SMALL["latent16k_small"]
    x = wl.make_inputs(w, device="cuda")
    hp = bench.HotPath(dsv, x, w, x.k_per_head, fused=True, rope="norm")
    hp.run()
    torch.cuda.synchronize()
    assert dsv.device_error()[0] == 0
    O, _, dQ, dK, dV, dwq, dwk = hp.results()
    pos, bands, one = wl.grid_positions(w.T, w.Hl, w.Wl).numpy(), wl.axis_bands(w.d), np.ones(w.d)
    for src, got in ((x.Q, hp.xr.Q), (x.K, hp.xr.K)):
        ref = oracle.rope_axes(to64(src), pos, bands, weight=one)
        _close(got, ref, _pair_size(ref), "rotated")
    fp, fc = (t.cpu().numpy() for t in hp.lists[:2])
    Q, K, V, dO = (to64(t) for t in (hp.xr.Q, hp.xr.K, x.V, x.dO))
    O_ref, _ = oracle.attn_fwd_groups(Q, K, V, fp, fc, w.block)
    gQ, gK, gV = oracle.attn_bwd_groups(Q, K, V, dO, fp, fc, w.block)
    assert rel_l2(to64(O), O_ref) <= O_REL_L2
    # The attention's gradients, element by element: P and dS are rounded to
    # bf16 (u = 2^-8 each), the fp32 part is e = 2^-12 of P, and D = dO . O takes
    # the error of the bf16 O, which dS carries as P * tol(D).  Where the softmax
    # is peaked, dP - D cancels and that is the largest term (3 % of dQ here in
    # norm, which a bound in norm alone would not separate from a slip).
    u, e, scale = 2.0 ** -8, 2.0 ** -12, w.d ** -0.5
    tq, tk, tv = u * np.abs(gQ), u * np.abs(gK), u * np.abs(gV)
    for h in range(w.H):
        mask = np.zeros((w.nb, w.nb), bool)
        for g in range(w.nb):
            mask[g, fc[fp[h * w.nb + g]:fp[h * w.nb + g + 1]]] = True
        mask = np.repeat(np.repeat(mask, w.block, 0), w.block, 1)
        q, k, v, do = (t[0, h] for t in (Q, K, V, dO))
        P = np.where(mask, scale * (q @ k.T), -np.inf)
        P = np.exp(P - P.max(-1, keepdims=True))
        P /= P.sum(-1, keepdims=True)
        tO = (u + e) * (P @ np.abs(v)) + u * np.abs(O_ref[0, h])
        dP = do @ v.T
        dS = P * (dP - np.sum(P * dP, -1, keepdims=True))
        tS = (u + 2 * e) * np.abs(dS) + P * (np.sum(np.abs(do) * tO, -1, keepdims=True) + e * (np.abs(do) @ np.abs(v).T))
        tv[0, h] += (u + 2 * e) * (P.T @ np.abs(do))
        tq[0, h] += scale * (tS @ np.abs(k))
        tk[0, h] += scale * (tS.T @ np.abs(q))
    assert np.all(np.abs(to64(dV) - gV) <= tv)
    # through the rotation (a pair's error at most sqrt(2) larger) and the norm's Jacobian, absolute values throughout
    for got, dw, src, g, t in ((dQ, dwq, x.Q, gQ, tq), (dK, dwk, x.K, gK, tk)):
        s64 = to64(src)
        ref, dwr = oracle.rope_axes_bwd(g, pos, bands, x=s64, weight=one)
        r = 1 / np.sqrt((s64 ** 2).mean(-1, keepdims=True) + 1e-6)
        xh, tr = s64 * r, _pair_size(t)
        tol = r * (tr + np.abs(xh) * np.mean(tr * np.abs(xh), -1, keepdims=True))
        gr = _pair_size(oracle.rope_axes_bwd(g, pos, bands))
        tol += 2.0 ** -20 * r * (gr + np.abs(xh) * np.mean(gr * np.abs(xh), -1, keepdims=True)) + u * np.abs(ref)
        assert np.all(np.abs(to64(got) - ref) <= tol), np.max(np.abs(to64(got) - ref) / tol)
        assert np.all(np.abs(to64(dw) - dwr) <= np.sum((tr + 2.0 ** -10 * gr) * np.abs(xh), axis=(0, 1, 2)))


def test_rope_launched_on_a_stream_that_is_not_current(dsv):
    """Results and workspace are allocated for the stream of the launch."""
    x, dy, pos = _rand(8, 1, 4, 300, 64), _rand(9, 1, 4, 300, 64), _grid_pos(3, 10, 10)
    w = torch.full((64,), 1.5, device="cuda")
    ref = (dsv.rope_axes(x, pos, (16, 24, 24), weight=w), *dsv.rope_axes_bwd(dy, pos, (16, 24, 24), x=x, weight=w))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(5):
        y = dsv.rope_axes(x, pos, (16, 24, 24), weight=w, stream=st)
        dx, dw = dsv.rope_axes_bwd(dy, pos, (16, 24, 24), x=x, weight=w, stream=st)
        junk = [torch.full((1 << 20,), 3.0, device="cuda") for _ in range(3)]       # the current stream's allocations
        st.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), ref))
        del junk


def _far_view(*tags):
    """[2, 2, 70, 64] views whose last batch lies wholly past 2^31 elements of a buffer of 4.3 GB each."""
    N = (1 << 23) + 4096
    for tag in tags:
        v = torch.empty(2, N, 2, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2)[:, :, -70:]
        assert (v[1, 0, 0].data_ptr() - v._base.data_ptr()) // 2 >= 1 << 31
        yield v if tag is None else v.copy_(_rand(tag, 2, 2, 70, 64))


def test_rope_rows_past_two_to_the_31_elements(dsv):
    """Inputs and outputs whose element offsets do not fit in 32 bits, forward and backward, with and without the norm."""
    pos, sec = _grid_pos(1, 7, 10, 5), (20, 20, 20)
    w = 1 + 0.25 * torch.randn(64, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    x, y = _far_view(6, None)
    near = x.clone()
    for weight in (None, w):
        want = dsv.rope_axes(near, pos, sec, weight=weight)
        assert torch.equal(dsv.rope_axes(x, pos, sec, weight=weight, out=y), want)
    ref = oracle.rope_axes(to64(near), pos.cpu().numpy(), sec, weight=to64(w))
    _close(y, ref, _pair_size(ref), "y")
    dy = y.copy_(_rand(7, 2, 2, 70, 64))
    dx, = _far_view(None)
    assert torch.equal(dsv.rope_axes_bwd(dy, pos, sec, dx=dx), dsv.rope_axes_bwd(dy.clone(), pos, sec))
    want, dww = dsv.rope_axes_bwd(dy.clone(), pos, sec, x=near, weight=w)
    got, dw = dsv.rope_axes_bwd(dy, pos, sec, x=x, weight=w, dx=dx)
    assert torch.equal(got, want) and torch.equal(dw, dww)
    ref, _ = oracle.rope_axes_bwd(to64(dy), pos.cpu().numpy(), sec, x=to64(near), weight=to64(w))
    x64 = to64(near)
    r = 1 / np.sqrt((x64 ** 2).mean(-1, keepdims=True) + 1e-6)
    g = oracle.rope_axes_bwd(to64(dy), pos.cpu().numpy(), sec)
    size = r * (_pair_size(g * to64(w)) + np.abs(x64 * r) * np.mean(np.abs(g * to64(w) * x64 * r), -1, keepdims=True))
    _close(got, ref, size, "dx")


@pytest.mark.parametrize("theta", [10000.0, 2.0, 1e6])
def test_rope_angles_are_as_good_as_stated(dsv, theta):
    """Sine and cosine of near and far positions, read in fp32 off the norm
    weight's gradient of one row (x = 1, dy = 1, 0, 1, 0, ...: cos, -sin, ...).

    The angle is good to 2 pi (|p| 2^-54 + 2^-25); sincospif is good to 2^-23, x^ = 1
    by rsqrtf to 2^-22, and two products are rounded: 2^-21 together."""
    import math
    from decimal import Decimal, getcontext
    getcontext().prec = 50
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582")
    d, sec = 64, (40, 20)
    x, dy = torch.ones(1, 1, 1, d, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 1, 1, d, device="cuda")
    dy[..., 0::2] = 1
    w = torch.ones(d, device="cuda")
    for p in ((0, 1), (1, -1), (3, 100), (-77, 4097), (65537, -1000003), (1 << 24, (1 << 24) + 1),
              ((1 << 31) - 1, -(1 << 31)), (123456789, -987654321)):
        _, dw = dsv.rope_axes_bwd(dy.to(torch.bfloat16), torch.tensor([p], dtype=torch.int32, device="cuda"), sec,
                                  theta=theta, x=x, weight=w, eps=1e-30)
        at = 0
        for a, c in zip(p, sec):
            for i in range(c // 2):
                turns = a * Decimal(theta) ** (Decimal(-2 * i) / c) / two_pi        # to 50 digits
                ang = float(turns - turns.to_integral_value()) * 2 * math.pi
                tol = 2 * math.pi * (abs(a) * 2.0 ** -54 + 2.0 ** -25) + 2.0 ** -21
                got = to64(dw)[2 * (at + i):2 * (at + i) + 2]
                assert abs(got[0] - math.cos(ang)) <= tol and abs(got[1] + math.sin(ang)) <= tol, (p, a, c, i)
            at += c // 2
    assert dsv.device_error()[0] == 0
