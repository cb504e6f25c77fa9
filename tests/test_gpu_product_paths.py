"""The 8-bit product behind every kernel that lets it start early (needs a GB300)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF, F32, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def dsv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from dynamic_block_sparse_projection_gb300 import binding
    binding.clear_device_error()
    return binding


def _rand(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def _codes(seed, *shape):
    """Numbers in e4m3, none of them infinite or NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randint(0, 120, shape, generator=g, device="cuda", dtype=torch.uint8).view(E4)


def _bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32)


def _packed(H, T, S, d, seed):
    q, k, v = (_rand(seed + i, H, T, d).to(BF) for i in range(3))
    ptr = torch.arange(S + 1, dtype=torch.int32, device="cuda") * (T // S)
    return q, k, v, ptr


def _behind_packed_fwd(dsv, H, T, S, d, tokens):
    """Keys whole (a work item for every SM): nothing of the call is behind its attention kernel."""
    q, k, v, ptr = _packed(H, T, S, d, 1)
    assert dsv.packed_attn_fwd_workspace_bytes(S, H, H, T, T, d) == 0
    out, lse = torch.empty_like(q), torch.empty(H, T, device="cuda")
    a, b = _codes(5, tokens, 128 * H), _codes(6, T, 128 * H)
    sa = torch.ones(H, tokens, device="cuda")

    def run(between):
        lse.fill_(float("nan"))
        dsv.packed_attn_fwd(q, k, v, ptr, ptr, out=out, lse=lse)
        between()
        return dsv.matmul_fp8(a, sa, b, lse)                # its lse: a scale for each row of b
    return run


def _behind_packed_bwd_without_queries(dsv, d):
    H, T = 8, 2560
    q, k, v, _ = _packed(H, T, 1, d, 1)
    kp, qp = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (T, 0))
    q, lse = q[:, :0].contiguous(), torch.empty(H, 0, device="cuda")
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    b = dv.view(-1).view(torch.uint8).view(-1, 128).view(E4)      # dv's own memory
    a, sa, sb = _codes(5, 1, 128), torch.ones(1, 1, device="cuda"), torch.ones(1, b.shape[0], device="cuda")

    def run(between):
        dv.fill_(1.0)
        dsv.packed_attn_bwd(q, k, v, q, q, lse, qp, kp, outs=(q, dk, dv))
        between()
        return dsv.matmul_fp8(a, sa, b, sb)
    return run


def _behind_norm_bwd(dsv, C):
    T, tokens = 500, 3
    x, dy = _rand(1, T, C), _rand(2, T, C).to(BF)
    stats = dsv.layer_norm(x)[1]
    dx = torch.empty_like(x)
    a, b, sa = _codes(5, tokens, 128 * T), _codes(6, C, 128 * T), torch.ones(T, tokens, device="cuda")

    def run(between):
        dx.fill_(float("nan"))
        dsv.layer_norm_bwd(dy, x, stats, dx=dx)             # no weight: no sums behind the rows
        between()
        return dsv.matmul_fp8(a, sa, b, dx)
    return run


@pytest.mark.parametrize("case", ["packed 64, two CTAs an SM", "packed 64", "packed 128", "no queries 64", "no queries 128",
                                  "norm 1160", "norm 1001"])
def test_product_directly_behind_a_kernel_that_lets_it_come_early(dsv, case):
    """The product reads what that kernel writes, and both allot tensor memory: the bits of the calls one by one."""
    kind, n = case.split(",")[0].split(" ")[0], int(case.split(",")[0].split(" ")[-1])
    if kind == "packed":                                    # one head's 24576 tokens: 192 tiles of the product
        run = _behind_packed_fwd(dsv, *((1, 24576, 192, n, 1) if "two" in case else (8, 2560, 1, n, 100)))
    elif kind == "no":
        run = _behind_packed_bwd_without_queries(dsv, n)
    else:
        run = _behind_norm_bwd(dsv, n)
    want = run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    assert not want.isnan().any()
    got = [run(lambda: None) for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(_bits(c), _bits(want)) for c in got)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        got = [run(lambda: None) for _ in range(3)]
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(_bits(c), _bits(want)) for c in got)
    assert dsv.device_error() == (0, 0)
