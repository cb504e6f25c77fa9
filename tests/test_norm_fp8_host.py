"""Host side of the layer norm, the 8-bit quantiser and the 8-bit product (CPU
only): the library refuses bad arguments before any launch, and the binding
checks shapes, types and devices."""
import pytest
import torch

FAKE = 1 << 20          # an aligned, never dereferenced address
FAR = [FAKE + (i << 32) for i in range(12)]


@pytest.fixture(scope="module")
def dsv():
    from dynamic_block_sparse_projection_gb300.build import build
    build()
    from dynamic_block_sparse_projection_gb300 import binding
    return binding


def test_norm_refusals(dsv):
    L, bad, uns, ok = dsv.lib, dsv.DSV_ERR_INVALID_ARG, dsv.DSV_ERR_UNSUPPORTED, dsv.DSV_OK
    R, BF, F = dsv.Rows, dsv.DSV_BF16, dsv.DSV_F32
    none = R(None, 0, 0)

    def f(p=(10, 64, 2), eps=1e-6, x=R(FAR[0], 64, BF), ptr=FAKE, w=FAKE, b=FAKE, y=R(FAR[1], 64, BF), st=FAKE):
        return L.dsv_layer_norm_fwd(x, dsv.Norm(*p, eps), ptr, w, b, y, st, None)

    for p in ((1 << 30, 64, 1), (10, 0, 1), (10, 16385, 1), (10, 64, 65536)):
        assert f(p) == uns, p
    for p in ((-1, 64, 1), (10, -1, 1), (10, 64, -1)):
        assert f(p) == bad, p
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        assert f(eps=eps) == bad
    assert f(w=None) == bad                                      # a bias alone
    assert f((11, 64, 2), ptr=None) == bad                       # equal parts of 11 rows
    assert f(ptr=FAKE + 2) == bad and f(w=FAKE + 1) == bad and f(b=FAKE + 2) == bad
    assert f(st=None) == bad and f(st=FAKE + 2) == bad
    assert f(x=none) == bad and f(y=none) == bad
    assert f(x=R(FAR[0], 63, BF)) == bad and f(y=R(FAR[1], 63, BF)) == bad      # rows overlap
    assert f(x=R(FAR[0] + 1, 64, BF)) == bad and f(x=R(FAR[0] + 2, 64, F)) == bad
    assert f(x=R(FAR[0], 64, dsv.DSV_E4M3)) == bad and f(x=R(FAR[0], 64, 7)) == bad
    assert f(y=R(FAR[1], 64, F)) == bad
    assert f(y=R(FAR[0], 72, BF)) == bad                         # x's address, other rows
    assert f(x=R(FAR[1], 64, F)) == bad                          # x's address, another type
    assert f((0, 64, 2), x=none, y=none, st=None) == ok          # no rows
    assert f((10, 64, 0), x=none, y=none, st=None) == ok         # no sequences

    n = dsv.layer_norm_bwd_workspace_bytes(10, 64, 2)
    assert n >= 3 * 2 * 64 * 4 and dsv.layer_norm_bwd_workspace_bytes(0, 64, 2) == 0
    assert L.dsv_layer_norm_bwd_workspace_bytes(dsv.Norm(10, 16385, 1, 1e-6)) == 0

    def g(p=(10, 64, 2), dy=R(FAR[2], 64, BF), x=R(FAR[0], 64, BF), st=FAKE, ptr=FAKE, w=FAKE, dx=R(FAR[3], 64, BF),
          dw=FAKE, db=FAKE, ws=FAKE, n=n):
        return L.dsv_layer_norm_bwd(dy, x, st, dsv.Norm(*p, 1e-6), ptr, w, dx, dw, db, ws, n, None)

    assert g((10, 16385, 2)) == uns and g((11, 64, 2), ptr=None) == bad
    assert g(dw=None) == bad and g(db=None) == bad and g(ws=None) == bad and g(n=n - 1) == bad and g(ws=FAKE + 64) == bad
    assert g(dy=none) == bad and g(x=none) == bad and g(dx=none) == bad and g(st=None) == bad
    assert g(dy=R(FAR[2], 64, F)) == bad and g(dx=R(FAR[3], 64, F)) == bad
    assert g(dx=R(FAR[0], 80, BF)) == bad and g(dx=R(FAR[2], 80, BF)) == bad
    assert g(x=R(FAR[2], 64, F), dx=R(FAR[2], 64, F)) == bad     # dx over a dy of another type


def test_quantize_refusals(dsv):
    L, bad, uns, ok = dsv.lib, dsv.DSV_ERR_INVALID_ARG, dsv.DSV_ERR_UNSUPPORTED, dsv.DSV_OK
    R, BF, F, E4, E5 = dsv.Rows, dsv.DSV_BF16, dsv.DSV_F32, dsv.DSV_E4M3, dsv.DSV_E5M2
    none = R(None, 0, 0)

    def f(r=40, c=100, rows=1, x=R(FAR[0], 100, BF), q=R(FAR[1], 112, E4), s=FAKE, qt=R(FAR[2], 48, E4), st=FAKE):
        return L.dsv_quantize_fp8(x, r, c, rows, q, s, qt, st, None)

    assert f(r=-1) == bad and f(c=-1) == bad and f(rows=2) == bad and f(rows=0) == bad
    assert f(r=2 ** 31 - 1) == uns and f(c=2 ** 31 - 128) == uns and f(r=2 ** 30, c=2 ** 30) == uns
    assert f(x=none) == bad and f(q=none) == bad and f(s=None) == bad and f(st=None) == bad and f(s=FAKE + 2) == bad
    assert f(x=R(FAR[0], 100, E4)) == bad and f(q=R(FAR[1], 112, BF)) == bad and f(qt=R(FAR[2], 48, E5)) == bad
    assert f(q=R(FAR[1] + 8, 112, E4)) == bad and f(q=R(FAR[1], 104, E4)) == bad and f(q=R(FAR[1], 96, E4)) == bad
    assert f(qt=R(FAR[2] + 8, 48, E4)) == bad and f(qt=R(FAR[2], 40, E4)) == bad and f(qt=R(FAR[2], 32, E4)) == bad
    assert f(qt=R(FAR[1], 48, E4)) == bad and f(q=R(FAR[0], 112, E4)) == bad
    assert f(x=R(FAR[0], 99, BF)) == bad and f(x=R(FAR[0] + 2, 100, F)) == bad
    for r, c in ((0, 100), (40, 0)):
        assert f(r, c, x=none, q=none, s=None, qt=none, st=None) == ok


def test_matmul_refusals(dsv):
    L, bad, uns, ok = dsv.lib, dsv.DSV_ERR_INVALID_ARG, dsv.DSV_ERR_UNSUPPORTED, dsv.DSV_OK
    R, BF, F, E4, E5 = dsv.Rows, dsv.DSV_BF16, dsv.DSV_F32, dsv.DSV_E4M3, dsv.DSV_E5M2
    none = R(None, 0, 0)

    def f(p=(40, 50, 100, 1, 128, 0), a=R(FAR[0], 112, E4), sa=FAKE, b=R(FAR[1], 112, E5), sb=FAKE, c=R(FAR[2], 50, BF)):
        return L.dsv_matmul_fp8(a, sa, b, sb, dsv.Matmul(*p), c, None)

    for p in ((-1, 50, 100, 1, 1, 0), (40, -1, 100, 1, 1, 0), (40, 50, -1, 1, 1, 0), (40, 50, 100, 2, 1, 0),
              (40, 50, 100, 1, 64, 0), (40, 50, 100, 1, 1, 2), (40, 50, 100, 1, 1, 1)):   # the last: bf16 accumulation
        assert f(p) == bad, p
    for p in ((2 ** 31 - 1, 1, 1, 1, 1, 0), (1, 2 ** 31 - 255, 1, 1, 1, 0), (1, 1, 2 ** 31 - 128, 1, 1, 0),
              (2 ** 30, 2 ** 30, 1, 1, 1, 0)):
        assert f(p) == uns, p
    assert f(a=none) == bad and f(b=none) == bad and f(c=none) == bad and f(sa=None) == bad and f(sb=None) == bad
    assert f(sa=FAKE + 2) == bad and f(sb=FAKE + 1) == bad
    assert f(a=R(FAR[0], 112, BF)) == bad and f(b=R(FAR[1], 112, F)) == bad and f(c=R(FAR[2], 50, E4)) == bad
    assert f(a=R(FAR[0] + 8, 112, E4)) == bad and f(a=R(FAR[0], 104, E4)) == bad and f(a=R(FAR[0], 96, E4)) == bad
    assert f(c=R(FAR[2], 49, BF)) == bad and f(c=R(FAR[2] + 1, 50, BF)) == bad and f(c=R(FAR[2] + 2, 50, F)) == bad
    assert f(c=R(FAR[0], 50, BF)) == bad and f(c=R(FAR[1], 50, BF)) == bad
    assert f((0, 50, 100, 1, 128, 0), none, None, none, None, none) == ok
    assert f((40, 0, 100, 1, 128, 0), none, None, none, None, none) == ok
    assert f((40, 50, 0, 1, 128, 1), none, None, none, None, R(FAR[2], 50, F)) == ok   # nothing to add


def test_binding_refusals(dsv):
    """Shapes and types, on tensors of the CPU (refused last, for their device)."""
    bf, f32, e4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
    x, w, ptr = torch.zeros(6, 8, dtype=bf), torch.zeros(2, 8), torch.zeros(3, dtype=torch.int32)
    st = torch.zeros(2, 6)
    with pytest.raises(ValueError, match="CUDA"):
        dsv.layer_norm(x, w, w, ptr)
    with pytest.raises(ValueError, match="CUDA"):
        dsv.layer_norm_bwd(x, x, st, w, ptr)
    for kw in (dict(weight=torch.zeros(7)), dict(weight=torch.zeros(4, 8)), dict(weight=w, seq_ptr=ptr[:2]),
               dict(weight=w[0], seq_ptr=ptr), dict(bias=w[0]), dict(weight=w, bias=w[0]), dict(seq_ptr=ptr[:0]),
               dict(out=x[:5]), dict(stats=st[:, :5])):
        with pytest.raises(ValueError):
            dsv.layer_norm(x, **kw)
    with pytest.raises(TypeError):
        dsv.layer_norm(x.half())
    with pytest.raises(TypeError):
        dsv.layer_norm([1.0])
    with pytest.raises(ValueError):
        dsv.layer_norm(torch.zeros(2, 3, 8, dtype=bf))
    for args, kw in (((x[:5], x, st), {}), ((x, x, st[:1]), {}), ((x, x, st), dict(dweight=w)),
                     ((x, x, st, w), dict(dweight=w[:1])), ((x, x, st, w), dict(dbias=w[0])), ((x, x, st), dict(dx=x[:5]))):
        with pytest.raises(ValueError):
            dsv.layer_norm_bwd(*args, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        dsv.quantize_fp8(x)
    with pytest.raises(ValueError):
        dsv.quantize_fp8(x, rows=64)
    with pytest.raises(TypeError):
        dsv.quantize_fp8(x, dtype=bf)
    with pytest.raises(TypeError):
        dsv.quantize_fp8(x.half())
    with pytest.raises(ValueError, match="outs"):
        dsv.quantize_fp8(x, transpose=True, outs=(x, x))
    with pytest.raises(ValueError, match="scale"):
        dsv.quantize_fp8(x, outs=(torch.zeros(6, 8, dtype=e4), torch.zeros(2, 6)))
    a, b = torch.zeros(200, 144, dtype=e4), torch.zeros(300, 144, dtype=e4)
    sa, sb = torch.zeros(2, 200), torch.zeros(2, 3)
    with pytest.raises(ValueError, match="CUDA"):
        dsv.matmul_fp8(a, sa, b, sb)
    for args, kw in (((a, sa, b[:, :128], sb), {}), ((a, sa[:1], b, sb), {}), ((a, sa, b, sb[:, :2]), {}),
                     ((a, sa, b, sb.t()), {}), ((a, sa, b, sb), dict(out=torch.zeros(200, 299))),
                     ((a, sa, b, sb), dict(accumulate=True))):
        with pytest.raises(ValueError):
            dsv.matmul_fp8(*args, **kw)
    for kw in (dict(out_dtype=torch.float16), dict(out=torch.zeros(200, 300, dtype=bf), accumulate=True)):
        with pytest.raises(TypeError):
            dsv.matmul_fp8(a, sa, b, sb, **kw)
    with pytest.raises(TypeError):
        dsv.matmul_fp8(torch.zeros(200, 144), sa, b, sb)


def test_binding_refuses_sizes_past_32_bits(dsv):
    """A size is not cut to its low 32 bits (2^32 + 1 rows would pass for one)."""
    many = 2 ** 32 + 1
    row = torch.zeros(1, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="32 bits"):
        dsv.layer_norm(row.expand(many, 8))
    a = torch.zeros(1, 16, dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="32 bits"):
        dsv.matmul_fp8(a.expand(many, 16), torch.zeros(1, 1).expand(1, many), a, torch.zeros(1, 1))


def test_benchmark_projection_arguments(capsys):
    import bench
    assert bench.parse_args([]).proj is None and bench.parse_args(["--proj", "fp8"]).proj == "fp8"
    with pytest.raises(SystemExit):
        bench.parse_args(["--proj", "fp8", "--impl", "reference"])
    assert "no oracle arm" in capsys.readouterr().err
