"""Host side of the rotary-position and packed-attention calls (CPU only): the
library refuses bad arguments before any launch, and the binding checks shapes
and hands over addresses, strides and sizes (recorded by stand-ins)."""
import contextlib
import ctypes

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


def _rope(dsv, B=2, H=4, N=100, d=64, sections=(20, 20, 20), theta=1e4, axes=None):
    return dsv.Rope(B, H, N, d, len(sections) if axes is None else axes,
                    (ctypes.c_int32 * 4)(*sections), theta)


def _v4(dsv, ptr, B=2, H=4, N=100, d=64):
    return dsv.View(ptr, H * N * d, N * d, d)


def test_rope_refusals(dsv):
    L, bad, uns = dsv.lib, dsv.DSV_ERR_INVALID_ARG, dsv.DSV_ERR_UNSUPPORTED
    x, y = _v4(dsv, FAR[0]), _v4(dsv, FAR[1])
    f = lambda r, x=x, y=y, pos=FAKE, pb=0, w=None, eps=1e-6: L.dsv_rope_axes_fwd(x, pos, pb, r, w, eps, y, None)  # noqa: E731
    ok = _rope(dsv)
    assert f(_rope(dsv, d=96)) == uns and f(_rope(dsv, H=1025)) == uns
    assert f(_rope(dsv, B=-1)) == bad
    assert f(_rope(dsv, axes=0)) == uns and f(_rope(dsv, axes=5)) == uns
    assert f(_rope(dsv, sections=(20, 21))) == bad and f(_rope(dsv, sections=(0, 20))) == bad
    assert f(_rope(dsv, sections=(40, 20, 10))) == bad                     # more than d channels
    for theta in (0.5, float("inf"), float("nan")):
        assert f(_rope(dsv, theta=theta)) == bad
    assert f(ok, pos=None) == bad and f(ok, pos=FAKE + 2) == bad and f(ok, pb=-1) == bad
    assert f(ok, x=dsv.View(None, 0, 0, 0)) == bad and f(ok, x=_v4(dsv, FAR[0] + 8)) == bad
    assert f(ok, x=dsv.View(FAR[0], 25600, 6400, 60)) == bad               # stride under d
    assert f(ok, x=dsv.View(FAR[0], 25600, 6400, 68)) == bad               # not a multiple of 8
    assert f(ok, y=dsv.View(FAR[1], 25600, 64, 64)) == bad                 # heads of the output overlap
    assert f(ok, y=dsv.View(FAR[0], 25600, 64, 256)) == bad                # same address, other strides
    assert f(ok, w=FAKE, eps=0.0) == bad and f(ok, w=FAKE, eps=float("nan")) == bad and f(ok, w=FAKE + 1) == bad
    assert f(_rope(dsv, N=0), x=dsv.View(None, 0, 0, 0), pos=None) == dsv.DSV_OK
    # backward
    ws = L.dsv_rope_axes_bwd_workspace_bytes(ok)
    assert ws >= 64 * 4 and L.dsv_rope_axes_bwd_workspace_bytes(_rope(dsv, d=96)) == 0
    dy, dx = _v4(dsv, FAR[2]), _v4(dsv, FAR[3])
    b = lambda dy=dy, x=x, w=FAKE, dx=dx, dw=FAKE, s=FAKE, n=ws: L.dsv_rope_axes_bwd(  # noqa: E731
        dy, x, FAKE, 0, ok, w, 1e-6, dx, dw, s, n, None)
    assert b(dw=None) == bad and b(s=None) == bad and b(n=ws - 1) == bad and b(s=FAKE + 64) == bad
    assert b(x=dsv.View(None, 0, 0, 0)) == bad and b(dy=dsv.View(None, 0, 0, 0)) == bad
    assert b(dx=dsv.View(FAR[0], 25600, 64, 256)) == bad


def _v3(dsv, ptr, H, T, d=128, token_major=False):
    return dsv.View(ptr, 0, d, H * d) if token_major else dsv.View(ptr, 0, T * d, d)


def test_packed_refusals(dsv):
    L, bad, uns = dsv.lib, dsv.DSV_ERR_INVALID_ARG, dsv.DSV_ERR_UNSUPPORTED
    P = dsv.Packed

    def f(p=P(2, 8, 4, 40, 30, 128), Q=None, K=None, V=None, qp=FAKE, kp=FAKE, causal=0, O=None, lse=FAKE, ws=FAKE,
          n=None):
        Q = _v3(dsv, FAR[0], 8, 40) if Q is None else Q
        K = _v3(dsv, FAR[1], 4, 30) if K is None else K
        V = _v3(dsv, FAR[2], 4, 30) if V is None else V
        O = _v3(dsv, FAR[3], 8, 40) if O is None else O
        n = L.dsv_packed_attn_fwd_workspace_bytes(p) if n is None else n
        return L.dsv_packed_attn_fwd(Q, K, V, p, qp, kp, causal, 0.0, O, lse, ws, n, None)

    none = dsv.View(None, 0, 0, 0)
    for p in (P(2, 8, 4, 40, 30, 96), P(2, 2048, 4, 40, 30, 128), P(2, 258, 2, 40, 30, 128),
              P(1 << 24, 8, 4, 2000000000, 30, 128)):
        assert f(p) == uns and L.dsv_packed_attn_fwd_workspace_bytes(p) == 0
    for p in (P(2, 8, 3, 40, 30, 128), P(2, 8, 0, 40, 30, 128), P(-1, 8, 4, 40, 30, 128), P(2, 8, 4, -1, 30, 128)):
        assert f(p) == bad
    assert f(qp=None) == bad and f(kp=FAKE + 1) == bad and f(lse=None) == bad and f(causal=2) == bad
    assert f(Q=none) == bad and f(K=none) == bad and f(V=none) == bad and f(O=none) == bad
    assert f(Q=_v3(dsv, FAR[0] + 8, 8, 40)) == bad
    assert f(K=dsv.View(FAR[1], 0, 0, 128)) == bad                         # a key head broadcast by stride 0
    assert f(O=dsv.View(FAR[3], 0, 128, 128)) == bad                       # heads of the output overlap
    assert f(O=_v3(dsv, FAR[0], 8, 40)) == bad                             # O over Q
    # few query tiles against long keys: the split needs its workspace
    p = P(1, 8, 4, 1, 30000, 128)
    need = L.dsv_packed_attn_fwd_workspace_bytes(p)
    assert need > 0
    long_k = dict(Q=_v3(dsv, FAR[0], 8, 1), O=_v3(dsv, FAR[3], 8, 1), K=_v3(dsv, FAR[1], 4, 30000),
                  V=_v3(dsv, FAR[2], 4, 30000))
    assert f(p, n=need - 1, **long_k) == bad and f(p, ws=None, **long_k) == bad and f(p, ws=FAKE + 64, **long_k) == bad
    assert L.dsv_packed_attn_fwd_workspace_bytes(P(1, 24, 24, 16384, 16384, 128)) == 0     # enough tiles: no split
    assert f(P(0, 8, 4, 40, 30, 128)) == dsv.DSV_OK and f(P(2, 8, 4, 0, 30, 128)) == dsv.DSV_OK

    def b(p=P(2, 8, 4, 40, 30, 128), dQ=None, dK=None, lse=FAKE, ws=FAKE, n=None, dO=None):
        n = L.dsv_packed_attn_bwd_workspace_bytes(p) if n is None else n
        return L.dsv_packed_attn_bwd(
            _v3(dsv, FAR[0], 8, 40), _v3(dsv, FAR[1], 4, 30), _v3(dsv, FAR[2], 4, 30), _v3(dsv, FAR[3], 8, 40),
            _v3(dsv, FAR[4], 8, 40) if dO is None else dO, lse, p, FAKE, FAKE, 0, 0.0,
            _v3(dsv, FAR[5], 8, 40) if dQ is None else dQ, _v3(dsv, FAR[6], 4, 30) if dK is None else dK,
            _v3(dsv, FAR[7], 4, 30), ws, n, None)

    need = L.dsv_packed_attn_bwd_workspace_bytes(P(2, 8, 4, 40, 30, 128))
    assert need >= 2 * 8 * 40 * 4
    assert b(n=need - 1) == bad and b(ws=None) == bad and b(ws=FAKE + 128) == bad and b(lse=None) == bad
    assert b(dO=none) == bad and b(dQ=none) == bad
    assert b(dQ=_v3(dsv, FAR[4], 8, 40)) == bad                            # dQ over dO
    assert b(dK=_v3(dsv, FAR[7], 4, 30)) == bad                            # dK over dV
    assert b(P(2, 8, 3, 40, 30, 128)) == bad and b(P(0, 8, 4, 40, 30, 128)) == dsv.DSV_OK


@pytest.fixture()
def fake(dsv, monkeypatch):
    calls = []

    class FakeLib:
        def __getattr__(self, name):
            if name.endswith("_workspace_bytes"):
                return lambda s: 512

            def fn(*args):
                calls.append((name, args))
                return 0
            return fn

    monkeypatch.setattr(dsv, "lib", FakeLib())
    monkeypatch.setattr(dsv, "_need", lambda *a, **k: None)
    monkeypatch.setattr(dsv, "_need_rows", lambda *a, **k: None)
    monkeypatch.setattr(dsv, "_stream", lambda dev, stream=None: 1234)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    return dsv, calls


def test_binding_rope(fake):
    dsv, calls = fake
    x = torch.zeros(2, 10, 4, 64, dtype=torch.bfloat16).transpose(1, 2)       # [B, H, N, d] over [B, N, H, d]
    pos = torch.zeros(10, 3, dtype=torch.int32)
    y = dsv.rope_axes(x, pos, (20, 20, 20))
    name, a = calls[-1]
    assert name == "dsv_rope_axes_fwd" and y.shape == x.shape
    assert (a[0].ptr, a[0].batch_stride, a[0].head_stride, a[0].token_stride) == (x.data_ptr(), 2560, 64, 256)
    assert a[2] == 0 and (a[3].B, a[3].H, a[3].N, a[3].d, a[3].axes) == (2, 4, 10, 64, 3) and a[4] is None
    assert list(a[3].section)[:3] == [20, 20, 20] and a[3].theta == 1e4 and a[6].ptr == y.data_ptr()
    w = torch.ones(64)
    assert dsv.rope_axes(x, torch.zeros(2, 10, 1, dtype=torch.int32), (64,), weight=w, out=x) is x
    assert calls[-1][1][2] == 10 and calls[-1][1][4] == w.data_ptr()
    dx, dw = dsv.rope_axes_bwd(y, torch.zeros(10, 2, dtype=torch.int32), (20, 20), x=x, weight=w)
    assert dx.shape == x.shape and dw.shape == (64,) and calls[-1][0] == "dsv_rope_axes_bwd"
    assert calls[-1][1][10] == 512
    assert isinstance(dsv.rope_axes_bwd(y, pos, (20, 20, 20)), torch.Tensor) and calls[-1][1][1].ptr is None
    for bad in (dict(pos=torch.zeros(10, 2, dtype=torch.int32)), dict(pos=torch.zeros(3, 10, 3, dtype=torch.int32)),
                dict(weight=torch.ones(32)), dict(out=torch.zeros(2, 4, 10, 32))):
        with pytest.raises(ValueError):
            dsv.rope_axes(**{**dict(x=x, pos=pos, sections=(20, 20, 20)), **bad})
    with pytest.raises(ValueError):
        dsv.rope_axes(x, torch.zeros(10, 5, dtype=torch.int32), (8,) * 5)
    with pytest.raises(ValueError, match="needs x"):
        dsv.rope_axes_bwd(y, pos, (20, 20, 20), weight=w)
    with pytest.raises(ValueError, match="without a weight"):
        dsv.rope_axes_bwd(y, pos, (20, 20, 20), dweight=w)


def test_binding_packed(fake):
    dsv, calls = fake
    bf = torch.bfloat16
    Q = torch.zeros(40, 8, 64, dtype=bf).transpose(0, 1)
    KV = torch.zeros(30, 8, 64, dtype=bf).transpose(0, 1)
    K, V = KV[:4], KV[4:]
    qp, kp = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    O, lse = dsv.packed_attn_fwd(Q, K, V, qp, kp, 0.5, causal=True)
    name, a = calls[-1]
    assert name == "dsv_packed_attn_fwd" and O.shape == Q.shape and lse.shape == (8, 40)
    assert (a[2].ptr, a[2].head_stride, a[2].token_stride) == (V.data_ptr(), 64, 512)
    assert (a[3].S, a[3].H, a[3].Hkv, a[3].Tq, a[3].Tk, a[3].d) == (2, 8, 4, 40, 30, 64)
    assert a[6] == 1 and a[7] == 0.5 and a[11] == 512 and a[12] == 1234
    g = dsv.packed_attn_bwd(Q, K, V, O, O, lse, qp, kp)
    assert calls[-1][0] == "dsv_packed_attn_bwd" and [t.shape for t in g] == [Q.shape, K.shape, V.shape]
    assert calls[-1][1][9] == 0 and calls[-1][1][10] == 0.0
    with pytest.raises(ValueError, match="workspace needs"):
        dsv.packed_attn_fwd(Q, K, V, qp, kp, workspace=torch.empty(100, dtype=torch.uint8))
    for args in ((Q, KV[:3], KV[:3], qp, kp), (Q, K, KV, qp, kp), (Q, K[:, :, :32], V, qp, kp),
                 (Q, K, V, qp, kp[:2]), (Q, K, V, qp[:0], kp), (Q[0], K, V, qp, kp)):
        with pytest.raises(ValueError):
            dsv.packed_attn_fwd(*args)
    with pytest.raises(ValueError):
        dsv.packed_attn_fwd(Q, K, V, qp, kp, lse=torch.empty(8, 41))
    with pytest.raises(ValueError):
        dsv.packed_attn_bwd(Q, K, V, O[:, :39], O, lse, qp, kp)
    with pytest.raises(ValueError):
        dsv.packed_attn_bwd(Q, K, V, O, O, lse, qp, kp, outs=(Q, K))


def test_binding_refuses_what_is_not_a_row_view(dsv):
    cpu = torch.zeros(2, 4, 10, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        dsv._need_rows(cpu, "x")
    with pytest.raises(TypeError):
        dsv._need_rows(cpu.float(), "x")
    with pytest.raises(TypeError):
        dsv._need_rows([1.0], "x")


def test_c_entries_check_their_arguments(dsv):
    """The C module's functions take ctypes' place: wrong counts, structures and values raise, nothing is called."""
    v, p = dsv.View(FAKE, 0, 64, 64), dsv.Packed(0, 0, 0, 0, 0, 64)
    good = [v, v, v, p, FAKE, FAKE, 0, 0.0, v, FAKE, None, 0, None]
    assert dsv.lib.dsv_packed_attn_fwd(*good) == dsv.DSV_OK             # no sequences: nothing to do
    with pytest.raises(TypeError, match="arguments"):
        dsv.lib.dsv_packed_attn_fwd(*good[:-1])
    for at, bad, err in ((0, p, TypeError), (3, v, TypeError), (0, 5, TypeError), (6, 1 << 40, OverflowError),
                         (7, "1", TypeError), (11, -1, OverflowError), (4, "x", TypeError)):
        with pytest.raises(err):
            dsv.lib.dsv_packed_attn_fwd(*good[:at], bad, *good[at + 1:])
    for name, n in (("dsv_packed_attn_bwd", 17), ("dsv_rope_axes_fwd", 8), ("dsv_rope_axes_bwd", 12)):
        with pytest.raises(TypeError, match=f"expected {n} arguments"):
            getattr(dsv.lib, name)()


def test_packed_gradient_of_keys_without_query_heads_is_refused(dsv):
    """No query heads beside key heads: dK and dV would be left unwritten."""
    L, P, none = dsv.lib, dsv.Packed, dsv.View(None, 0, 0, 0)

    def b(p):
        k = [_v3(dsv, a, 4, 30) for a in FAR[1:3]]
        dk = [_v3(dsv, a, 4, 30) for a in FAR[6:8]]
        return L.dsv_packed_attn_bwd(none, *k, none, none, None, p, FAKE, FAKE, 0, 0.0, none, *dk, None, 0, None)

    assert b(P(2, 0, 4, 40, 30, 128)) == dsv.DSV_ERR_INVALID_ARG
    assert b(P(2, 0, 4, 0, 30, 128)) == dsv.DSV_ERR_INVALID_ARG
    # nothing to write: no keys, no sequences, no heads at all
    for p in (P(2, 0, 4, 40, 0, 128), P(0, 0, 4, 40, 30, 128), P(2, 0, 0, 40, 30, 128)):
        assert b(p) == dsv.DSV_OK
    assert L.dsv_packed_attn_fwd(none, none, none, P(2, 0, 4, 40, 30, 128), FAKE, FAKE, 0, 0.0, none, None, None, 0,
                                 None) == dsv.DSV_OK


def test_rope_refuses_token_counts_whose_last_tile_leaves_32_bits(dsv):
    L = dsv.lib
    for N in (2 ** 31 - 1, 2 ** 31 - 16, 2 ** 31 - 32):
        for d in (64, 128):
            r = _rope(dsv, B=1, H=1, N=N, d=d, sections=(d,))
            x, y = (dsv.View(a, 0, d, d) for a in FAR[:2])
            assert L.dsv_rope_axes_fwd(x, FAKE, 0, r, None, 1e-6, y, None) == dsv.DSV_ERR_UNSUPPORTED
            assert L.dsv_rope_axes_bwd(x, x, FAKE, 0, r, None, 1e-6, y, None, None, 0, None) == dsv.DSV_ERR_UNSUPPORTED
            assert L.dsv_rope_axes_bwd_workspace_bytes(r) == 0
    # below that, and below the limit on all rows, sizes are taken
    assert L.dsv_rope_axes_bwd_workspace_bytes(_rope(dsv, B=1, H=1, N=2 ** 31 - 33, sections=(64,))) > 0
    assert L.dsv_rope_axes_bwd_workspace_bytes(_rope(dsv, B=1, H=17, N=2 ** 31 - 33, sections=(64,))) == 0


def test_binding_refuses_sizes_past_32_bits(fake):
    """A size is not cut to its low 32 bits (2^32 + 1 keys would pass for one)."""
    dsv, calls = fake
    many, bf = 2 ** 32 + 1, torch.bfloat16
    row, ptr = torch.zeros(1, 1, 64, dtype=bf), torch.zeros(2, dtype=torch.int32)
    far, far_ptr = row.expand(1, many, 64), torch.zeros(1, dtype=torch.int32).expand(many + 1)
    for args in ((row, far, far, ptr, ptr), (far, row, row, ptr, ptr), (row, row, row, far_ptr, far_ptr)):
        with pytest.raises(ValueError, match="32 bits"):
            dsv.packed_attn_fwd(*args)
        with pytest.raises(ValueError, match="32 bits"):
            dsv.packed_attn_bwd(*args[:3], args[0], args[0], torch.zeros(1).expand(1, args[0].shape[1]), *args[3:])
    pos = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError, match="32 bits"):
        dsv.rope_axes(far[None], pos.expand(many, 1), (64,))
    with pytest.raises(ValueError, match="32 bits"):
        dsv.rope_axes(row[None], pos, (2 ** 32 + 64,))
    for f in (dsv.packed_attn_fwd_workspace_bytes, dsv.packed_attn_bwd_workspace_bytes):
        with pytest.raises(ValueError, match="32 bits"):
            f(1, 1, 1, 1, many, 64)
    assert not calls


def test_c_module_is_that_of_this_interpreter(dsv, monkeypatch, tmp_path):
    """The module's file carries the interpreter's tag, so one of another version neither counts as built nor is loaded."""
    import importlib.machinery
    import os
    import shutil

    from dynamic_block_sparse_projection_gb300 import build
    assert build.CALLS == dsv._CALLS_PATH and build.CALLS.name == "dsv_calls" + importlib.machinery.EXTENSION_SUFFIXES[0]
    other = tmp_path / "dsv_calls.cpython-399-other-linux-gnu.so"
    shutil.copy(build.CALLS, other)
    os.utime(other)
    assert build.up_to_date()
    monkeypatch.setattr(build, "CALLS", tmp_path / build.CALLS.name)
    assert not build.up_to_date()
    monkeypatch.setattr(dsv, "_CALLS_PATH", build.CALLS)
    with pytest.raises(ImportError, match="not built for this interpreter"):
        dsv._load_calls().row_views


def test_calls_of_the_library_do_not_need_the_c_module(dsv, tmp_path):
    """A tree whose C module is missing still has every call that does not go through it."""
    import shutil
    import subprocess
    import sys
    from pathlib import Path
    pkg = Path(dsv.__file__).parent
    shutil.copytree(pkg, tmp_path / pkg.name, ignore=shutil.ignore_patterns("dsv_calls*", "*.o", "__pycache__", "csrc"))
    code = f"""
import torch
from {pkg.name} import binding as d
assert d.status_string(0) and d.lib.dsv_version() > 0 and d.packed_attn_fwd_workspace_bytes(1, 1, 1, 1, 9000, 64) > 0
x = torch.zeros(1, 1, 4, 64, dtype=torch.bfloat16)
d._need_rows = lambda *a, **k: None
d._need = lambda *a, **k: None
try:
    d.rope_axes(x, torch.zeros(4, 1, dtype=torch.int32), (64,))
except ImportError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0 and "not built for this interpreter" in r.stdout, r.stdout + r.stderr
