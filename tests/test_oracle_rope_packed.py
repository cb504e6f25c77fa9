"""Pins of the fp64 oracle's rotary positions and packed attention against
things other than itself: hand-worked values, invariants, torch's fp64 softmax
and autograd, and central differences (CPU only)."""
import numpy as np
import pytest
import torch

import oracle
from dynamic_block_sparse_projection_gb300 import workloads as wl


def _case(rng, H, Hkv, d, ql, kl):
    qp, kp = np.concatenate([[0], np.cumsum(ql)]), np.concatenate([[0], np.cumsum(kl)])
    Q, dO = (rng.standard_normal((H, qp[-1], d)) for _ in range(2))
    K, V = (rng.standard_normal((Hkv, kp[-1], d)) for _ in range(2))
    return Q, K, V, dO, qp, kp


def test_rope_hand_worked():
    # d = 6, bands of 4 and 2 channels, theta = 100: frequencies 1, 100^(-1/2) = 0.1 and 1
    x = np.arange(1.0, 7.0).reshape(1, 1, 1, 6)
    y = oracle.rope_axes(x, np.array([[2, 3]]), (4, 2), theta=100.0)[0, 0, 0]
    want = []
    for (a, b), ang in (((1, 2), 2.0), ((3, 4), 0.2), ((5, 6), 3.0)):
        want += [a * np.cos(ang) - b * np.sin(ang), a * np.sin(ang) + b * np.cos(ang)]
    assert np.allclose(y, want, rtol=0, atol=1e-14)


def test_rope_invariants(rng):
    x = rng.standard_normal((2, 3, 10, 64))
    pos = rng.integers(-50, 1000, (10, 3))
    y = oracle.rope_axes(x, pos, (20, 20, 20))
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))                     # lengths stay
    assert np.array_equal(y[..., 60:], x[..., 60:])                            # channels behind the bands
    assert np.array_equal(oracle.rope_axes(x, 0 * pos, (20, 20, 20)), x)
    # q . k depends on the difference of the positions alone
    q, k = x[:, :, :5], x[:, :, 5:]
    a = (oracle.rope_axes(q, pos[:5], (20, 20, 20)) * oracle.rope_axes(k, pos[5:], (20, 20, 20))).sum(-1)
    b = (oracle.rope_axes(q, pos[:5] + 77, (20, 20, 20)) * oracle.rope_axes(k, pos[5:] + 77, (20, 20, 20))).sum(-1)
    assert np.allclose(a, b, atol=1e-9)
    # per-batch positions
    pb = np.stack([pos, pos + 3])
    yb = oracle.rope_axes(x, pb, (20, 20, 20))
    assert np.array_equal(yb[0], y[0]) and np.array_equal(yb[1], oracle.rope_axes(x, pos + 3, (20, 20, 20))[1])


def test_rope_angles_are_the_embedding_s(rng):
    """A unit pair (1, 0) turned by the oracle is (cos, sin) of the sinusoidal
    embedding the workloads add, whose pairs are (sin, cos)."""
    T, Hl, Wl, d = 3, 4, 5, 64
    pe = wl.posemb_3d(T, Hl, Wl, d).numpy().astype(np.float64)
    n = np.arange(T * Hl * Wl)
    pos = np.stack([n // (Hl * Wl), (n // Wl) % Hl, n % Wl], 1)
    x = np.zeros((1, 1, len(n), d))
    x[..., 0::2] = 1.0
    y = oracle.rope_axes(x, pos, (20, 20, 20))[0, 0]
    assert np.allclose(y[:, 0:60:2], pe[:, 1:60:2], atol=1e-6) and np.allclose(y[:, 1:60:2], pe[:, 0:60:2], atol=1e-6)


@pytest.mark.parametrize("norm", [False, True])
def test_rope_gradient_against_differences_and_autograd(rng, norm):
    x, dy = (rng.standard_normal((1, 2, 4, 16)) for _ in range(2))
    w = 1 + 0.3 * rng.standard_normal(16) if norm else None
    pos, sec, eps = rng.integers(0, 9, (4, 2)), (8, 4), 1e-3
    got = oracle.rope_axes_bwd(dy, pos, sec, x=x, weight=w, eps=eps)
    dx, dw = got if norm else (got, None)
    f = lambda x_, w_: (oracle.rope_axes(x_, pos, sec, weight=w_, eps=eps) * dy).sum()   # noqa: E731
    h = 1e-6
    u = rng.standard_normal(x.shape)
    assert np.isclose((f(x + h * u, w) - f(x - h * u, w)) / (2 * h), (dx * u).sum(), rtol=1e-7)
    if norm:
        v = rng.standard_normal(16)
        assert np.isclose((f(x, w + h * v) - f(x, w - h * v)) / (2 * h), (dw * v).sum(), rtol=1e-7)
        tx = torch.tensor(x, requires_grad=True)
        tw = torch.tensor(w, requires_grad=True)
        xn = torch.nn.functional.rms_norm(tx, (16,), tw, eps)
        xn.backward(torch.tensor(oracle.rope_axes_bwd(dy, pos, sec)))
        assert np.allclose(tx.grad.numpy(), dx) and np.allclose(tw.grad.numpy(), dw)


@pytest.mark.parametrize("causal", [False, True])
def test_packed_attention_against_torch(rng, causal):
    Q, K, V, dO, qp, kp = _case(rng, 4, 2, 8, (5, 1, 0, 7), (9, 1, 3, 7))
    O, lse = oracle.packed_attn_fwd(Q, K, V, qp, kp, causal)
    dQ, dK, dV = oracle.packed_attn_bwd(Q, K, V, dO, qp, kp, causal)
    tq, tk, tv = (torch.tensor(t, requires_grad=True) for t in (Q, K, V))
    out = []
    for s in range(4):
        a, b, c, e = qp[s], qp[s + 1], kp[s], kp[s + 1]
        k, v = (t[:, c:e].repeat_interleave(2, 0) for t in (tk, tv))
        i = torch.arange(b - a)[:, None] + (e - c) - (b - a)
        m = (torch.arange(e - c)[None] <= i) if causal else None
        out.append(torch.nn.functional.scaled_dot_product_attention(tq[:, a:b], k, v, attn_mask=m))
    out = torch.cat(out, 1)
    assert np.allclose(out.detach().numpy(), O)
    out.backward(torch.tensor(dO))
    for got, t in ((dQ, tq), (dK, tk), (dV, tv)):
        assert np.allclose(got, t.grad.numpy())
    # keys of the sequence without queries
    assert not dK[:, 10:13].any() and not dV[:, 10:13].any()


def test_packed_attention_rows_without_keys(rng):
    """Causal with fewer keys than queries: the first Lq - Lk rows see nothing."""
    Q, K, V, dO, qp, kp = _case(rng, 1, 1, 8, (6, 2), (4, 0))
    O, lse = oracle.packed_attn_fwd(Q, K, V, qp, kp, True)
    assert not O[:, :2].any() and np.all(np.isneginf(lse[:, :2])) and np.all(np.isfinite(lse[:, 2:6]))
    assert not O[:, 6:].any() and np.all(np.isneginf(lse[:, 6:]))
    assert np.allclose(O[0, 2], V[0, 0]) and np.isclose(lse[0, 2], Q[0, 2] @ K[0, 0] / np.sqrt(8))
    dQ, _, _ = oracle.packed_attn_bwd(Q, K, V, dO, qp, kp, True)
    assert not dQ[:, :2].any() and not dQ[:, 6:].any() and np.all(np.isfinite(dQ))


def test_packed_gradient_against_differences(rng):
    Q, K, V, dO, qp, kp = _case(rng, 4, 2, 8, (5, 3), (6, 2))
    grads = oracle.packed_attn_bwd(Q, K, V, dO, qp, kp, True, 0.3)
    f = lambda q, k, v: (oracle.packed_attn_fwd(q, k, v, qp, kp, True, 0.3)[0] * dO).sum()   # noqa: E731
    h = 1e-6
    for i in range(3):
        u = [np.zeros_like(t) for t in (Q, K, V)]
        u[i] = rng.standard_normal(u[i].shape)
        num = (f(*(t + h * e for t, e in zip((Q, K, V), u))) - f(*(t - h * e for t, e in zip((Q, K, V), u)))) / (2 * h)
        assert np.isclose(num, (grads[i] * u[i]).sum(), rtol=1e-6)


def test_packing_is_one_sequence_at_a_time(rng):
    Q, K, V, dO, qp, kp = _case(rng, 2, 1, 8, (5, 3), (4, 6))
    O, lse = oracle.packed_attn_fwd(Q, K, V, qp, kp, True)
    for s in range(2):
        a, b, c, e = qp[s], qp[s + 1], kp[s], kp[s + 1]
        o, l = oracle.packed_attn_fwd(Q[:, a:b], K[:, c:e], V[:, c:e], [0, b - a], [0, e - c], True)
        assert np.array_equal(o, O[:, a:b]) and np.array_equal(l, lse[:, a:b])
