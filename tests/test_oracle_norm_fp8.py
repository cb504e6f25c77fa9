"""Pins of the fp64 oracle's layer norm, 8-bit blocks and product against
things other than itself: torch's fp64 layer norm and autograd, torch's 8-bit
types, hand-worked values (CPU only)."""
import numpy as np
import pytest
import torch

import oracle


def test_layer_norm_is_torchs(rng):
    x, w, b = rng.standard_normal((11, 24)) * 3 + 5, rng.standard_normal((3, 24)), rng.standard_normal((3, 24))
    ptr = [0, 4, 4, 11]
    y, mean, rstd = oracle.layer_norm(x, w, b, ptr, eps=1e-5)
    dy = rng.standard_normal(x.shape)
    tx, tw, tb = (torch.tensor(v, requires_grad=True) for v in (x, w, b))
    parts = [torch.nn.functional.layer_norm(tx[i:j], (24,), tw[s], tb[s], 1e-5)
             for s, (i, j) in enumerate(zip(ptr[:-1], ptr[1:]))]
    ty = torch.cat(parts)
    assert np.allclose(y, ty.detach().numpy(), rtol=0, atol=1e-12)
    ty.backward(torch.tensor(dy))
    for got, t in zip(oracle.layer_norm_bwd(dy, x, mean, rstd, w, ptr), (tx, tw, tb)):
        assert np.allclose(got, t.grad.numpy(), rtol=0, atol=1e-12)
    # one weight, and none
    y1 = oracle.layer_norm(x, w[0], b[0], eps=1e-5)[0]
    assert np.allclose(y1, torch.nn.functional.layer_norm(tx, (24,), tw[0], tb[0], 1e-5).detach().numpy(), atol=1e-12)
    assert np.allclose(oracle.layer_norm(x)[0], (x - x.mean(-1, keepdims=True)) / np.sqrt(x.var(-1, keepdims=True) + 1e-6))
    # equal parts without pointers; rows outside the sequences
    assert np.array_equal(oracle.layer_norm(x[:9], w, b)[0], oracle.layer_norm(x[:9], w, b, [0, 3, 6, 9])[0])
    assert np.isnan(oracle.layer_norm(x, w, b, [2, 4, 5, 9])[0][[0, 1, 9, 10]]).all()


@pytest.mark.parametrize("to,dtype", [("e4m3", torch.float8_e4m3fn), ("e5m2", torch.float8_e5m2)])
def test_round_fp8_is_torchs(to, dtype, rng):
    codes = torch.arange(256, dtype=torch.uint8).view(dtype).double().numpy()
    codes = np.sort(codes[np.isfinite(codes)])
    assert codes[-1] == oracle.FP8_TYPES[to][2]
    halves = (codes[1:] + codes[:-1]) / 2
    v = np.concatenate([codes, halves, rng.standard_normal(1000) * 10, rng.standard_normal(1000) * 2.0 ** -9])
    assert np.array_equal(oracle.round_fp8(v, to), torch.tensor(v).float().to(dtype).double().numpy())


def test_quantize_hand_worked(rng):
    x = np.zeros((3, 130))
    x[0, 5], x[0, 6] = 448.0, 1.0        # the largest value itself: scale 1
    x[1, 0] = 448.5                      # just past it: scale 2
    x[2, 129] = -0.875                   # 1.75 / 2: scale 2^-9, q = -448
    q, s = oracle.quantize_fp8(x)
    assert s.tolist() == [[1.0, 2.0, 1.0], [1.0, 1.0, 2.0 ** -9]]
    assert q[0, 5] == 448 and q[1, 0] == 224 and q[2, 129] == -448
    q, s = oracle.quantize_fp8(x, rows=128)
    assert s.tolist() == [[2.0], [2.0 ** -9]] and q[0, 5] == 224 and q[0, 6] == 0.5
    x = rng.standard_normal((200, 300)) * np.exp(rng.standard_normal((200, 1)))
    for rows in (1, 128):
        q, s = oracle.quantize_fp8(x, rows)
        back = oracle.dequantize_fp8(q, s)
        top = np.abs(q).reshape(200, 300).max()
        assert 224 < top <= 448
        # half a step of an element, or of the least normal number of its block
        row = np.arange(200) // rows
        least = s[np.arange(300) // 128][:, row].T * 2.0 ** -6
        assert np.all(np.abs(back - x) <= 2.0 ** -4 * np.maximum(np.abs(x), least))


def test_product_is_that_of_the_values(rng):
    a, b = rng.standard_normal((5, 200)), rng.standard_normal((7, 200))
    qa, sa = oracle.quantize_fp8(a)
    qb, sb = oracle.quantize_fp8(b, rows=128)
    want = np.zeros((5, 7))
    for m in range(5):
        for n in range(7):
            for k in range(200):
                want[m, n] += qa[m, k] * sa[k // 128, m] * qb[n, k] * sb[k // 128, 0]
    assert np.allclose(oracle.matmul_fp8(qa, sa, qb, sb), want, rtol=0, atol=1e-12)
