"""Pins of oracle/train_step.py: torch float64 autograd, torch's E4M3 type and AdamW, finite differences and
hand values (CPU)."""
import numpy as np
import pytest
import torch

from oracle import train_step as S

KINDS = [(True, True), (True, False), (False, True), (False, False)]


def test_choose_by_hand():
    l = np.array([[0.0, 2.0, 1.0, 3.0, -1.0, 3.0, 0.5, 0.0]])
    assert S.choose(l, None, 3, 1, 1, True).tolist() == [[3, 5, 1]]
    b = np.zeros(8)
    b[0] = 1.0
    assert S.choose(l, b, 2, 1, 1, True).tolist() == [[0, 3]]
    # groups of two: sums of both scores; the third has s(-1) + s(3), the second s(1) + s(3)
    assert S.choose(l, None, 2, 4, 1, True).tolist() == [[3, 2]]
    assert S.choose(l, None, 3, 4, 2, True).tolist() == [[3, 1, 2]]
    # a shut expert, equal values, a NaN
    b[:] = 0.0
    b[3] = -np.inf
    assert S.choose(l, b, 2, 1, 1, False).tolist() == [[5, 1]]
    assert S.choose(np.zeros((1, 5)), None, 3, 1, 1, True).tolist() == [[0, 1, 2]]
    assert S.choose(np.array([[np.nan, -np.inf, 1.0]]), None, 3, 1, 1, True).tolist() == [[2, 1, 0]]


def test_move_bias_by_hand():
    assert S.move_bias([4, 0, 2, 2], 0.5, np.array([0.0, 0.0, 1.0, -1.0])).tolist() == [-0.5, 0.5, 1.0, -1.0]


@pytest.mark.parametrize("sigmoid,renormalize", KINDS)
def test_gates_against_autograd(sigmoid, renormalize):
    r = np.random.default_rng(3)
    l, dg, scale = r.standard_normal((7, 12)) * 3, r.standard_normal((7, 4)), 2.5
    idx = S.choose(l, r.standard_normal(12) * 0.1, 4, 3, 2, sigmoid)
    t = torch.tensor(l, requires_grad=True)
    s = t.sigmoid() if sigmoid else t.softmax(1)
    g = s.gather(1, torch.tensor(idx))
    if renormalize:
        g = g / g.sum(1, keepdim=True)
    g = g * scale
    (g * torch.tensor(dg)).sum().backward()
    np.testing.assert_allclose(S.gates(l, idx, sigmoid, renormalize, scale), g.detach().numpy(), rtol=1e-13)
    dl = S.gates_bwd(dg, l, idx, sigmoid, renormalize, scale)
    np.testing.assert_allclose(dl, t.grad.numpy(), rtol=1e-10, atol=1e-14)
    h = 1e-6
    for _ in range(6):
        i, e = r.integers(7), r.integers(12)
        up, down = l.copy(), l.copy()
        up[i, e] += h
        down[i, e] -= h
        d = ((S.gates(up, idx, sigmoid, renormalize, scale) - S.gates(down, idx, sigmoid, renormalize, scale)) * dg).sum()
        assert abs(d / (2 * h) - dl[i, e]) < 1e-8 * max(1.0, np.abs(dl).max())


def test_gates_that_underflow():
    l = np.array([[-900.0, -901.0, -2000.0], [-np.inf, -np.inf, 0.0]])
    g = S.gates(l, np.array([[0, 1], [0, 1]]), True, True, 1.0)
    e = 1.0 / (1.0 + np.exp(-1.0))
    np.testing.assert_allclose(g, [[e, 1 - e], [0.0, 0.0]], rtol=1e-12)


def test_e4m3_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(S.E4M3, t)
    r = np.random.default_rng(5)
    mid = (S.E4M3[:0x7E] + S.E4M3[1:0x7F]) / 2
    v = np.concatenate([mid, -mid, S.E4M3[:0x7F], r.uniform(-448, 448, 4000), r.standard_normal(4000) * 2.0 ** -7])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(S.e4m3(v), want)


def test_quantizers_and_product():
    r = np.random.default_rng(6)
    x = r.standard_normal((5, 256)) * np.exp(r.standard_normal((5, 1)))
    x[2, :128] = 0.0
    codes, s = S.quantize_rows(x)
    assert codes.shape == (5, 256) and s.shape == (2, 5)
    y = S.rows_of(codes, s)
    top = np.abs(x.reshape(5, 2, 128)).max(2).T
    assert np.all(np.abs(y - x) <= np.maximum(np.abs(x) * 2.0 ** -4, np.repeat(top.T, 128, 1) / 448 * 2.0 ** -10) * (1 + 1e-12))
    assert s[0, 2] == S.TINY / 448 and not codes[2, :128].any()
    w = r.standard_normal((2, 128, 256))
    cw, sw = S.quantize_weights(w)
    ct, st = S.quantize_weights(w.transpose(0, 2, 1))
    np.testing.assert_array_equal(ct, cw.transpose(0, 2, 1))
    np.testing.assert_array_equal(st, sw.transpose(0, 2, 1))
    out, size, tops = S.grouped_product(y, S.weights_of(cw, sw), [1, 1, 4])
    assert np.isnan(out[0]).all() and np.isnan(out[4]).all()
    np.testing.assert_allclose(out[1:4], y[1:4] @ S.weights_of(cw, sw)[1].T)
    assert np.all(np.abs(out[1:4]) <= size[1:4]) and np.all(size[1:4] <= 8 * tops[1:4])


def test_adamw_is_torchs():
    r = np.random.default_rng(7)
    p0 = r.standard_normal(50)
    t = torch.tensor(p0, requires_grad=True)
    opt = torch.optim.AdamW([t], lr=0.01, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
    p, m, v = p0, np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = r.standard_normal(50)
        t.grad = torch.tensor(g)
        opt.step()
        p, m, v = S.adamw(p, g, m, v, 0.01, 0.9, 0.95, 1e-8, step, 0.1)
        np.testing.assert_allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14)
    assert S.clip(None, 1.0) == 1.0 and S.clip(0.25, 1.0) == 1.0
    assert abs(S.clip(16.0, 1.0) - 1.0 / (4.0 + 1e-6)) < 1e-15
