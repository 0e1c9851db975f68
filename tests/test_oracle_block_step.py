"""Pins of the oracle of the block norms, the vocabulary loss and gradient clipping: torch float64
autograd of the plain formulas, central finite differences, and hand values."""
import numpy as np
import pytest
import torch

from oracle import block_step as S


def _norm_case(T, d, gate_rows, seed):
    rng = np.random.default_rng(seed)
    r = lambda *s: rng.standard_normal(s)
    gate = r(-(-T // gate_rows), d) if gate_rows else None
    return dict(x=r(T, d), y=r(T, d), w_in=1 + 0.1 * r(d), w_out=1 + 0.1 * r(d), gate=gate, dout=r(T, d), dxn=r(T, d))


@pytest.mark.parametrize("T,d,gate_rows", [(1, 8, 0), (5, 16, 5), (7, 24, 3), (6, 8, 1)])
def test_norms_match_autograd(T, d, gate_rows):
    c = _norm_case(T, d, gate_rows, T + d)
    a, eps = 0.7, 1e-6
    t = {k: None if v is None else torch.tensor(v, requires_grad=True) for k, v in c.items()}
    xn = t["x"] * torch.rsqrt(t["x"].pow(2).mean(1, keepdim=True) + eps) * t["w_in"]
    g = t["gate"][torch.arange(T) // gate_rows] if gate_rows else 1.0
    out = a * t["x"] + g * (t["y"] * torch.rsqrt(t["y"].pow(2).mean(1, keepdim=True) + eps) * t["w_out"])
    got_xn, r_in = S.norm_in(c["x"], c["w_in"], eps)
    got_out, r_out = S.norm_out(c["y"], c["x"], c["w_out"], c["gate"], gate_rows, a, eps)
    assert np.allclose(got_xn, xn.detach().numpy(), atol=1e-12)
    assert np.allclose(got_out, out.detach().numpy(), atol=1e-12)
    (xn * torch.tensor(c["dxn"]) + out * torch.tensor(c["dout"])).sum().backward()
    dy, dw_out, dgate = S.norm_out_bwd(c["dout"], c["y"], c["w_out"], c["gate"], gate_rows, r_out)
    dx, dw_in = S.norm_in_bwd(c["dxn"], c["x"], c["w_in"], r_in, c["dout"], a)
    for got, name in ((dy, "y"), (dx, "x"), (dw_out, "w_out"), (dw_in, "w_in"), (dgate, "gate")):
        if got is not None:
            assert np.allclose(got, t[name].grad.numpy(), atol=1e-11), name


def test_norm_gradients_match_differences():
    c = _norm_case(4, 8, 2, 3)
    a, eps, h = 0.5, 1e-3, 1e-5
    f = lambda y: (S.norm_out(y, c["x"], c["w_out"], c["gate"], 2, a, eps)[0] * c["dout"]).sum()
    r = S.rms_rstd(c["y"], eps)
    dy, _, _ = S.norm_out_bwd(c["dout"], c["y"], c["w_out"], c["gate"], 2, r)
    for i, j in ((0, 0), (3, 7), (2, 5)):
        e = np.zeros_like(c["y"])
        e[i, j] = h
        assert abs((f(c["y"] + e) - f(c["y"] - e)) / (2 * h) - dy[i, j]) < 1e-7


def test_norm_hand_values():
    xn, r = S.norm_in([[3.0, 4.0]], [1.0, 2.0], 0.0)   # mean of squares 12.5
    assert np.allclose(r, 1 / np.sqrt(12.5)) and np.allclose(xn, [[3 / np.sqrt(12.5), 8 / np.sqrt(12.5)]])
    out, _ = S.norm_out([[0.0, 0.0]], [[1.0, 2.0]], [1.0, 1.0], None, 1, 0.5, 1e-6)
    assert np.array_equal(out, [[0.5, 1.0]])


@pytest.mark.parametrize("T,V,d", [(1, 1, 8), (6, 5, 8), (9, 33, 16)])
def test_vocab_loss_matches_autograd(T, V, d):
    rng = np.random.default_rng(V)
    h, w = rng.standard_normal((T, d)), rng.standard_normal((V, d))
    target = rng.integers(0, V, T)
    if T > 2:
        target[1], target[2] = -100, V
    dloss = rng.standard_normal(T)
    loss, lse = S.vocab_loss(h, w, target)
    ok = (target >= 0) & (target < V)
    th, tw = torch.tensor(h, requires_grad=True), torch.tensor(w, requires_grad=True)
    ref = torch.nn.functional.cross_entropy(th @ tw.T, torch.tensor(np.where(ok, target, -100)), reduction="none")
    assert np.allclose(loss, ref.detach().numpy(), atol=1e-12)
    (ref * torch.tensor(dloss)).sum().backward()
    dh, dw = S.vocab_loss_bwd(h, w, target, dloss)
    assert np.allclose(dh, th.grad.numpy(), atol=1e-12) and np.allclose(dw, tw.grad.numpy(), atol=1e-12)
    assert np.all(dh[~ok] == 0) and np.all(loss[~ok] == 0)


def test_vocab_loss_hand_values():
    loss, lse = S.vocab_loss([[0.0, 0.0]], [[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]], [2])
    assert np.allclose(loss, np.log(3)) and np.allclose(lse, np.log(3))   # equal logits: log V
    loss, _ = S.vocab_loss([[1.0, 0.0]], [[0.0, 9.0], [2.0, 9.0]], [1])
    assert np.allclose(loss, np.log(1 + np.exp(-2.0)))


def test_vocab_loss_gradient_matches_differences():
    rng = np.random.default_rng(0)
    h, w, target, dloss = rng.standard_normal((3, 4)), rng.standard_normal((7, 4)), np.array([6, 0, 3]), np.array([1.0, -2.0, 0.5])
    f = lambda a, b: (S.vocab_loss(a, b, target)[0] * dloss).sum()
    dh, dw = S.vocab_loss_bwd(h, w, target, dloss)
    e = 1e-6
    for i, j in ((0, 0), (2, 3)):
        p = np.zeros_like(h)
        p[i, j] = e
        assert abs((f(h + p, w) - f(h - p, w)) / (2 * e) - dh[i, j]) < 1e-8
    for i, j in ((6, 0), (0, 1), (5, 2)):
        p = np.zeros_like(w)
        p[i, j] = e
        assert abs((f(h, w + p) - f(h, w - p)) / (2 * e) - dw[i, j]) < 1e-8


def test_clip_matches_torch():
    rng = np.random.default_rng(1)
    grads = [rng.standard_normal(n) for n in (3, 1, 40)]
    for max_norm in (0.5, 1e3):
        ps = [torch.zeros(len(g), dtype=torch.float64, requires_grad=True) for g in grads]
        for p, g in zip(ps, grads):
            p.grad = torch.tensor(g)
        ref = torch.nn.utils.clip_grad_norm_(ps, max_norm)
        got, norm = S.clip(grads, max_norm)
        assert abs(norm - float(ref)) < 1e-12
        assert all(np.allclose(a, p.grad.numpy(), atol=1e-12) for a, p in zip(got, ps))


def test_clip_hand_values():
    got, norm = S.clip([[3.0], [4.0]], 1.0)
    assert norm == 5.0 and np.allclose([got[0][0], got[1][0]], [0.6, 0.8], atol=1e-6)
    got, norm = S.clip([[np.inf], [4.0]], 1.0)   # nothing is scaled
    assert np.isinf(norm) and got[1][0] == 4.0


def test_clip_of_a_norm_beyond_fp32():
    got, norm = S.clip([[3e38, -3e38]], 1.0)   # reported in fp32 as infinite: nothing is scaled
    assert norm > 4e38 and got[0].tolist() == [3e38, -3e38]
    got, norm = S.clip([[2e38, 2e38]], 1e30)
    assert np.allclose(got[0], 1e30 / np.sqrt(2), rtol=1e-12)
