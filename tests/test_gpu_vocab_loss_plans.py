"""The vocabulary loss in every way its products are cut (tests/vocab_loss_sizes.py), against the formulas
in float64 on the GPU: loss, lse, dh and dw whole, with a bound for each element."""
import pytest
import torch

from mixture_experts_layer_20_amd import libmoe as L
from tests.gpu_helpers import DEV, log
from tests.vocab_loss_sizes import PLANS

pytestmark = pytest.mark.gpu

DT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step, relative


def make_data(T, d, V, dtype, seed):
    """Logits with a deviation of 2.5: a row's probability lies on some dozens of words, so that a word or
    a row left out shows in the sums."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=g)
    h, w = rnd(T, d).to(TORCH[dtype]), (2.5 / d ** 0.5 * rnd(V, d)).to(TORCH[dtype])
    target = torch.randint(0, V, (T,), device=DEV, generator=g)
    target[torch.rand(T, device=DEV, generator=g) < 0.1] = -100
    target[0], target[1], target[2] = V - 1, V, 0   # the last word, one past it, the first
    return h, w, target.to(torch.int32), rnd(T)


def run_loss(h, w, target, dloss, dtype):
    (T, d), V, dt = h.shape, w.shape[0], DT[dtype]
    nan = lambda *s, t=torch.float32: torch.full(s, float("nan"), dtype=t, device=DEV)
    ws = lambda n: torch.full((max(int(n), 256),), 0xFF, dtype=torch.uint8, device=DEV)
    loss, lse, dh, dw = nan(T), nan(T), nan(T, d, t=h.dtype), nan(V, d, t=h.dtype)
    wf, wb = ws(L.moe_vocab_loss_workspace_size(T, d, V, dt)), ws(L.moe_vocab_loss_bwd_workspace_size(T, d, V, dt))
    L.moe_vocab_loss(h, w, target, T, d, V, dt, loss, lse, wf, wf.numel())
    L.moe_vocab_loss_bwd(h, w, target, lse, dloss, T, d, V, dt, dh, dw, wb, wb.numel())
    torch.cuda.synchronize()
    return loss, lse, dh, dw


def within(name, got, ref, bound):
    got = got.double()
    assert bool(torch.isfinite(got).all()), f"{name}: a value is not finite"
    over = ((got - ref).abs() - bound).max()
    assert float(over) <= 0, f"{name}: {float((got - ref).abs().max()):.3e} off, bound exceeded by {float(over):.3e}"


def check_loss(h, w, target, dloss, dtype, got):
    """A product of K terms accumulated in fp32 is off by at most 2 K u sum |a b| (a matrix instruction
    may round inside as well as on its way out); the exponentials and the joins of the sums add some
    2^-20 relative; P is rounded to the storage type, then the outputs are."""
    (T, d), V, half = h.shape, w.shape[0], HALF[dtype] * (1 + 1e-3)
    h, w, t = h.double(), w.double(), target.long()
    l = h @ w.t()
    lse = torch.logsumexp(l, 1)
    ok = (t >= 0) & (t < V)
    rows = torch.nonzero(ok)[:, 0]
    loss = torch.zeros_like(lse)
    loss[rows] = lse[rows] - l[rows, t[rows]]
    e_l = 2 * d * U * (h.abs() @ w.abs().t()).amax(1)
    e_lse = e_l + 2.0 ** -20 + 4 * U * lse.abs()
    within("lse", got[1], lse, e_lse)
    within("loss", got[0], loss, 2 * e_lse + 4 * U * loss.abs())
    p = l.sub_(lse[:, None]).exp_()
    dl = torch.where(ok, dloss.double(), torch.zeros_like(lse))[:, None]
    e_P = p * (e_l + e_lse + 2.0 ** -20)[:, None]
    p[rows, t[rows]] -= 1.0
    e_P = dl.abs() * (e_P + half * p.abs() + 2 * U)
    P = p * dl
    del l, p
    A = P.abs()
    dh = P @ w
    within("dh", got[2], dh, e_P @ w.abs() + 2 * V * U * (A @ w.abs()) + half * dh.abs() + 2.0 ** -120)
    dw = P.t() @ h
    within("dw", got[3], dw, e_P.t() @ h.abs() + 2 * T * U * (A.t() @ h.abs()) + half * dw.abs() + 2.0 ** -120)
    assert not got[0][~ok].any() and not got[2][~ok].any()


@pytest.mark.parametrize("T,d,V,dtype", [c[:4] for c in PLANS])
def test_vocab_loss_as_it_is_cut(T, d, V, dtype):
    log(f"vocab loss plan {dtype} T={T} d={d} V={V}")
    data = make_data(T, d, V, dtype, T + V)
    check_loss(*data, dtype, run_loss(*data, dtype))


def test_the_bound_shows_what_is_left_out():
    """The check itself, on the oracle's side: gradients without the last words, without the last rows'
    terms or without a word that matters are outside the bounds."""
    log("vocab loss: the bound")
    T, d, V = 600, 136, 4000
    h, w, target, dloss = make_data(T, d, V, "bf16", 5)
    got = run_loss(h, w, target, dloss, "bf16")
    check_loss(h, w, target, dloss, "bf16", got)
    short = make_data(T, d, V, "bf16", 5)[1]
    short[-256:] = 0
    x, y, t = h.double(), w.double(), target.long()
    p = torch.softmax(x @ y.t(), 1)
    at = torch.nonzero((t >= 0) & (t < V))[:, 0]
    p[at, t[at]] -= 1
    keep = torch.zeros(T, 1, dtype=torch.float64, device=DEV)
    keep[at] = dloss.double()[at, None]
    P = p * keep
    top = P.abs().amax(0).argmax()
    for name, bad in (("dh", (P @ short.double(), P.t() @ x)), ("dw", (P @ y, P[:-100].t() @ x[:-100]))):
        with pytest.raises(AssertionError, match=name):
            check_loss(h, w, target, dloss, "bf16", (got[0], got[1], bad[0].to(h.dtype), bad[1].to(h.dtype)))
    P[:, top] = 0
    with pytest.raises(AssertionError, match="dh"):
        check_loss(h, w, target, dloss, "bf16", (got[0], got[1], (P @ y).to(h.dtype), got[3]))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,V", [(300, 65536, 700), (5, 65536, 9), (3, 8, 1 << 22), (1 << 22, 8, 64)])
def test_vocab_loss_at_its_limits(T, d, V, dtype):
    """The widest rows, the most words and the most tokens that the calls take."""
    log(f"vocab loss limits {dtype} T={T} d={d} V={V}")
    data = make_data(T, d, V, dtype, 11)
    check_loss(*data, dtype, run_loss(*data, dtype))
