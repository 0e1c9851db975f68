"""The block norms, the vocabulary loss and gradient clipping on the GPU against the float64 oracle.

Tolerances are bounds, computed from the data where they depend on it: u = 2^-24 (half a step of fp32)
for every fp32 operation of a sum, and half a step of the storage type for every rounding to it."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_20_amd import inputs as I
from mixture_experts_layer_20_amd import layer as LY
from mixture_experts_layer_20_amd import libmoe as L
from oracle import block_step as S
from oracle import moe_oracle as O
from tests.gpu_helpers import DEV, as_dtype_values, assert_close, dev_tensor, log, tnp

pytestmark = pytest.mark.gpu

DT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}
U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}   # half a step, relative
EPS = 1e-6


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


def empty(*shape, dtype="f32"):
    """Filled with NaN: a value that is not written shows."""
    return torch.full(shape, float("nan"), dtype=torch.bfloat16 if dtype == "bf16" else torch.float32, device=DEV)


def ws_of(n):
    return torch.full((max(int(n), 256),), 0xFF, dtype=torch.uint8, device=DEV)   # NaN in every type


def within(name, got, ref, bound):
    """|got - ref| <= bound, element by element (bound broadcasts)."""
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    over = np.abs(got - ref) - bound
    assert np.all(np.isfinite(got)), f"{name}: a value is not finite"
    assert np.max(over, initial=-1.0) <= 0, f"{name}: {np.max(np.abs(got - ref)):.3e} off, bound exceeded by {np.max(over):.3e}"


# ------------------------------------------------------------------------------------------- norms
# A row statistic adds d squares: at most 64 in a lane (d <= 16384), then 8 levels of a tree, a
# division and a root: its relative error is under STAT = 80 u; a normalised value has three more
# roundings.  The mean m of u_j n_j adds terms with such errors: off by at most 2 STAT mean |u n|.
STAT = 80 * U


def norm_data(T, d, dtype, gate_rows, seed):
    rng = np.random.default_rng(seed)
    v = lambda *s, f=1.0, o=0.0: as_dtype_values(o + f * rng.standard_normal(s), dtype)
    c = dict(x=v(T, d) * 1.0, y=v(T, d, f=3.0), w_in=v(d, f=0.1, o=1.0), w_out=v(d, f=0.1, o=1.0), dout=v(T, d), dxn=v(T, d),
             gate=v(-(-T // gate_rows), d, f=0.3, o=0.5) if gate_rows else None)
    return c, {k: None if a is None else dev_tensor(a, dtype) for k, a in c.items()}


NORM_SIZES = [(1, 8, 0), (1, 4096, 1), (3, 520, 2), (7, 2048, 1), (129, 1000, 100), (130, 2056, 64), (1031, 128, 1031),
              (2050, 64, 3), (40, 8192, 17), (9, 16384, 0), (600, 4104, 600), (5000, 16, 700)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,gate_rows", NORM_SIZES)
def test_norms_match_oracle(dtype, T, d, gate_rows):
    log(f"norms {dtype} T={T} d={d} gate_rows={gate_rows}")
    a = 0.75
    c, t = norm_data(T, d, dtype, gate_rows, T + d)
    xn, out, r_in, r_out = empty(T, d, dtype=dtype), empty(T, d, dtype=dtype), empty(T), empty(T)
    L.moe_norm_in(t["x"], t["w_in"], T, d, EPS, DT[dtype], xn, r_in)
    L.moe_norm_out(t["y"], t["x"], t["w_out"], t["gate"], gate_rows, a, EPS, T, d, DT[dtype], out, r_out)
    ref_xn, ref_ri = S.norm_in(c["x"], c["w_in"], EPS)
    ref_out, ref_ro = S.norm_out(c["y"], c["x"], c["w_out"], c["gate"], gate_rows, a, EPS)
    half = HALF[dtype]
    within("rstd_in", tnp(r_in), ref_ri, STAT * ref_ri)
    within("rstd_out", tnp(r_out), ref_ro, STAT * ref_ro)
    within("xn", tnp(xn), ref_xn, (STAT + 4 * U + half) * np.abs(ref_xn))
    normed = np.abs(ref_out - a * c["x"].astype(np.float64))
    within("out", tnp(out), ref_out, (STAT + 6 * U) * normed + 3 * U * np.abs(a * c["x"]) + half * (1 + 1e-4) * np.abs(ref_out)
           + 2.0 ** -120)

    # backward, from the device's own statistics
    dy, dx = empty(T, d, dtype=dtype), empty(T, d, dtype=dtype)
    dw_in, dw_out = empty(d), empty(d)
    dgate = empty(*c["gate"].shape) if gate_rows else None
    ws = ws_of(L.moe_norm_bwd_workspace_size(T, d))
    L.moe_norm_out_bwd(t["dout"], t["y"], t["w_out"], t["gate"], gate_rows, r_out, T, d, DT[dtype], dy, dw_out, dgate, ws,
                       ws.numel())
    ws2 = ws_of(L.moe_norm_bwd_workspace_size(T, d))
    L.moe_norm_in_bwd(t["dxn"], t["x"], t["w_in"], r_in, t["dout"], a, T, d, DT[dtype], dx, dw_in, ws2, ws2.numel())
    ref_dy, ref_dwo, ref_dg = S.norm_out_bwd(c["dout"], c["y"], c["w_out"], c["gate"], gate_rows, ref_ro)
    ref_dx, ref_dwi = S.norm_in_bwd(c["dxn"], c["x"], c["w_in"], ref_ri, c["dout"], a)
    g = S.gate_of_rows(c["gate"], gate_rows, T, d)

    def through(u, v, r):   # bound of r (u - n m)
        n = v * r[:, None]
        m = np.abs(u * n).mean(axis=1, keepdims=True)
        return r[:, None] * (np.abs(u) * (STAT + 8 * U) + np.abs(n) * m * (4 * STAT + 8 * U))

    within("dy", tnp(dy), ref_dy, through(c["dout"] * g * c["w_out"], c["y"], ref_ro) + half * (1 + 1e-4) * np.abs(ref_dy))
    within("dx", tnp(dx), ref_dx, through(c["dxn"] * c["w_in"], c["x"], ref_ri) + 3 * U * np.abs(a * c["dout"])
           + half * (1 + 1e-4) * np.abs(ref_dx))
    col = (T + 16) * U + STAT   # a column adds at most T terms with a statistic in each
    n_out, n_in = c["y"] * ref_ro[:, None], c["x"] * ref_ri[:, None]
    within("dw_out", tnp(dw_out), ref_dwo, col * np.abs(c["dout"] * g * n_out).sum(axis=0))
    within("dw_in", tnp(dw_in), ref_dwi, col * np.abs(c["dxn"] * n_in).sum(axis=0))
    if gate_rows:
        each = np.zeros(c["gate"].shape)
        np.add.at(each, np.arange(T) // gate_rows, np.abs(c["dout"] * n_out * c["w_out"]))
        within("dgate", tnp(dgate), ref_dg, col * each)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,k,shared,gate_rows", [(1, 4096, 4, True, 0), (37, 1000, 8, True, 10), (5, 16, 1, False, 5),
                                                     (300, 2048, 3, False, 1), (20, 16384, 2, True, 0)])
def test_combine_norm_out_matches_oracle(dtype, T, d, k, shared, gate_rows):
    log(f"combine norm {dtype} T={T} d={d} k={k} shared={shared} gate_rows={gate_rows}")
    rng = np.random.default_rng(T + k)
    c, t = norm_data(T, d, dtype, gate_rows, T + d)
    yp = as_dtype_values(rng.standard_normal((T * k, d)), dtype)
    gates = rng.random((T, k)).astype(np.float32)
    pos = rng.permutation(T * k).astype(np.int32)
    sh = as_dtype_values(rng.standard_normal((T, d)), dtype) if shared else None
    rows = yp.astype(np.float64)[pos].reshape(T, k, d)
    y = (rows * gates[:, :, None].astype(np.float64)).sum(axis=1) + (sh if shared else 0.0)
    size = (np.abs(rows) * gates[:, :, None]).sum(axis=1) + (np.abs(sh) if shared else 0.0)
    ref, ref_r = S.norm_out(y, c["x"], c["w_out"], c["gate"], gate_rows, 1.0, EPS)
    dev = [dev_tensor(yp, dtype), f32(gates), torch.from_numpy(pos).to(DEV), dev_tensor(sh, dtype) if shared else None]
    y_dev, out, r = empty(T, d, dtype=dtype), empty(T, d, dtype=dtype), empty(T)
    L.moe_combine_norm_out(*dev, t["x"], t["w_out"], t["gate"], gate_rows, 1.0, EPS, T, d, k, DT[dtype], y_dev, out, r)
    half = HALF[dtype]
    e_y = (2 * k + 2) * U * size   # every product and sum rounded once
    within("y", tnp(y_dev), y, e_y + half * (1 + 1e-4) * np.abs(y))
    e_r = STAT + (e_y * np.abs(y)).mean(axis=1) * ref_r ** 2
    within("rstd", tnp(r), ref_r, e_r * ref_r)
    g = np.abs(S.gate_of_rows(c["gate"], gate_rows, T, d) * c["w_out"])
    bound = g * ref_r[:, None] * (e_y + np.abs(y) * (e_r[:, None] + 6 * U)) + 3 * U * np.abs(c["x"])
    within("out", tnp(out), ref, bound + half * (1 + 1e-4) * np.abs(ref))
    # without the stash and the statistic: the same output
    out2 = empty(T, d, dtype=dtype)
    L.moe_combine_norm_out(*dev, t["x"], t["w_out"], t["gate"], gate_rows, 1.0, EPS, T, d, k, DT[dtype], None, out2, None)
    assert torch.equal(out, out2)
    # the rounded rows are those of moe_combine
    if d % 8 == 0:
        comb = empty(T, d, dtype=dtype)
        L.moe_combine(*dev, T, d, k, DT[dtype], comb)
        within("combine", tnp(comb), y, e_y + half * (1 + 1e-4) * np.abs(y))


def test_norm_rows_of_zeros_and_extreme_scales():
    """A row of zeros normalises to zeros (eps keeps the root finite) with a finite gradient; rows of
    1e-15 and 1e15 keep their statistics."""
    log("norms: zero and extreme rows")
    T, d = 3, 256
    rng = np.random.default_rng(0)
    x = rng.standard_normal((T, d)).astype(np.float32) * np.array([[0.0], [1e-15], [1e15]], np.float32)
    w = np.ones(d, np.float32)
    for eps in (1e-6, 1e-36):
        xn, r = empty(T, d), empty(T)
        L.moe_norm_in(f32(x), f32(w), T, d, eps, L.MOE_F32, xn, r)
        ref, ref_r = S.norm_in(x, w, float(np.float32(eps)))
        within("rstd", tnp(r), ref_r, STAT * ref_r)
        within("xn", tnp(xn), ref, (STAT + 8 * U) * np.abs(ref))
        dx, dw, ws = empty(T, d), empty(d), ws_of(L.moe_norm_bwd_workspace_size(T, d))
        L.moe_norm_in_bwd(f32(np.ones((T, d))), f32(x), f32(w), r, None, 1.0, T, d, L.MOE_F32, dx, dw, ws, ws.numel())
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_norms_of_more_rows_than_one_grid():
    """2^20 workgroups of four rows, and five rows more."""
    log("norms: many rows")
    T, d = (1 << 22) + 5, 8
    rng = np.random.default_rng(1)
    x = rng.standard_normal((T, d)).astype(np.float32)
    w = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    xd, xn, out, r = f32(x), empty(T, d), empty(T, d), empty(T)
    L.moe_norm_in(xd, f32(w), T, d, EPS, L.MOE_F32, xn, r)
    ref, _ = S.norm_in(x, w, EPS)
    within("xn", tnp(xn), ref, (STAT + 4 * U) * np.abs(ref))
    L.moe_norm_out(xd, xn, f32(w), None, 1, 0.0, EPS, T, d, L.MOE_F32, out, None)
    assert torch.equal(out, xn)


def test_norm_offsets_beyond_32_bits():
    log("norms: 4.9e9 elements")
    T, d, n = 600_000, 8192, 3
    x = torch.zeros(T, d, dtype=torch.bfloat16, device=DEV)
    xn, r = torch.empty_like(x), empty(T)
    c, t = norm_data(n, d, "bf16", 0, 5)
    x[-n:] = t["x"]
    L.moe_norm_in(x, t["w_in"], T, d, EPS, L.MOE_BF16, xn, r)
    ref, ref_r = S.norm_in(c["x"], c["w_in"], EPS)
    within("xn", tnp(xn[-n:]), ref, (STAT + 4 * U + HALF["bf16"]) * np.abs(ref))
    assert not xn[:10].any()
    g = torch.zeros_like(x)
    g[-n:] = t["dxn"]
    dw, ws = empty(d), ws_of(L.moe_norm_bwd_workspace_size(T, d))
    L.moe_norm_in_bwd(g, x, t["w_in"], r, None, 1.0, T, d, L.MOE_BF16, xn, dw, ws, ws.numel())
    _, ref_dw = S.norm_in_bwd(c["dxn"], c["x"], c["w_in"], ref_r, None, 1.0)
    # three rows have terms: the sums add at most those, whatever their order, and zeros exactly
    within("dw", tnp(dw), ref_dw, (n * U + STAT) * np.abs(c["dxn"] * c["x"] * ref_r[:, None]).sum(axis=0))


def test_norms_without_rows():
    log("norms: no rows")
    d = 64
    dw = empty(d)
    z = torch.zeros(0, d, device=DEV)
    w = torch.ones(d, device=DEV)
    L.moe_norm_in_bwd(None, None, w, None, None, 1.0, 0, d, L.MOE_F32, None, dw, None, 0)
    assert torch.equal(dw, torch.zeros(d, device=DEV))
    dw.fill_(float("nan"))
    L.moe_norm_out_bwd(None, None, w, None, 1, None, 0, d, L.MOE_F32, z, dw, None, None, 0)
    assert torch.equal(dw, torch.zeros(d, device=DEV))


# -------------------------------------------------------------------------------------------- loss

def loss_data(T, d, V, dtype, ignored, seed, scale=0.05):
    rng = np.random.default_rng(seed)
    h = as_dtype_values(rng.standard_normal((T, d)), dtype)
    w = as_dtype_values(scale * rng.standard_normal((V, d)), dtype)
    target = rng.integers(0, V, T).astype(np.int32)
    target[rng.random(T) < ignored] = -100
    if T > 3:
        target[0], target[1], target[2] = V - 1, V, 0   # the last word, one past it, the first
    dloss = rng.standard_normal(T).astype(np.float32)
    return h, w, target, dloss


def run_loss(h, w, target, dloss, dtype):
    (T, d), V = h.shape, w.shape[0]
    hd, wd, td = dev_tensor(h, dtype), dev_tensor(w, dtype), torch.from_numpy(target).to(DEV)
    loss, lse = empty(T), empty(T)
    ws = ws_of(L.moe_vocab_loss_workspace_size(T, d, V, DT[dtype]))
    L.moe_vocab_loss(hd, wd, td, T, d, V, DT[dtype], loss, lse, ws, ws.numel())
    dh, dw = empty(T, d, dtype=dtype), empty(V, d, dtype=dtype)
    wsb = ws_of(L.moe_vocab_loss_bwd_workspace_size(T, d, V, DT[dtype]))
    L.moe_vocab_loss_bwd(hd, wd, td, lse, f32(dloss), T, d, V, DT[dtype], dh, dw, wsb, wsb.numel())
    torch.cuda.synchronize()
    return loss, lse, dh, dw


def check_loss(h, w, target, dloss, dtype, got):
    """A product of K terms accumulated in fp32 is off by at most 2 K u sum |a b| (a matrix
    instruction may round inside as well as on its way out); the exponentials and the joins of the
    sums add some 2^-20 relative; P is rounded to the storage type, then the outputs are."""
    (T, d), V = h.shape, w.shape[0]
    h64, w64 = h.astype(np.float64), w.astype(np.float64)
    loss, lse = S.vocab_loss(h, w, target)
    dh, dw = S.vocab_loss_bwd(h, w, target, dloss)
    e_l = 2 * d * U * (np.abs(h64) @ np.abs(w64).T).max(axis=1)      # every logit of the row
    e_lse = e_l + 2.0 ** -20 + 4 * U * np.abs(lse)
    within("lse", tnp(got[1]), lse, e_lse)
    within("loss", tnp(got[0]), loss, 2 * e_lse + 4 * U * np.abs(loss))
    ok = (target >= 0) & (target < V)
    assert np.all(tnp(got[0])[~ok] == 0)
    p = np.exp(h64 @ w64.T - lse[:, None])
    P = p.copy()
    P[ok, target[ok]] -= 1.0
    dl = np.where(ok, np.abs(dloss.astype(np.float64)), 0.0)[:, None]
    e_P = dl * (p * (e_l + e_lse + 2.0 ** -20)[:, None] + HALF[dtype] * np.abs(P) * (1 + 1e-3) + 2 * U)
    P = np.abs(P) * dl
    within("dh", tnp(got[2]), dh, e_P @ np.abs(w64) + 2 * V * U * (P @ np.abs(w64)) + HALF[dtype] * (1 + 1e-3) * np.abs(dh)
           + 2.0 ** -120)
    within("dw", tnp(got[3]), dw, e_P.T @ np.abs(h64) + 2 * T * U * (P.T @ np.abs(h64)) + HALF[dtype] * (1 + 1e-3) * np.abs(dw)
           + 2.0 ** -120)
    assert np.all(tnp(got[2])[~ok] == 0)


LOSS_SIZES = [(1, 8, 1, 0.0), (1, 4096, 1000, 0.0), (2, 64, 127, 0.0), (5, 72, 129, 0.3), (63, 256, 257, 0.0),
              (130, 136, 1000, 0.5), (257, 512, 513, 0.1), (300, 1000, 301, 0.0), (64, 2048, 4099, 0.2), (513, 64, 8200, 0.0),
              (700, 200, 16421, 0.1), (2500, 72, 4001, 0.2), (4097, 136, 300, 0.1), (1030, 1032, 3000, 0.1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,V,ignored", LOSS_SIZES)
def test_vocab_loss_matches_oracle(dtype, T, d, V, ignored):
    log(f"vocab loss {dtype} T={T} d={d} V={V} ignored={ignored}")
    data = loss_data(T, d, V, dtype, ignored, T + V)
    check_loss(*data, dtype, run_loss(*data, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_vocab_loss_over_several_pieces(dtype):
    """More words than one piece of the backward holds (at least 4096 words and 2^26 elements of P)."""
    T, d, V = 16390, 24, 4500
    log(f"vocab loss {dtype} several pieces T={T} d={d} V={V}")
    data = loss_data(T, d, V, dtype, 0.1, 5)
    check_loss(*data, dtype, run_loss(*data, dtype))


def test_vocab_loss_with_dw_split_over_the_rows():
    """Many rows against few words and columns: the large tiles split dw's sum as well as dh's."""
    T, d, V = 4100, 520, 9001
    log(f"vocab loss bf16 dw split T={T} d={d} V={V}")
    data = loss_data(T, d, V, "bf16", 0.1, 6)
    check_loss(*data, "bf16", run_loss(*data, "bf16"))


def _gpu_reference(h, w, target, dloss, rows):
    """Loss, dh of the first and last rows and dw in float64 on the GPU, a block of rows at a time."""
    T, V = h.shape[0], w.shape[0]
    w64, dw, loss, dh = w.double(), torch.zeros(w.shape, dtype=torch.float64, device=DEV), [], []
    for t0 in range(0, T, rows):
        hb, tb = h[t0:t0 + rows].double(), target[t0:t0 + rows].long()
        l = hb @ w64.t()
        lse = torch.logsumexp(l, 1)
        at = torch.arange(len(tb), device=DEV)
        loss.append(lse - l[at, tb])
        p = torch.exp(l - lse[:, None])
        p[at, tb] -= 1.0
        p *= dloss[t0:t0 + rows, None].double()
        dw += p.t().contiguous() @ hb
        if t0 == 0 or t0 + rows >= T:
            dh.append((p @ w64)[:1] if t0 == 0 else (p @ w64)[-1:])
    return torch.cat(loss), torch.cat(dh), dw


@pytest.mark.parametrize("T,d,V", [(530_000, 64, 4096), (24, 4096, 600_000)])
def test_vocab_loss_offsets_beyond_32_bits(T, d, V):
    """P of 2.2e9 elements; w and dw of 2.5e9.  The layer's tolerance: the sums are far longer than the
    terms that matter, and the bound by terms would say nothing."""
    log(f"vocab loss bf16 T={T} d={d} V={V}")
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    h = torch.randn(T, d, device=DEV, generator=g).to(torch.bfloat16)
    w = (0.1 * torch.randn(V, d, device=DEV, generator=g)).to(torch.bfloat16)
    target = torch.randint(0, V, (T,), device=DEV, generator=g).to(torch.int32)
    target[-1] = V - 1
    dloss = torch.rand(T, device=DEV, generator=g)
    loss, lse, dh, dw = empty(T), empty(T), torch.empty_like(h), torch.empty_like(w)
    ws = torch.empty(L.moe_vocab_loss_workspace_size(T, d, V, 1), dtype=torch.uint8, device=DEV)
    L.moe_vocab_loss(h, w, target, T, d, V, L.MOE_BF16, loss, lse, ws, ws.numel())
    ws = torch.empty(L.moe_vocab_loss_bwd_workspace_size(T, d, V, 1), dtype=torch.uint8, device=DEV)
    L.moe_vocab_loss_bwd(h, w, target, lse, dloss, T, d, V, L.MOE_BF16, dh, dw, ws, ws.numel())
    ref_loss, ref_dh, ref_dw = _gpu_reference(h, w, target, dloss, 65536)
    if T == 24:
        ref_dh = torch.cat([ref_dh[:1], ref_dh[:1]])   # one block: its first row
    err = lambda a, b: float((a.double() - b).abs().max() / b.abs().max())
    assert err(loss, ref_loss) < 1e-5
    assert err(dh[:1], ref_dh[:1]) < 2e-2 and (T == 24 or err(dh[-1:], ref_dh[1:]) < 2e-2)
    assert err(dw, ref_dw) < 2e-2 and err(dw[-1], ref_dw[-1]) < 2e-2


def test_vocab_loss_with_no_target_at_all_and_confident_rows():
    log("vocab loss: all ignored; confident rows")
    T, d, V = 70, 128, 500
    h, w, target, dloss = loss_data(T, d, V, "bf16", 0.0, 9)
    loss, lse, dh, dw = run_loss(h, w, np.full(T, -1, np.int32), dloss, "bf16")
    assert not loss.any() and not dh.any() and not dw.any()
    # logits of some hundred: exponentials would overflow without the maximum
    h, w, target, dloss = loss_data(T, d, V, "bf16", 0.0, 10, scale=8.0)
    data = (h, w, target, dloss)
    check_loss(*data, "bf16", run_loss(*data, "bf16"))
    # the gradient of an ignored row's loss is not read
    target[5] = -100
    dloss[5] = np.nan
    loss, lse, dh, dw = run_loss(h, w, target, dloss, "bf16")
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all() and not dh[5].any()


def test_vocab_loss_gradient_of_the_mean_is_not_biased():
    """Every token's dloss is 1 / n and no target is likely: the gradient is the targets' rows, and the
    rounding of 1 / n in P (up to 2^-9, the same in every row) must not show in it.  P's element of a
    target is 1 - p with its sign: bf16 steps by 2^-8 below 1, so for p < 2^-9 it rounds to 1 and is off
    by p, always outwards; for the other words and the outputs the roundings go either way."""
    log("vocab loss: mean's gradient")
    T, d, V = 300, 64, 5000
    h, w, _, _ = loss_data(T, d, V, "bf16", 0.0, 12)
    target = np.random.default_rng(1).permutation(V)[:T].astype(np.int32)
    for n in (T, 307, 509):   # 1 / n rounds to bf16 by up to half a step
        dloss = np.full(T, 1.0 / n, np.float32)
        _, _, _, dw = run_loss(h, w, target, dloss, "bf16")
        _, ref = S.vocab_loss_bwd(h, w, target, dloss)
        got, ref = tnp(dw)[target].astype(np.float64), ref[target]
        p = np.exp(-S.vocab_loss(h, w, target)[0])
        assert p.max() < 2.0 ** -9
        # the signed mean error of 300 x 64 independent roundings, each under 2^-8, stays below 6 sigma
        signed = ((got - ref) * np.sign(ref)).sum() / np.abs(ref).sum()
        assert abs(signed) < 6 * 2.0 ** -8 / np.sqrt(3 * T * d) + p.mean() * 1.5, signed   # |h| differs by row


def test_vocab_loss_scales_of_dloss():
    """dloss of very different sizes among the rows, tiny everywhere, infinite in one row."""
    log("vocab loss: dloss scales")
    T, d, V = 66, 64, 300
    h, w, target, dloss = loss_data(T, d, V, "f32", 0.0, 13)
    for f in (10.0 ** np.linspace(-12, 0, T), np.full(T, 1e-30)):
        data = (h, w, target, (dloss * f).astype(np.float32))
        check_loss(*data, "f32", run_loss(*data, "f32"))
    dloss[7] = np.inf
    _, _, dh, _ = run_loss(h, w, target, dloss, "f32")
    ref, _ = S.vocab_loss_bwd(h, w, target, np.where(np.arange(T) == 7, 0.0, dloss))
    rows = np.arange(T) != 7
    assert not np.isfinite(tnp(dh)[7]).all()
    assert_close("dh of the other rows", tnp(dh)[rows], ref[rows], 1e-5)


def test_vocab_loss_without_tokens():
    log("vocab loss: no tokens")
    w = torch.ones(100, 64, device=DEV)
    dw = empty(100, 64)
    L.moe_vocab_loss_bwd(None, w, None, None, None, 0, 64, 100, L.MOE_F32, None, dw, None, 0)
    assert not dw.any()


def test_vocab_loss_gradient_matches_differences():
    log("vocab loss: differences")
    T, d, V = 20, 64, 300
    h, w, target, dloss = loss_data(T, d, V, "f32", 0.2, 3, scale=0.3)
    _, _, dh, dw = run_loss(h, w, target, dloss, "f32")
    f = lambda a, b: (S.vocab_loss(a, b, target)[0] * dloss.astype(np.float64)).sum()
    e = 1e-5
    for name, a, grad, at in (("h", h, dh, (4, 7)), ("w", w, dw, (int(target[0]), 3)), ("w", w, dw, (11, 63))):
        p = np.zeros(a.shape)
        p[at] = e
        hi, lo = (f(h + p, w), f(h - p, w)) if name == "h" else (f(h, w + p), f(h, w - p))
        # the difference is off by e^2/6 times a third derivative (under 10) and 1e-12 / e of rounding
        assert abs((hi - lo) / (2 * e) - float(grad[at])) < 1e-6 + 1e-4 * abs(float(grad[at]))


# ---------------------------------------------------------------------------------------- clipping

def clip_data(sizes, seed, scale=1.0):
    rng = np.random.default_rng(seed)
    types = ["bf16" if i % 2 else "f32" for i in range(len(sizes))]
    vals = [as_dtype_values(scale * (1 + i % 3) * rng.standard_normal(n), t) for i, (n, t) in enumerate(zip(sizes, types))]
    return types, vals


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [0, 4096, 0, 4097, 100003], [3] * 250, [5_000_011, 1, 999], []])
def test_clip_matches_oracle(sizes, max_norm):
    log(f"clip sizes={sizes[:5]} of {len(sizes)} max_norm={max_norm}")
    types, vals = clip_data(sizes, len(sizes))
    grads = [dev_tensor(v, t) for v, t in zip(vals, types)]
    outs = [torch.full_like(g, float("nan")) for g in grads]
    ref, ref_norm = S.clip(vals, float(np.float32(max_norm)))
    lst = L.grad_list(grads, outs)
    ws, norm = ws_of(L.moe_grad_workspace_size(lst)), empty(1)
    L.moe_grad_clip(lst, max_norm, norm, ws, ws.numel())
    within("norm", tnp(norm), [ref_norm], 2 * U * ref_norm)   # double sums, rounded once
    for o, r, t, g, v in zip(outs, ref, types, grads, vals):
        within("out", tnp(o), r, (3 * U + HALF[t]) * np.abs(r) + (2.0 ** -133 if t == "bf16" else 2.0 ** -149))
        assert np.array_equal(tnp(g), v)   # the input is left as it was
        if max_norm > 1e8:
            assert np.array_equal(tnp(o), v)
    # in place, through the two separate calls: the same bits
    inplace = [g.clone() for g in grads]
    lst2 = L.grad_list(inplace)
    sumsq = torch.full((1,), float("nan"), dtype=torch.float64, device=DEV)
    norm2, norm3 = empty(1), empty(1)
    L.moe_grad_norm(lst2, sumsq, norm2, ws, ws.numel())
    L.moe_grad_scale(lst2, sumsq, max_norm, norm3)
    assert torch.equal(norm, norm2) and torch.equal(norm, norm3)
    assert abs(float(sumsq) - ref_norm ** 2) <= 1e-12 * ref_norm ** 2
    assert all(torch.equal(a, b) for a, b in zip(inplace, outs))


def test_clip_of_extreme_and_non_finite_gradients():
    log("clip: extreme and non-finite")
    run = lambda v, m: _clip_once([f32(v)], m)
    outs, norm = run(np.full(1000, 1e25), 1.0)       # squares beyond fp32's range
    assert abs(norm / (1e25 * np.sqrt(1000)) - 1) < 1e-6 and abs(float(outs[0][0]) * np.sqrt(1000) - 1) < 1e-6
    outs, norm = run(np.full(1000, 1e-30), 1.0)      # squares below it
    assert abs(norm / (1e-30 * np.sqrt(1000)) - 1) < 1e-6
    for bad in (np.inf, np.nan):
        v = np.ones(1000, np.float32)
        v[500] = bad
        outs, norm = run(v, 0.1)
        assert not np.isfinite(norm)
        assert torch.equal(outs[0][:500], torch.ones(500, device=DEV))   # nothing is scaled
    outs, norm = run(np.zeros(10), 1.0)
    assert norm == 0.0 and not outs[0].any()


def _clip_once(grads, max_norm):
    outs = [torch.full_like(g, float("nan")) for g in grads]
    lst = L.grad_list(grads, outs)
    ws, norm = ws_of(L.moe_grad_workspace_size(lst)), empty(1)
    L.moe_grad_clip(lst, max_norm, norm, ws, ws.numel())
    return outs, float(norm)


def test_clip_of_a_norm_summed_over_ranks():
    """Two halves of the gradients, as two ranks hold them: each rank's sum of squares, added, scales
    both as one list does."""
    log("clip: two ranks' lists")
    types, vals = clip_data([1000, 50_001, 33, 7], 4)
    grads = [dev_tensor(v, t) for v, t in zip(vals, types)]
    whole, norm = _clip_once(grads, 1.0)
    lists = [L.grad_list([g.clone() for g in grads[:2]]), L.grad_list([g.clone() for g in grads[2:]])]
    sums = []
    for l in lists:
        s, ws = torch.empty(1, dtype=torch.float64, device=DEV), ws_of(L.moe_grad_workspace_size(l))
        L.moe_grad_norm(l, s, None, ws, ws.numel())
        sums.append(s)
    total = sums[0] + sums[1]
    for l in lists:
        L.moe_grad_scale(l, total, 1.0, None)
    got = lists[0].tensors[0] + lists[1].tensors[0]
    for a, b, t in zip(got, whole, types):   # the two sums of squares may differ in their last bits
        assert torch.allclose(a.float(), b.float(), rtol=2 * HALF[t] + 1e-7, atol=0)


# ------------------------------------------------------------------------------------------- guards

class Guarded:
    """Tensors and workspaces with a run of known bytes behind each, which no call may change."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=torch.float32, fill=0):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        raw = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device=DEV)
        t = raw[:n].view(dtype).view(*shape)
        t.fill_(fill)
        self.all.append((raw, n))
        return t

    def copy(self, t):
        g = self(*t.shape, dtype=t.dtype)
        g.copy_(t)
        return g

    def check(self):
        torch.cuda.synchronize()
        for i, (raw, n) in enumerate(self.all):
            assert bool((raw[n:] == 0x5A).all()), f"bytes behind buffer {i} changed"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,V,k,gate_rows", [(1, 8, 1, 1, 1), (65, 264, 333, 3, 7), (300, 1032, 12345, 4, 300),
                                                (1029, 2056, 2047, 2, 100), (4097, 520, 9001, 1, 0)])
def test_nothing_is_written_behind_outputs_and_workspaces(dtype, T, d, V, k, gate_rows):
    log(f"guards {dtype} T={T} d={d} V={V}")
    G, dt, td = Guarded(), DT[dtype], torch.bfloat16 if dtype == "bf16" else torch.float32
    rnd = lambda *s: G.copy(torch.randn(*s, device=DEV).to(td))
    x, y, dout, w, gate = rnd(T, d), rnd(T, d), rnd(T, d), rnd(d), rnd(-(-T // gate_rows), d) if gate_rows else None
    xn, out, dy, dx, yc = (G(T, d, dtype=td) for _ in range(5))
    r1, r2, dw1, dw2 = G(T), G(T), G(d), G(d)
    dgate = G(*gate.shape) if gate_rows else None
    n = L.moe_norm_bwd_workspace_size(T, d)
    ws = G(n, dtype=torch.uint8)
    L.moe_norm_in(x, w, T, d, EPS, dt, xn, r1)
    L.moe_norm_out(y, x, w, gate, gate_rows, 1.0, EPS, T, d, dt, out, r2)
    L.moe_norm_out_bwd(dout, y, w, gate, gate_rows, r2, T, d, dt, dy, dw1, dgate, ws, n)
    L.moe_norm_in_bwd(dout, x, w, r1, dout, 1.0, T, d, dt, dx, dw2, ws, n)
    yp, tg = rnd(T * k, d), G.copy(torch.rand(T, k, device=DEV))
    pos = G.copy(torch.randperm(T * k, device=DEV).to(torch.int32))
    L.moe_combine_norm_out(yp, tg, pos, y, x, w, gate, gate_rows, 1.0, EPS, T, d, k, dt, yc, out, r2)
    words, target = rnd(V, d), G.copy(torch.randint(0, V, (T,), device=DEV).to(torch.int32))
    loss, lse, dl = G(T), G(T), G(T, fill=1.0)
    nf, nb = L.moe_vocab_loss_workspace_size(T, d, V, dt), L.moe_vocab_loss_bwd_workspace_size(T, d, V, dt)
    wf, wb, dh, dw = G(nf, dtype=torch.uint8), G(nb, dtype=torch.uint8), G(T, d, dtype=td), G(V, d, dtype=td)
    L.moe_vocab_loss(x, words, target, T, d, V, dt, loss, lse, wf, nf)
    L.moe_vocab_loss_bwd(x, words, target, lse, dl, T, d, V, dt, dh, dw, wb, nb)
    grads = [dh, dw, dw1, dw2, G(1, dtype=td, fill=3.0)]
    lst = L.grad_list(grads, [G(*g.shape, dtype=g.dtype) for g in grads])
    ng, norm, sq = L.moe_grad_workspace_size(lst), G(1), G(1, dtype=torch.float64)
    wg = G(ng, dtype=torch.uint8)
    L.moe_grad_clip(lst, 0.1, norm, wg, ng)
    L.moe_grad_norm(lst, sq, norm, wg, ng)
    L.moe_grad_scale(lst, sq, 0.1, norm)
    G.check()
    assert all(bool(torch.isfinite(t).all()) for t in (xn, out, dy, dx, dw1, dw2, loss, dh, dw))


# --------------------------------------------------------------------------------- the run of them

def block_case(T=200, d=256, E=8, k=2, f=256, fs=128, dtype="bf16", gate_rows=64, routing="learned", V=777, seed=2):
    cfg = I.CONFIGS["tiny64e_learned_skew"].with_(name="block", T=T, d=d, E=E, k=k, f=f, fs=fs, dtype=dtype,
                                                  routing=routing, bias_std=0.0, seed=seed)
    inp = I.make_inputs(cfg)
    rng = np.random.default_rng(seed + 100)
    v = lambda *s, f=1.0, o=0.0: as_dtype_values(o + f * rng.standard_normal(s), dtype)
    extra = dict(norm_in=v(d, f=0.1, o=1.0), norm_out=v(d, f=0.1, o=1.0))
    if gate_rows:
        extra["norm_gate"] = v(-(-T // gate_rows), d, f=0.3, o=0.5)
    head, target = v(V, d, f=0.05), rng.integers(0, V, T).astype(np.int32)
    target[rng.random(T) < 0.2] = -100
    params = {**LY.upload_inputs(inp, DEV), **{n: dev_tensor(a, dtype) for n, a in extra.items()}}
    return cfg, I.values(inp), extra, params, head, target


class TrainStep:
    """norm -> layer -> combine, norm, gate, residual -> vocabulary loss -> all the way back -> clipping."""

    def __init__(self, cfg, params, head, target, gate_rows, res_scale, max_norm, **kw):
        self.cfg, self.max_norm = cfg, max_norm
        T, d, V = cfg.T, cfg.d, head.shape[0]
        self.lay = LY.MoELayer(cfg, params, block_norm=True, gate_rows=gate_rows or None, res_scale=res_scale, **kw)
        self.w, self.target = dev_tensor(head, cfg.dtype), torch.from_numpy(target).to(DEV)
        ok = (target >= 0) & (target < V)
        self.dloss = f32(ok / max(1, ok.sum()))
        dt = DT[cfg.dtype]
        self.ws = ws_of(L.moe_vocab_loss_workspace_size(T, d, V, dt))
        self.wsb = ws_of(L.moe_vocab_loss_bwd_workspace_size(T, d, V, dt))
        self.loss, self.lse = empty(T), empty(T)
        self.dh, self.dw = empty(T, d, dtype=cfg.dtype), empty(V, d, dtype=cfg.dtype)
        lay = self.lay
        self.list = L.grad_list(lay.gradients() + [self.dw])
        self.wsg, self.norm = ws_of(L.moe_grad_workspace_size(self.list)), empty(1)

    def run(self):
        c, V, dt = self.cfg, self.w.shape[0], DT[self.cfg.dtype]
        out = self.lay.forward()
        L.moe_vocab_loss(out, self.w, self.target, c.T, c.d, V, dt, self.loss, self.lse, self.ws, self.ws.numel())
        L.moe_vocab_loss_bwd(out, self.w, self.target, self.lse, self.dloss, c.T, c.d, V, dt, self.dh, self.dw, self.wsb,
                             self.wsb.numel())
        self.lay.backward(self.dh)
        if self.max_norm:
            L.moe_grad_clip(self.list, self.max_norm, self.norm, self.wsg, self.wsg.numel())

    def outputs(self):
        return [self.lay.bufs["out"], self.loss, self.lse, self.dh, self.lay.bufs["dx"], self.norm] + self.list.tensors[0]


@pytest.mark.parametrize("dtype,gate_rows,fs,routing", [("f32", 64, 128, "learned"), ("bf16", 64, 128, "learned"),
                                                         ("bf16", 0, 0, "random")])
def test_train_step_matches_oracle(dtype, gate_rows, fs, routing):
    """The whole run against the oracle's, with the layer tests' tolerance; the oracle takes the
    device's rounded block input, so routing is decided on the same values."""
    log(f"train step {dtype} gate_rows={gate_rows} fs={fs} {routing}")
    a = 0.8
    cfg, vals, extra, params, head, target = block_case(dtype=dtype, gate_rows=gate_rows, fs=fs, routing=routing)
    s = TrainStep(cfg, params, head, target, gate_rows, a, max_norm=None)
    s.run()
    torch.cuda.synchronize()
    b = s.lay.bufs
    tol = {"f32": 2e-5, "bf16": 2e-2}[dtype]
    xn, r_in = S.norm_in(vals["x"], extra["norm_in"], EPS)
    assert_close("xn", tnp(b["xn"]), xn, tol)
    sub = dict(vals, x=tnp(b["xn"]))
    fwd = O.run_layer(cfg.with_(backward=False), sub)[0]
    gate = extra.get("norm_gate")
    out, r_out = S.norm_out(fwd["out"], vals["x"], extra["norm_out"], gate, gate_rows, a, EPS)
    assert_close("out", tnp(b["out"]), out, tol)
    loss, lse = S.vocab_loss(tnp(b["out"]), head, target)
    assert_close("loss", tnp(s.loss), loss, 1e-5)
    dl = tnp(s.dloss)
    dh, dw = S.vocab_loss_bwd(tnp(b["out"]), head, target, dl)
    assert_close("dh", tnp(s.dh), dh, tol)
    assert_close("dw", tnp(s.dw), dw, tol)
    dy, dwo, dg = S.norm_out_bwd(tnp(s.dh), fwd["out"], extra["norm_out"], gate, gate_rows, r_out)
    assert_close("dblock", tnp(b["dblock"]), dy, tol)
    assert_close("dnorm_out", tnp(b["dnorm_out"]), dwo, tol)
    if gate is not None:
        assert_close("dnorm_gate", tnp(b["dnorm_gate"]), dg, tol)
    bwd = O.run_layer(cfg, dict(sub, dout=tnp(b["dblock"])))[1]
    assert_close("dw1", tnp(b["dw1"]), bwd["dW1"], tol)
    assert_close("dw2", tnp(b["dw2"]), bwd["dW2"], tol)
    assert_close("dxn", tnp(b["dxn"]), bwd["dx"], tol)
    dx, dwi = S.norm_in_bwd(tnp(b["dxn"]), vals["x"], extra["norm_in"], r_in, tnp(s.dh), a)
    assert_close("dx", tnp(b["dx"]), dx, tol)
    assert_close("dnorm_in", tnp(b["dnorm_in"]), dwi, tol)
    # clipping the layer's own gradients in place
    before = [g.clone() for g in s.lay.gradients()]
    norm = S.grad_norm([tnp(g) for g in before])
    got = s.lay.clip_gradients(norm / 3)
    assert abs(float(got) / norm - 1) < 1e-6
    for g, o in zip(s.lay.gradients(), before):
        ref = tnp(o).astype(np.float64) / 3
        half = HALF["bf16" if g.dtype == torch.bfloat16 else "f32"]
        # c = max_norm / (norm + 1e-6): the 1e-6 and the rounding of max_norm to fp32
        within("clipped", tnp(g), ref, (half + 4 * U + 1e-6 / norm) * np.abs(ref) + 2.0 ** -133)


def test_layer_without_block_norm_is_unchanged_by_it():
    """The block with the norms on, fed its own normalised input, computes what the plain layer does."""
    log("layer with and without norms")
    cfg, vals, extra, params, head, target = block_case(gate_rows=0)
    normed = LY.MoELayer(cfg, params, block_norm=True)
    normed.forward()
    plain = LY.MoELayer(cfg, dict(params, x=normed.bufs["xn"].clone()))
    plain.forward()
    assert torch.equal(normed.bufs["y"], plain.bufs["y"]) and torch.equal(normed.bufs["y_block"], plain.bufs["out"])
    dout = torch.randn(cfg.T, cfg.d, device=DEV).to(torch.bfloat16)
    normed.backward(dout)
    plain.backward(normed.bufs["dblock"])
    assert torch.equal(normed.bufs["dxn"], plain.bufs["dx"])
    assert all(torch.equal(normed.bufs[n], plain.bufs[n]) for n in ("dw1", "dw3", "dw2", "dws1", "dwr"))


def test_mxfp8_block_runs_and_clips():
    log("mxfp8 block")
    cfg, vals, extra, params, head, target = block_case(gate_rows=64)
    s = TrainStep(cfg, params, head, target, 64, 1.0, 0.01, precision="mxfp8")
    s.run()
    assert float(s.norm) > 0.01 and all(torch.isfinite(t).all() for t in s.outputs())


def test_train_step_in_a_graph_and_on_another_stream():
    """The run captured once and replayed, with eager runs between the replays, and an eager run on a
    side stream: every output bit-equal each time."""
    log("train step: graph, stream")
    cfg, vals, extra, params, head, target = block_case()
    s = TrainStep(cfg, params, head, target, 64, 0.8, 0.01)
    s.run()
    torch.cuda.synchronize()
    ref = [t.clone() for t in s.outputs()]
    same = lambda: all(torch.equal(a, b) for a, b in zip(ref, s.outputs()))

    def spoil():
        for t in s.outputs():
            t.fill_(float("nan"))
        for t in (s.ws, s.wsb, s.wsg, s.lay.bufs["ws_norm"]):
            t.fill_(0xFF)
        torch.cuda.synchronize()

    side = torch.cuda.Stream()
    spoil()
    with torch.cuda.stream(side):
        s.run()
    side.synchronize()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    for i in range(4):
        spoil()
        graph.replay()
        torch.cuda.synchronize()
        assert same(), f"replay {i}"
        spoil()
        s.run()
        torch.cuda.synchronize()
        assert same(), f"eager run {i}"


def test_layers_that_share_buffers():
    """Blocks run one after the other over the same buffers, their gates of different shapes, give the
    gradients that each gives over buffers of its own."""
    log("layers over shared buffers")
    cfg, vals, extra, params, head, target = block_case(gate_rows=1)
    rows = [1, 64, cfg.T, 0]   # the fewest gate rows, and none, after the most
    cases = []
    for r in rows:
        p = dict(params)
        gate = p.pop("norm_gate")
        if r:
            p["norm_gate"] = gate[:-(-cfg.T // r)].contiguous()
        cases.append((p, r or None))
    dout = torch.randn(cfg.T, cfg.d, device=DEV).to(torch.bfloat16)
    own = [LY.MoELayer(cfg, p, block_norm=True, gate_rows=r) for p, r in cases]
    bufs = LY.Buffers.allocate(cfg, params["x"].device)
    shared = [LY.MoELayer(cfg, p, bufs=bufs, block_norm=True, gate_rows=r) for p, r in cases]
    for a, b in zip(own, shared):
        for lay in (a, b):
            lay.forward()
            lay.backward(dout)
            lay.clip_gradients(0.01)
        torch.cuda.synchronize()
        assert torch.equal(a.bufs["dx"], b.bufs["dx"]) and torch.equal(a.grad_norm, b.grad_norm)
        assert all(torch.equal(g, h) for g, h in zip(a.gradients(), b.gradients()))
        gate = b.bufs["dnorm_gate"]
        assert gate is None if "norm_gate" not in b.p else torch.equal(gate, a.bufs["dnorm_gate"])


@pytest.mark.parametrize("dtype,T,d,V", [("bf16", 1990, 1000, 3990), ("f32", 1990, 512, 3990), ("bf16", 190, 2000, 20000),
                                         ("bf16", 16400, 136, 4500), ("f32", 16400, 136, 4500)])
def test_vocab_loss_in_larger_tiles(dtype, T, d, V):
    """Products of some hundred tiles of 128x128, whose last rows and columns are ragged; the last two
    go through two pieces of the vocabulary."""
    log(f"vocab loss {dtype} larger tiles T={T} d={d} V={V}")
    data = loss_data(T, d, V, dtype, 0.1, 9)
    check_loss(*data, dtype, run_loss(*data, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("T,d,gate_rows", [(300, 200, 300), (1000, 1000, 0), (65, 72, 33), (5, 8, 0), (300, 5000, 299),
                                           (1024, 2048, 128), (77, 24, 11), (70, 3000, 8), (1023, 104, 1), (33, 16384, 20)])
def test_norms_of_few_rows(dtype, T, d, gate_rows):
    """Where the column sums are formed beside the rows, and (4 gate rows are the most) where not."""
    test_norms_match_oracle(dtype, T, d, gate_rows)
