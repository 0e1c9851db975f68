"""Values and sizes at which routing by scores, the block-scaled 8-bit products and AdamW could go wrong, on the
GPU against the float64 oracle."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_20_amd import libmoe as L
from oracle import train_step as S
from tests.test_gpu_train_step import BF, DEV, F, HYPER, SIG, SOFT, Case, check_route, np64, put, route_bwd, sums_bound

pytestmark = pytest.mark.gpu
VALUES = torch.from_numpy(S.E4M3)


# ---- AdamW --------------------------------------------------------------------------------------------


@pytest.mark.parametrize("what", ["code", "scale", "infinite scale"])
def test_adamw_keeps_a_lost_first_moment(what):
    """A NaN that m alone holds is m's block's: it gets a scale of NaN, v's does not, and nothing else is lost."""
    n = 2048 + 300
    c = Case([n], [torch.float32], [torch.float32], 8, False, seed=10)
    blocks = -(-n // 128)
    for at in (200, n - 5):   # a block of wide accesses, one of the tail
        if what == "code":
            c.m[0][at] = 0x7F
        else:
            c.sc[0][at // 128] = float("nan") if what == "scale" else float("inf")
            c.m[0][at // 128 * 128:][:128].clamp_(min=1)   # codes above zero, or all of them: 0 times infinity is NaN too
    L.moe_adamw(c.list(0.0), seed=3, **HYPER)
    c.check_guards()
    p, m, v, sc, _ = c.results(0)
    bad = torch.isnan(sc).view(2, blocks)
    lost = torch.zeros(blocks, dtype=torch.bool, device=DEV)
    lost[[200 // 128, (n - 5) // 128]] = True
    assert torch.equal(bad[0], lost) and not bad[1].any()
    ends = ~torch.isfinite(p)
    where = torch.zeros(n, dtype=torch.bool, device=DEV)
    if what == "code":
        where[[200, n - 5]] = True
    else:
        where = lost.repeat_interleave(128)[:n]
    assert torch.equal(ends, where)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("nan", [0x7FFFFFFF, 0xFFFFFFFF, 0x7FC00000, 0x7FC0FFFF])
def test_adamw_keeps_nan_in_random_rounding(nan, bits):
    """A NaN gradient makes its bf16 parameter, which has no master copy, a NaN: whatever the NaN's payload and
    the random bits that are added to it."""
    n = 2048 + 77   # wide accesses and a tail
    c = Case([n], [torch.bfloat16], [torch.float32], bits, False, seed=9)
    at = torch.arange(0, n, 3, device=DEV)
    c.g[0].view(torch.int32)[at] = nan - (1 << 32) if nan >= 1 << 31 else nan
    L.moe_adamw(c.list(0.0), seed=3, **HYPER)
    c.check_guards()
    bad = torch.isnan(c.results(0)[0])
    assert bad[at].all() and bad.sum() == len(at)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("nan", [0x7FFFFFFF, 0xFFFFFFFF])
def test_adamw_keeps_nan_of_a_state_in_random_rounding(nan, bits):
    """As before, with the NaN in m, or in the scale of one of its blocks."""
    n = 2048 + 77
    c = Case([n], [torch.bfloat16], [torch.float32], bits, False, seed=11)
    state, at = (c.m[0], torch.arange(0, n, 3, device=DEV)) if bits == 32 else (c.sc[0], torch.arange(0, 17, 2, device=DEV))
    state.view(torch.int32)[at] = nan - (1 << 32) if nan >= 1 << 31 else nan
    L.moe_adamw(c.list(0.0), seed=3, **HYPER)
    where = torch.zeros(n if bits == 32 else 17, dtype=torch.bool, device=DEV)
    where[at] = True
    assert torch.equal(torch.isnan(c.results(0)[0]), where if bits == 32 else where.repeat_interleave(128)[:n])


def quantized_at_random(y, gen):
    """E4M3 values around y in [0, 448], up with the probability of the rest; a positive one not to zero."""
    step = torch.exp2(torch.floor(torch.log2(y.clamp(min=2.0 ** -6))) - 3)
    q = torch.floor(y / step + torch.rand(y.shape, dtype=y.dtype, device=DEV, generator=gen)) * step
    return torch.where(y > 0, q.clamp(min=2.0 ** -9), q).clamp(max=448.0)


@pytest.mark.parametrize("beta2,steps", [(0.95, 200), (0.999, 2000)])
def test_adamw_long_runs_of_8_bit_states(beta2, steps):
    """What accumulates in v over many steps: the mean of the root is kept in each rounding, so v's own comes out a few
    per cent high, as it does for the rule in float64 with other random bits.  Blocks of 128 are independent: the mean
    over n / 128 of them is within six of its standard deviations, of either side."""
    n = 1 << 17
    gen = torch.Generator(device=DEV).manual_seed(13)
    p, g = torch.zeros(n, device=DEV), torch.zeros(n, device=DEV)
    m, v, sc, _ = L.adamw_states([p], 8)
    t = L.adamw_list([p], [g], m, v, sc)
    rule, exact, first = (torch.zeros(n, dtype=torch.float64, device=DEV) for _ in range(3))
    for step in range(1, steps + 1):
        g.normal_(0.0, 1e-3, generator=gen)
        L.moe_adamw(t, 1e-3, 0.9, beta2, 1e-8, step, seed=step)
        sq = g.double().square()
        exact = beta2 * exact + (1 - beta2) * sq
        first = 0.9 * first + 0.1 * g.double()
        root = (beta2 * rule + (1 - beta2) * sq).sqrt().view(-1, 128)
        scale = root.amax(1, keepdim=True) / 448
        rule = (quantized_at_random(root / scale, gen) * scale).view(-1).square()
    s = sc[0].double().view(2, -1).repeat_interleave(128, 1)
    values = VALUES.to(DEV)
    got, moment = (values[v[0].long()] * s[1]).square(), values[m[0].long()] * s[0]
    per = lambda x: (x / exact).view(-1, 128).mean(1)
    a, b = per(got), per(rule)
    off = 6 * (a.var() / a.numel() + b.var() / b.numel()).sqrt()
    assert (a.mean() - b.mean()).abs() <= off, (a.mean().item(), b.mean().item(), off.item())
    assert 1.0 <= b.mean() <= 1.1
    d = ((moment - first) / exact.sqrt()).view(-1, 128).mean(1)   # m's own roundings have the right mean
    assert d.mean().abs() <= 6 * (d.var() / d.numel()).sqrt()


@pytest.mark.parametrize("bits", [32, 8])
def test_adamw_of_more_than_2_32_elements(bits):
    """Chunks of two steps and offsets beyond 32 bits: contents that repeat give results that repeat."""
    P, n = 1 << 20, (1 << 32) + (3 << 20) + 2 * 2048 + 77
    c = Case([P], [torch.float32], [torch.float32], bits, False, seed=14)

    def repeated(t, period, size):
        out = torch.empty(size, dtype=t.dtype, device=DEV)
        whole = size // period * period
        out[:whole].view(-1, period).copy_(t[:period])
        out[whole:].copy_(t[:size - whole])
        return out

    def repeats(t, want, equal):
        whole = t.numel() // want.numel() * want.numel()
        for part in t[:whole].view(-1, want.numel()).split(512):
            assert equal(part, want)
        return equal(t[whole:], want[:t.numel() - whole])

    blocks, whole = -(-n // 128), P // 128
    p, g = repeated(c.p[0], P, n), repeated(c.g[0], P, n)
    m, v = repeated(c.m[0], P, n), repeated(c.v[0], P, n)
    sc = None
    if bits == 8:
        sc = torch.empty(2, blocks, device=DEV)
        for row in range(2):
            sc[row] = repeated(c.sc[0].view(2, -1)[row], whole, blocks)
        sc = sc.view(-1)
    big = L.adamw_list([p], [g], [m], [v], [sc])
    L.moe_adamw(c.list(0.0), seed=3, **HYPER)
    L.moe_adamw(big, seed=3, **HYPER)
    same = lambda a, b: torch.equal(a, b.expand_as(a))
    want = c.results(0)
    assert repeats(p, want[0], same)
    if bits == 32:
        assert repeats(m, want[1], same) and repeats(v, want[2], same)
        return
    # codes of the same values with other random bits: the one below or the one above
    near = lambda a, b: ((a & 0x7F).to(torch.int8) - (b & 0x7F).to(torch.int8)).abs().amax() <= 1
    last = blocks - 1   # the last block is part of one: its scale is its own
    for row in range(2):
        assert repeats(sc.view(2, -1)[row][:last], want[3].view(2, -1)[row], same)
    cut = last * 128
    assert repeats(m[:cut], want[1], near) and repeats(v[:cut], want[2], near)


def test_adamw_of_32_bit_states_rounds_to_nearest():
    """From a parameter of zero, a step is -(lr / bc1) m / (sqrt(v) / sqrt(bc2) + eps) of the new m and v, each operation
    rounded once.  (numpy's roots of doubles, rounded to float, are roots rounded to nearest; torch's of floats on the CPU
    need not be.  The sum with eps is formed in double and rounded twice, which differs once in 2^29.)"""
    n = 20000
    c = Case([n], [torch.float32], [torch.float32], 32, False, seed=15)
    c.p[0].zero_()
    L.moe_adamw(c.list(0.0), seed=3, **HYPER)
    p, m, v = (t.cpu().numpy() for t in c.results(0)[:3])
    f32 = np.float32
    root, factor = np.sqrt(v.astype(np.float64)).astype(f32), f32((1.0 - HYPER["beta2"] ** HYPER["step"]) ** -0.5)
    den = (root.astype(np.float64) * np.float64(factor) + np.float64(f32(HYPER["eps"]))).astype(f32)
    np.testing.assert_array_equal(p, -f32(HYPER["lr"] / (1.0 - HYPER["beta1"] ** HYPER["step"])) * (m / den))


# ---- routing by scores --------------------------------------------------------------------------------

@pytest.mark.parametrize("score", [SIG, SOFT])
@pytest.mark.parametrize("E,groups,topk_groups", [(32, 4, 2), (96, 8, 3), (256, 8, 4), (48, 6, 3), (255, 15, 4)])
@pytest.mark.parametrize("size", [8.0, 4096.0, 2.0 ** 20])
def test_route_groups_of_opposite_biases(E, groups, topk_groups, score, size):
    """A group's two largest scores that cancel: their sum is small, what fp32 loses of each of them is not."""
    r = np.random.default_rng(int(size) + E)
    T, k = 1024, 2
    l = r.standard_normal((T, E)).astype(np.float32)
    b = np.full((groups, E // groups), -4 * size, np.float32)
    b[:, 0], b[:, 1] = size, -size
    b = np.take_along_axis(b, np.argsort(r.random(b.shape), axis=1), axis=1)
    check_route(l, b.reshape(-1), k, groups, topk_groups, score, 1, 1.0)


@pytest.mark.parametrize("score,renorm", [(SIG, 1), (SIG, 0), (SOFT, 1), (SOFT, 0)])
def test_route_backward_of_an_expert_named_twice(score, renorm):
    """A choice that a caller made: each of a token's places has its own gate and gradient, also where two name one
    expert."""
    r = np.random.default_rng(21)
    T, d, E, k, scale = 70, 64, 12, 4, 1.5
    logits, idx = put(r.standard_normal((T, E)) * 2), put(r.integers(0, E, (T, k)), torch.int32)
    idx[:, 2] = idx[:, 0]
    x, w, dgate = put(r.standard_normal((T, d))), put(r.standard_normal((E, d)) * 0.3), put(r.standard_normal((T, k)))
    dw, dx = route_bwd(dgate, logits, idx, x, w, score, renorm, scale)
    l, dg, i = np64(logits), np64(dgate), idx.cpu().numpy().astype(np.int64)
    dl, g = S.gates_bwd(dg, l, i, score == SIG, renorm, scale), S.gates(l, i, score == SIG, renorm, 1.0)
    # terms of a logit's gradient, and their roundings: the gates' own, k differences and products
    size = np.zeros_like(dl)
    if score == SOFT and not renorm:
        size += scale * S.scores(l, False) * (g * np.abs(dg)).sum(1, keepdims=True)
    inner = np.abs(dg) + ((g * np.abs(dg)).sum(1, keepdims=True) if renorm else 0.0)
    np.add.at(size, (np.arange(T)[:, None], i), scale * g * inner)
    e_dl = (12 * np.abs(l).max() + 100) * F * size
    x64, w64 = np64(x), np64(w)
    # each place is a term of its own in the sums: their magnitudes, not those of what is left of two
    tol_dw = e_dl.T @ np.abs(x64) + (T + 8) * F * (size.T @ np.abs(x64))
    tol_dx = e_dl @ np.abs(w64) + (E + 8) * F * (size @ np.abs(w64))
    assert np.all(np.abs(np64(dw) - dl.T @ x64) <= tol_dw * 1.01 + 1e-30)
    assert np.all(np.abs(np64(dx) - dl @ w64) <= tol_dx * 1.01 + 1e-30)


# ---- products -------------------------------------------------------------------------------------------

def rows_of(codes, scales):
    return VALUES.to(DEV)[codes.long()] * scales.double().t().repeat_interleave(128, 1)


def weights_of(codes, scales):
    return VALUES.to(DEV)[codes.long()] * scales.double().repeat_interleave(128, 1).repeat_interleave(128, 2)


def grouped_product(a, b, offsets):
    """S.grouped_product on the device: the product, the sum of magnitudes, the sum of each eight's largest."""
    M, N = a.shape[0], b.shape[1]
    out, size, tops = (torch.full((M, N), float("nan"), dtype=torch.float64, device=DEV) for _ in range(3))
    top = lambda t: t.abs().view(*t.shape[:-1], -1, 8).amax(-1)
    for g, (r0, r1) in enumerate(zip(offsets, offsets[1:])):
        if r1 > r0:
            out[r0:r1] = a[r0:r1] @ b[g].t()
            size[r0:r1] = a[r0:r1].abs() @ b[g].abs().t()
            tops[r0:r1] = top(a[r0:r1]) @ top(b[g]).t()
    return out, size, tops


def cut(sizes, first, behind):
    """Offsets of groups of these sizes, with rows before and behind them that belong to none."""
    offsets = [first]
    for n in sizes:
        offsets.append(offsets[-1] + n)
    return offsets[-1] + behind, offsets


# Row tiles of 256 whose last ones fill 1 to 4 quarters in turn, groups of one tile and of several, empty ones.
RAGGED = [300, 70, 0, 513, 190, 250, 1, 400, 129, 256, 0, 60, 700, 64, 65, 333, 512, 128, 449, 5, 210, 600, 90, 385]
TILED = [(*cut(RAGGED, 3, 7), 8192, 128), (*cut(RAGGED, 0, 0), 8192, 384), (*cut([2000, 1900, 30, 2100], 0, 1), 8192, 256)]


def row_tiles(offsets):
    return sum(-(-(b - a) // 256) for a, b in zip(offsets, offsets[1:]))


def operands(M, G, N, K, seed, sources=1, scale=1.0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    codes = lambda *s: torch.randint(0, 256, s, device=DEV, generator=gen, dtype=torch.int32).to(torch.uint8)
    keep = lambda c: torch.where((c & 0x7F) == 0x7F, c - 1, c)   # no NaN
    factor = lambda *s: scale * torch.exp(0.5 * torch.randn(*s, device=DEV, generator=gen))
    t = [keep(codes(M, K)), factor(K // 128, M)]
    for _ in range(sources):
        t += [keep(codes(G, N, K)), factor(G, N // 128, K // 128)]
    return t


def outputs(M, N, count=1):
    return [torch.full((M + 1, N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(count)]


def within(got, want, e, M):
    """got against want, whose rows of no group are NaN, with an error of e before the one rounding to bf16."""
    inside = ~torch.isnan(want[:, 0])
    assert (got[:M][~inside] == 7.0).all() and (got[M] == 7.0).all()
    err = (got[:M].double() - want).abs()[inside]
    tol = (e * (1 + BF) + BF * want.abs())[inside] + 1e-30
    assert (err <= tol).all(), (err / tol).max().item()


def several_tiles(offsets, columns):
    """Whether every workgroup of the persistent product, one for each CU, gets two tiles at least."""
    assert row_tiles(offsets) * columns >= 2 * torch.cuda.get_device_properties(0).multi_processor_count + 8


@pytest.mark.parametrize("M,offsets,N,K", TILED)
def test_product_of_many_tiles(M, offsets, N, K):
    several_tiles(offsets, N // 256)
    G = len(offsets) - 1
    t, off = operands(M, G, N, K, M + K), put(np.array(offsets), torch.int32)
    out, = outputs(M, N)
    L.moe_fp8_gemm_rows(*t, None, None, 0, off, G, M, N, K, L.MOE_MX_EPI_STORE, out, None, None, None, None, None, 0)
    want, size, tops = grouped_product(rows_of(*t[:2]), weights_of(*t[2:]), offsets)
    within(out, want, sums_bound(size, tops, K), M)


@pytest.mark.parametrize("M,offsets,N,K", TILED)
def test_product_of_many_tiles_and_two_sources(M, offsets, N, K):
    several_tiles(offsets, N // 256)
    G, kb = len(offsets) - 1, K // 128
    for K2 in (128, 256):
        Ks = K + K2
        t, off = operands(M, G, N, Ks, M + Ks), put(np.array(offsets), torch.int32)
        one, two = outputs(M, N, 2)
        part = lambda v, lo, hi: v[:, :, lo:hi].clone(memory_format=torch.contiguous_format)
        tail = (off, G, M, N, Ks, L.MOE_MX_EPI_STORE)
        L.moe_fp8_gemm_rows(*t[:2], part(t[2], 0, K), part(t[3], 0, kb), part(t[2], K, Ks), part(t[3], kb, Ks // 128), K, *tail,
                            two, None, None, None, None, None, 0)
        want, size, tops = grouped_product(rows_of(*t[:2]), weights_of(*t[2:]), offsets)
        within(two, want, sums_bound(size, tops, Ks), M)
        L.moe_fp8_gemm_rows(*t, None, None, 0, *tail, one, None, None, None, None, None, 0)
        assert torch.equal(one, two)


@pytest.mark.parametrize("M,offsets,N,K", TILED)
def test_product_of_many_tiles_swiglu(M, offsets, N, K):
    several_tiles(offsets, N // 128)
    G = len(offsets) - 1
    # E4M3's codes have a root mean square of 90: gates of a few units
    t, off = operands(M, G, N, K, M + K + 1, 2, K ** -0.25 / 90.0), put(np.array(offsets), torch.int32)
    o = outputs(M, N, 3)
    L.moe_fp8_gemm_rows(*t, 0, off, G, M, N, K, L.MOE_MX_EPI_SWIGLU, *o, None, None, None, 0)
    A = rows_of(*t[:2])
    (ga, size_a, top_a), (up, size_u, top_u) = (grouped_product(A, weights_of(*w), offsets) for w in (t[2:4], t[4:]))
    ea, eu = sums_bound(size_a, top_a, K), sums_bound(size_u, top_u, K)
    act = ga / (1.0 + torch.exp(-ga))
    h = act * up
    # silu's slope is below 1.1; an exponential of an argument rounded |a| half steps, a reciprocal, two products
    eh = 1.1 * ea * (up.abs() + eu) + act.abs() * eu + (8 * ga.abs() + 24) * F * h.abs()
    for got, want, e in zip(o, (ga, up, h), (ea, eu, eh)):
        within(got, want, e, M)


@pytest.mark.parametrize("M,offsets,N,K", TILED)
def test_product_of_many_tiles_swiglu_backward(M, offsets, N, K):
    several_tiles(offsets, N // 256)
    G = len(offsets) - 1
    t, off = operands(M, G, N, K, M + K + 2, 1, K ** -0.25 / 90.0), put(np.array(offsets), torch.int32)
    gen = torch.Generator(device=DEV).manual_seed(M)
    ga, up = ((2 * torch.randn(M, N, device=DEV, generator=gen)).to(torch.bfloat16) for _ in range(2))
    out, = outputs(M, 2 * N)
    L.moe_fp8_gemm_rows(*t, None, None, 0, off, G, M, N, K, L.MOE_MX_EPI_SWIGLU_BWD, out, None, None, ga, up, None, 0)
    dh, size, tops = grouped_product(rows_of(*t[:2]), weights_of(*t[2:]), offsets)
    e, A, U = sums_bound(size, tops, K), ga.double(), up.double()
    sg = 1.0 / (1.0 + torch.exp(-A))
    fa, fb = U * sg * (1.0 + A * (1.0 - sg)), A * sg
    # 1 + a (1 - sg) cancels where it is near zero: its terms are counted by themselves
    slack_a = (8 * A.abs() + 24) * F * dh.abs() * U.abs() * sg * (1.0 + A.abs())
    slack_b = (8 * A.abs() + 24) * F * (dh * fb).abs()
    within(out[:, :N], dh * fa, e * fa.abs() + slack_a, M)
    within(out[:, N:], dh * fb, e * fb.abs() + slack_b, M)


FEW = [(1, [0, 1]), (9, [0, 9]), (40, [0, 3, 3, 20, 40])]


@pytest.mark.parametrize("K", [2048, 2944])
@pytest.mark.parametrize("M,offsets", FEW)
def test_product_of_few_rows_and_long_sums(M, offsets, K):
    """A wave's share of K in steps of 4, 2 and 1 blocks; a second source from within a step of 4 on."""
    G, N = len(offsets) - 1, 256
    t, off = operands(M, G, N, K, M + K, 2, K ** -0.25 / 90.0), put(np.array(offsets), torch.int32)
    A = rows_of(*t[:2])
    (ga, size_a, top_a), (up, size_u, top_u) = (grouped_product(A, weights_of(*w), offsets) for w in (t[2:4], t[4:]))
    ea, eu = sums_bound(size_a, top_a, K), sums_bound(size_u, top_u, K)
    one, = outputs(M, N)
    tail = (off, G, M, N, K)
    L.moe_fp8_gemm_rows(*t[:4], None, None, 0, *tail, L.MOE_MX_EPI_STORE, one, None, None, None, None, None, 0)
    within(one, ga, ea, M)
    part = lambda v, lo, hi: v[:, :, lo:hi].clone(memory_format=torch.contiguous_format)
    for kb in (1, 2, 7, K // 128 - 1):
        two, = outputs(M, N)
        L.moe_fp8_gemm_rows(*t[:2], part(t[2], 0, 128 * kb), part(t[3], 0, kb), part(t[2], 128 * kb, K), part(t[3], kb, K // 128),
                            128 * kb, *tail, L.MOE_MX_EPI_STORE, two, None, None, None, None, None, 0)
        assert torch.equal(one, two)
    o = outputs(M, N, 3)
    L.moe_fp8_gemm_rows(*t, 0, *tail, L.MOE_MX_EPI_SWIGLU, *o, None, None, None, 0)
    act = ga / (1.0 + torch.exp(-ga))
    eh = 1.1 * ea * (up.abs() + eu) + act.abs() * eu + (8 * ga.abs() + 24) * F * (act * up).abs()
    for got, want, e in zip(o, (ga, up, act * up), (ea, eu, eh)):
        within(got, want, e, M)


@pytest.mark.parametrize("G", [65, 129, 1024])
@pytest.mark.parametrize("N,per", [(256, 2), (256, 12), (384, 12)])
def test_product_of_many_groups(N, per, G):
    """More groups than a wave has lanes, most of them of few rows, a third of them empty: all three kernels' lists."""
    r, K = np.random.default_rng(G + N), 256
    sizes = (r.poisson(1.5 * per, G) * (r.random(G) < 0.67)).tolist()
    M, offsets = cut(sizes, 5, 9)
    assert (M > 8 * G) == (per == 12)
    t, off = operands(M, G, N, K, G, 2, K ** -0.25 / 90.0), put(np.array(offsets), torch.int32)
    A = rows_of(*t[:2])
    (ga, size_a, top_a), (up, size_u, top_u) = (grouped_product(A, weights_of(*w), offsets) for w in (t[2:4], t[4:]))
    ea, eu = sums_bound(size_a, top_a, K), sums_bound(size_u, top_u, K)
    one, o = outputs(M, N)[0], outputs(M, N, 3)
    L.moe_fp8_gemm_rows(*t[:4], None, None, 0, off, G, M, N, K, L.MOE_MX_EPI_STORE, one, None, None, None, None, None, 0)
    L.moe_fp8_gemm_rows(*t, 0, off, G, M, N, K, L.MOE_MX_EPI_SWIGLU, *o, None, None, None, 0)
    act = ga / (1.0 + torch.exp(-ga))
    eh = 1.1 * ea * (up.abs() + eu) + act.abs() * eu + (8 * ga.abs() + 24) * F * (act * up).abs()
    for got, want, e in zip((one, *o), (ga, ga, up, act * up), (ea, ea, eu, eh)):
        within(got, want, e, M)
