"""Values and sizes at which routing by scores, the block-scaled 8-bit products and AdamW could go wrong, on the
GPU against the float64 oracle."""
import pytest
import torch

from mixture_experts_layer_20_amd import libmoe as L
from tests.test_gpu_train_step import DEV, HYPER, Case

pytestmark = pytest.mark.gpu


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
