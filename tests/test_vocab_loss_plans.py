"""How the vocabulary loss cuts its products, asked on the host (CPU): the sizes that the GPU tests run
reach every kernel."""
import pytest

from mixture_experts_layer_20_amd import libmoe as L
from tests.vocab_loss_sizes import FORWARD, PLANS

DT = {"f32": L.MOE_F32, "bf16": L.MOE_BF16}


@pytest.mark.parametrize("T,d,V,dtype,logits,dh,dw,pieces,dh_split,dw_split", PLANS)
def test_size_is_cut_as_the_gpu_test_needs_it(T, d, V, dtype, logits, dh, dw, pieces, dh_split, dw_split):
    p = L.moe_vocab_loss_plan(T, d, V, DT[dtype])
    assert (p.logits_tile, p.dh_tile, p.dw_tile) == (logits, dh, dw)
    assert (p.pieces > 1, p.dh_splits > 1, p.dw_splits > 1) == (pieces, dh_split, dw_split)


@pytest.mark.parametrize("T,d,V,dtype,tile", FORWARD)
def test_forward_takes_the_tiles_that_the_gpu_test_needs(T, d, V, dtype, tile):
    assert L.moe_vocab_loss_plan(T, d, V, DT[dtype]).fwd_tile == tile


def test_sizes_cover_the_kernels():
    cut = [c[3:] for c in PLANS]
    large = [c for c in PLANS if c[5] == c[6] == 256]
    assert {(c[2], c[3]) for c in cut if c[0] == "bf16"} >= {(64, 64), (64, 256), (128, 128), (128, 256), (256, 64), (256, 128),
                                                             (256, 256)}
    assert {(c[2], c[3]) for c in cut if c[0] == "f32"} == {(64, 64), (128, 128)}
    assert {(c[7], c[8], c[9]) for c in large} >= {(False, True, True), (True, True, True), (True, True, False),
                                                   (True, False, False)}
    whole = [c for c in large if c[0] % 256 == c[1] % 256 == c[2] % 256 == 0]
    assert {c[9] for c in whole if c[7]} == {False, True} and {c[8] for c in whole if c[7]} == {False, True}


def test_plan_of_the_pieces():
    p = L.moe_vocab_loss_plan(8192, 4096, 65536, L.MOE_BF16)
    assert (p.piece_words, p.pieces, p.fwd_tile, p.dh_tile, p.dw_tile) == (8192, 8, 256, 256, 256)
    p = L.moe_vocab_loss_plan(0, 64, 100, L.MOE_F32)
    assert not any(getattr(p, n) for n, _ in p._fields_)
    for args, status in (((4, 60, 100, L.MOE_BF16), L.MOE_ERR_UNSUPPORTED), ((4, 64, 0, L.MOE_BF16), L.MOE_ERR_INVALID_VALUE),
                         ((4, 64, 100, 5), L.MOE_ERR_INVALID_VALUE)):
        with pytest.raises(L.MoEError) as e:
            L.moe_vocab_loss_plan(*args)
        assert e.value.status == status
    assert L.lib().moe_vocab_loss_plan(4, 64, 100, L.MOE_F32, None) == L.MOE_ERR_INVALID_VALUE
