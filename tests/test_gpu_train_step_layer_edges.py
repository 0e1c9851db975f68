"""The MoE layer's steps of training where something is out of the ordinary (GPU)."""
import pytest
import torch

from mixture_experts_layer_20_amd import inputs as I
from mixture_experts_layer_20_amd import layer as LY
from oracle import train_step as S
from tests.gpu_helpers import DEV
from tests.test_gpu_train_step import check_adamw, np64
from tests.test_gpu_train_step_layer import CASES

pytestmark = pytest.mark.gpu


class Before:
    """What check_adamw reads: a layer's parameters, gradients and states before a step, and its own after it."""

    def __init__(self, lay, bits):
        rows = lay._adamw.tensors
        flat = lambda ts: [None if t is None else t.clone().flatten() for t in ts]
        self.bits = bits
        self.p, self.g, self.m, self.v, self.sc, self.w = (flat(r) for r in rows[:6])
        self.results = lambda i: [None if r[i] is None else r[i].flatten() for r in rows[6:]]


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_without_a_norm_does_not_count(bits):
    """The step after one whose norm is NaN or infinite is the one that the formulas number so: the first, the second."""
    lay = LY.MoELayer(CASES["ragged"], LY.upload_inputs(I.make_inputs(CASES["ragged"]), DEV))
    lay.make_adamw(bits)
    hyper = dict(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8)
    made = 0
    for bad in (float("nan"), None, float("inf"), None, None):
        lay.step()
        if bad is not None:
            lay.gradients()[-1].view(-1)[5] = bad
        c = Before(lay, bits)
        lay.adamw_step(**hyper, max_norm=1e9, seed=made)
        if bad is None:
            made += 1
            torch.cuda.synchronize()
            for i in range(len(c.p)):
                check_adamw(c, i, 0.0, S.clip(np64(lay.grad_norm)[0] ** 2, 1e9), dict(**hyper, step=made))
        else:
            assert all(torch.equal(a, b) for i in range(len(c.p)) for a, b in zip((c.p[i], c.m[i], c.v[i]), c.results(i)))
        if made != 2:   # read now and then: a step finds out by itself
            assert lay.steps == made
    assert lay.steps == made == 3
    lay.steps = 10                      # as after a restart
    lay.step()
    c = Before(lay, bits)
    lay.adamw_step(**hyper)             # without a norm: every call is a step
    for i in range(len(c.p)):
        check_adamw(c, i, 0.0, 1.0, dict(**hyper, step=11))
    assert lay.steps == 11


def test_captured_steps_repeat_their_number():
    """A graph of a clipped step: each replay is the step of the number that it was captured with."""
    cfg = CASES["no_shared"]
    one, other = (LY.MoELayer(cfg, LY.upload_inputs(I.make_inputs(cfg), DEV)) for _ in range(2))
    hyper = dict(lr=0.01, beta1=0.9, beta2=0.95, eps=1e-8, max_norm=0.5, seed=3)
    for lay in (one, other):
        lay.make_adamw(8)
        lay.step()
        lay.adamw_step(**hyper)
        assert lay.steps == 1
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        other.step()
        other.adamw_step(**hyper)
    for _ in range(3):
        one.steps = 1
        one.step()
        one.adamw_step(**hyper)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(one._adamw.tensors, other._adamw.tensors):
            assert all(x is None or torch.equal(x, y) for x, y in zip(a, b))
        assert torch.equal(one.grad_norm, other.grad_norm)
