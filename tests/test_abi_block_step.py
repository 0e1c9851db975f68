"""Refusals of the block norms, the vocabulary loss and the gradient calls: every bad argument is
turned away on the host, before anything is enqueued (CPU)."""
import ctypes

import pytest
import torch

from mixture_experts_layer_20_amd import layer as LY
from mixture_experts_layer_20_amd import libmoe as L
from mixture_experts_layer_20_amd.inputs import MoEConfig

FAKE = 1 << 20   # a non-null pointer value; never dereferenced, the checks fail first
BF, F32 = L.MOE_BF16, L.MOE_F32
INVALID, UNSUPPORTED, WORKSPACE = L.MOE_ERR_INVALID_VALUE, L.MOE_ERR_UNSUPPORTED, L.MOE_ERR_WORKSPACE


def expect(status, fn, *args):
    with pytest.raises(L.MoEError) as ei:
        fn(*args)
    assert ei.value.status == status, str(ei.value)
    assert L.last_error() != ""


def test_norm_forward_refusals():
    f = L.moe_norm_in
    expect(INVALID, f, FAKE, FAKE, 4, 16, 1e-6, 7, FAKE, None)
    expect(INVALID, f, FAKE, FAKE, -1, 16, 1e-6, BF, FAKE, None)
    expect(INVALID, f, FAKE, FAKE, 4, 0, 1e-6, BF, FAKE, None)
    expect(UNSUPPORTED, f, FAKE, FAKE, 4, 12, 1e-6, BF, FAKE, None)
    expect(UNSUPPORTED, f, FAKE, FAKE, 4, 16392, 1e-6, BF, FAKE, None)
    expect(UNSUPPORTED, f, FAKE, FAKE, 1 << 31, 16, 1e-6, BF, FAKE, None)
    expect(INVALID, f, FAKE, FAKE, 4, 16, -1e-6, BF, FAKE, None)
    expect(INVALID, f, FAKE, FAKE, 4, 16, float("nan"), BF, FAKE, None)
    expect(INVALID, f, None, FAKE, 4, 16, 1e-6, BF, FAKE, None)
    expect(INVALID, f, FAKE, FAKE + 2, 4, 16, 1e-6, BF, FAKE, None)
    expect(INVALID, f, FAKE, FAKE, 4, 16, 1e-6, BF, FAKE, FAKE + 4)
    f(None, None, 0, 16, 1e-6, BF, None, None)   # no rows: nothing to do
    g = L.moe_norm_out
    expect(INVALID, g, FAKE, FAKE, FAKE, FAKE, 0, 1.0, 1e-6, 4, 16, BF, FAKE, None)      # gate_rows
    expect(INVALID, g, FAKE, None, FAKE, None, 0, 1.0, 1e-6, 4, 16, BF, FAKE, None)
    expect(INVALID, g, FAKE, FAKE, FAKE, FAKE + 8, 4, 1.0, 1e-6, 4, 16, BF, FAKE, None)
    g(None, None, None, None, 0, 1.0, 1e-6, 0, 16, F32, None, None)
    c = L.moe_combine_norm_out
    args = lambda k=2, pos=FAKE, y=None, T=4: (FAKE, FAKE, pos, None, FAKE, FAKE, None, 1, 1.0, 1e-6, T, 16, k, BF, y,
                                               FAKE, None)
    expect(INVALID, c, *args(k=0))
    expect(UNSUPPORTED, c, *args(k=9))
    expect(INVALID, c, *args(pos=None))
    expect(INVALID, c, *args(y=FAKE + 2))
    expect(UNSUPPORTED, c, *args(k=8, T=(1 << 30) - 1))


def test_norm_backward_refusals():
    need = L.moe_norm_bwd_workspace_size(100, 64)
    assert need > 0 and L.moe_norm_bwd_workspace_size(0, 64) == 0 and L.moe_norm_bwd_workspace_size(4, 1 << 20) == 0
    o = L.moe_norm_out_bwd
    args = lambda gate=None, rows=1, dgate=None, ws=FAKE, n=need, rstd=FAKE, dw=FAKE: (
        FAKE, FAKE, FAKE, gate, rows, rstd, 100, 64, BF, FAKE, dw, dgate, ws, n)
    expect(WORKSPACE, o, *args(n=need - 1))
    expect(WORKSPACE, o, *args(ws=None))
    expect(INVALID, o, *args(gate=FAKE))              # gate without dgate
    expect(INVALID, o, *args(dgate=FAKE))             # dgate without gate
    expect(INVALID, o, *args(gate=FAKE, dgate=FAKE, rows=0))
    expect(INVALID, o, *args(rstd=None))
    expect(INVALID, o, *args(dw=FAKE + 4))
    i = L.moe_norm_in_bwd
    expect(WORKSPACE, i, FAKE, FAKE, FAKE, FAKE, None, 1.0, 100, 64, BF, FAKE, FAKE, FAKE, need - 1)
    expect(INVALID, i, FAKE, FAKE, FAKE, FAKE, FAKE + 2, 1.0, 100, 64, BF, FAKE, FAKE, FAKE, need)
    expect(INVALID, i, FAKE, FAKE, FAKE, FAKE, None, 1.0, 100, 64, BF, FAKE, None, FAKE, need)
    assert L.moe_workspace_bytes(L.MOE_OP_NORM_BWD, 100, 64, 8, 2, 128, 0) == need


def test_vocab_loss_refusals():
    need = L.moe_vocab_loss_workspace_size(100, 64, 1000, BF)
    assert need > 0 and L.moe_vocab_loss_workspace_size(100, 60, 1000, BF) == 0
    f = L.moe_vocab_loss
    args = lambda T=100, d=64, V=1000, dt=BF, h=FAKE, loss=FAKE, n=need: (h, FAKE, FAKE, T, d, V, dt, loss, FAKE, FAKE, n)
    expect(WORKSPACE, f, *args(n=need - 1))
    expect(UNSUPPORTED, f, *args(d=60))
    expect(UNSUPPORTED, f, *args(d=1 << 17))
    expect(UNSUPPORTED, f, *args(V=(1 << 22) + 1))
    expect(UNSUPPORTED, f, *args(T=(1 << 22) + 1))
    expect(UNSUPPORTED, f, *args(T=1 << 20, V=1 << 16))
    expect(UNSUPPORTED, f, *args(d=1 << 16, V=1 << 20))
    expect(UNSUPPORTED, f, *args(d=1 << 16, T=1 << 20))
    expect(INVALID, f, *args(V=0))
    expect(INVALID, f, *args(T=-1))
    expect(INVALID, f, *args(dt=3))
    expect(INVALID, f, *args(h=None))
    expect(INVALID, f, *args(loss=FAKE + 4))
    f(None, FAKE, None, 0, 64, 1000, BF, None, None, None, 0)
    b = L.moe_vocab_loss_bwd
    need = L.moe_vocab_loss_bwd_workspace_size(100, 64, 1000, F32)
    bargs = lambda lse=FAKE, dw=FAKE, n=need: (FAKE, FAKE, FAKE, lse, FAKE, 100, 64, 1000, F32, FAKE, dw, FAKE, n)
    expect(WORKSPACE, b, *bargs(n=need - 1))
    expect(INVALID, b, *bargs(lse=None))
    expect(INVALID, b, *bargs(dw=None))
    expect(INVALID, b, *bargs(dw=FAKE + 2))


class List:
    """A gradient list from addresses."""

    def __init__(self, *items):   # (grad, out, n, dt)
        self.array = (L.Grad * max(1, len(items)))(*[L.Grad(*i) for i in items])
        self.count, self.ptr = len(items), ctypes.cast(self.array, ctypes.c_void_p)


def test_gradient_refusals():
    A = 1 << 20
    ok = List((A, A, 1000, BF), (A + 4096, A + 8192, 10, F32), (None, None, 0, F32))
    need = L.moe_grad_workspace_size(ok)
    assert need >= 3 * 8
    clip = lambda l, m=1.0, n=1 << 20, ws=FAKE: L.moe_grad_clip(l, m, None, ws, n)
    expect(WORKSPACE, clip, ok, 1.0, need - 1)
    expect(WORKSPACE, clip, ok, 1.0, need, None)
    for m in (0.0, -1.0, float("nan")):
        expect(INVALID, clip, ok, m)
        expect(INVALID, L.moe_grad_scale, ok, FAKE, m, None)
    expect(INVALID, clip, List((A, A, -1, BF)))
    expect(INVALID, clip, List((A, A, 8, 5)))
    expect(INVALID, clip, List((None, A, 8, BF)))
    expect(INVALID, clip, List((A, None, 8, BF)))
    expect(INVALID, clip, List((A + 2, A + 2, 8, BF)))
    expect(UNSUPPORTED, clip, List((A, A, 1 << 42, BF)))
    # a tensor listed twice, an out on another tensor's gradient or out, an out that begins inside its own gradient
    expect(INVALID, clip, List((A, A, 8, BF), (A, A, 8, BF)))
    expect(INVALID, clip, List((A, A + 4096, 8, BF), (A + 64, A + 4096, 8, BF)))
    expect(INVALID, clip, List((A, A + 64, 8, BF), (A + 64, A + 4096, 8, BF)))
    expect(INVALID, clip, List((A, A + 16, 64, BF)))
    expect(INVALID, L.moe_grad_scale, List((A, A, 8, BF), (A, A, 8, BF)), FAKE, 1.0, None)
    expect(INVALID, L.moe_grad_scale, ok, None, 1.0, None)
    expect(INVALID, L.moe_grad_norm, ok, None, None, FAKE, need)
    expect(INVALID, L.moe_grad_norm, ok, FAKE + 8, None, FAKE, need)
    expect(WORKSPACE, L.moe_grad_norm, ok, FAKE, None, FAKE, need - 1)
    # the same gradient read twice into two outs is no overlap; the workspace check is what turns it away
    expect(WORKSPACE, clip, List((A, A + 4096, 8, BF), (A, A + 8192, 8, BF)), 1.0, 0)


def test_gradient_list_checks_its_tensors():
    a = torch.zeros(8)
    with pytest.raises(ValueError):
        L.grad_list([a], [torch.zeros(8, dtype=torch.bfloat16)])
    with pytest.raises(ValueError):
        L.grad_list([a], [torch.zeros(9)])
    with pytest.raises(ValueError):
        L.grad_list([a], [])
    with pytest.raises(ValueError):
        L.grad_list([torch.zeros(4, 4).t()[:, :2]])
    with pytest.raises(ValueError):
        L.grad_list([torch.zeros(8, dtype=torch.float64)])


def test_layer_refuses_norm_weights_of_another_shape_or_type():
    cfg = MoEConfig("t", 6, 256, 4, 2, 128, 0, "f32", "random", 0.0, False)
    z = torch.zeros
    p = dict(x=z(6, 256), logits=z(6, 4), norm_in=z(256), norm_out=z(256), norm_gate=z(2, 256))
    make = lambda **k: LY.MoELayer(cfg, {**p, **k}, block_norm=True, gate_rows=3)
    make()
    for bad in (dict(norm_gate=z(3, 256)), dict(norm_in=z(128)), dict(norm_out=z(256, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            make(**bad)
    with pytest.raises(ValueError):
        make().clip_gradients(1.0)   # no backward


def test_layers_that_share_buffers_keep_their_own_gate_gradient():
    """A second layer over the same buffers, with fewer gate rows or none, must not take away or shrink
    what the first one's backward writes; tensors of equal shapes stay the same ones."""
    cfg = MoEConfig("t", 6, 256, 4, 2, 128, 0, "f32", "random", 0.0, True)
    z = torch.zeros
    p = dict(x=z(6, 256), logits=z(6, 4), norm_in=z(256), norm_out=z(256), dout=z(6, 256))
    first = LY.MoELayer(cfg, dict(p, norm_gate=z(6, 256)), block_norm=True, gate_rows=1)
    held = {n: first.bufs[n] for n in ("xn", "rstd_in", "rstd_out", "y_block", "dblock", "dxn", "dnorm_in", "dnorm_out",
                                       "ws_norm")}
    second = LY.MoELayer(cfg, dict(p, norm_gate=z(1, 256)), bufs=first.bufs, block_norm=True)
    third = LY.MoELayer(cfg, p, bufs=first.bufs, block_norm=True)
    LY.MoELayer(cfg, p, bufs=first.bufs)
    assert first.gradients()[-1].shape == (6, 256) and second.gradients()[-1].shape == (1, 256)
    assert len(third.gradients()) == len(first.gradients()) - 1
    assert all(first.bufs[n] is t for n, t in held.items())


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    """With the device in use (here only said to be), host tensors and another device's are turned away."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    t = torch.zeros(64)
    target, grads = torch.zeros(8, dtype=torch.int32), L.grad_list([t])
    calls = [lambda: L.moe_norm_in(t, t, 8, 8, 0.0, F32, t, None),
             lambda: L.moe_norm_out(t, t, t, None, 1, 1.0, 0.0, 8, 8, F32, t, None),
             lambda: L.moe_combine_norm_out(t, t, target, None, t, t, None, 1, 1.0, 0.0, 8, 8, 1, F32, None, t, None),
             lambda: L.moe_norm_out_bwd(t, t, t, None, 1, t, 8, 8, F32, t, t, None, t, 256),
             lambda: L.moe_norm_in_bwd(t, t, t, t, None, 1.0, 8, 8, F32, t, t, t, 256),
             lambda: L.moe_vocab_loss(t, t, target, 8, 8, 8, F32, t, t, t, 256),
             lambda: L.moe_vocab_loss_bwd(t, t, target, t, t, 8, 8, 8, F32, t, t, t, 256),
             lambda: L.moe_grad_norm(grads, t, None, t, 256), lambda: L.moe_grad_scale(grads, t, 1.0, None),
             lambda: L.moe_grad_clip(grads, 1.0, None, t, 256)]
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()
    with pytest.raises(ValueError, match="different devices"):
        L.grad_list([t, torch.zeros(8, device="meta")])


@pytest.mark.parametrize("norm", [False, True])
def test_layer_with_a_backward_over_forward_buffers(norm):
    """Buffers without the backward's tensors serve a forward, whatever the configuration says."""
    cfg = MoEConfig("t", 6, 256, 4, 2, 128, 0, "f32", "random", 0.0, True)
    z = torch.zeros
    p = dict(x=z(6, 256), logits=z(6, 4), norm_in=z(256), norm_out=z(256), dout=z(6, 256))
    bufs = LY.Buffers.allocate(cfg.with_(backward=False), torch.device("cpu"))
    assert "dw1" not in bufs.t
    LY.MoELayer(cfg, p, bufs=bufs, block_norm=norm)


def test_clipping_workspace_is_made_once_when_it_is_needed(monkeypatch):
    cfg = MoEConfig("t", 6, 256, 4, 2, 128, 0, "f32", "random", 0.0, True)
    z = torch.zeros
    lay = LY.MoELayer(cfg, dict(x=z(6, 256), logits=z(6, 4), dout=z(6, 256)))
    before = set(lay.bufs.t)
    calls = []
    monkeypatch.setattr(L, "moe_grad_clip", lambda *a: calls.append(a))
    lay.clip_gradients(1.0)
    lay.clip_gradients(2.0)
    (grads, _, norm, ws, n), second = calls[0], calls[1]
    assert ws.numel() == n >= L.moe_grad_workspace_size(grads) and norm is lay.grad_norm
    assert second[3] is ws and set(lay.bufs.t) == before


class OnDevice(torch.Tensor):
    """A tensor that says it is on device 1, with an address that nothing reads."""

    @staticmethod
    def __new__(cls):
        return torch.Tensor._make_subclass(cls, torch.zeros(64))

    def get_device(self):
        return 1

    def data_ptr(self):
        return FAKE


def _calls(t, grads):
    """Each call over the tensors ``t`` (a function of a tensor's place in the call), and how many it takes."""
    return [(4, lambda s: L.moe_norm_in(t(0), t(1), 8, 8, 0.0, F32, t(2), t(3), s)),
            (6, lambda s: L.moe_norm_out(t(0), t(1), t(2), t(3), 1, 1.0, 0.0, 8, 8, F32, t(4), t(5), s)),
            (10, lambda s: L.moe_combine_norm_out(t(0), t(1), t(2), t(3), t(4), t(5), t(6), 1, 1.0, 0.0, 8, 8, 1, F32, t(7),
                                                  t(8), t(9), s)),
            (9, lambda s: L.moe_norm_out_bwd(t(0), t(1), t(2), t(3), 1, t(4), 8, 8, F32, t(5), t(6), t(7), t(8), 1 << 20, s)),
            (8, lambda s: L.moe_norm_in_bwd(t(0), t(1), t(2), t(3), t(4), 1.0, 8, 8, F32, t(5), t(6), t(7), 1 << 20, s)),
            (6, lambda s: L.moe_vocab_loss(t(0), t(1), t(2), 8, 8, 8, F32, t(3), t(4), t(5), 1 << 20, s)),
            (8, lambda s: L.moe_vocab_loss_bwd(t(0), t(1), t(2), t(3), t(4), 8, 8, 8, F32, t(5), t(6), t(7), 1 << 20, s)),
            (3, lambda s: L.moe_grad_norm(grads, t(0), t(1), t(2), 1 << 20, s)),
            (2, lambda s: L.moe_grad_scale(grads, t(0), 1.0, t(1), s)),
            (2, lambda s: L.moe_grad_clip(grads, 1.0, t(0), t(1), 1 << 20, s))]


class FakeStream:
    device_index, cuda_stream = 1, 0


@pytest.mark.parametrize("stream,initialized", [(None, True), (None, False), (FakeStream(), True), (FakeStream(), False),
                                                (64, True)])
def test_every_tensor_of_a_call_must_be_on_its_device(monkeypatch, stream, initialized):
    """One tensor of the call on the host, each in turn, with the stream by default (also before anything
    used the device), given, or given as a handle: refused before libmoe is called."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: initialized)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    reached = []
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: 0, raising=False)
    monkeypatch.setattr(L, "_call", lambda name, *a: reached.append(name))
    host, device, grads = torch.zeros(64), OnDevice(), L.grad_list([OnDevice()])
    off = [None]
    t = lambda i: host if i == off[0] else device
    for n, call in _calls(t, grads):
        off[0] = None
        call(stream)
        assert reached.pop()
        for off[0] in range(n):
            with pytest.raises(ValueError):
                call(stream)
            assert not reached
    off[0] = None
    for n, call in _calls(t, L.grad_list([torch.zeros(64)]))[-3:]:
        with pytest.raises(ValueError):
            call(stream)
        assert not reached
