"""Refusals of the selective-SSM calls, on the host: the C entry points reject
bad arguments before anything is launched (every call below carries at least
one, so the fake addresses are never used), and the wrappers reject tensors of
the wrong shape, type, layout or device."""
import ctypes

import pytest
import torch

from fft_long_convolution_flashconv_b200 import _lib, api

P, P2, P3, P4, P5, P6 = (0x10000000 + (i << 32) for i in range(6))  # fake, far apart, never dereferenced
EINVAL, EUNSUP = _lib.FC_EINVAL, _lib.FC_EUNSUPPORTED
F16 = _lib.FC_F16


def _err():
    return _lib.load().fc_last_error().decode()


def _ll(*v):
    return (ctypes.c_longlong * len(v))(*v)


def conv_fwd(**kw):
    a = dict(x=P, w=P2, bias=P3, y=P4, B=2, H=3, L=40, K=4, silu=1, lengths=None, strides=None, sin=None, sout=None,
             dtype=F16)
    a.update(kw)
    return _lib.load().short_conv_fwd(*a.values(), None)


def conv_bwd(**kw):
    a = dict(dy=P, x=P2, w=P3, bias=P3, dx=P4, dw=P5, db=P5, B=2, H=3, L=40, K=4, silu=1, lengths=None, strides=None,
             sin=None, dsout=None, dsin=None, ws=P6, wsb=1 << 20, dtype=F16)
    a.update(kw)
    return _lib.load().short_conv_bwd(*a.values(), None)


def conv_step(**kw):
    a = dict(x=P, state=P2, w=P3, bias=P3, y=P4, B=2, H=3, K=4, silu=1, slots=None, S=2, xs=3, dtype=F16)
    a.update(kw)
    return _lib.load().short_conv_step(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(K=0), EUNSUP, "K must"), (dict(K=9), EUNSUP, "K must"), (dict(B=0), EINVAL, ">= 1"),
    (dict(L=0), EINVAL, ">= 1"), (dict(L=(1 << 30) + 1), EUNSUP, "2^30"), (dict(H=1 << 30, B=4), EUNSUP, "2^31"),
    (dict(dtype=3), EINVAL, "dtype"), (dict(x=None), EINVAL, "null"), (dict(w=None), EINVAL, "null"),
    (dict(y=None), EINVAL, "y must"), (dict(y=P4 + 8), EINVAL, "16-byte"), (dict(x=P + 1), EINVAL, "aligned"),
    (dict(y=P + 64), EINVAL, "overlap"), (dict(strides=_ll(-1, 40)), EINVAL, "strides"),
    (dict(strides=_ll(1 << 60, 40)), EINVAL, "strides"), (dict(sin=P2, sout=P2), EINVAL, "overlap"),
    (dict(strides=_ll((P4 - P) // 2, 40)), EINVAL, "overlap"),  # the second batch row of x would lie in y
])
def test_short_conv_fwd_refusals(bad, status, word):
    assert conv_fwd(**bad) == status
    assert word in _err()


@pytest.mark.parametrize("bad,status,word", [
    (dict(dy=None), EINVAL, "null"), (dict(dw=None), EINVAL, "null"), (dict(dx=P2 + 16), EINVAL, "overlap"),
    (dict(ws=None), EINVAL, "workspace"), (dict(ws=P6 + 16), EINVAL, "256-byte"), (dict(wsb=8), EINVAL, "too small"),
    (dict(strides=_ll(120, 40, -3, 40)), EINVAL, "strides"), (dict(dsin=P4), EINVAL, "overlap"),
    (dict(K=9), EUNSUP, "K must"),
])
def test_short_conv_bwd_refusals(bad, status, word):
    assert conv_bwd(**bad) == status
    assert word in _err()


@pytest.mark.parametrize("bad,status,word", [
    (dict(S=3), EINVAL, "without slots"), (dict(S=0, slots=P5), EINVAL, "pool"), (dict(B=65536), EUNSUP, "65535"),
    (dict(state=None), EINVAL, "state"), (dict(y=P2 + 2), EINVAL, "overlap"), (dict(slots=P5 + 2), EINVAL, "slots"),
    (dict(xs=-1), EINVAL, "x_stride"), (dict(y=P), EINVAL, "overlap"),
])
def test_short_conv_step_refusals(bad, status, word):
    assert conv_step(**bad) == status
    assert word in _err()


def scan_fwd(**kw):
    a = dict(u=P, delta=P2, A=P3, Bt=P4, Ct=P4 + 4096, D=P3, bias=P3, z=None, y=P5, B=2, H=6, L=40, N=8, G=2, sp=1,
             lengths=None, strides=None, sin=None, sout=None, ckpt=None, ws=None, wsb=0, dtype=F16)
    a.update(kw)
    return _lib.load().selective_scan_fwd(*a.values(), None)


def scan_bwd(**kw):
    q = 1 << 20
    a = dict(dy=P, u=P + q, delta=P2, A=P3, Bt=P4, Ct=P4 + 4096, D=P3, bias=P3, z=None, ckpt=P2 + q, du=P5,
             ddelta=P5 + q, dA=P5 + 2 * q, dB=P5 + 3 * q, dC=P5 + 4 * q, dD=P5 + 5 * q, db=P5 + 6 * q, dz=None, B=2, H=6,
             L=40, N=8, G=2, sp=1, lengths=None, strides=None, dsout=None, dsin=None, ws=P6, wsb=1 << 30, dtype=F16)
    a.update(kw)
    return _lib.load().selective_scan_bwd(*a.values(), None)


def scan_step(**kw):
    a = dict(u=P, delta=P2, A=P3, Bt=P4, Ct=P4 + 4096, D=P3, bias=P3, z=None, state=P6, y=P5, B=2, H=6, N=8, G=2, sp=1,
             slots=None, S=2, strides=None, dtype=F16)
    a.update(kw)
    return _lib.load().selective_scan_step(*a.values(), None)


@pytest.mark.parametrize("bad,status,word", [
    (dict(N=0), EINVAL, "N, G"), (dict(N=257), EUNSUP, "256"), (dict(G=4), EINVAL, "multiple"),
    (dict(G=0), EINVAL, "N, G"), (dict(u=None), EINVAL, "null"), (dict(A=None), EINVAL, "null"),
    (dict(Ct=None), EINVAL, "null"), (dict(A=P3 + 2), EINVAL, "aligned"), (dict(y=P5 + 2), EINVAL, "16-byte"),
    (dict(y=P2), EINVAL, "overlap"), (dict(y=P4), EINVAL, "overlap"), (dict(z=P5), EINVAL, "overlap"),
    (dict(ckpt=P5), EINVAL, "ckpt"), (dict(sin=P6, sout=P6), EINVAL, "state_out"), (dict(dtype=-1), EINVAL, "dtype"),
    (dict(strides=_ll(*[240, 40] * 3, 640, -320, 40, 640, 320, 40)), EINVAL, "strides"),
    (dict(L=1 << 30, B=1, H=256, N=256, G=256), EUNSUP, "2^37"),
])
def test_selective_scan_fwd_refusals(bad, status, word):
    assert scan_fwd(**bad) == status
    assert word in _err()


@pytest.mark.parametrize("bad,status,word", [
    (dict(ckpt=None), EINVAL, "null"), (dict(dB=None), EINVAL, "null"), (dict(z=P6 + (1 << 31)), EINVAL, "z and dz"),
    (dict(dz=P6 + (1 << 31)), EINVAL, "z and dz"), (dict(du=P2), EINVAL, "overlaps an input"),
    (dict(ddelta=P5), EINVAL, "two gradients"), (dict(ws=None), EINVAL, "workspace"),
    (dict(wsb=64), EINVAL, "too small"), (dict(N=300), EUNSUP, "256"), (dict(dA=P5 + 2), EINVAL, "aligned"),
])
def test_selective_scan_bwd_refusals(bad, status, word):
    assert scan_bwd(**bad) == status
    assert word in _err()


@pytest.mark.parametrize("bad,status,word", [
    (dict(S=5), EINVAL, "without slots"), (dict(state=None), EINVAL, "state"), (dict(y=P6), EINVAL, "overlaps"),
    (dict(u=P6), EINVAL, "overlaps"), (dict(B=70000, S=70000), EUNSUP, "65535"), (dict(G=5), EINVAL, "multiple"),
])
def test_selective_scan_step_refusals(bad, status, word):
    assert scan_step(**bad) == status
    assert word in _err()


@pytest.mark.parametrize("bad,status,word", [
    (dict(G=5), EINVAL, "multiple"), (dict(G=0), EINVAL, "multiple"), (dict(C=8193 * 2), EUNSUP, "8192"),
    (dict(eps=0.0), EINVAL, "eps"), (dict(eps=float("nan")), EINVAL, "eps"), (dict(x=P + 2), EINVAL, "16-byte"),
    (dict(y=P), EINVAL, "overlap"), (dict(y=None), EINVAL, "y must"), (dict(gate=P4), EINVAL, "overlap"),
    (dict(L=0), EINVAL, ">= 1"),
])
def test_group_norm_act_refusals(bad, status, word):
    a = dict(x=P, w=P2, bias=P2, gate=None, y=P4, B=2, L=5, C=12, G=2, eps=1e-5, cm=0, dtype=F16)
    a.update(bad)
    assert _lib.load().group_norm_act_fwd(*a.values(), None) == status
    assert word in _err()


def test_group_norm_act_bwd_refusals():
    def call(**kw):
        a = dict(dy=P, x=P2, w=P3, bias=P3, gate=None, dx=P4, dw=P5, db=P5, dgate=None, B=2, L=5, C=12, G=2, eps=1e-5,
                 cm=0, ws=P6, wsb=1 << 20, dtype=F16)
        a.update(kw)
        return _lib.load().group_norm_act_bwd(*a.values(), None)
    for bad, word in ((dict(gate=P6), "gate and dgate"), (dict(dx=P), "overlaps"), (dict(wsb=4), "too small"),
                      (dict(ws=P6 + 8), "256-byte"), (dict(dy=None), "non-null"),
                      (dict(gate=P6 + (1 << 20), dgate=P4), "dx and dgate")):
        assert call(**bad) == EINVAL
        assert word in _err(), word


def test_workspace_sizes():
    lib = _lib.load()
    # one partial dB and dC for each 16 channels of a group
    assert lib.selective_scan_bwd_workspace(2, 64, 100, 8, 2) >= 2 * 2 * 2 * 2 * 8 * 100 * 4
    assert lib.selective_scan_bwd_workspace(2, 63, 100, 8, 2) == 0
    assert lib.selective_scan_ckpt_bytes(2, 3, 65, 4) == 2 * 3 * 2 * 4 * 4
    assert lib.short_conv_bwd_workspace(2, 3, 40, 9) == 0
    assert lib.group_norm_act_bwd_workspace(1, 1, 12, 5, 0) == 0


# ------------------------------------------------------------------ the wrappers
def test_wrappers_refuse_wrong_tensors():
    x, w = torch.zeros(2, 3, 8), torch.zeros(3, 4)
    with pytest.raises(ValueError, match="CUDA"):
        api.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="shape"):
        api.short_conv_fwd(x, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="float32"):
        api.short_conv_fwd(x, w.double())
    with pytest.raises(ValueError, match="last axis"):
        api.short_conv_fwd(torch.zeros(2, 8, 3).transpose(1, 2), w)
    with pytest.raises(ValueError, match="dtype"):
        api.short_conv_fwd(x.double(), w)
    with pytest.raises(ValueError, match="state_in"):
        api.short_conv_fwd(x, w, state_in=torch.zeros(2, 3, 4))
    with pytest.raises(ValueError, match="lengths"):
        api.short_conv_fwd(x, w, lengths=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="dy"):
        api.short_conv_bwd(torch.zeros(2, 3, 9), x, w)
    with pytest.raises(ValueError, match="slots"):
        api.short_conv_step(x[..., 0].contiguous(), torch.zeros(2, 3, 3), w, slots=torch.zeros(3, dtype=torch.int32))
    u, A, Bt = torch.zeros(2, 6, 8), torch.zeros(6, 4), torch.zeros(2, 2, 4, 8)
    with pytest.raises(ValueError, match="CUDA"):
        api.selective_scan_fwd(u, u, A, Bt, Bt)
    with pytest.raises(ValueError, match="Ct"):
        api.selective_scan_fwd(u, u, A, Bt, Bt[:, :, :3])
    with pytest.raises(ValueError, match="delta"):
        api.selective_scan_fwd(u, u.half(), A, Bt, Bt)
    with pytest.raises(ValueError, match="B x G x N"):
        api.selective_scan_fwd(u, u, A, Bt[0], Bt)
    with pytest.raises(ValueError, match="ckpt"):
        api.selective_scan_bwd(u, u, u, A, Bt, Bt, torch.zeros(7))
    with pytest.raises(ValueError, match="state"):
        api.selective_scan_step(u[..., 0], u[..., 0], A, Bt[..., 0], Bt[..., 0], torch.zeros(2, 6, 5))
    with pytest.raises(ValueError, match="groups"):
        api.group_norm_act_fwd(torch.zeros(1, 2, 10), 3)
    with pytest.raises(ValueError, match="contiguous"):
        api.group_norm_act_fwd(torch.zeros(2, 10, 4).transpose(1, 2), 2)
    with pytest.raises(ValueError, match="gate"):
        api.group_norm_act_fwd(torch.zeros(1, 2, 10), 2, gate=torch.zeros(1, 2, 9))


def test_wrappers_refuse_tensors_of_another_device():
    meta = torch.zeros(3, 4, device="meta")

    class Fake:  # a tensor as the device check sees it
        def __init__(self, device):
            self.device = torch.device(device)
    with pytest.raises(ValueError, match="different devices"):
        api._device(Fake("cuda:0"), None, Fake("cuda:1"))
    with pytest.raises(ValueError, match="CUDA"):
        api._device(meta)
    assert api._device(Fake("cuda:1"), None, Fake("cuda:1")) == torch.device("cuda:1")


@pytest.mark.parametrize("H", [(1 << 30) + 1, (1 << 31) - 2])
@pytest.mark.parametrize("call,kw", [
    (conv_fwd, {"L": 1}), (conv_bwd, {"L": 1}), (conv_step, {"S": 1}), (scan_fwd, {"L": 1, "G": 1}),
    (scan_bwd, {"L": 1, "G": 1}), (scan_step, {"S": 1, "G": 1}),
])
def test_more_channels_than_an_int_index_holds(call, kw, H):
    # a block's last channel lies up to a block past H; y is bad too, so nothing can launch
    kw = dict(kw, B=1, H=H, **({"dx": None} if call is conv_bwd else {"du": None} if call is scan_bwd else {"y": None}))
    assert call(**kw) == EUNSUP
    assert "H = " in _err() and "2^30" in _err()
