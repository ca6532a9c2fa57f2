"""Every output of the selective-SSM calls laid over every input and every other
output: refused on the host, with both names."""
import itertools

import pytest
import torch

import test_selective_abi_host as T
from fft_long_convolution_flashconv_b200 import _lib

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="the addresses are fake: host only")
STEP = 1 << 36  # further apart than any array here is long


def norm_fwd(**kw):
    a = dict(x=0, weight=0, bias=0, gate=0, y=0, B=2, L=5, C=12, G=2, eps=1e-5, cm=0, dtype=T.F16)
    a.update(kw)
    return _lib.load().group_norm_act_fwd(*a.values(), None)


def norm_bwd(**kw):
    a = dict(dy=0, x=0, weight=0, bias=0, gate=0, dx=0, dweight=0, dbias=0, dgate=0, B=2, L=5, C=12, G=2, eps=1e-5, cm=0,
             ws=0, wsb=1 << 20, dtype=T.F16)
    a.update(kw)
    return _lib.load().group_norm_act_bwd(*a.values(), None)


# the call, its inputs and its outputs: argument of the helper -> name in the message
SCAN = dict(u="u", delta="delta", A="A", Bt="Bt", Ct="Ct", D="D", bias="dt_bias", z="z")
CALLS = [
    (T.conv_fwd, dict(x="x", w="w", bias="bias", lengths="lengths", sin="state_in"), dict(y="y", sout="state_out")),
    (T.conv_bwd, dict(dy="dy", x="x", w="w", bias="bias", lengths="lengths", sin="state_in", dsout="dstate_out"),
     dict(dx="dx", dw="dw", db="dbias", dsin="dstate_in", ws="workspace")),
    (T.conv_step, dict(x="x", w="w", bias="bias", slots="slots"), dict(y="y", state="state")),
    # (its workspace, which is for segments of rows, has no bytes at the one SM that a host without a GPU counts)
    (T.scan_fwd, dict(SCAN, lengths="lengths", sin="state_in"), dict(y="y", sout="state_out", ckpt="ckpt")),
    (T.scan_bwd, dict(SCAN, dy="dy", ckpt="ckpt", lengths="lengths", dsout="dstate_out"),
     dict(du="du", ddelta="ddelta", dA="dA", dB="dB", dC="dC", dD="dD", db="ddt_bias", dz="dz", dsin="dstate_in",
          ws="workspace")),
    (T.scan_step, dict(SCAN, slots="slots"), dict(y="y", state="state")),
    (norm_fwd, dict(x="x", weight="weight", bias="bias", gate="gate"), dict(y="y")),
    (norm_bwd, dict(dy="dy", x="x", weight="weight", bias="bias", gate="gate"),
     dict(dx="dx", dweight="dweight", dbias="dbias", dgate="dgate", ws="workspace")),
]


def _cases():
    for call, ins, outs in CALLS:
        for o, i in itertools.chain(itertools.product(outs, ins), itertools.combinations(outs, 2)):
            yield pytest.param(call, ins, outs, o, i, id=f"{call.__name__}-{o}-over-{i}")


@pytest.mark.parametrize("call,ins,outs,over,under", list(_cases()))
def test_overlap_is_refused(call, ins, outs, over, under):
    names = {**ins, **outs}
    args = {a: STEP * (k + 1) for k, a in enumerate(names)}
    args[over] = args[under]  # the same first element: aligned for either
    assert call(**args) == T.EINVAL
    msg = T._err()
    assert "overlaps" in msg and names[over] in msg and names[under] in msg
