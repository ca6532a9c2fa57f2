"""Selective-SSM calls whose sizes or values reach parts of the kernels that
ordinary ones do not: references, magnitudes and tolerances are those of
test_selective_gpu.py, where they are derived."""
import numpy as np
import pytest
import torch

import test_selective_gpu as T
from fft_long_convolution_flashconv_b200 import api

pytestmark = pytest.mark.gpu
_cuda = T._cuda

GRADS = ("du", "ddelta", "dA", "dB", "dC", "dD", "ddt_bias", "dz", "dstate_in")


def scan_bwd(c, p, args, ckpt):
    return api.selective_scan_bwd(T.cu(p["dy"]), args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"], ckpt,
                                  T.cu(c["D"]), T.cu(c["dt_bias"]), args["z"], c["softplus"], T.cu(c["n"]),
                                  T.cu(c["dso"]), need_dstate_in=True)


@pytest.mark.parametrize("B,H,L,N,dtype,sizes", [(1, 3, 1500, 16, "f32", (1e3, 3e4, 6e4, 1e8)),
                                                 (2, 5, 1100, 20, "bf16", (1e3, 3e4, 6e4))])
def test_large_steps_among_small_ones_in_segments(B, H, L, N, dtype, sizes):
    """Some steps that reset the state, among steps of about 0.01: what lies between such a step and a segment's end
    (backward: its start) keeps its small distances."""
    assert api.selective_scan_workspace_bytes(B, H, L, N, 1) > 0  # the row is cut into segments
    c = T.scan_case(B, H, L, N, 1, dtype, 23, ("D", "gate", "state", "raw"))
    rng = np.random.default_rng(6)
    dt = rng.uniform(0.005, 0.02, (B, H, L))
    for k in range(0, L, 64):  # one such step in every third block of a row, in any of its lanes
        hit = rng.random((B, H)) < 0.34
        at = np.minimum(k + rng.integers(0, 64, (B, H)), L - 1)
        for b, h in zip(*np.nonzero(hit)):
            dt[b, h, at[b, h]] = rng.choice(sizes)
    c["delta"] = torch.tensor(dt).to(T.DT[dtype])
    want, mag = T.scan_want(c)
    args, (y, state, ckpt) = T.call_fwd(c, return_state=True, return_ckpt=True)
    # Arguments |dt A| above 88 give zero on both sides; below, one step adds 88 * 2^-21 to a term, twice that where
    # two meet.  A distance to a segment's end is a sum of positive steps with at most 16 + 2 + 24 roundings, 42 * 88 *
    # 2^-24 = 2.2e-4 of a term, which takes the place of the k 2^-22 of k decays in kappa(L) (2.6e-4 at 1100).
    k = T.kappa(L) + 2 * 88 * 2.0 ** -21
    T.close(y, want["y"], mag["y"], k, "y")
    T.close(state, want["state"], mag["state"], k, "state")
    for name, g in zip(GRADS, scan_bwd(c, c, args, ckpt)):
        if name != "ddt_bias":
            T.close(g, want[name], mag[name], 2 * k, name)


def test_workspace_over_an_output_is_refused():
    c = T.scan_case(1, 3, 1500, 4, 1, "f32", 2, ("D",))
    a = [c[k].cuda() for k in ("u", "delta", "A", "Bt", "Ct", "D")]
    need = api.selective_scan_workspace_bytes(1, 3, 1500, 4, 1)
    assert need > 0
    ws = torch.zeros(need + 3 * 1500 * 4, dtype=torch.uint8, device="cuda")
    out = ws.view(torch.float32)[need // 4 - 4:][:3 * 1500].view(1, 3, 1500)  # begins inside the workspace
    with pytest.raises(Exception, match="y and workspace: one overlaps the other"):
        api.selective_scan_fwd(*a, workspace=ws, out=out)
    out = ws.view(torch.float32)[need // 4:][:3 * 1500].view(1, 3, 1500)  # right behind what the call uses
    assert torch.equal(api.selective_scan_fwd(*a, workspace=ws, out=out), api.selective_scan_fwd(*a))
