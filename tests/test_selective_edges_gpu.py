"""Selective-SSM calls whose sizes or values reach parts of the kernels that
ordinary ones do not: references, magnitudes and tolerances are those of
test_selective_gpu.py, where they are derived."""
import numpy as np
import pytest
import torch

import test_selective_gpu as T
from fft_long_convolution_flashconv_b200 import _lib, api

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


@pytest.mark.parametrize("L", [90, 1500])
def test_growing_states(L):
    """A above zero: states that grow by up to e^35 in one piece and in segments."""
    assert (api.selective_scan_workspace_bytes(1, 3, L, 4, 1) > 0) == (L == 1500)
    c = T.scan_case(1, 3, L, 4, 1, "f32", 41, ("D", "gate", "state", "raw"))
    rng = np.random.default_rng(3)
    c["A"] = torch.tensor(rng.uniform(0.05, 0.5, (3, 4)), dtype=torch.float32)
    c["delta"] = torch.tensor(rng.uniform(0.001, 70 / L, (1, 3, L)), dtype=torch.float32)  # sum dt A <= 35
    want, mag = T.scan_want(c)
    args, (y, state, ckpt) = T.call_fwd(c, return_state=True, return_ckpt=True)
    # |sum dt A| <= 35 over the row instead of 32: 3 * 2^-21 more, within kappa's 96 * 2^-21 of slack
    T.close(y, want["y"], mag["y"], T.kappa(L), "y")
    T.close(state, want["state"], mag["state"], T.kappa(L), "state")
    for name, g in zip(GRADS, scan_bwd(c, c, args, ckpt)):
        if name != "ddt_bias":
            T.close(g, want[name], mag[name], T.kappa(L, True), name)


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


# ------------------------------------------------------------------ sixteen steps a lane
def scan_want_on_gpu(c):
    """scan_want with its 64-bit steps on the GPU (some thousand channels)."""
    with torch.device("cuda"):
        want, mag = T.scan_want({k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()})
    return ({k: v.detach().cpu() for k, v in d.items()} for d in (want, mag))


@pytest.mark.parametrize("B,H,L,N,G,dtype,segments,view,opts", [
    # rows on 16-byte boundaries; a last group of channels that is not full; two chunks of states
    (5, 2000, 136, 16, 1, "f16", False, False, ("D", "bias", "gate", "state", "ragged")),
    (4, 2404, 200, 20, 2, "bf16", False, False, ("D", "bias", "gate", "state", "ragged")),
    (3, 3200, 200, 4, 1, "f32", False, False, ("D", "gate", "state", "ragged", "raw")),
    # rows on two-byte boundaries: blocks inside the sequence load together
    (5, 1920, 203, 16, 1, "f16", False, False, ("D", "bias", "gate", "state", "ragged")),
    (2, 5000, 269, 33, 1, "bf16", False, False, ("bias", "state")),
    # rows of both kinds, NaN around them, and fp32 rows on four-byte boundaries
    (5, 1920, 200, 5, 1, "f16", False, True, ("D", "bias", "gate", "state", "ragged")),
    (3, 3201, 150, 3, 3, "f32", False, True, ("D", "bias", "gate", "state", "ragged")),
    # in segments, both kinds of rows
    (1, 1600, 1504, 4, 1, "bf16", True, False, ("D", "bias", "gate", "state")),
    (1, 1600, 1501, 4, 1, "f16", True, False, ("D", "bias", "gate", "state")),
])
def test_scan_of_sixteen_steps_a_lane(B, H, L, N, G, dtype, segments, view, opts):
    """Batches that fill the GPU take the form with sixteen steps a lane; its kept states feed the backward pass."""
    assert _lib.load().fc_debug_scan_lane_steps(B, H, L, N, G) == 16
    assert (api.selective_scan_workspace_bytes(B, H, L, N, G) > 0) == segments
    c = T.scan_case(B, H, L, N, G, dtype, L + N, opts)
    if segments:
        c["dt_bias"] = torch.full((H,), -7.0)  # decays to e^-1 and so over the row: segments matter to one another
    want, mag = scan_want_on_gpu(c)
    p = T.poison(c)
    # Sums over a group's channels have up to 200 more roundings of 2^-24 than kappa's tens: 1.2e-5, where kappa's
    # count of k 2^-21 for an error of k 2^-22 leaves L 2^-22 (3.2e-5 at 136).
    args, (y, state, ckpt) = T.call_fwd(p, view=view, return_state=True, return_ckpt=True)
    T.close(y, want["y"], mag["y"], T.kappa(L), "y")
    T.close(state, want["state"], mag["state"], T.kappa(L), "state")
    _, plain = T.call_fwd(p, view=view)  # without kept states: another kernel, the same arithmetic
    assert torch.equal(plain, y)
    for k, g in zip(GRADS, scan_bwd(c, p, args, ckpt)):
        if g is None:
            assert k not in want
        else:
            T.close(g, want[k], mag[k], T.kappa(L, True), k)


# ------------------------------------------------------------------ short convolution of aligned rows
@pytest.mark.parametrize("B,H,L,K,dtype,silu,bias,state,ragged", [
    (3, 5, 1024, 4, "f16", True, True, True, False),   # one block of 32 threads a row, every vector inside
    (5, 6, 1024, 4, "bf16", True, True, True, True),   # rows that end inside a thread's vectors
    (2, 3, 4096, 8, "f16", True, True, True, False),
    (2, 4, 5128, 3, "f32", True, False, True, True),   # the last block of a row is not full
    (2, 3, 1024, 1, "f32", False, True, False, False),
    (3, 2, 1040, 7, "bf16", False, True, True, True),
    (2, 3, 2048, 2, "f16", True, True, True, False),
    (1, 3, 8192, 5, "f32", True, True, True, False),
    (2, 2, 4104, 6, "bf16", True, True, False, False),
    (2, 600, 1024, 4, "f16", True, True, True, True),  # one part a channel, several items a thread
])
def test_short_conv_of_aligned_rows(B, H, L, K, dtype, silu, bias, state, ragged):
    x, w, bi, past, dy, dso, n = T.conv_case(B, H, L, K, dtype, silu, bias, state, ragged, seed=L + K)
    ns = [L if n is None else int(n[b]) for b in range(B)]
    zeros = torch.zeros(B, H, K - 1, dtype=torch.float64)
    dbl = lambda t: None if t is None else t.double()  # noqa: E731

    def run(f):
        """Outputs, states and gradients in 64 bits, of the formula (f = identity) or of its magnitudes (f = abs)."""
        on = f is not torch.abs
        X, W, P = (f(t.double()).requires_grad_() for t in (x, w, zeros if past is None else past))
        bb = None if bi is None else f(bi.double()).requires_grad_()
        rows = [T.conv_ref(X[b], W, bb, silu and on, P[b], ns[b]) for b in range(B)]
        y, s = torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
        scale = 1 if on else (1 + y.detach()) * 1.1  # silu' < 1.1, and dc's own error is relative to |dy| (1 + M)
        loss = (y * f(dbl(dy)) * scale).sum() + (s * f(dbl(dso))).sum()
        leaves = [X, W, P] + ([] if bb is None else [bb])
        g = torch.autograd.grad(loss, leaves, allow_unused=True)
        g = [torch.zeros_like(a) if v is None else v for a, v in zip(leaves, g)]
        return y.detach(), s.detach(), g + [None] * (4 - len(g))

    want, wstate, grads = run(lambda t: t)
    mag, _, mags = run(torch.abs)
    for b in range(B):  # padding may hold anything
        x[b, :, ns[b]:] = T.NAN
        dy[b, :, ns[b]:] = T.NAN
    kap = 64 * 2.0 ** -22
    a = (x.cuda(), w.cuda(), T.cu(bi), silu, T.cu(past), T.cu(n))
    y, s = api.short_conv_fwd(*a, return_state=True)
    T.close(y, want, mag * (1 + mag), kap, "y")
    assert torch.equal(s.cpu().double(), wstate)
    dx, dw, db, dp = api.short_conv_bwd(dy.cuda(), *a, T.cu(dso), need_dstate_in=True)
    for name, g, r, m, k in (("dx", dx, grads[0], mags[0], kap), ("dstate_in", dp, grads[2], mags[2], kap),
                             ("dw", dw, grads[1], mags[1], kap + 512 * 2.0 ** -24),
                             ("dbias", db, grads[3], mags[3], kap + 512 * 2.0 ** -24)):
        assert (g is None) == (r is None)
        if g is not None:
            T.close(g, r, m, k, name)


# ------------------------------------------------------------------ group norm
@pytest.mark.parametrize("B,L,C,G,dtype,opts,cm", [
    # groups of 513 to 1024 channels: four vectors a lane of one warp
    (2, 37, 768, 1, "f16", ("w", "b", "gate"), False),
    (1, 33, 1024, 1, "f32", ("w", "b", "gate"), False),
    (3, 50, 1544, 2, "bf16", ("w", "b"), False),       # groups of 772
    (2, 65, 1040, 2, "f16", ("w", "gate"), False),     # groups of 520
    (1, 20, 519, 1, "f32", ("b", "gate"), False),
    # more groups than the GPU holds: every thread takes several
    (5, 1000, 640, 1, "f16", ("w", "b", "gate"), False),
    (2, 12000, 64, 1, "f16", ("w", "b", "gate"), False),
    (1, 3000, 384, 1, "bf16", ("w", "b"), False),
    (1, 700, 1100, 1, "f32", ("w", "b", "gate"), False),
    (2, 400, 2050, 1, "bf16", ("w", "b"), False),
    (1, 80001, 32, 1, "f16", ("w", "b", "gate"), True),
])
def test_group_norm_of_wide_groups_and_many_tokens(B, L, C, G, dtype, opts, cm):
    T.test_group_norm_act(B, L, C, G, dtype, opts, cm)
