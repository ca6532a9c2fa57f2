"""The selective-SSM kernels (short causal convolution, selective scan, group
norm with SiLU) against plain step-by-step forms in 64 bits.

Tolerances are fixed beforehand from the arithmetic.  An output is compared as
|got - want| <= half a step of its type at want + kappa * M, where M is the
same formula with the absolute value of every term (so cancellation does not
hide behind the result's size) and kappa counts fp32 roundings.  A term of the
scan that is carried k steps is a product of k factors exp(dt A), each with a
relative error of 2^-22 (special function unit) + |dt A| 2^-21 (argument: dt's
own error 2^-22, product and scaling); terms with sum |dt A| > 32 are below
e^-32 of M.  So a term's relative error is below (k 2^-22 + 32 2^-21) + some
tens of roundings: kappa = (L + 128) 2^-21 for one recurrence and twice that
for gradients, which pass through two.  The convolution and the norm have a
fixed number of roundings per term (their exponentials' arguments stay below 16
in size): kappa = 64 * 2^-22 and, for sums over tokens (tree and chain of up
to some hundred), 512 * 2^-24."""
import numpy as np
import pytest
import torch

from fft_long_convolution_flashconv_b200 import api

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    torch.cuda.set_device(0)
    yield
    torch.cuda.synchronize()


def close(got, want, mag, kappa, what=""):
    g, w, m = got.detach().double().cpu(), want.detach().double(), mag.detach().double().abs()
    assert g.shape == w.shape, (what, g.shape, w.shape)
    step = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * step * 2  # half a step below the normal range, and its twin
    tol = step * w.abs() * (1 + kappa) + (1 + step) * kappa * m + tiny
    bad = ~((g - w).abs() <= tol)
    assert not bad.any(), (what, int(bad.sum()), float(((g - w).abs() / tol.clamp(min=1e-300))[bad].max()))


def rand(rng, *shape, std=1.0, dtype=torch.float32):
    return torch.tensor(rng.normal(0, std, shape), dtype=torch.float64).to(dtype)


def lens(rng, B, L):
    n = rng.integers(0, L + 1, B)
    n[0] = L
    if B > 1:
        n[1] = 0
    return torch.tensor(n, dtype=torch.int32)


def cu(t):
    return None if t is None else t.cuda()


# ------------------------------------------------------------------ short convolution
def conv_ref(x, w, bias, silu, past, n):
    """One batch row (H x L), n valid steps: y (H x L) and the last K-1 inputs."""
    H, L = x.shape
    K = w.shape[1]
    seq = torch.cat([past, x[:, :n]], 1)
    pre = torch.zeros(H, n, dtype=torch.float64) + (0 if bias is None else bias[:, None])
    for j in range(K):
        pre = pre + w[:, j:j + 1] * seq[:, K - 1 - j:K - 1 - j + n]
    y = pre * torch.sigmoid(pre) if silu else pre
    return torch.cat([y, torch.zeros(H, L - n, dtype=torch.float64)], 1), seq[:, n:]


def conv_case(B, H, L, K, dtype, silu, bias, state, ragged, seed):
    rng = np.random.default_rng(seed)
    d = DT[dtype]
    x = rand(rng, B, H, L, dtype=d)
    w = rand(rng, H, K, std=0.5)
    bi = rand(rng, H, std=0.5) if bias else None
    past = rand(rng, B, H, K - 1, dtype=d) if state else None
    dy, dso = rand(rng, B, H, L, dtype=d), rand(rng, B, H, K - 1, dtype=d)
    n = lens(rng, B, L) if ragged else None
    return x, w, bi, past, dy, dso, n


@pytest.mark.parametrize("B,H,L,K,dtype,silu,bias,state,ragged", [
    (2, 5, 1, 4, "f32", True, True, True, False),
    (3, 7, 2, 4, "f16", True, True, True, True),      # shorter than the window
    (2, 3, 8, 8, "bf16", False, False, True, True),
    (2, 3, 129, 1, "f32", True, True, False, True),   # one tap: no state
    (4, 6, 1000, 4, "bf16", True, True, True, True),
    (2, 4, 1025, 3, "f16", True, False, False, False),
    (1, 2, 2048, 8, "f32", False, True, True, False),
    (5, 300, 24, 5, "f16", True, True, True, True),
    (1, 1, 5000, 2, "f32", True, True, True, False),
    (3, 2, 64, 6, "f16", True, True, False, False),
    (2, 9, 77, 7, "bf16", True, True, True, True),
])
def test_short_conv(B, H, L, K, dtype, silu, bias, state, ragged):
    x, w, bi, past, dy, dso, n = conv_case(B, H, L, K, dtype, silu, bias, state, ragged, seed=L * 10 + K)
    # 64-bit reference, with gradients by torch's differentiation of the formula
    X, Wd = x.double().requires_grad_(), w.double().requires_grad_()
    bd = None if bi is None else bi.double().requires_grad_()
    Pd = (torch.zeros(B, H, K - 1, dtype=torch.float64) if past is None else past.double()).requires_grad_()
    ns = [L if n is None else int(n[b]) for b in range(B)]
    rows = [conv_ref(X[b], Wd, bd, silu, Pd[b], ns[b]) for b in range(B)]
    want, wstate = torch.stack([r[0] for r in rows]), torch.stack([r[1] for r in rows])
    loss = (want * dy.double()).sum() + (wstate * dso.double()).sum()
    leaves = [X, Wd, Pd] + ([bd] if bd is not None else [])
    gX, gW, gP, *gb = torch.autograd.grad(loss, leaves, allow_unused=True)
    zero = lambda g, like: torch.zeros_like(like) if g is None else g  # noqa: E731
    # magnitudes: |w| * |x|; silu' is below 1.1
    ab = [conv_ref(x[b].double().abs(), w.double().abs(), None if bi is None else bi.double().abs(), False,
                   Pd[b].detach().abs(), ns[b])[0] for b in range(B)]
    mag = torch.stack(ab)
    Xa, Wa = x.double().abs().requires_grad_(), w.double().abs().requires_grad_()
    Pa = Pd.detach().abs().requires_grad_()
    ra = [conv_ref(Xa[b], Wa, None, False, Pa[b], ns[b]) for b in range(B)]
    # dc's own error is relative to |dy| (1 + M) 1.1: fold (1 + M) in
    la = (torch.stack([r[0] for r in ra]) * dy.double().abs() * (1 + mag) * 1.1).sum() \
        + (torch.stack([r[1] for r in ra]) * dso.double().abs()).sum()
    mX, mW, mP = torch.autograd.grad(la, [Xa, Wa, Pa], allow_unused=True)

    wide = torch.full((B, 2 * H, L + 3), NAN, dtype=DT[dtype])  # x and dy as strided views
    wide[:, H:, :L] = x
    if n is not None:  # padding may hold anything
        for b in range(B):
            wide[b, :, ns[b]:] = NAN
            dy[b, :, ns[b]:] = NAN
    xv = wide.cuda()[:, H:, :L]
    kap = 64 * 2.0 ** -22
    y, s = api.short_conv_fwd(xv, w.cuda(), cu(bi), silu, cu(past), cu(n), return_state=True)
    close(y, want, mag * (1 + mag), kap, "y")
    assert torch.equal(s.cpu().double(), wstate.detach())
    dx, dw, db, dp = api.short_conv_bwd(dy.cuda(), xv, w.cuda(), cu(bi), silu, cu(past), cu(n), cu(dso),
                                        need_dstate_in=True)
    close(dx, zero(gX, X), zero(mX, Xa), kap, "dx")
    close(dp, zero(gP, Pd), zero(mP, Pa), kap, "dstate_in")
    close(dw, zero(gW, Wd), zero(mW, Wa), kap + 512 * 2.0 ** -24, "dw")
    if bi is not None:
        mb = (torch.nan_to_num(dy.double()).abs() * (1 + mag) * 1.1).sum((0, 2))
        close(db, zero(gb[0], bd), mb, kap + 512 * 2.0 ** -24, "dbias")
    else:
        assert db is None
    # the same call, the same bits
    again = api.short_conv_bwd(dy.cuda(), xv, w.cuda(), cu(bi), silu, cu(past), cu(n), cu(dso), need_dstate_in=True)
    for a, b in zip((dx, dw, db, dp), again):
        assert a is None or torch.equal(a, b)


def test_short_conv_many_rows_sum_over_splits():
    """Few channels and many rows: the weight gradient is joined from parts."""
    rng = np.random.default_rng(3)
    B, H, L, K = 6, 2, 4096, 4
    x, dy, w = rand(rng, B, H, L), rand(rng, B, H, L), rand(rng, H, K, std=0.5)
    X, Wd = x.double().requires_grad_(), w.double().requires_grad_()
    z = torch.zeros(H, K - 1, dtype=torch.float64)
    want = torch.stack([conv_ref(X[b], Wd, None, True, z, L)[0] for b in range(B)])
    gX, gW = torch.autograd.grad((want * dy.double()).sum(), [X, Wd])
    dx, dw, _ = api.short_conv_bwd(dy.cuda(), x.cuda(), w.cuda())
    # sums of 24576 terms of size about 1 in chains of at most some hundred: 512 * 2^-24 of the absolute sum
    close(dw, gW, torch.full_like(gW, float((dy.abs() * 1.1).sum() / H * 1.0)), 512 * 2.0 ** -24, "dw")
    close(dx, gX, torch.full_like(gX, 8.0), 64 * 2.0 ** -22, "dx")


@pytest.mark.parametrize("B,H,K,dtype,S", [(1, 5, 4, "f16", 1), (9, 130, 4, "bf16", 12), (3, 7, 1, "f32", 3),
                                           (20, 33, 8, "f32", 64)])
def test_short_conv_step(B, H, K, dtype, S):
    rng = np.random.default_rng(B * H)
    d = DT[dtype]
    wide = rand(rng, B, 2 * H, dtype=d)
    x, w, bi, state = wide[:, H:], rand(rng, H, K, std=0.5), rand(rng, H, std=0.5), rand(rng, S, H, K - 1, dtype=d)
    slots = None
    if S > B:
        sl = rng.permutation(S)[:B]
        if B > 4:
            sl[2], sl[3] = -1, S          # padded rows
            sl[4] = sl[0]                 # a slot that an earlier row holds: padded as well
        slots = torch.tensor(sl, dtype=torch.int32)
    dev = state.cuda()
    xd = wide.cuda()[:, H:]
    y = api.short_conv_step(xd, dev, w.cuda(), bi.cuda(), slots=cu(slots))
    want, wst, seen = torch.zeros(B, H, dtype=torch.float64), state.clone(), set()
    mag = torch.zeros(B, H, dtype=torch.float64)
    for b in range(B):
        s = b if slots is None else int(slots[b])
        if s < 0 or s >= S or s in seen:
            continue
        seen.add(s)
        r, _ = conv_ref(x[b].double()[:, None], w.double(), bi.double(), True, state[s].double(), 1)
        m, _ = conv_ref(x[b].double().abs()[:, None], w.double().abs(), bi.double().abs(), False,
                        state[s].double().abs(), 1)
        want[b], mag[b] = r[:, 0], m[:, 0] * (1 + m[:, 0])
        wst[s] = torch.cat([state[s], x[b][:, None]], 1)[:, 1:]
    close(y, want, mag, 64 * 2.0 ** -22, "y")
    assert torch.equal(dev.cpu(), wst)


# ------------------------------------------------------------------ selective scan
def scan_ref(u, dta, dtb, A, Bt, Ct, D, act, x0, ns):
    """Step by step; dta: the step size in the decay, dtb: in the input term.  Returns (y, state)."""
    B, H, L = u.shape
    N, E = A.shape[1], H // Bt.shape[1]
    ys, xs = [], []
    for b in range(B):
        x, row = x0[b], []
        Bh, Ch = Bt[b].repeat_interleave(E, 0), Ct[b].repeat_interleave(E, 0)  # H x N x L
        for t in range(ns[b]):
            x = torch.exp(dta[b, :, t, None] * A) * x + (dtb[b, :, t] * u[b, :, t])[:, None] * Bh[..., t]
            row.append((x * Ch[..., t]).sum(-1) + (D * u[b, :, t] if D is not None else 0))
        row = torch.stack(row, -1) if row else torch.zeros(H, 0, dtype=torch.float64)
        if act is not None:
            row = row * act[b, :, :ns[b]]
        ys.append(torch.cat([row, torch.zeros(H, L - ns[b], dtype=torch.float64)], -1))
        xs.append(x)
    return torch.stack(ys), torch.stack(xs)


def scan_case(B, H, L, N, G, dtype, seed, opts):
    rng = np.random.default_rng(seed)
    d = DT[dtype]
    c = dict(u=rand(rng, B, H, L, dtype=d), delta=rand(rng, B, H, L, std=0.7, dtype=d),
             Bt=rand(rng, B, G, N, L, dtype=d), Ct=rand(rng, B, G, N, L, dtype=d),
             A=-torch.tensor(np.arange(1, N + 1) * np.exp(rng.normal(0, 0.1, (H, N))), dtype=torch.float32),
             D=rand(rng, H) if "D" in opts else None,
             dt_bias=torch.tensor(rng.uniform(-6, -2, H), dtype=torch.float32) if "bias" in opts else None,
             z=rand(rng, B, H, L, dtype=d) if "gate" in opts else None,
             x0=rand(rng, B, H, N) if "state" in opts else None,
             n=lens(rng, B, L) if "ragged" in opts else None,
             dy=rand(rng, B, H, L, dtype=d), dso=rand(rng, B, H, N), softplus="raw" not in opts)
    if "raw" in opts:  # step sizes given directly
        c["delta"] = torch.tensor(rng.uniform(0.001, 0.3, (B, H, L)), dtype=torch.float64).to(d)
    return c


def wide_view(t, pad, fill=NAN):
    """t (its values on the GPU) as a view of a wider tensor: odd strides, NaN around it."""
    shape = list(t.shape)
    shape[1] += 1
    shape[-1] += pad
    w = torch.full(shape, fill, dtype=t.dtype)
    w[:, 1:, ..., :t.shape[-1]] = t
    return w.cuda()[:, 1:, ..., :t.shape[-1]]


SCANS = [
    (1, 1, 1, 1, 1, "f32", ("D", "bias")),
    (2, 3, 1, 16, 1, "f16", ("D", "bias", "gate", "state", "ragged")),
    (2, 6, 7, 4, 2, "f32", ("D", "bias", "gate", "state", "ragged")),
    (3, 18, 64, 16, 1, "bf16", ("D", "bias", "gate")),
    (2, 40, 65, 5, 2, "f32", ("bias", "state", "ragged")),
    (2, 17, 130, 16, 1, "f16", ("D", "bias", "gate", "state")),
    (1, 33, 200, 17, 1, "f32", ("D", "state", "raw")),
    (4, 8, 127, 33, 4, "bf16", ("D", "bias", "gate", "state", "ragged")),
    (1, 4, 300, 64, 1, "f32", ("D", "bias", "gate", "state", "ragged")),
    (1, 2, 40, 256, 2, "f16", ("D", "bias", "state")),
    (1, 70, 520, 16, 1, "f16", ("D", "bias", "gate", "state", "ragged")),
    (2, 16, 513, 8, 1, "bf16", ("D", "bias", "gate", "state")),
]


def scan_want(c, grads=True):
    """Reference outputs, gradients and their magnitudes (64 bits, CPU)."""
    B, H, L = c["u"].shape
    ns = [L if c["n"] is None else int(c["n"][b]) for b in range(B)]
    leaf = lambda k: None if c[k] is None else c[k].double().requires_grad_()  # noqa: E731
    u, delta, A, Bt, Ct, D, bias, z = (leaf(k) for k in ("u", "delta", "A", "Bt", "Ct", "D", "dt_bias", "z"))
    N = A.shape[1]
    x0 = torch.zeros(B, H, N, dtype=torch.float64).requires_grad_() if c["x0"] is None else leaf("x0")
    raw = delta + (0 if bias is None else bias[:, None])
    dt = torch.log1p(torch.exp(raw)) if c["softplus"] else raw
    act = None if z is None else z * torch.sigmoid(z)
    y, x = scan_ref(u, dt, dt, A, Bt, Ct, D, act, x0, ns)
    names = [("du", u), ("ddelta", delta), ("dA", A), ("dB", Bt), ("dC", Ct), ("dD", D), ("ddt_bias", bias), ("dz", z),
             ("dstate_in", x0)]
    out = {"y": y, "state": x}
    if grads:
        loss = (y * c["dy"].double()).sum() + (x * c["dso"].double()).sum()
        have = [(k, v) for k, v in names if v is not None]
        for (k, v), g in zip(have, torch.autograd.grad(loss, [v for _, v in have], allow_unused=True)):
            out[k] = torch.zeros_like(v) if g is None else g
    # magnitudes: the same sums over absolute values
    pos = lambda t: t.detach().abs().requires_grad_()  # noqa: E731
    ua, Ba, Ca, xa, dta, dtb = pos(u), pos(Bt), pos(Ct), pos(x0), dt.detach().clone().requires_grad_(), pos(dt)
    Da = None if D is None else pos(D)
    Aa = A.detach().clone().requires_grad_()
    aa = None if act is None else pos(act)
    ya, sa = scan_ref(ua, dta, dtb, Aa, Ba, Ca, Da, aa, xa, ns)
    mag = {"y": ya, "state": sa}
    if grads:
        la = (ya * c["dy"].double().abs()).sum() + (sa * c["dso"].double().abs()).sum()
        vs = [ua, dta, dtb, Aa, Ba, Ca, xa] + [v for v in (Da, aa) if v is not None]
        gs = dict(zip([id(v) for v in vs], torch.autograd.grad(la, vs, allow_unused=True)))
        get = lambda v: torch.zeros_like(v) if gs[id(v)] is None else gs[id(v)].abs()  # noqa: E731
        ds = torch.sigmoid(raw.detach()) if c["softplus"] else torch.ones_like(raw)
        mag.update(du=get(ua), ddelta=(get(dta) + get(dtb)) * ds, dA=get(Aa), dB=get(Ba), dC=get(Ca), dstate_in=get(xa))
        mag["ddt_bias"] = mag["ddelta"].sum((0, 2))
        if D is not None:
            mag["dD"] = get(Da)
        if z is not None:
            mag["dz"] = get(aa) * 1.1  # |silu'| < 1.1
            # silu's own error: relative 2^-20 of a value that multiplies y
    return out, mag


def kappa(L, grads=False):
    return (L + 128) * 2.0 ** -21 * (2 if grads else 1)


def call_fwd(c, view=True, **kw):
    f = (lambda t, pad=3: None if t is None else wide_view(t, pad)) if view else (lambda t, pad=0: cu(t))
    args = dict(u=f(c["u"]), delta=f(c["delta"], 0), z=f(c["z"], 1), Bt=f(c["Bt"], 2), Ct=f(c["Ct"]))
    if view and args["Bt"] is not None:
        args["Ct"] = cu(c["Ct"])
    y = api.selective_scan_fwd(args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"], cu(c["D"]),
                               cu(c["dt_bias"]), args["z"], c["softplus"], cu(c["x0"]), cu(c["n"]), **kw)
    return args, y


def poison(c):
    """NaN behind every row's end."""
    p = dict(c)
    if c["n"] is not None:
        for k in ("u", "delta", "z", "dy", "Bt", "Ct"):
            if c[k] is not None:
                p[k] = c[k].clone()
                for b in range(len(c["n"])):
                    p[k][b, ..., int(c["n"][b]):] = NAN
    return p


@pytest.mark.parametrize("B,H,L,N,G,dtype,opts", SCANS)
def test_selective_scan(B, H, L, N, G, dtype, opts):
    c = scan_case(B, H, L, N, G, dtype, B * 1000 + L, opts)
    want, mag = scan_want(c)
    p = poison(c)
    args, (y, state, ckpt) = call_fwd(p, return_state=True, return_ckpt=True)
    close(y, want["y"], mag["y"], kappa(L), "y")
    close(state, want["state"], mag["state"], kappa(L), "state")
    got = api.selective_scan_bwd(p["dy"].cuda(), args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"], ckpt,
                                 cu(c["D"]), cu(c["dt_bias"]), args["z"], c["softplus"], cu(c["n"]), cu(c["dso"]),
                                 need_dstate_in=True)
    for k, g in zip(("du", "ddelta", "dA", "dB", "dC", "dD", "ddt_bias", "dz", "dstate_in"), got):
        if g is None:
            assert k not in want
        else:
            close(g, want[k], mag[k], kappa(L, True), k)
    again = api.selective_scan_bwd(p["dy"].cuda(), args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"],
                                   ckpt, cu(c["D"]), cu(c["dt_bias"]), args["z"], c["softplus"], cu(c["n"]),
                                   cu(c["dso"]), need_dstate_in=True)
    for a, b in zip(got, again):
        assert a is None or torch.equal(a, b)


def test_selective_scan_gradient_against_differences():
    """Directional derivatives of the 64-bit forward by central differences against the kernel's gradients."""
    c = scan_case(2, 6, 70, 8, 2, "f32", 5, ("D", "bias", "gate", "state"))
    args, (y, ckpt) = call_fwd(c, view=False, return_ckpt=True)
    got = api.selective_scan_bwd(c["dy"].cuda(), args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"], ckpt,
                                 cu(c["D"]), cu(c["dt_bias"]), args["z"], dstate_out=c["dso"].cuda(),
                                 need_dstate_in=True)
    keys = ("u", "delta", "A", "Bt", "Ct", "D", "dt_bias", "z", "x0")
    rng = np.random.default_rng(1)

    def loss(e, k, v):
        q = {kk: (t.double() if torch.is_tensor(t) and t.is_floating_point() else t) for kk, t in c.items()}
        q[k] = q[k] + e * v
        dt = torch.log1p(torch.exp(q["delta"] + q["dt_bias"][:, None]))
        yy, xx = scan_ref(q["u"], dt, dt, q["A"], q["Bt"], q["Ct"], q["D"], q["z"] * torch.sigmoid(q["z"]), q["x0"],
                          [70, 70])
        return float((yy * q["dy"]).sum() + (xx * q["dso"]).sum())

    for k, g in zip(keys, got):
        v = torch.tensor(rng.normal(size=tuple(c[k].shape)))
        e = 1e-5
        diff = (loss(e, k, v) - loss(-e, k, v)) / (2 * e)
        have = g.double().cpu()
        # differences: e^2 times third derivatives and 2^-52 |loss| / e, both below 1e-7 of the terms' sum
        tol = (kappa(70, True) + 1e-6) * float((have * v).abs().sum()) + 1e-6
        assert abs(diff - float((have * v).sum())) <= tol, k


@pytest.mark.parametrize("B,H,N,G,dtype,S,opts", [
    (1, 5, 16, 1, "f32", 1, ("D", "bias", "gate")), (9, 40, 16, 2, "bf16", 12, ("D", "bias", "gate")),
    (3, 7, 5, 1, "f16", 3, ("bias",)), (20, 34, 64, 2, "f32", 64, ("D", "bias", "gate")),
    (6, 3, 200, 1, "f32", 8, ("D", "raw")), (2, 130, 1, 1, "f16", 2, ("D", "bias", "gate")),
])
def test_selective_scan_step(B, H, N, G, dtype, S, opts):
    c = scan_case(B, H, 1, N, G, dtype, S + N, opts)
    rng = np.random.default_rng(N)
    state = rand(rng, S, H, N)
    slots = None
    if S > B:
        sl = rng.permutation(S)[:B]
        if B > 4:
            sl[2], sl[3], sl[4] = -7, S, sl[0]
        slots = torch.tensor(sl, dtype=torch.int32)
    seen, live = set(), []
    for b in range(B):
        s = b if slots is None else int(slots[b])
        live.append(0 <= s < S and s not in seen)
        seen.add(s)
    c["x0"] = torch.stack([state[(b if slots is None else int(slots[b])) if live[b] else 0] for b in range(B)])
    want, mag = scan_want(c, grads=False)
    dev = state.cuda()
    tok = lambda t: None if t is None else t[..., 0].cuda()  # noqa: E731
    wide = torch.full((B, 2 * H), NAN, dtype=DT[dtype])
    wide[:, :H] = c["u"][..., 0]
    y = api.selective_scan_step(wide.cuda()[:, :H], tok(c["delta"]), c["A"].cuda(), c["Bt"].cuda()[..., 0],
                                tok(c["Ct"]), dev, cu(c["D"]), cu(c["dt_bias"]), tok(c["z"]), c["softplus"], cu(slots))
    ok = torch.tensor(live)
    close(y, torch.where(ok[:, None], want["y"][..., 0].detach(), torch.zeros(())), mag["y"][..., 0], kappa(1), "y")
    wst, mst = state.double(), state.double().abs()
    for b in range(B):
        if live[b]:
            wst[b if slots is None else int(slots[b])] = want["state"][b].detach()
            mst[b if slots is None else int(slots[b])] = mag["state"][b].detach()
    close(dev, wst, mst, kappa(1), "state")
    untouched = [s for s in range(S) if s not in {b if slots is None else int(slots[b]) for b in range(B) if live[b]}]
    assert torch.equal(dev.cpu()[untouched], state[untouched])


def test_scan_in_pieces_and_by_tokens_equals_whole():
    """One sequence whole, in two calls joined by the state, and token by token."""
    c = scan_case(2, 20, 96, 16, 1, "f32", 9, ("D", "bias", "gate"))
    want, mag = scan_want(c, grads=False)
    rng = np.random.default_rng(4)
    w, bi = rand(rng, 20, 4, std=0.5).cuda(), rand(rng, 20, std=0.1).cuda()
    a = {k: c[k].cuda() for k in ("u", "delta", "z", "Bt", "Ct", "A", "D", "dt_bias")}
    cut = 41
    ys, state = [], None
    for lo, hi in ((0, cut), (cut, 96)):
        y, state = api.selective_scan_fwd(a["u"][..., lo:hi], a["delta"][..., lo:hi], a["A"], a["Bt"][..., lo:hi],
                                          a["Ct"][..., lo:hi], a["D"], a["dt_bias"], a["z"][..., lo:hi],
                                          state_in=state, return_state=True)
        ys.append(y)
    close(torch.cat(ys, -1), want["y"], mag["y"], kappa(96), "pieces")
    close(state, want["state"], mag["state"], kappa(96), "state")
    x = torch.zeros(2, 20, 16, device="cuda")
    ring = torch.zeros(2, 20, 3, device="cuda")
    whole = api.short_conv_fwd(a["u"], w, bi)
    for t in range(96):
        tok = [v[..., t].contiguous() for v in (a["u"], a["delta"], a["z"], a["Bt"], a["Ct"])]
        y = api.selective_scan_step(tok[0], tok[1], a["A"], tok[3], tok[4], x, a["D"], a["dt_bias"], tok[2])
        close(y, want["y"][..., t], mag["y"][..., t], kappa(96), f"token {t}")
        assert torch.allclose(api.short_conv_step(tok[0], ring, w, bi), whole[..., t], atol=1e-5, rtol=0)


# ------------------------------------------------------------------ group norm with SiLU
def norm_ref(x, G, w, bias, gate, eps):
    """x, gate: B x L x C."""
    B, L, C = x.shape
    xs = x.reshape(B, L, G, C // G)
    mean = xs.mean(-1, keepdim=True)
    xh = ((xs - mean) / torch.sqrt(((xs - mean) ** 2).mean(-1, keepdim=True) + eps)).reshape(B, L, C)
    n = xh * (1 if w is None else w) + (0 if bias is None else bias)
    v = n if gate is None else gate
    return n * torch.sigmoid(v) * (1 if gate is None else gate), xh, n


@pytest.mark.parametrize("cm", [False, True])
@pytest.mark.parametrize("B,L,C,G,dtype,opts", [
    (1, 1, 1, 1, "f32", ("w", "b")),
    (2, 3, 10, 2, "f32", ("w", "b", "gate")),      # groups of 5
    (2, 64, 128, 2, "f16", ("w", "b")),
    (1, 65, 768, 12, "bf16", ("w", "b", "gate")),
    (3, 70, 96, 4, "f16", ("w", "gate")),          # groups of 24
    (2, 40, 200, 1, "f32", ("b",)),
    (1, 20, 520, 2, "f16", ("w", "b", "gate")),    # groups of 260
    (1, 9, 1100, 1, "f32", ("w", "b", "gate")),
    (2, 5, 2050, 1, "bf16", ()),
    (1, 3, 8192, 1, "f32", ("w", "b", "gate")),
    (4, 300, 64, 1, "f16", ("w", "b", "gate")),
    (1, 33, 36, 3, "f32", ("w", "b")),             # groups of 12
    (1, 1, 64, 1, "f16", ("w", "b", "gate")),      # one group: most of its block has nothing to do
    (1, 3, 32, 2, "f32", ("w", "b")),
    (2, 128, 32, 1, "bf16", ("w", "b", "gate")),   # whole tiles of tokens and channels
    (1, 192, 256, 2, "f16", ("w", "b")),
    (1, 64, 512, 2, "f32", ("w", "gate")),
    (2, 256, 128, 2, "f16", ("w", "b", "gate")),
])
def test_group_norm_act(B, L, C, G, dtype, opts, cm):
    rng = np.random.default_rng(C + L)
    d, eps = DT[dtype], 1e-5
    x, dy = rand(rng, B, L, C, std=1.5, dtype=d), rand(rng, B, L, C, dtype=d)
    gate = rand(rng, B, L, C, dtype=d) if "gate" in opts else None
    w = 1 + rand(rng, C, std=0.2) if "w" in opts else None
    bias = rand(rng, C, std=0.2) if "b" in opts else None
    leaf = lambda t: None if t is None else t.double().requires_grad_()  # noqa: E731
    X, Wd, bd, gd = leaf(x), leaf(w), leaf(bias), leaf(gate)
    want, xh, n = norm_ref(X, G, Wd, bd, gd, eps)
    have = [t for t in (X, Wd, bd, gd) if t is not None]
    gr = dict(zip([id(t) for t in have], torch.autograd.grad((want * dy.double()).sum(), have)))
    lay = (lambda t: None if t is None else t.transpose(1, 2).contiguous().cuda()) if cm else cu
    kw = dict(weight=cu(w), bias=cu(bias), gate=lay(gate), channel_major=cm)
    # n's error: a few roundings of (|x| + |mean|) rstd |w| + |bias|; silu and its slope are below 1.1 (1 + |.|)
    M = C // G
    xs = x.double().reshape(B, L, G, M)
    rstd = 1 / torch.sqrt(xs.var(-1, unbiased=False, keepdim=True) + eps)
    mxh = ((xs.abs() + xs.abs().mean(-1, keepdim=True)) * rstd).reshape(B, L, C)
    mn = mxh * (1 if w is None else w.double().abs()) + (0 if bias is None else bias.double().abs())
    ga = None if gate is None else gate.double().abs()
    fac = 1.1 * (1 + mn) if gate is None else 1.1 * ga
    kap = 64 * 2.0 ** -22
    y = api.group_norm_act_fwd(lay(x), G, **kw)
    close(y, want, mn * fac, kap, "y")
    dx, dw, db, dg = api.group_norm_act_bwd(dy.cuda(), lay(x), G, **kw)
    back = (lambda t: t.transpose(1, 2)) if cm else (lambda t: t)
    # |dn| <= |dy| fac'; each of dx's three terms is below rstd (|e| + mean|e| (1 + |xh| |xh'|))
    dnm = dy.double().abs() * 1.1 * ((1 + mn) if gate is None else ga)
    e = (dnm * (1 if w is None else w.double().abs())).reshape(B, L, G, M)
    h = mxh.reshape(B, L, G, M)
    mdx = (rstd * (e + e.mean(-1, keepdim=True) + h * (e * h).mean(-1, keepdim=True))).reshape(B, L, C)
    close(back(dx), gr[id(X)], mdx, 2 * kap, "dx")
    for g, leaf_, m, name in ((dw, Wd, (dnm * mxh).sum((0, 1)), "dw"), (db, bd, dnm.sum((0, 1)), "dbias")):
        assert (g is None) == (leaf_ is None)
        if g is not None:
            close(g, gr[id(leaf_)], m, kap + 512 * 2.0 ** -24, name)
    assert (dg is None) == (gate is None)
    if dg is not None:
        close(back(dg), gr[id(gd)], dy.double().abs() * mn * 1.1, 2 * kap, "dgate")
    again = api.group_norm_act_bwd(dy.cuda(), lay(x), G, **kw)
    for a, b in zip((dx, dw, db, dg), again):
        assert a is None or torch.equal(a, b)


def test_group_norm_constant_and_large_offset():
    """A group of equal values (variance 0) and values far from zero next to their spread."""
    x = torch.full((1, 4, 64), 3.0)
    x[0, 1] = 1000 + torch.arange(64) / 64.0
    y = api.group_norm_act_fwd(x.cuda(), 1)
    want, _, _ = norm_ref(x.double(), 1, None, None, None, 1e-5)
    assert torch.equal(y[0, 0].cpu(), torch.zeros(64))
    # xh's error: 2^-24 * 1000 / 0.29 from the mean's rounding, silu' < 1.1
    assert float((y.cpu().double() - want).abs().max()) < 1.1 * 8 * 2.0 ** -24 * 1000 / 0.28


# ------------------------------------------------------------------ the operators together
def _block(p, x, lengths, state=None, need=False):
    """A gated selective-SSM block: convolution, scan, norm by heads (token-major)."""
    conv_s, scan_s = state if state is not None else (None, None)
    c, cs = api.short_conv_fwd(x, p["w"], p["cb"], state_in=conv_s, lengths=lengths, return_state=True)
    y, ss, ck = api.selective_scan_fwd(c, p["delta"], p["A"], p["Bt"], p["Ct"], p["D"], p["dtb"], state_in=scan_s,
                                       lengths=lengths, return_state=True, return_ckpt=True)
    o = api.group_norm_act_fwd(y, p["G"], p["nw"], p["nb"], p["z"], channel_major=True)
    return (o, (cs, ss), (c, y, ck)) if need else (o, (cs, ss))


def _block_case(dtype, B, H, L, N):
    rng = np.random.default_rng(17)
    d = DT[dtype]
    p = dict(w=rand(rng, H, 4, std=0.5), cb=rand(rng, H, std=0.1), delta=rand(rng, B, H, L, std=0.5, dtype=d),
             A=-torch.arange(1, N + 1).float().repeat(H, 1), Bt=rand(rng, B, 1, N, L, dtype=d),
             Ct=rand(rng, B, 1, N, L, dtype=d), D=rand(rng, H), dtb=torch.full((H,), -3.0), z=rand(rng, B, H, L, dtype=d),
             nw=1 + rand(rng, H, std=0.1), nb=rand(rng, H, std=0.1), G=2)
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in p.items()}, rand(rng, B, H, L, dtype=d).cuda()


def test_block_trains_and_generates():
    """Forward and backward of the block in fp32 against 64-bit differentiation, then generation from its states."""
    B, H, L, N = 2, 24, 50, 8
    p, x = _block_case("f32", B, H, L + 6, N)
    lengths = torch.tensor([50, 31], dtype=torch.int32, device="cuda")
    first = {k: (v[..., :L] if torch.is_tensor(v) and v.dim() > 2 else v) for k, v in p.items()}
    first["z"] = first["z"].contiguous()
    o, (cs, ss), (c, y, ck) = _block(first, x[..., :L], lengths, need=True)
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(0)).cuda()
    gy, gnw, gnb, gz = api.group_norm_act_bwd(do, y, 2, p["nw"], p["nb"], first["z"], channel_major=True)
    gc, gd, gA, gB, gC, gD, gdtb, _ = api.selective_scan_bwd(gy, c, first["delta"], p["A"], first["Bt"], first["Ct"],
                                                            ck, p["D"], p["dtb"], lengths=lengths)
    gx, gw, gcb = api.short_conv_bwd(gc, x[..., :L], p["w"], p["cb"], lengths=lengths)
    q = {k: v.double().cpu().requires_grad_() if torch.is_tensor(v) else v for k, v in first.items()}
    X = x[..., :L].double().cpu().requires_grad_()
    ns = lengths.tolist()
    past = torch.zeros(H, 3, dtype=torch.float64)
    cr = torch.stack([conv_ref(X[b], q["w"], q["cb"], True, past, ns[b])[0] for b in range(B)])
    dt = torch.log1p(torch.exp(q["delta"] + q["dtb"][:, None]))
    yr, _ = scan_ref(cr, dt, dt, q["A"], q["Bt"], q["Ct"], q["D"], None, torch.zeros(B, H, N, dtype=torch.float64), ns)
    orf, _, _ = norm_ref(yr.transpose(1, 2), 2, q["nw"], q["nb"], q["z"].transpose(1, 2), 1e-5)
    leaves = [X, q["w"], q["cb"], q["delta"], q["A"], q["Bt"], q["Ct"], q["D"], q["dtb"], q["nw"], q["nb"], q["z"]]
    refs = torch.autograd.grad((orf * do.double().cpu()).sum(), leaves)
    # rows behind a sequence's end have variance 0: rstd = 316, so fp32 roundings of zeros stay zeros; elsewhere
    # three operators of kappa <= 2 (50 + 128) 2^-21 each, against each gradient's largest value with a factor 8 for
    # the cancellation in sums of about a hundred terms of mixed sign
    tol = 3 * 2 * (L + 128) * 2.0 ** -21 * 8
    for g, r in zip((gx, gw, gcb, gd, gA, gB, gC, gD, gdtb, gnw, gnb, gz), refs):
        assert float((g.double().cpu() - r).abs().max()) <= tol * float(r.abs().max())
    assert float((o.double().cpu() - orf.detach()).abs().max()) <= tol * float(orf.detach().abs().max())
    # generation: six tokens a row from the prompt's states, against one run over prompt and tokens
    for b in range(B):
        n = ns[b]
        row = {k: (torch.cat([v[b:b + 1, ..., :n], v[b:b + 1, ..., L:]], -1).contiguous()
                   if torch.is_tensor(v) and v.dim() > 2 else v) for k, v in p.items()}
        xr = torch.cat([x[b:b + 1, :, :n], x[b:b + 1, :, L:]], -1).contiguous()
        whole, _ = _block(row, xr, None)
        cst, sst = cs[b:b + 1].clone(), ss[b:b + 1].clone()
        for t in range(n, n + 6):
            ct = api.short_conv_step(xr[..., t].contiguous(), cst, p["w"], p["cb"])
            yt = api.selective_scan_step(ct, row["delta"][..., t].contiguous(), p["A"], row["Bt"][..., t],
                                         row["Ct"][..., t], sst, p["D"], p["dtb"])
            ot = api.group_norm_act_fwd(yt[:, None], 2, p["nw"], p["nb"], row["z"][:, None, :, t].contiguous())
            assert float((ot[:, 0] - whole[:, t]).abs().max()) <= tol * float(whole.abs().max())


def test_block_in_a_graph_on_another_stream():
    """Captured and replayed on new inputs, and run on a side stream: the same bits as eager calls."""
    p, x = _block_case("f16", 2, 32, 200, 16)
    p["z"] = p["z"].contiguous()
    static = x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        warm, _ = _block(p, static, None)
    torch.cuda.current_stream().wait_stream(s)
    eager, _ = _block(p, x, None)
    assert torch.equal(warm, eager)
    dy = torch.randn(eager.shape, device="cuda").half()

    def step():
        o, _, (c, y, ck) = _block(p, static, None, need=True)
        gy, gw, _, _ = api.group_norm_act_bwd(dy, y, 2, p["nw"], p["nb"], p["z"], channel_major=True)
        gc, *g = api.selective_scan_bwd(gy, c, p["delta"], p["A"], p["Bt"], p["Ct"], ck, p["D"], p["dtb"])
        gx, gk, _ = api.short_conv_bwd(gc, static, p["w"], p["cb"])
        return [o, gw, gx, gk, *[t for t in g if t is not None]]

    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for k in range(2):
        static.copy_(x * (k + 1) * 0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a, b)


def test_decode_in_a_graph():
    """The step calls captured with a slot map that changes between replays."""
    B, H, N, S = 4, 24, 16, 6
    c = scan_case(B, H, 1, N, 1, "bf16", 3, ("D", "bias", "gate"))
    tok = [c[k][..., 0].contiguous().cuda() for k in ("u", "delta", "Bt", "Ct", "z")]
    A, D, bias = c["A"].cuda(), c["D"].cuda(), c["dt_bias"].cuda()
    pool = torch.randn(S, H, N, device="cuda")
    slots = torch.tensor([3, -1, 0, 5], dtype=torch.int32, device="cuda")
    run = lambda st: api.selective_scan_step(tok[0], tok[1], A, tok[2], tok[3], st, D, bias, tok[4], slots=slots)  # noqa: E731
    run(pool.clone())
    torch.cuda.synchronize()
    live = pool.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = run(live)
    for sl in ([3, -1, 0, 5], [1, 2, 1, 4]):
        slots.copy_(torch.tensor(sl, dtype=torch.int32))
        live.copy_(pool)
        graph.replay()
        eager = pool.clone()
        ye = run(eager)
        assert torch.equal(y, ye) and torch.equal(live, eager)


def test_offsets_past_31_bits():
    """A B x H x L beyond 2^31 elements: the last row of the convolution and of the norm."""
    B, H, L = 2, 1056, 1 << 20  # 2.2e9 elements
    x = torch.zeros(B, H, L, dtype=torch.float16, device="cuda")
    w = torch.full((H, 4), 0.25, device="cuda")
    x[1, H - 1] = torch.randn(L, generator=torch.Generator("cuda").manual_seed(1), device="cuda").half()
    y = api.short_conv_fwd(x, w)
    want = api.short_conv_fwd(x[1:, H - 1:], w[:1])
    assert torch.equal(y[1, H - 1], want[0, 0]) and not bool(y[0].any())
    del y
    A = torch.full((H, 1), -1.0, device="cuda")
    ones = torch.ones(B, 1, 1, L, dtype=torch.float16, device="cuda")
    s, state = api.selective_scan_fwd(x, x, A, ones, ones, return_state=True)
    one, ostate = api.selective_scan_fwd(x[1:, H - 1:], x[1:, H - 1:], A[:1], ones[1:], ones[1:], return_state=True)
    # Other sizes may be cut into other segments, so the bits may differ.  With dt about 0.8 and A = -1 what is more
    # than 128 steps old is below e^-100; states stay below 10.
    # Both sides are rounded, half a step (2^-11 in fp16) each: together one step of the value, besides kappa * 10.
    w = one[0, 0].double()
    assert bool(((s[1, H - 1].double() - w).abs() <= 2 * 2.0 ** -11 * w.abs() * (1 + kappa(128)) + kappa(128) * 10).all())
    assert float((state[1, H - 1] - ostate[0, 0]).abs().max()) <= kappa(128) * 10


# ------------------------------------------------------------------ long rows, other callers' ways
@pytest.mark.parametrize("B,H,L,N,G,dtype", [(3, 5, 1000, 16, 1, "f32"), (2, 34, 777, 20, 2, "f16"),
                                             (1, 1, 1500, 3, 1, "bf16")])
def test_scan_in_segments(B, H, L, N, G, dtype):
    """Few channels and many steps: rows are cut into segments; lengths end in the first, a middle and the last one."""
    assert api.selective_scan_workspace_bytes(B, H, L, N, G) > 0
    c = scan_case(B, H, L, N, G, dtype, 77, ("D", "bias", "gate", "state", "ragged"))
    if B == 3:
        c["n"] = torch.tensor([L, 70, 530], dtype=torch.int32)
    # decays down to e^-1 over the whole row, so that segments matter to one another
    c["dt_bias"] = torch.full((H,), -7.0)
    want, mag = scan_want(c)
    p = poison(c)
    args, (y, state, ckpt) = call_fwd(p, return_state=True, return_ckpt=True)
    close(y, want["y"], mag["y"], kappa(L), "y")
    close(state, want["state"], mag["state"], kappa(L), "state")
    got = api.selective_scan_bwd(p["dy"].cuda(), args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"], ckpt,
                                 cu(c["D"]), cu(c["dt_bias"]), args["z"], True, cu(c["n"]), cu(c["dso"]),
                                 need_dstate_in=True)
    for k, g in zip(("du", "ddelta", "dA", "dB", "dC", "dD", "ddt_bias", "dz", "dstate_in"), got):
        close(g, want[k], mag[k], kappa(L, True), k)


def test_scan_extreme_step_sizes_and_gates():
    """Step sizes from e^-30 to 30 (a decays to nothing, or not at all), gates of +-100."""
    c = scan_case(2, 8, 90, 8, 1, "f32", 21, ("D", "gate", "state"))
    rng = np.random.default_rng(8)
    c["delta"] = torch.tensor(rng.uniform(-30, 30, (2, 8, 90)), dtype=torch.float32)
    c["z"] = torch.tensor(rng.choice([-100.0, -20.0, 0.0, 20.0, 100.0], (2, 8, 90)), dtype=torch.float32)
    want, mag = scan_want(c)
    args, (y, state, ckpt) = call_fwd(c, return_state=True, return_ckpt=True)
    # a's argument |dt A| goes up to 30 * 11: where a is above 2^-126 its relative error is below 88 * 2^-21 a step,
    # and only one such step can be in a term that is above e^-88; exp(-x) for a gate of -100 is zero or below 2^-126
    k = kappa(90) + 2 * 88 * 2.0 ** -21
    close(y, want["y"], mag["y"] + 2.0 ** -100, k, "y")
    close(state, want["state"], mag["state"], k, "state")
    got = api.selective_scan_bwd(c["dy"].cuda(), args["u"], args["delta"], c["A"].cuda(), args["Bt"], args["Ct"], ckpt,
                                 cu(c["D"]), None, args["z"], dstate_out=cu(c["dso"]), need_dstate_in=True)
    for name, g in zip(("du", "ddelta", "dA", "dB", "dC", "dD", None, "dz", "dstate_in"), got):
        if name:
            # silu' of +-100 is 1 or below e^-99 * 100: its own error is covered by an absolute 2^-100
            close(g, want[name], mag[name] + 2.0 ** -100, 2 * k, name)


def test_expanded_inputs_given_outputs_and_workspaces():
    c = scan_case(3, 12, 700, 8, 1, "f16", 5, ("D", "bias", "gate"))
    one = {k: c[k].cuda() for k in ("u", "delta", "A", "Bt", "Ct", "D", "dt_bias", "z")}
    args = (one["u"], one["delta"], one["A"], one["Bt"][:1].expand(3, 1, 8, 700), one["Ct"][:1].expand(3, 1, 8, 700),
            one["D"], one["dt_bias"], one["z"])
    dense = [a.contiguous() for a in args]
    want = api.selective_scan_fwd(*dense)
    out = torch.full_like(want, NAN)
    need = api.selective_scan_workspace_bytes(3, 12, 700, 8, 1)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    y = api.selective_scan_fwd(*args, workspace=ws, out=out)
    assert y.data_ptr() == out.data_ptr() and torch.equal(y, want)
    if need:
        with pytest.raises(Exception, match="workspace too small"):
            api.selective_scan_fwd(*args, workspace=ws[:need - 1].clone())
    with pytest.raises(ValueError, match="out"):
        api.selective_scan_fwd(*args, out=out[:, :, :-1])
    with pytest.raises(Exception, match="16-byte"):
        api.selective_scan_fwd(*args, out=torch.empty(want.numel() + 1, dtype=want.dtype, device="cuda")[1:].view_as(want))
    x = one["u"][:, :1].expand(3, 12, 700)  # one channel for all, by stride
    w = torch.randn(12, 4, device="cuda")
    assert torch.equal(api.short_conv_fwd(x, w), api.short_conv_fwd(x.contiguous(), w))
    dy = torch.randn(3, 12, 1, device="cuda").half().expand(3, 12, 700)
    with pytest.raises(ValueError, match="last axis"):
        api.short_conv_bwd(dy, x, w)
    bw = torch.empty(api.short_conv_bwd_workspace_bytes(3, 12, 700, 4), dtype=torch.uint8, device="cuda")
    a = api.short_conv_bwd(dy.contiguous(), x, w, workspace=bw)
    b = api.short_conv_bwd(dy.contiguous(), x.contiguous(), w)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_a_batch_of_padding_touches_nothing():
    B, H, N, S = 5, 20, 16, 3
    slots = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    u = torch.full((B, H), NAN, device="cuda")
    Bt = torch.full((B, 1, N), NAN, device="cuda")
    A, w = -torch.ones(H, N, device="cuda"), torch.ones(H, 4, device="cuda")
    state, ring = torch.randn(S, H, N, device="cuda"), torch.randn(S, H, 3, device="cuda")
    s0, r0 = state.clone(), ring.clone()
    assert not bool(api.selective_scan_step(u, u, A, Bt, Bt, state, slots=slots).any())
    assert not bool(api.short_conv_step(u, ring, w, slots=slots).any())
    assert torch.equal(state, s0) and torch.equal(ring, r0)


def test_two_streams_and_two_graphs_side_by_side():
    """Backward passes on two streams at once, and two captured ones replayed side by side, each with its own
    workspace, give the bits of calls made one after the other."""
    def case(seed):
        c = scan_case(2, 48, 900, 16, 1, "bf16", seed, ("D", "bias", "gate"))
        d = {k: c[k].cuda() for k in ("u", "delta", "A", "Bt", "Ct", "D", "dt_bias", "z", "dy")}

        def run():
            y, ck = api.selective_scan_fwd(d["u"], d["delta"], d["A"], d["Bt"], d["Ct"], d["D"], d["dt_bias"], d["z"],
                                           return_ckpt=True)
            g = api.selective_scan_bwd(d["dy"], d["u"], d["delta"], d["A"], d["Bt"], d["Ct"], ck, d["D"], d["dt_bias"],
                                       d["z"])
            return [y, *g]
        return run
    runs = [case(1), case(2)]
    want = [[t.clone() for t in r()] for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i] = runs[i]()
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))
    graphs, res = [], []
    for i, s in enumerate(streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            res.append(runs[i]())
        graphs.append(g)
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for o, w in zip(res, want):
        assert all(torch.equal(a, b) for a, b in zip(o, w))


def test_lengths_outside_the_row_count_as_its_ends():
    c = scan_case(3, 6, 150, 4, 1, "f32", 31, ("D", "bias"))
    a = [c[k].cuda() for k in ("u", "delta", "A", "Bt", "Ct", "D", "dt_bias")]
    w = torch.randn(6, 4, generator=torch.Generator().manual_seed(2)).cuda()
    n = torch.tensor([1000, -5, 40], dtype=torch.int32, device="cuda")
    m = torch.tensor([150, 0, 40], dtype=torch.int32, device="cuda")
    for f in (lambda k: api.selective_scan_fwd(*a, lengths=k, return_state=True),
              lambda k: api.short_conv_fwd(a[0], w, lengths=k, return_state=True),
              lambda k: api.short_conv_bwd(a[0], a[1], w, lengths=k)[:2]):
        for x, y in zip(f(n), f(m)):
            assert torch.equal(x, y)
