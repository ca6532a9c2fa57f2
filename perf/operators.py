"""Cases of the selective-SSM operators: the short causal convolution, the
selective scan (prompts, training, single tokens) and the group norm with an
activation.

A case is one pass a user's program makes: a prompt, a training step (forward
and backward) or one generated token for a batch of requests.  ``run`` makes it
in elementary torch operations in 32 bits, or, with ``own`` set, through
``fft_long_convolution_flashconv_b200.api``; ``exact`` gives the same outputs
step by step in 64 bits.

Notation: dt = softplus(delta + dt_bias), a_n = exp(dt A_n),
x_n <- a_n x_n + dt B_n u, y = (sum_n C_n x_n + D u) silu(z).
"""
import math

import torch
import torch.nn.functional as F

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ cases
def _conv(name, kind, B, H, L, K, dtype, ragged=False, state=False, pool=0):
    return dict(name=name, op="conv", kind=kind, B=B, H=H, L=L, K=K, dtype=dtype, ragged=ragged, state=state, pool=pool)


def _scan(name, kind, B, H, L, N, G, dtype, gate=True, ragged=False, state=False, pool=0):
    return dict(name=name, op="scan", kind=kind, B=B, H=H, L=L, N=N, G=G, dtype=dtype, gate=gate, ragged=ragged,
                state=state, pool=pool)


def _norm(name, kind, B, L, C, G, dtype, gate, channel_major):
    return dict(name=name, op="norm", kind=kind, B=B, L=L, C=C, G=G, dtype=dtype, gate=gate,
                channel_major=channel_major)


def listed():
    return [
        # one request generating: latency of the convolution's update
        _conv("conv-step-one", "step", 1, 768, 1, 4, "f16", pool=1),
        # one long document, with the state handed to generation
        _conv("conv-prompt-long", "prompt", 1, 2560, 65536, 4, "f16", state=True),
        # a training step at the H3 layer's shape
        _conv("conv-train", "train", 8, 768, 1024, 4, "f16"),
        # one request generating: latency of the scan's update
        _scan("scan-step-one", "step", 1, 768, 1, 16, 1, "bf16", pool=1),
        # a server's batch: requests in slots of a state pool, some rows padded
        _scan("scan-step-many", "step", 256, 2560, 1, 16, 1, "bf16", pool=320),
        # a batch of prompts of one length at the H3 layer's shape
        _scan("scan-prompt", "prompt", 8, 768, 1024, 16, 1, "f16"),
        # prompts of several lengths padded to an odd longest one, a large state, two groups, no gate, continued
        _scan("scan-prompt-ragged", "prompt", 5, 1000, 2047, 64, 2, "bf16", gate=False, ragged=True, state=True),
        # one long document
        _scan("scan-prompt-long", "prompt", 1, 2560, 65536, 16, 1, "f16", state=True),
        # a training step on long sequences
        _scan("scan-train", "train", 4, 1024, 8192, 16, 1, "bf16"),
        # a small training step in fp32 with odd sizes, padded rows and groups
        _scan("scan-train-odd", "train", 3, 100, 777, 8, 4, "f32", ragged=True, state=True),
        # the H3 mixer's output (12 heads of 64), training step
        _norm("norm-train", "train", 8, 2048, 768, 12, "f16", False, False),
        # a scan's output over a long document, gated, to token-major for the output projection
        _norm("norm-gate-long", "prompt", 1, 65536, 2560, 40, "f16", True, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["conv", "scan", "scan", "norm"])
    kind = rng.choice(["prompt", "train"] if op == "norm" else ["prompt", "train", "step"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "norm":
        G = rng.choice([1, 2, 8, 12, 40])
        C = G * rng.choice([16, 40, 64, 128])
        B, L = _log(rng, 1, 8), _log(rng, 1, 8192)
        L = min(L, 2 ** 26 // (B * C))
        c = _norm("", kind, B, L, C, G, dtype, rng.random() < 0.5, rng.random() < 0.5)
    else:
        H = _log(rng, 32, 2560)
        B = _log(rng, 1, 256) if kind == "step" else _log(rng, 1, 8)
        L = 1 if kind == "step" else min(_log(rng, 1, 8192), 2 ** 26 // (B * H))
        pool = B + rng.randrange(0, 64) if kind == "step" else 0
        ragged, state = rng.random() < 0.5, rng.random() < 0.5
        if op == "conv":
            c = _conv("", kind, B, H, L, rng.randrange(1, 9), dtype, ragged, state, pool)
        else:
            G = rng.choice([1, 1, 2, 4])
            H = max(1, H // G) * G
            N = rng.choice([1, 4, 8, 16, 16, 16, 24, 32, 64])
            # bounded by the listed prompts and training steps
            while B * H * L * N > (2 ** 29 if kind == "train" else 2 ** 30):
                L = L // 2 + 1
            c = _scan("", kind, B, H, L, N, G, dtype, rng.random() < 0.7, ragged, state, pool)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 7919 + 13)
    dt = _DT[case["dtype"]]
    kind = case["kind"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "norm":
        B, L, C = case["B"], case["L"], case["C"]
        shape = (B, C, L) if case["channel_major"] else (B, L, C)
        s["x"] = (normal(*shape) * 1.5 + 0.1).to(dt)
        s["gate"] = normal(*shape).to(dt) if case["gate"] else None
        s["weight"] = 1 + normal(C, std=0.1)
        s["bias"] = normal(C, std=0.1)
        if kind == "train":
            s["dy"] = normal(B, L, C).to(dt)
        return s
    B, H, L = case["B"], case["H"], case["L"]
    step = kind == "step"
    if step:
        S = case["pool"]
        # each request's place in the pool; every eighth row of a batch is padding
        slots = torch.randperm(S, generator=gen, device="cuda")[:B].to(torch.int32)
        if B >= 8:
            slots[7::8] = -1
        s["slots"] = slots if S > 1 else None
    s["lengths"] = None
    if case["ragged"] and not step:
        s["lengths"] = (uniform(B) * (L + 1)).to(torch.int32).clamp(0, L)
        s["lengths"][0] = L
    if case["op"] == "conv":
        K = case["K"]
        s["w"] = normal(H, K, std=1 / math.sqrt(K))
        s["bias"] = normal(H, std=0.1)
        # x is one half of the input projection's output
        s["x"] = normal(B, 2 * H).to(dt)[:, :H] if step else normal(B, 2 * H, L).to(dt)[:, :H]
        if step:
            s["state"] = normal(S, H, K - 1).to(dt)
        else:
            s["state_in"] = normal(B, H, K - 1).to(dt) if case["state"] else None
            if kind == "train":
                s["dy"] = normal(B, H, L).to(dt)
        return s
    N, G = case["N"], case["G"]
    # dt between 1e-3 and 1e-1 through its bias, A = -(1..N) as trained models drift from it
    t0 = torch.exp(uniform(H) * math.log(100.0) + math.log(1e-3))
    s["dt_bias"] = t0 + torch.log(-torch.expm1(-t0))
    s["A"] = -torch.arange(1, N + 1, device="cuda").float()[None] * torch.exp(normal(H, N, std=0.1))
    s["D"] = 1 + normal(H, std=0.1)
    tail = () if step else (L,)
    s["u"] = normal(B, H, *tail).to(dt)
    s["delta"] = normal(B, H, *tail, std=0.7).to(dt)
    s["z"] = normal(B, 2 * H, *tail).to(dt)[:, H:] if case["gate"] else None
    # Bt and Ct are halves of one projection's output
    bc = normal(B, 2, G, N, *tail).to(dt)
    s["Bt"], s["Ct"] = bc[:, 0], bc[:, 1]
    if step:
        s["state"] = normal(S, H, N)
    else:
        s["state_in"] = normal(B, H, N) if case["state"] else None
        if kind == "train":
            s["dy"] = normal(B, H, L).to(dt)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if own:
        return _run_own(s, c)
    if c["op"] == "norm":
        return _plain_norm(s, c)
    if c["op"] == "conv":
        return _plain_conv_step(s, c) if c["kind"] == "step" else _plain_conv(s, c)
    return _plain_scan_step(s, c) if c["kind"] == "step" else _plain_scan(s, c)


def _run_own(s, c):
    from fft_long_convolution_flashconv_b200 import api
    train = c["kind"] == "train"
    if c["op"] == "norm":
        args = dict(weight=s["weight"], bias=s["bias"], gate=s["gate"], channel_major=c["channel_major"])
        y = api.group_norm_act_fwd(s["x"], c["G"], **args)
        if not train:
            return y
        return (y, *api.group_norm_act_bwd(s["dy"], s["x"], c["G"], **args))
    if c["op"] == "conv":
        if c["kind"] == "step":
            return api.short_conv_step(s["x"], s["state"], s["w"], s["bias"], slots=s["slots"]), s["state"]
        kw = dict(state_in=s["state_in"], lengths=s["lengths"])
        y, state = api.short_conv_fwd(s["x"], s["w"], s["bias"], return_state=True, **kw)
        if not train:
            return y, state
        return (y, state, *api.short_conv_bwd(s["dy"], s["x"], s["w"], s["bias"], **kw))
    p = dict(D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
    if c["kind"] == "step":
        return api.selective_scan_step(s["u"], s["delta"], s["A"], s["Bt"], s["Ct"], s["state"], slots=s["slots"],
                                       **p), s["state"]
    p["lengths"] = s["lengths"]
    if not train:
        return api.selective_scan_fwd(s["u"], s["delta"], s["A"], s["Bt"], s["Ct"], state_in=s["state_in"],
                                      return_state=True, **p)
    y, ckpt = api.selective_scan_fwd(s["u"], s["delta"], s["A"], s["Bt"], s["Ct"], state_in=s["state_in"],
                                     return_ckpt=True, **p)
    return (y, *api.selective_scan_bwd(s["dy"], s["u"], s["delta"], s["A"], s["Bt"], s["Ct"], ckpt,
                                       need_dstate_in=True, **p))


# ------------------------------------------------------------------ plain forms, 32 bits
def _valid(s, L):
    """B x 1 x L truth values (all true without lengths)."""
    t = torch.arange(L, device="cuda")
    if s["lengths"] is None:
        return torch.ones(1, 1, L, dtype=torch.bool, device="cuda")
    return (t[None] < s["lengths"][:, None])[:, None]


def _masked(ok, x):
    return torch.where(ok, x.float(), torch.zeros((), device="cuda"))


def _dsilu(x):
    g = torch.sigmoid(x)
    return g * (1 + x * (1 - g))


def _plain_conv(s, c):
    B, H, L, K = c["B"], c["H"], c["L"], c["K"]
    dt = s["x"].dtype
    ok = _valid(s, L)
    x = _masked(ok, s["x"])
    past = s["state_in"].float() if s["state_in"] is not None else x.new_zeros(B, H, K - 1)
    xp = torch.cat([past, x], -1)
    n = torch.full((B,), L, device="cuda") if s["lengths"] is None else s["lengths"].long()
    # the K - 1 inputs before each row's end
    at = (n[:, None] + torch.arange(K - 1, device="cuda"))[:, None].expand(B, H, K - 1)
    state = torch.gather(xp, 2, at).to(dt)
    win = xp.unfold(-1, K, 1)  # win[..., t, j] = x[t - (K - 1) + j]
    w = s["w"].flip(1)
    pre = (win * w[:, None]).sum(-1) + s["bias"][:, None]
    y = _masked(ok, pre * torch.sigmoid(pre)).to(dt)
    if c["kind"] == "prompt":
        return y, state
    dc = _masked(ok, s["dy"]) * _dsilu(pre)
    dx = (F.pad(dc, (0, K - 1)).unfold(-1, K, 1) * s["w"][:, None]).sum(-1)
    dw = (dc[..., None] * win).sum((0, 2)).flip(1)
    return y, state, _masked(ok, dx).to(dt), dw, dc.sum((0, 2))


def _plain_conv_step(s, c):
    at, live = _slots(s, c)
    new = torch.cat([s["state"][at].float(), s["x"].float()[..., None]], -1)
    pre = (new * s["w"].flip(1)).sum(-1) + s["bias"]
    s["state"][at[live]] = new[live][..., 1:].to(s["x"].dtype)
    return _masked(live[:, None], pre * torch.sigmoid(pre)).to(s["x"].dtype), s["state"]


def _slots(s, c):
    slots = torch.arange(c["B"], device="cuda") if s["slots"] is None else s["slots"].long()
    return slots.clamp(min=0), slots >= 0


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(torch.clamp(x, max=20))))


def _recur(a, b):
    """x[t] = a[t] x[t-1] + b[t] along the last axis, by doubling."""
    n = 1
    while n < a.shape[-1]:
        b = torch.cat([b[..., :n], b[..., n:] + a[..., n:] * b[..., :-n]], -1)
        a = torch.cat([a[..., :n], a[..., n:] * a[..., :-n]], -1)
        n *= 2
    return b


def _plain_scan(s, c):
    B, H, L, N, G = c["B"], c["H"], c["L"], c["N"], c["G"]
    E = H // G
    io = s["u"].dtype
    ok = _valid(s, L)
    u, delta = _masked(ok, s["u"]), _masked(ok, s["delta"])
    Bt, Ct = (_masked(ok[:, :, None], s[k])[:, :, None] for k in ("Bt", "Ct"))  # B x G x 1 x N x L
    raw = delta + s["dt_bias"][:, None]
    dt = _masked(ok, _softplus(raw))
    wide = (B, G, E, 1, L)
    A = s["A"].reshape(G, E, N, 1)
    a = torch.exp(dt.reshape(wide) * A)
    b = (dt * u).reshape(wide) * Bt
    x0 = s["state_in"].reshape(B, G, E, N, 1) if s["state_in"] is not None else b.new_zeros(B, G, E, N, 1)
    b[..., :1] += a[..., :1] * x0
    x = _recur(a, b)
    del b
    y0 = (Ct * x).sum(3).reshape(B, H, L) + s["D"][:, None] * u
    z = None if s["z"] is None else _masked(ok, s["z"])
    y = (y0 if z is None else y0 * z * torch.sigmoid(z)).to(io)
    if c["kind"] == "prompt":
        return y, x[..., -1].reshape(B, H, N).clone()
    dy = _masked(ok, s["dy"])
    dyp = dy if z is None else dy * z * torch.sigmoid(z)
    g = Ct * dyp.reshape(wide)
    later = torch.cat([a[..., 1:], torch.zeros_like(a[..., :1])], -1).flip(-1)  # a[t+1], reversed in time
    g = _recur(later, g.flip(-1)).flip(-1)
    del later
    ax = a * torch.cat([x0, x[..., :-1]], -1)
    gB = (g * Bt).sum(3).reshape(B, H, L)
    q = g * ax
    ddt = u * gB + (q * A).sum(3).reshape(B, H, L)
    ddelta = _masked(ok, ddt * torch.sigmoid(raw))
    dA = (q * dt.reshape(wide)).sum((0, 4)).reshape(H, N)
    dB = (g * (dt * u).reshape(wide)).sum(2)
    dC = (x * dyp.reshape(wide)).sum(2)
    du = _masked(ok, s["D"][:, None] * dyp + dt * gB)
    return (y, du.to(io), ddelta.to(io), dA, _masked(ok[:, :, None], dB).to(io), _masked(ok[:, :, None], dC).to(io),
            (dyp * u).sum((0, 2)), ddelta.sum((0, 2)), None if z is None else (dy * y0 * _dsilu(z)).to(io),
            (a[..., 0] * g[..., 0]).reshape(B, H, N))


def _plain_scan_step(s, c):
    B, H, N, G = c["B"], c["H"], c["N"], c["G"]
    at, live = _slots(s, c)
    dt = _softplus(s["delta"].float() + s["dt_bias"])
    u = s["u"].float()
    Bt, Ct = (s[k].float()[:, :, None].expand(B, G, H // G, N).reshape(B, H, N) for k in ("Bt", "Ct"))
    x = torch.exp(dt[..., None] * s["A"]) * s["state"][at] + (dt * u)[..., None] * Bt
    s["state"][at[live]] = x[live]
    y = (Ct * x).sum(-1) + s["D"] * u
    if s["z"] is not None:
        z = s["z"].float()
        y = y * z * torch.sigmoid(z)
    return _masked(live[:, None], y).to(s["u"].dtype), s["state"]


def _plain_norm(s, c):
    B, L, C, G = c["B"], c["L"], c["C"], c["G"]
    io = s["x"].dtype
    tokens = (lambda t: t.transpose(1, 2)) if c["channel_major"] else (lambda t: t)
    x = tokens(s["x"]).float().reshape(B, L, G, C // G)
    d = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt((d * d).mean(-1, keepdim=True) + 1e-5)
    w, bias = s["weight"].reshape(G, -1), s["bias"].reshape(G, -1)
    xh = d * r
    n = xh * w + bias
    gate = None if s["gate"] is None else tokens(s["gate"]).float().reshape(n.shape)
    act = n * torch.sigmoid(n) if gate is None else n * gate * torch.sigmoid(gate)
    y = act.reshape(B, L, C).to(io)
    if c["kind"] == "prompt":
        return y
    dy = s["dy"].float().reshape(n.shape)
    dn = dy * _dsilu(n) if gate is None else dy * gate * torch.sigmoid(gate)
    h = dn * w
    dx = r * (h - h.mean(-1, keepdim=True) - xh * (h * xh).mean(-1, keepdim=True))
    back = lambda t: tokens(t.reshape(B, L, C)).to(io).contiguous()  # noqa: E731
    return (y, back(dx), (dn * xh).sum((0, 1)).reshape(C), dn.sum((0, 1)).reshape(C),
            None if gate is None else back(dy * n * _dsilu(gate)))


# ------------------------------------------------------------------ the definitions, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in s.items()}
    with torch.no_grad():
        return {"norm": _exact_norm, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](d, case)


def _sig(x):
    return 1 / (1 + torch.exp(-x))


def _exact_norm(d, c):
    x, gate = d["x"], d["gate"]
    if c["channel_major"]:
        x, gate = x.permute(0, 2, 1), None if gate is None else gate.permute(0, 2, 1)
    B, L, C = x.shape
    y, dx, dg = (torch.empty(B, L, C, dtype=torch.float64, device="cuda") for _ in range(3))
    dw, db = torch.zeros_like(d["weight"]), torch.zeros_like(d["bias"])
    M = C // c["G"]
    for k in range(0, C, M):  # group by group
        xs, w = x[..., k:k + M], d["weight"][k:k + M]
        mean = xs.sum(-1, keepdim=True) / M
        std = torch.sqrt(((xs - mean) ** 2).sum(-1, keepdim=True) / M + 1e-5)
        h = (xs - mean) / std
        n = h * w + d["bias"][k:k + M]
        v = n if gate is None else gate[..., k:k + M]
        sv = _sig(v)
        y[..., k:k + M] = n * sv if gate is None else n * v * sv
        if c["kind"] == "train":
            dy = d["dy"][..., k:k + M]
            ds = sv + v * sv * (1 - sv)
            dn = dy * ds if gate is None else dy * v * sv
            if gate is not None:
                dg[..., k:k + M] = dy * n * ds
            dw[k:k + M], db[k:k + M] = (dn * h).sum((0, 1)), dn.sum((0, 1))
            e = dn * w
            dx[..., k:k + M] = (e - e.sum(-1, keepdim=True) / M - h * (e * h).sum(-1, keepdim=True) / M) / std
    if c["kind"] == "prompt":
        return y
    if c["channel_major"]:
        dx, dg = dx.permute(0, 2, 1).contiguous(), dg.permute(0, 2, 1).contiguous()
    return y, dx, dw, db, None if gate is None else dg


def _exact_conv(d, c):
    B, H, L, K = c["B"], c["H"], c["L"], c["K"]
    w, bias, x = d["w"], d["bias"], d["x"]
    if c["kind"] == "step":
        slots = list(range(B)) if d["slots"] is None else d["slots"].tolist()
        y, state = torch.zeros_like(x), d["state"].clone()
        for b, slot in enumerate(slots):
            if slot < 0:
                continue
            pre = bias + w[:, 0] * x[b]
            for j in range(1, K):
                pre = pre + w[:, j] * state[slot, :, K - 1 - j]
            y[b] = pre * _sig(pre)
            state[slot] = torch.cat([state[slot], x[b][:, None]], 1)[:, 1:]
        return y, state
    y, dx = torch.zeros(B, H, L, dtype=torch.float64, device="cuda"), torch.zeros(B, H, L, dtype=torch.float64, device="cuda")
    state = torch.zeros(B, H, K - 1, dtype=torch.float64, device="cuda")
    dw, db = torch.zeros_like(w), torch.zeros_like(bias)
    for b in range(B):
        n = L if d["lengths"] is None else int(d["lengths"][b])
        past = torch.zeros_like(state[b]) if d["state_in"] is None else d["state_in"][b]
        seq = torch.cat([past, x[b][:, :n]], 1)
        state[b] = seq[:, n:]
        pre = bias[:, None] + torch.zeros(H, n, dtype=torch.float64, device="cuda")
        for j in range(K):
            pre = pre + w[:, j:j + 1] * seq[:, K - 1 - j:K - 1 - j + n]
        y[b, :, :n] = pre * _sig(pre)
        if c["kind"] == "train":
            dc = d["dy"][b][:, :n] * (_sig(pre) + pre * _sig(pre) * (1 - _sig(pre)))
            db += dc.sum(1)
            for j in range(K):
                dw[:, j] += (dc * seq[:, K - 1 - j:K - 1 - j + n]).sum(1)
                if n > j:
                    dx[b, :, :n - j] += w[:, j:j + 1] * dc[:, j:]
    return (y, state, dx, dw, db) if c["kind"] == "train" else (y, state)


def _exact_scan(d, c):
    B, H, L, N, G = c["B"], c["H"], c["L"], c["N"], c["G"]
    if c["kind"] == "step":
        slots = list(range(B)) if d["slots"] is None else d["slots"].tolist()
        y, state = torch.zeros_like(d["u"]), d["state"].clone()
        for b, slot in enumerate(slots):
            if slot < 0:
                continue
            dt = torch.log1p(torch.exp(d["delta"][b] + d["dt_bias"]))
            Bt, Ct = (d[k][b].repeat_interleave(H // G, 0) for k in ("Bt", "Ct"))
            state[slot] = torch.exp(dt[:, None] * d["A"]) * state[slot] + (dt * d["u"][b])[:, None] * Bt
            y[b] = (state[slot] * Ct).sum(1) + d["D"] * d["u"][b]
            if d["z"] is not None:
                y[b] *= d["z"][b] * _sig(d["z"][b])
        return y, state
    train = c["kind"] == "train"
    n = torch.full((B,), L, device="cuda") if d["lengths"] is None else d["lengths"]
    live = (torch.arange(L, device="cuda")[:, None] < n)  # L x B
    # time first, so that a step reads neighbouring values; what lies behind a row's end is not used
    first = lambda t, fill=0.0: torch.where(live.reshape(L, B, *([1] * (t.dim() - 2))), t.movedim(-1, 0), fill).contiguous()  # noqa: E731
    u, raw = first(d["u"]), first(d["delta"] + d["dt_bias"][:, None], -math.inf)
    Bt, Ct = first(d["Bt"]), first(d["Ct"])
    dt = torch.log1p(torch.exp(raw))
    A = d["A"]
    x = torch.zeros(B, H, N, dtype=torch.float64, device="cuda") if d["state_in"] is None else d["state_in"].clone()
    y0 = torch.empty(L, B, H, dtype=torch.float64, device="cuda")
    kept = torch.empty(L + 1, B, H, N, dtype=torch.float64, device="cuda") if train else None
    dtu = dt * u
    per = lambda v: v.unsqueeze(2).expand(B, G, H // G, N).reshape(B, H, N)  # noqa: E731  groups to channels
    for t in range(L):
        if train:
            kept[t] = x
        x = torch.exp(dt[t][..., None] * A) * x + dtu[t][..., None] * per(Bt[t])
        torch.sum(x * per(Ct[t]), -1, out=y0[t])
    y0 += d["D"] * u
    z = None if d["z"] is None else first(d["z"])
    act = 1.0 if z is None else z * _sig(z)
    last = lambda v: v.movedim(0, -1).contiguous()  # noqa: E731
    if not train:
        return last(y0 * act), x
    kept[L] = x
    dy = first(d["dy"])
    dyp = dy * act
    ddt, du = torch.empty_like(dyp), torch.empty_like(dyp)
    dB, dC = torch.empty_like(Bt), torch.empty_like(Ct)
    dA, r = torch.zeros_like(A), torch.zeros_like(x)
    for t in range(L - 1, -1, -1):
        g = per(Ct[t]) * dyp[t][..., None] + r
        dC[t] = (dyp[t][..., None] * kept[t + 1]).reshape(B, G, H // G, N).sum(2)
        dB[t] = (g * dtu[t][..., None]).reshape(B, G, H // G, N).sum(2)
        gB = (g * per(Bt[t])).sum(-1)
        r = g * torch.exp(dt[t][..., None] * A)
        q = r * kept[t]
        du[t] = d["D"] * dyp[t] + dt[t] * gB
        ddt[t] = u[t] * gB + (q * A).sum(-1)
        dA += (q * dt[t][..., None]).sum(0)
    # behind a row's end nothing came in: no gradient but the state's, which passes through
    dB, dC = (v * live[:, :, None, None] for v in (dB, dC))
    ddelta = ddt * _sig(raw)
    dz = None if z is None else last(dy * y0 * (_sig(z) + z * _sig(z) * (1 - _sig(z))))
    return (last(y0 * act), last(du), last(ddelta), dA, last(dB), last(dC), (dyp * u).sum((0, 1)), ddelta.sum((0, 1)), dz, r)


# ------------------------------------------------------------------ floors
def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    B, L, kind = case["B"], case["L"], case["kind"]
    if case["op"] == "norm":
        C, gate = case["C"], 1 if case["gate"] else 0
        n = B * L * C
        arrays = 2 + gate if kind == "prompt" else 4 + 2 * gate  # x, gate, y; dy, dx, dgate
        return {"bytes": n * e * arrays + 8 * C * (1 if kind == "prompt" else 2), "flops": n * (14 if kind == "prompt" else 45)}
    H = case["H"]
    n = B * H * L
    if case["op"] == "conv":
        K = case["K"]
        tail = B * H * (K - 1) * e
        small = H * (K + 1) * 4
        if kind == "step":
            return {"bytes": n * e * 2 + 2 * tail + small, "flops": n * (2 * K + 6)}
        if kind == "prompt":
            return {"bytes": n * e * 2 + tail * (2 if case["state"] else 1) + small, "flops": n * (2 * K + 6)}
        return {"bytes": n * e * 4 + tail * (2 if case["state"] else 1) + 2 * small, "flops": n * (8 * K + 20)}
    N, G, gate = case["N"], case["G"], 1 if case["gate"] else 0
    state = B * H * N * 4
    small = H * (N + 2) * 4
    bc = 2 * B * G * N * L * e
    if kind == "step":
        return {"bytes": n * e * (3 + gate) + 2 * state + bc + small, "flops": n * (7 * N + 12)}
    ins = state if case["state"] else 0
    if kind == "prompt":
        return {"bytes": n * e * (3 + gate) + bc + state + ins + small, "flops": n * (7 * N + 12)}
    # u, delta, z, dy in; y, du, ddelta, dz out
    return {"bytes": n * e * (6 + 2 * gate) + 2 * bc + state + ins + 2 * small, "flops": n * (26 * N + 40)}
