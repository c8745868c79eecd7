"""What is measured of the gated linear recurrence and the gated linear unit: their cases, plain forms and 64-bit values.

The gated linear recurrence, per batch b and channel d, with w_t = exp(log_w_t):

    h_t = w_t h_{t-1} + s(w_t) x_t        y_t = h_t        s = 1, 1 - w ("mix") or sqrt(1 - w^2) ("norm")

for whole prompts, single tokens and the gradients; the gated linear unit h = act(x Wg) * (x Wu), the wide half of a
gated feed-forward block, forward and backward. The plain forms are elementary torch operations in float32.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
INPUTS = ("plain", "mix", "norm")
ACTS = ("sigmoid", "silu", "gelu", "relu2")


def listed():
    return [
        # one short chat prompt from a fresh state: latency is what counts
        {"name": "scan-short", "op": "scan", "B": 1, "T": 77, "D": 768, "dtype": "bf16", "input": "plain", "state": False,
         "ragged": False},
        # one long document, float32: few channels, the sequence has to be spread over the chip
        {"name": "scan-one-long-f32", "op": "scan", "B": 1, "T": 32767, "D": 1024, "dtype": "f32", "input": "norm",
         "state": True, "ragged": False},
        # the largest: a padded batch of long prompts of a wide model, resumed from their states
        {"name": "scan-large", "op": "scan", "B": 8, "T": 8192, "D": 4096, "dtype": "bf16", "input": "mix", "state": True,
         "ragged": True},
        # one token for a few chats
        {"name": "scan-step-small", "op": "scan_step", "B": 4, "D": 768, "dtype": "bf16", "input": "plain"},
        # one token for a large serving batch
        {"name": "scan-step-large", "op": "scan_step", "B": 512, "D": 4096, "dtype": "bf16", "input": "norm"},
        # a training step's gradients at a small model's context
        {"name": "scan-grad-train", "op": "scan_grad", "B": 8, "T": 4096, "D": 1024, "dtype": "bf16", "input": "mix",
         "state": False, "ragged": False},
        # gradients in float32 over a padded batch, a width that is no power of two
        {"name": "scan-grad-ragged-f32", "op": "scan_grad", "B": 3, "T": 515, "D": 1000, "dtype": "f32", "input": "norm",
         "state": True, "ragged": True},
        # one generated token: the weights' bytes are what counts
        {"name": "glu-token", "op": "glu", "M": 1, "D": 2048, "F": 5504, "dtype": "bf16", "act": "silu", "pre": False},
        # a prompt through the widest layer
        {"name": "glu-prompt", "op": "glu", "M": 8192, "D": 4096, "F": 10944, "dtype": "bf16", "act": "silu", "pre": False},
        # a float32 training forward at odd sizes, pre-activations kept
        {"name": "glu-odd-f32", "op": "glu", "M": 515, "D": 770, "F": 2049, "dtype": "f32", "act": "gelu", "pre": True},
        # a training step's gradients, 32768 tokens of a small model
        {"name": "glu-grad-train", "op": "glu_grad", "M": 32768, "D": 768, "F": 2048, "dtype": "bf16", "act": "silu"},
        # gradients of a small batch in float32, squared ReLU
        {"name": "glu-grad-f32", "op": "glu_grad", "M": 1000, "D": 512, "F": 1365, "dtype": "f32", "act": "relu2"},
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A number of channels: mostly a multiple of 64 or 8, as models have them, and any (odd ones too) now and then."""
    n, kind = _between(rng, lo, hi), rng.random()
    if kind < 0.5 and n >= 64:
        return n // 64 * 64
    return n // 8 * 8 if kind < 0.75 and n >= 8 else n


def draw(rng):
    op = rng.choice(["scan", "scan", "scan_step", "scan_grad", "glu", "glu", "glu_grad"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    half = 2 if dtype == "f32" else 1
    if op == "scan_step":
        return {"op": op, "B": _between(rng, 1, 512 // half), "D": _width(rng, 16, 4096), "dtype": dtype,
                "input": rng.choice(INPUTS)}
    if op in ("scan", "scan_grad"):
        most = 8 * 8192 * 4096 // half // (1 if op == "scan" else 4)
        D = _width(rng, 16, 4096)
        T = min(_between(rng, 1, 32768), most // D)
        B = _between(rng, 1, max(1, min(16, most // (D * T))))
        return {"op": op, "B": B, "T": T, "D": D, "dtype": dtype, "input": rng.choice(INPUTS),
                "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}
    most = 8192 * 4096 * 10944 // (1 if op == "glu" else 2) // (8 if dtype == "f32" else 1)
    D, F = _width(rng, 16, 4096), _width(rng, 16, 10944)
    M = _between(rng, 1, max(1, min(32768, most // (D * F))))
    case = {"op": op, "M": M, "D": D, "F": F, "dtype": dtype, "act": rng.choice(ACTS)}
    if op == "glu":
        case["pre"] = rng.random() < 0.5
    return case


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    dtype = DTYPES[case["dtype"]]
    s = {"op": case["op"]}
    if case["op"] in ("glu", "glu_grad"):
        M, D, F = case["M"], case["D"], case["F"]
        s["act"], s["pre"] = case["act"], case.get("pre", False)
        s["x"] = normal(M, D, dtype=dtype)
        s["w_gate"], s["w_up"] = (normal(D, F, scale=D ** -0.5, dtype=dtype) for _ in range(2))
        if case["op"] == "glu_grad":  # what the forward left
            s["gate"], s["up"] = ((s["x"].float() @ s[n].float()).to(dtype) for n in ("w_gate", "w_up"))
            s["dh"] = normal(M, F, dtype=dtype)
        return s
    B, T, D = case["B"], case.get("T", 1), case["D"]
    s["input"] = case["input"]
    s["x"] = normal(B, T, D, dtype=dtype)
    # decays of a gate, from fast to slow channels, and now and then a reset where packed sequences meet
    u = torch.rand((B, T, D), generator=g, device="cuda") * 2.0 - torch.linspace(1.5, 8.0, D, device="cuda")
    s["log_w"] = -torch.exp(u)
    s["log_w"].masked_fill_((torch.rand((B, T), generator=g, device="cuda") < 1e-3)[..., None], -math.inf)
    s["state"] = normal(B, D) if case.get("state", True) else None
    s["lens"] = None
    if case.get("ragged"):
        s["lens"] = ((0.5 + 0.5 * torch.rand((B,), generator=g, device="cuda")) * T).to(torch.int32)
    if case["op"] == "scan_grad":
        s["dy"] = normal(B, T, D, dtype=dtype)
        s["dstate"] = normal(B, D) if case["state"] else None
    return s


def _scan(a, b):
    """b[t] <- b[t] + a[t] b[t-1] + a[t] a[t-1] b[t-2] + ... along dimension 1, by doubling; a and b are overwritten."""
    d, T = 1, a.shape[1]
    while d < T:
        b[:, d:] = b[:, d:] + a[:, d:] * b[:, :-d]
        a[:, d:] = a[:, d:] * a[:, :-d]
        d *= 2
    return b


def _scale(log_w, kind):
    """s(w) and its derivative to log w."""
    if kind == "plain":
        return torch.ones((), device="cuda"), torch.zeros((), device="cuda")
    if kind == "mix":
        return -torch.expm1(log_w), -log_w.exp()
    s = torch.sqrt(-torch.expm1(2 * log_w))
    return s, -torch.exp(2 * log_w) / s


def _kept(s, T):
    """[B, T, 1] truth values: the tokens before each sequence's end."""
    return (torch.arange(T, device="cuda")[None, :] < s["lens"][:, None].clamp(0, T))[..., None]


def _states(s):
    """h of every token; behind a sequence's end it stays."""
    x, lw = s["x"].float(), s["log_w"]
    w, b = lw.exp(), _scale(lw, s["input"])[0] * x
    if s["lens"] is not None:
        keep = _kept(s, x.shape[1])
        w, b = torch.where(keep, w, 1.0), torch.where(keep, b, 0.0)
    if s["state"] is not None:
        b[:, 0] += w[:, 0] * s["state"]
    return _scan(w, b)


def _prompt(s):
    h = _states(s)
    y = h if s["lens"] is None else torch.where(_kept(s, h.shape[1]), h, 0.0)
    return {"y": y.to(s["x"].dtype), "state": h[:, -1].clone()}


def _step(s):
    lw = s["log_w"][:, 0]
    h = lw.exp() * s["state"] + _scale(lw, s["input"])[0] * s["x"][:, 0].float()
    return {"y": h[:, None].to(s["x"].dtype), "state": h}


def _scan_grad(s):
    x, lw, dy = s["x"].float(), s["log_w"], s["dy"].float()
    B, T, D = x.shape
    first = torch.zeros((B, D), device="cuda") if s["state"] is None else s["state"]
    before = torch.cat([first[:, None], _states(s)[:, :-1]], 1)
    w = lw.exp()
    if s["lens"] is not None:
        keep = _kept(s, T)
        w, dy = torch.where(keep, w, 1.0), torch.where(keep, dy, 0.0)
    if s["dstate"] is not None:
        dy[:, -1] += s["dstate"]
    later = torch.cat([w[:, 1:], torch.ones((B, 1, D), device="cuda")], 1)
    g = _scan(later.flip(1), dy.flip(1)).flip(1)
    scale, slope = _scale(lw, s["input"])
    dstate = w[:, 0] * g[:, 0]
    dx, dlw = scale * g, (w * before + slope * x) * g
    if s["lens"] is not None:
        dx, dlw = torch.where(keep, dx, 0.0), torch.where(keep, dlw, 0.0)
    return {"dx": dx.to(s["x"].dtype), "dlog_w": dlw, "dstate_in": dstate}


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "relu2":
        r = g.clamp_min(0)
        return r * r, 2 * r
    if kind == "gelu":
        c = 0.5 * (1 + torch.erf(g * math.sqrt(0.5)))
        return g * c, c + g * torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    e = 1 / (1 + torch.exp(-g))
    return (e, e * (1 - e)) if kind == "sigmoid" else (g * e, e * (1 + g * (1 - e)))


def _glu(s):
    x, dt = s["x"].float(), s["x"].dtype
    g, u = x @ s["w_gate"].float(), x @ s["w_up"].float()
    h = (_act(g, s["act"])[0] * u).to(dt)
    return {"h": h, "gate": g.to(dt), "up": u.to(dt)} if s["pre"] else {"h": h}


def _glu_grad(s):
    x, g, u, dh, dt = s["x"].float(), s["gate"].float(), s["up"].float(), s["dh"].float(), s["x"].dtype
    a, slope = _act(g, s["act"])
    dg, du = dh * u * slope, dh * a
    dx = dg @ s["w_gate"].float().t() + du @ s["w_up"].float().t()
    return {"dx": dx.to(dt), "dw_gate": (x.t() @ dg).to(dt), "dw_up": (x.t() @ du).to(dt)}


def run(state):
    s = state
    if own:
        from linear_rnn_amd import wkv
        if s["op"] in ("glu", "glu_grad"):
            act = {"sigmoid": wkv.RWKV7_ACT_SIGMOID, "silu": wkv.RWKV7_ACT_SILU, "gelu": wkv.RWKV7_ACT_GELU,
                   "relu2": wkv.RWKV7_ACT_RELU2}[s["act"]]
            if s["op"] == "glu_grad":
                return wkv.glu_backward(s["x"], s["w_gate"], s["w_up"], s["gate"], s["up"], s["dh"], act=act)
            h, gate, up = wkv.glu(s["x"], s["w_gate"], s["w_up"], act=act, want_pre=s["pre"])
            return {"h": h, "gate": gate, "up": up} if s["pre"] else {"h": h}
        kind = {"plain": wkv.RWKV7_INPUT_PLAIN, "mix": wkv.RWKV7_INPUT_MIX, "norm": wkv.RWKV7_INPUT_NORM}[s["input"]]
        if s["op"] == "scan":
            y, out = wkv.gscan(s["x"], s["log_w"], state_in=s["state"], lens=s["lens"], input=kind)
            return {"y": y, "state": out}
        if s["op"] == "scan_step":
            y, out = wkv.gscan_step(s["x"], s["log_w"], s["state"], input=kind)
            return {"y": y, "state": out}
        return wkv.gscan_backward(s["x"], s["log_w"], s["dy"], state_in=s["state"], lens=s["lens"],
                                  dstate_out=s["dstate"], input=kind)
    return {"scan": _prompt, "scan_step": _step, "scan_grad": _scan_grad, "glu": _glu, "glu_grad": _glu_grad}[s["op"]](s)


def work(case):
    e = {"bf16": 2, "f32": 4}[case["dtype"]]
    if case["op"] in ("glu", "glu_grad"):
        M, D, F = case["M"], case["D"], case["F"]
        if case["op"] == "glu":
            return {"bytes": e * (M * D + 2 * D * F + M * F * (3 if case["pre"] else 1)), "flops": 4 * M * D * F}
        return {"bytes": e * (2 * M * D + 4 * D * F + 3 * M * F), "flops": 8 * M * D * F}
    B, T, D = case["B"], case.get("T", 1), case["D"]
    n, states = B * T * D, 4 * B * D
    read = 0.75 if case.get("ragged") else 1.0  # of a padded batch's tokens, on average
    if case["op"] == "scan_grad":
        return {"bytes": n * (read * (2 * e + 4) + e + 4) + states * (1 + 2 * bool(case["state"])), "flops": 12 * n * read}
    return {"bytes": n * (read * (e + 4) + e) + states * (1 + bool(case.get("state", True))), "flops": 5 * n * read}


def exact(case, seed):
    """Token by token and product by product in float64, from the definitions."""
    s = prepare(case, seed)
    f = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    if s["op"] in ("glu", "glu_grad"):
        def phi(g):  # the activation in terms of torch's own float64 functions
            return {"sigmoid": torch.sigmoid, "silu": lambda t: t * torch.sigmoid(t),
                    "gelu": lambda t: t * torch.special.ndtr(t), "relu2": lambda t: torch.relu(t) ** 2}[s["act"]](g)

        if s["op"] == "glu":
            g, u = f["x"].matmul(f["w_gate"]), f["x"].matmul(f["w_up"])
            h = phi(g).mul_(u)
            return {"h": h, "gate": g, "up": u} if s["pre"] else {"h": h}
        g = f["gate"].requires_grad_(True)
        a = phi(g)
        (slope,) = torch.autograd.grad(a.sum(), g)
        dg, du = slope * f["up"] * f["dh"], a.detach() * f["dh"]
        dx = torch.addmm(du.matmul(f["w_up"].t()), dg, f["w_gate"].t())
        return {"dx": dx, "dw_gate": f["x"].t().matmul(dg), "dw_up": f["x"].t().matmul(du)}
    B, T, D = s["x"].shape
    live = torch.ones((T, B, 1), dtype=torch.bool, device="cuda")
    if s.get("lens") is not None:
        live = (torch.arange(T, device="cuda")[:, None] < s["lens"][None, :])[..., None]
    one = torch.ones((), dtype=torch.float64, device="cuda")
    none = torch.zeros((), dtype=torch.float64, device="cuda")

    def at(t):
        """Decay, input scale and its slope of token t."""
        lw = f["log_w"][:, t]
        w = torch.exp(lw)
        if s["input"] == "plain":
            return w, one, none
        if s["input"] == "mix":
            return w, -torch.expm1(lw), -w
        scale = (-torch.expm1(2 * lw)).sqrt()
        return w, scale, -w * w / scale

    h = f["state"].clone() if s["state"] is not None else torch.zeros((B, D), dtype=torch.float64, device="cuda")
    back = s["op"] == "scan_grad"
    out = torch.zeros((B, T, D), dtype=torch.float64, device="cuda")
    for t in range(T):
        w, scale, _ = at(t)
        if back:
            out[:, t] = h  # the state before this token
        h = torch.where(live[t], w * h + scale * f["x"][:, t], h)
        if not back:
            out[:, t] = torch.where(live[t], h, none)
    if not back:
        return {"y": out, "state": h}
    g = f["dstate"].clone() if s["dstate"] is not None else torch.zeros_like(h)
    dx = torch.zeros_like(out)
    for t in range(T - 1, -1, -1):
        w, scale, slope = at(t)
        here = g + f["dy"][:, t]
        dx[:, t] = torch.where(live[t], scale * here, none)
        out[:, t] = torch.where(live[t], here * (w * out[:, t] + slope * f["x"][:, t]), none)
        g = torch.where(live[t], w * here, g)
    return {"dx": dx, "dlog_w": out, "dstate_in": g}
