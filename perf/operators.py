"""What is measured of the linear attention and layer norm operators: their cases, plain forms and 64-bit values.

Linear attention with a decay for each head, per batch b and head h, with a float32 state S [value, key]:

    S_t = exp(log_w_t) S_{t-1} + v_t k_t^T        y_t = S_t r_t

for whole prompts, single tokens and the gradients; layer norm over groups of channels, forward and backward. The
plain forms are elementary torch operations in float32 (cumulative log decays in float64).
"""
import math

import torch

own = False

N = 64  # head size
CHUNK = 64  # tokens in a chunk of the plain form
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # one short chat prompt of a 12-head model from a fresh state: latency is what counts
        {"name": "prefill-short", "op": "prefill", "B": 1, "T": 77, "H": 12, "dtype": "bf16", "decay": "head",
         "state": False, "ragged": False},
        # one long prompt of a 32-head model: few heads, the sequence has to be spread over the chip
        {"name": "prefill-one-long", "op": "prefill", "B": 1, "T": 8191, "H": 32, "dtype": "bf16", "decay": "head",
         "state": False, "ragged": False},
        # a padded batch of prompts resumed from their states, float32
        {"name": "prefill-ragged-f32", "op": "prefill", "B": 6, "T": 1500, "H": 16, "dtype": "f32", "decay": "token",
         "state": True, "ragged": True},
        # the largest: four long sequences of a 64-head model, a decay for each token
        {"name": "prefill-large", "op": "prefill", "B": 4, "T": 16384, "H": 64, "dtype": "bf16", "decay": "token",
         "state": True, "ragged": False},
        # one token for a few chats
        {"name": "step-small", "op": "step", "B": 4, "H": 12, "dtype": "bf16", "decay": "head"},
        # one token for a large serving batch
        {"name": "step-large", "op": "step", "B": 512, "H": 32, "dtype": "bf16", "decay": "token"},
        # a training step's gradients at the 12-head model's context
        {"name": "backward-train", "op": "backward", "B": 8, "T": 4096, "H": 12, "dtype": "bf16", "decay": "token",
         "state": True, "ragged": False},
        # gradients in float32 over a padded batch, one learned decay for each head
        {"name": "backward-ragged-f32", "op": "backward", "B": 3, "T": 515, "H": 16, "dtype": "f32", "decay": "head",
         "state": False, "ragged": True},
        # the norm before a projection: float32 residual stream in, bfloat16 out
        {"name": "norm-residual", "op": "norm", "M": 32768, "D": 768, "G": 1, "x": "f32", "y": "bf16"},
        # the norm of one prompt's heads, bfloat16
        {"name": "norm-heads", "op": "norm", "M": 77, "D": 768, "G": 12, "x": "bf16", "y": "bf16"},
        # training: gradients of the norm over a wide residual stream
        {"name": "norm-grad-wide", "op": "norm_grad", "M": 16384, "D": 4096, "G": 1, "x": "bf16", "y": "bf16"},
        # training: gradients of the norm over heads, float32
        {"name": "norm-grad-heads", "op": "norm_grad", "M": 8191, "D": 1024, "G": 16, "x": "f32", "y": "f32"},
    ]


def _between(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi], odd more often than not."""
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(lo, min(hi, n | 1 if rng.random() < 0.6 else n))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "step", "backward", "backward", "norm", "norm_grad"])
    if op in ("prefill", "backward"):
        most = 4 * 16384 * 64 if op == "prefill" else 8 * 4096 * 12
        dtype = rng.choice(["bf16", "bf16", "f32"])
        most = most // 2 if dtype == "f32" else most
        H = _between(rng, 1, 64)
        T = max(1, min(_between(rng, 1, 16384), most // H))
        B = _between(rng, 1, max(1, min(16, most // (H * T))))
        return {"op": op, "B": min(B, max(1, most // (H * T))), "T": T, "H": H, "dtype": dtype,
                "decay": rng.choice(["head", "token"]), "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}
    if op == "step":
        return {"op": op, "B": _between(rng, 1, 512), "H": _between(rng, 1, 32), "dtype": rng.choice(["bf16", "f32"]),
                "decay": rng.choice(["head", "token"])}
    if rng.random() < 0.4:  # the norm of heads of 64 channels
        G = _between(rng, 2, 64)
        D = 64 * G
    elif rng.random() < 0.3:  # a few groups of any size
        G = rng.choice([2, 3, 4, 8])
        D = G * _between(rng, 8, 1024)
    else:
        G, D = 1, _between(rng, 64, 16384)
    M = _between(rng, 1, min(65536, (16384 * 4096) // D))
    return {"op": op, "M": M, "D": D, "G": G, "x": rng.choice(["bf16", "f32"]), "y": rng.choice(["bf16", "f32"])}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)

    s = {"op": case["op"]}
    if case["op"] in ("norm", "norm_grad"):
        M, D, G = case["M"], case["D"], case["G"]
        s["G"], s["eps"], s["y"] = G, (64e-5 if G > 1 else 1e-5), DTYPES[case["y"]]
        # rows of different sizes and with an offset, as a residual stream has them
        x = normal(M, D) * torch.exp(normal(M, 1, scale=0.5)) + normal(1, D, scale=0.5)
        s["x"] = x.to(DTYPES[case["x"]])
        s["weight"], s["bias"] = 1 + normal(D, scale=0.2), normal(D, scale=0.2)
        if case["op"] == "norm_grad":
            s["dy"] = normal(M, D, dtype=s["y"])
            xg = s["x"].double().view(M, G, D // G)
            s["mean"] = xg.mean(-1)
            s["rstd"] = torch.rsqrt((xg - s["mean"][..., None]).square().mean(-1) + s["eps"]).float()
            s["mean"] = s["mean"].float()
        return s
    B, T, H, dtype = case["B"], case.get("T", 1), case["H"], DTYPES[case["dtype"]]
    s["r"], s["v"] = normal(B, T, H, N, dtype=dtype), normal(B, T, H, N, dtype=dtype)
    s["k"] = normal(B, T, H, N, scale=0.125, dtype=dtype)
    if case["decay"] == "token":  # decays of a gate, and now and then a reset where packed sequences meet
        u = torch.rand((B, T, H), generator=g, device="cuda") * 4.5 - 5.0
        s["log_w"] = -torch.exp(u)
        s["log_w"][torch.rand((B, T, H), generator=g, device="cuda") < 1e-3] = -math.inf
    else:
        s["log_w"] = -torch.exp(torch.rand((H,), generator=g, device="cuda") * 4.5 - 5.0)
    s["state"] = normal(B, H, N, N, scale=0.1) if case.get("state", True) else None
    s["lens"] = None
    if case.get("ragged"):
        share = 0.5 + 0.5 * torch.rand((B,), generator=g, device="cuda")
        s["lens"] = (share * T).to(torch.int32)
    if case["op"] == "backward":
        s["dy"] = normal(B, T, H, N, dtype=dtype)
        s["dstate"] = normal(B, H, N, N, scale=0.1) if case["state"] else None
    return s


def _kept(s, T):
    """[B, T, 1] truth values: the tokens before each sequence's end."""
    at = torch.arange(T, device="cuda")
    return (at[None, :] < s["lens"][:, None].clamp(0, T))[..., None]


def _chunks(x, keep):
    """[B, T, H, N] to float32 [B, H, chunks, CHUNK, N], zeros behind each sequence's end."""
    B, T, H, n = x.shape
    x = x.float()
    if keep is not None:
        x = torch.where(keep[..., None], x, torch.zeros((), device="cuda"))
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, -T % CHUNK))
    return x.view(B, -1, CHUNK, H, n).permute(0, 3, 1, 2, 4).contiguous()


def _tokens(x, T, dtype):
    """Back to [B, T, H, N]."""
    B, H, c, _, n = x.shape
    return x.permute(0, 2, 3, 1, 4).reshape(B, c * CHUNK, H, n)[:, :T].to(dtype)


def _decays(s, B, T, H, keep):
    """Cumulative log decays in float64: inside each chunk [B, H, chunks, CHUNK], and of whole chunks [B, H, chunks].
    A decay of zero (log -inf) is held as -1e4: the exponential of any sum with it is zero all the same."""
    lw = s["log_w"].double().clamp_min(-1e4)
    lw = lw.expand(B, T, H)
    if keep is not None:
        lw = torch.where(keep, lw, torch.zeros((), device="cuda", dtype=torch.float64))
    lw = torch.nn.functional.pad(lw, (0, 0, 0, -T % CHUNK)).view(B, -1, CHUNK, H).permute(0, 3, 1, 2)
    c = lw.cumsum(-1)
    return c, c[..., -1].cumsum(-1)


def _between_chunks(E):
    """What is left at the start of chunk m (row m; one more for the end) of what chunk l (column l) added."""
    start = torch.nn.functional.pad(E, (1, 0))
    d = start[..., :, None] - E[..., None, :]
    n = E.shape[-1]
    before = torch.arange(n + 1, device="cuda")[:, None] > torch.arange(n, device="cuda")[None, :]
    return torch.where(before, d, torch.full((), -math.inf, device="cuda", dtype=torch.float64)).exp().float(), start.exp().float()


def _inside(c):
    d = c[..., :, None] - c[..., None, :]
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device="cuda").tril()
    return torch.where(low, d, torch.full((), -math.inf, device="cuda", dtype=torch.float64)).exp().float()


def _states(v, k, c, E, first):
    """The state at the start of each chunk and after the last: [B, H, chunks + 1, N, N]."""
    left = (c[..., -1:] - c).exp().float()[..., None]
    added = (v * left).transpose(-1, -2) @ k
    B, H, n = E.shape
    over, from_first = _between_chunks(E)
    S = (over @ added.view(B, H, n, N * N)).view(B, H, n + 1, N, N)
    return S if first is None else S + from_first[..., None, None] * first[:, :, None]


def _prefill(s):
    B, T, H, _ = s["r"].shape
    keep = None if s["lens"] is None else _kept(s, T)
    r, k, v = (_chunks(s[n], keep) for n in "rkv")
    c, E = _decays(s, B, T, H, keep)
    S = _states(v, k, c, E, s["state"])
    y = ((r @ k.transpose(-1, -2)) * _inside(c)) @ v
    y = y + c.exp().float()[..., None] * (r @ S[:, :, :-1].transpose(-1, -2))
    return {"y": _tokens(y, T, s["r"].dtype), "state": S[:, :, -1].contiguous()}


def _step(s):
    r, k, v = (s[n][:, 0].float() for n in "rkv")
    w = s["log_w"].exp().expand(r.shape[0], 1, r.shape[1])[:, 0, :, None, None]
    S = w * s["state"] + v[..., None] * k[..., None, :]
    return {"y": (S @ r[..., None])[..., 0][:, None].to(s["r"].dtype), "state": S}


def _backward(s):
    B, T, H, _ = s["r"].shape
    keep = None if s["lens"] is None else _kept(s, T)
    r, k, v, dy = (_chunks(s[n], keep) for n in ("r", "k", "v", "dy"))
    c, E = _decays(s, B, T, H, keep)
    n = E.shape[-1]
    S = _states(v, k, c, E, s["state"])[:, :, :-1]
    # the state's gradient after each chunk, and (first) before the first
    e = c.exp().float()[..., None]
    added = (dy * e).transpose(-1, -2) @ r
    start = torch.nn.functional.pad(E, (1, 0))
    d = start[..., None, :-1] - start[..., :, None]  # from the end of chunk m - 1 to the start of chunk l
    after = torch.arange(n, device="cuda")[None, :] >= torch.arange(n + 1, device="cuda")[:, None]
    over = torch.where(after, d, torch.full((), -math.inf, device="cuda", dtype=torch.float64)).exp().float()
    G = (over @ added.view(B, H, n, N * N)).view(B, H, n + 1, N, N)
    if s["dstate"] is not None:
        G = G + (E[..., -1:] - start).exp().float()[..., None, None] * s["dstate"][:, :, None]
    dstate, G = G[:, :, 0].contiguous(), G[:, :, 1:]
    left = (c[..., -1:] - c).exp().float()[..., None]
    D = _inside(c)
    A = r @ k.transpose(-1, -2)
    P = (dy @ v.transpose(-1, -2)) * D
    dr_in, dk_in = e * (dy @ S), left * (v @ G)
    dr, dk = P @ k + dr_in, P.transpose(-1, -2) @ r + dk_in
    dv = (A * D).transpose(-1, -2) @ dy + left * (k @ G.transpose(-1, -2))
    W = (A * P).tril(-1).double()
    a = W.sum(-1) - W.sum(-2) + (r * dr_in).sum(-1).double()
    b = (k * dk_in).sum(-1).double()
    x = c[..., -1].exp() * (S * G).sum((-1, -2)).double()
    dlw = a.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + x[..., None]
    dlw = dlw.permute(0, 2, 3, 1).reshape(B, -1, H)[:, :T]
    if keep is not None:
        dlw = torch.where(keep, dlw, torch.zeros((), device="cuda", dtype=torch.float64))
    dlw = dlw.sum((0, 1)) if s["log_w"].dim() == 1 else dlw
    dt = s["r"].dtype
    return {"dr": _tokens(dr, T, dt), "dlog_w": dlw.float(), "dk": _tokens(dk, T, dt), "dv": _tokens(dv, T, dt),
            "dstate_in": dstate}


def _norm(s):
    M, D = s["x"].shape
    x = s["x"].float().view(M, s["G"], -1)
    mean = x.mean(-1, keepdim=True)
    rstd = torch.rsqrt((x - mean).square().mean(-1, keepdim=True) + s["eps"])
    y = ((x - mean) * rstd).view(M, D) * s["weight"] + s["bias"]
    return {"y": y.to(s["y"]), "mean": mean[..., 0], "rstd": rstd[..., 0]}


def _norm_grad(s):
    M, D = s["x"].shape
    G = s["G"]
    xh = (s["x"].float().view(M, G, -1) - s["mean"][..., None]) * s["rstd"][..., None]
    dy = s["dy"].float()
    g = (dy * s["weight"]).view(M, G, -1)
    dx = (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True)) * s["rstd"][..., None]
    return {"dx": dx.view(M, D).to(s["x"].dtype), "dweight": (dy * xh.view(M, D)).sum(0), "dbias": dy.sum(0)}


def run(state):
    s = state
    if own:
        from linear_rnn_amd import wkv
        if s["op"] == "prefill":
            y, out = wkv.linattn(s["r"], s["log_w"], s["k"], s["v"], state_in=s["state"], lens=s["lens"])
            return {"y": y, "state": out}
        if s["op"] == "step":
            y, out = wkv.linattn_step(s["r"], s["log_w"], s["k"], s["v"], s["state"])
            return {"y": y, "state": out}
        if s["op"] == "backward":
            return wkv.linattn_backward(s["r"], s["log_w"], s["k"], s["v"], s["dy"], state_in=s["state"],
                                        lens=s["lens"], dstate_out=s["dstate"])
        if s["op"] == "norm":
            y, mean, rstd = wkv.layernorm(s["x"], s["weight"], s["bias"], groups=s["G"], eps=s["eps"], out_dtype=s["y"])
            return {"y": y, "mean": mean, "rstd": rstd}
        return wkv.layernorm_backward(s["x"], s["weight"], s["mean"], s["rstd"], s["dy"], groups=s["G"])
    return {"prefill": _prefill, "step": _step, "backward": _backward, "norm": _norm, "norm_grad": _norm_grad}[s["op"]](s)


def work(case):
    size = {"bf16": 2, "f32": 4}
    if case["op"] in ("norm", "norm_grad"):
        n, ex, ey = case["M"] * case["D"], size[case["x"]], size[case["y"]]
        stats = 8 * case["M"] * case["G"]
        if case["op"] == "norm":
            return {"bytes": n * (ex + ey) + stats + 8 * case["D"], "flops": 8 * n}
        return {"bytes": n * (2 * ex + ey) + stats + 12 * case["D"], "flops": 14 * n}
    B, T, H = case["B"], case.get("T", 1), case["H"]
    th, e = B * T * H, size[case["dtype"]]
    read = 0.75 if case.get("ragged") else 1.0  # of a padded batch's tokens, on average
    decay = 4 * (th * read if case["decay"] == "token" else H)
    states = B * H * N * N * 4
    if case["op"] == "step":
        return {"bytes": 2 * states + th * 4 * N * e + decay, "flops": th * 5 * N * N}
    if case["op"] == "prefill":
        return {"bytes": th * N * e * (3 * read + 1) + decay + states * (1 + bool(case["state"])),
                "flops": th * read * 4 * N * N}
    return {"bytes": th * N * e * (4 * read + 3) + 2 * decay + states * (1 + 2 * bool(case["state"])),
            "flops": th * read * 10 * N * N}


def exact(case, seed):
    """The recurrence and the norms in float64, token by token and from their definitions."""
    s = prepare(case, seed)
    f = {n: t.double() for n, t in s.items() if isinstance(t, torch.Tensor)}
    if s["op"] in ("norm", "norm_grad"):
        M, D = s["x"].shape
        G, n = s["G"], D // s["G"]
        x, w = f["x"].view(M, G, n), f["weight"].view(G, n)
        if s["op"] == "norm":
            mean = x.sum(-1) / n
            var = (x * x).sum(-1) / n - mean * mean
            y = w * ((x - mean[..., None]) / (var + s["eps"]).sqrt()[..., None]) + f["bias"].view(G, n)
            return {"y": y.view(M, D), "mean": mean, "rstd": 1 / (var + s["eps"]).sqrt()}
        dy, mean, rstd = f["dy"].view(M, G, n), f["mean"][..., None], f["rstd"][..., None]
        # through y = w xh + b, xh = (x - mean) rstd, then through the mean and the variance
        dxh = dy * w
        dvar = -0.5 * (dxh * (x - mean)).sum(-1, keepdim=True) * rstd ** 3
        dmean = -(dxh * rstd).sum(-1, keepdim=True)
        dx = dxh * rstd + dvar * 2 * (x - mean) / n + dmean / n
        return {"dx": dx.view(M, D), "dweight": (dy * (x - mean) * rstd).sum(0).view(D), "dbias": dy.sum(0).view(D)}
    B, T, H, _ = s["r"].shape
    w = f["log_w"].exp().expand(B, T, H)
    S = f["state"].clone() if s["state"] is not None else torch.zeros((B, H, N, N), dtype=torch.float64, device="cuda")
    live = None
    if s.get("lens") is not None:
        live = (torch.arange(T, device="cuda")[:, None] < s["lens"][None, :]).double()[..., None, None]  # [T, B, 1, 1]
        w = torch.where(live[..., 0].permute(1, 0, 2) > 0, w, 1.0)
    r, k, v = f["r"], f["k"], f["v"]
    if live is not None:
        m = live.permute(1, 0, 2, 3)
        r, k, v = r * m, k * m, v * m
    first, second = torch.zeros_like(r), torch.zeros_like(r)
    back = s["op"] == "backward"
    dy = f["dy"] * (m if live is not None else 1.0) if back else None
    for t in range(T):
        S = S * w[:, t, :, None, None] + v[:, t, :, :, None] * k[:, t, :, None, :]
        if back:
            first[:, t] = (S * dy[:, t, :, :, None]).sum(-2)
        else:
            first[:, t] = (S * r[:, t, :, None, :]).sum(-1)
    if not back:
        return {"y": first, "state": S}
    G = f["dstate"].clone() if s["dstate"] is not None else torch.zeros_like(S)
    third = torch.zeros_like(r)
    at_end = (S * G).sum((-1, -2))
    for t in range(T - 1, -1, -1):
        G = G + dy[:, t, :, :, None] * r[:, t, :, None, :]
        second[:, t] = (G * v[:, t, :, :, None]).sum(-2)
        third[:, t] = (G * k[:, t, :, None, :]).sum(-1)
        G = G * w[:, t, :, None, None]
    # scaling every later token's decay path: log_w_t moves r_s.dr_s and k_s.dk_s of the tokens from t on
    move = (r * first).sum(-1) - (k * second).sum(-1)
    dlw = move.flip(1).cumsum(1).flip(1) + at_end[:, None]
    if live is not None:
        dlw = dlw * live[:, :, :, 0].permute(1, 0, 2)
    if s["log_w"].dim() == 1:
        dlw = dlw.sum((0, 1))
    return {"dr": first, "dlog_w": dlw, "dk": second, "dv": third, "dstate_in": G}
