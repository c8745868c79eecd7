"""Plain float64 implementation of the linear attention with a decay for each head, token by token,
with the sums of magnitudes that its rounding errors are measured against.

Nothing here uses the package: torch on the CPU, float64 throughout.
"""
import torch

F64 = torch.float64


def make(B, T, H, dtype, decay, seed, state=True, resets=0.0, lw_range=(-5.0, -0.5)):
    """Seeded inputs: r, v ~ N(0,1), k ~ N(0,1)/8, log_w = -exp(U(lw_range)), states ~ N(0, 0.1^2)."""
    g = torch.Generator().manual_seed(seed)

    def n(*shape, scale=1.0):
        return torch.randn(shape, generator=g) * scale

    x = {"r": n(B, T, H, 64).to(dtype), "k": n(B, T, H, 64, scale=0.125).to(dtype), "v": n(B, T, H, 64).to(dtype),
         "dy": n(B, T, H, 64).to(dtype)}
    shape = (H,) if decay == "head" else (B, T, H)
    lo, hi = lw_range
    x["log_w"] = -torch.exp(torch.rand(shape, generator=g) * (hi - lo) + lo)
    if resets:
        x["log_w"][torch.rand(shape, generator=g) < resets] = -float("inf")
    x["state_in"] = n(B, H, 64, 64, scale=0.1) if state else None
    x["dstate_out"] = n(B, H, 64, 64, scale=0.1) if state else None
    x["lens"] = None
    return x


def _inputs(x, names):
    B, T, H, _ = x["r"].shape
    out = {n: x[n].to(F64) for n in names}
    w = x["log_w"].to(F64).exp().expand(B, T, H).clone()
    if x["lens"] is not None:
        live = torch.arange(T)[None, :] < x["lens"].clamp(0, T)[:, None]
        for n in names:
            out[n] = torch.where(live[:, :, None, None], out[n], torch.zeros((), dtype=F64))
        w = torch.where(live[:, :, None], w, torch.ones((), dtype=F64))
    return out, w


def _state(s, B, H):
    return torch.zeros((B, H, 64, 64), dtype=F64) if s is None else s.to(F64)


def _scan(r, w, k, v, S):
    ys = []
    for t in range(r.shape[1]):
        S = w[:, t, :, None, None] * S + v[:, t, :, :, None] * k[:, t, :, None, :]
        ys.append((S * r[:, t, :, None, :]).sum(-1))
    return (torch.stack(ys, 1) if ys else torch.zeros_like(r)), S


def forward(x):
    """(y, state_out) and the same sums over magnitudes."""
    B, T, H, _ = x["r"].shape
    f, w = _inputs(x, ("r", "k", "v"))
    S = _state(x["state_in"], B, H)
    y, s = _scan(f["r"], w, f["k"], f["v"], S)
    ya, sa = _scan(f["r"].abs(), w, f["k"].abs(), f["v"].abs(), S.abs())
    return y, s, ya, sa


def _reverse(f, w, S, G):
    """Gradients from the definition (the states of every token kept)."""
    T = w.shape[1]
    states = [S]
    for t in range(T):
        S = w[:, t, :, None, None] * S + f["v"][:, t, :, :, None] * f["k"][:, t, :, None, :]
        states.append(S)
    out = {n: torch.zeros_like(f["r"]) for n in ("dr", "dk", "dv")}
    out["dlog_w"] = torch.zeros_like(w)
    for t in range(T - 1, -1, -1):
        G = G + f["dy"][:, t, :, :, None] * f["r"][:, t, :, None, :]
        out["dr"][:, t] = (states[t + 1] * f["dy"][:, t, :, :, None]).sum(-2)
        out["dk"][:, t] = (G * f["v"][:, t, :, :, None]).sum(-2)
        out["dv"][:, t] = (G * f["k"][:, t, :, None, :]).sum(-1)
        out["dlog_w"][:, t] = w[:, t] * (states[t] * G).sum((-1, -2))
        G = w[:, t, :, None, None] * G
    out["dstate_in"] = G
    return out


def backward(x):
    """The gradients and the same sums over magnitudes; dlog_w in log_w's layout."""
    B, T, H, _ = x["r"].shape
    f, w = _inputs(x, ("r", "k", "v", "dy"))
    S, G = _state(x["state_in"], B, H), _state(x["dstate_out"], B, H)
    out = _reverse(f, w, S, G)
    mag = _reverse({n: t.abs() for n, t in f.items()}, w, S.abs(), G.abs())
    if x["lens"] is not None:
        live = torch.arange(T)[None, :] < x["lens"].clamp(0, T)[:, None]
        for o in (out, mag):
            o["dlog_w"] = torch.where(live[:, :, None], o["dlog_w"], torch.zeros((), dtype=F64))
    if x["log_w"].dim() == 1:
        for o in (out, mag):
            o["dlog_w"] = o["dlog_w"].sum((0, 1))
    return out, mag


# ---- tolerances, from the arithmetic of the kernels
#
# Sums run in float32 (unit 2^-24). The longest chain of an output has at most 64 (channels) + 32
# (tokens) + 64 (channels of the state product) terms inside 32 tokens, each entering as up to six
# products of bfloat16 pieces, and up to 8 roundings for each of the T / 32 times that a state is
# scaled, added and split: 6 * 160 + 8 * ceil(T / 32) roundings of at most 2^-24 of the sum of the
# magnitudes. Decay factors: an exponential to 2 units in the last place of an argument rounded to
# 2^-24 of its size, which for arguments to -16 adds 16 + 2 units, below that the factor itself is
# under 2^-23: within the same count. What pieces leave out: 2^-24 (three pieces: 4 dropped
# products, in the same count) or 2^-16 for each of the two factors of a product (two pieces, only
# where the output is bfloat16). The output's own rounding: 2^-8 (bfloat16) of the value.
#
# Underflow: a decay factor under 2^-126, the smallest normal float32, may be 0, so it is off by at most
# 2^-126, and so is a product of factors. It multiplies a sum of at most 2^13 terms (64 * 64 of a state
# product and the tokens), each a product of at most four inputs under 8 in magnitude, 2^12: together 2^-101.
U32 = 2.0 ** -24
UNDERFLOW = 2.0 ** -101


def roundings(T):
    return 6 * 160 + 8 * -(-T // 32) + 32


def limit(ref, mag, T, bf16):
    return (2.0 ** -8 * ref.abs() if bf16 else 0.0) + (2.0 ** -15 if bf16 else 0.0) * mag + roundings(T) * U32 * mag + UNDERFLOW


def check(name, got, ref, mag, T, bf16):
    """Every element within its bound, and, as errors of both signs add as the root of their squares, the whole
    within sqrt(roundings) units (bfloat16 outputs: their rounding is uniform, so 2^-8 / sqrt(3) on average at
    most)."""
    got = got.detach().cpu().to(F64)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert torch.isfinite(got).all(), name
    if not got.numel():
        return
    over = (got - ref).abs() - limit(ref, mag, T, bf16)
    assert over.max() <= 0, "%s: %g over its bound" % (name, float(over.max()))
    unit = (2.0 ** -8 / 3 ** 0.5 * ref.norm() if bf16 else 0.0) + roundings(T) ** 0.5 * U32 * mag.norm() + \
        UNDERFLOW * mag.numel() ** 0.5
    err = float((got - ref).norm())
    assert err <= float(unit), "%s: 2-norm of the error %g, bound %g" % (name, err, float(unit))
