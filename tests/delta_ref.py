"""The gated delta rule and the norm with the residual's addition in float64, one
token and one row at a time; inputs; and the bounds the GPU results are held to."""
import numpy as np

from mixer_ref import bf16

# Bounds, per element.  An output stored in bf16 is rounded once (half a step, 2^-8 of
# the value; float32 2^-24).  Behind it, for a column p of a head's state (its dstate
# values for one channel), with c_p the largest |S_p| (2-norm) and |v_p| that the
# sequence meets:
#  - a block of 64 tokens reads the column at its keys (operands of 22 bits, sums over
#    up to 256 states: 2^-22 c_p a row), goes through T, whose entries are at most one
#    for keys no longer than one (64 rows of random errors: sqrt(64)), and writes the
#    rows back (64 keys again: sqrt(64)): 2^-22 64 c_p = 2^-16 c_p a block;
#  - a step's transition is no longer than one, so blocks' errors add up at random:
#    sqrt(blocks), decays aside.
# State: E c_p with E = 2^-16 sqrt(blocks).  y: E c_p |q^|.  Backwards the same holds for
# the gradient of a column, g_p the largest |dS_p| of the sequence:
#  - dv: E g_p;  dq^: sum_p |dy_p| E c_p;  dk^: three products of the two, sum_p 3 E c_p g_p;
#  - dbeta, the log decay: sum_p 2 E c_p g_p each, and the log decay's running sum over 64
#    rows adds its terms' own roundings, 64 2^-24 sum_p c_p g_p: below another E;
#  - dA, ddt_bias: the rows' bounds added up.
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
BLOCK = 2.0 ** -16


def _q(dtype):
    return bf16 if dtype == "bf16" else lambda a: np.asarray(a, dtype=np.float32).astype(np.float64)


def delta_inputs(rng, tokens, nseq, H, G, P, N, dtype, nslots, bias=True, state=True, kstd=1.0):
    q = _q(dtype)
    f = lambda a: np.asarray(a, dtype=np.float32).astype(np.float64)  # noqa: E731
    x = dict(q=q(rng.standard_normal((tokens, G * N)) * kstd), k=q(rng.standard_normal((tokens, G * N)) * kstd),
             v=q(rng.standard_normal((tokens, H * P))), dt=q(rng.standard_normal((tokens, H))),
             beta=q(rng.standard_normal((tokens, H))), A=f(-rng.uniform(1, 16, H)),
             dt_bias=f(np.log(np.expm1(rng.uniform(1e-3, 1e-1, H)))) if bias else None,
             dy=q(rng.standard_normal((tokens, H * P))))
    if state:
        x["state"] = f(rng.standard_normal((nslots, H, P, N)) * 0.3)
    return x


def _sig(v):
    return 1 / (1 + np.exp(-v))


class How:
    def __init__(self, softplus=True, sigmoid=True, norm=True, eps=1e-6, scale=None):
        self.softplus, self.sigmoid, self.norm, self.eps, self.scale = softplus, sigmoid, norm, eps, scale

    def kw(self):
        return dict(dt_softplus=self.softplus, beta_sigmoid=self.sigmoid, qk_norm=self.norm, eps=self.eps,
                    scale=self.scale)


def rows(x, G, how):
    """Normalised rows and scalars, every head its own: q, k [T, H, N], v [T, H, P], a, b, dt [T, H]."""
    T, H = x["dt"].shape
    N, P = x["q"].shape[1] // G, x["v"].shape[1] // H
    scale = N ** -0.5 if how.scale is None else how.scale
    q, k = x["q"].reshape(T, G, N), x["k"].reshape(T, G, N)
    lq = np.sqrt((q * q).sum(2, keepdims=True) + how.eps) if how.norm else np.ones((T, G, 1))
    lk = np.sqrt((k * k).sum(2, keepdims=True) + how.eps) if how.norm else np.ones((T, G, 1))
    raw = x["dt"] + (0 if x["dt_bias"] is None else x["dt_bias"])
    dt = np.logaddexp(0, raw) if how.softplus else raw
    wide = lambda v: np.repeat(v, H // G, 1)  # noqa: E731
    return dict(q=wide(q / lq * scale), k=wide(k / lk), lq=lq, lk=lk, scale=scale, v=x["v"].reshape(T, H, P), raw=raw,
                dt=dt, a=np.exp(dt * x["A"]), b=_sig(x["beta"]) if how.sigmoid else x["beta"])


def _walk(r, lo, hi, S):
    """One sequence: the states before every token and the last, u, c_p."""
    before, us, c = [], [], np.linalg.norm(S, axis=2)
    for t in range(lo, hi):
        before.append(S)
        old = S * r["a"][t][:, None, None]
        u = r["b"][t][:, None] * (r["v"][t] - np.matmul(old, r["k"][t][:, :, None])[..., 0])
        S = old + u[:, :, None] * r["k"][t][:, None, :]
        us.append(u)
        c = np.maximum(c, np.maximum(np.linalg.norm(S, axis=2), np.abs(r["v"][t])))
    return before, us, S, c


def err(lo, hi):
    return BLOCK * np.sqrt(max(1, -(-(hi - lo) // 64)))


def delta(x, cu, G, how, slots=None, has=None):
    """y (NaN where no sequence writes it), the states after, and both bounds without the half step."""
    r = rows(x, G, how)
    T, H, P = r["v"].shape
    y, yb = np.full((T, H * P), np.nan), np.zeros((T, H * P))
    state = x["state"].copy() if "state" in x else None
    sb = np.zeros_like(state) if state is not None else None
    N = r["q"].shape[2]
    for s in range(len(cu) - 1):
        lo, hi = cu[s], cu[s + 1]
        slot = s if slots is None else slots[s]
        if state is not None and not 0 <= slot < len(state):
            continue
        S = x["state"][slot] if state is not None and has is not None and has[s] else np.zeros((H, P, N))
        before, us, end, c = _walk(r, lo, hi, S)
        states = before[1:] + [end]
        for i, t in enumerate(range(lo, hi)):
            y[t] = np.matmul(states[i], r["q"][t][:, :, None])[..., 0].reshape(-1)
            yb[t] = (err(lo, hi) * c * np.linalg.norm(r["q"][t], axis=1)[:, None]).reshape(-1)
        if state is not None:
            state[slot], sb[slot] = end, (err(lo, hi) * c)[..., None] if hi > lo else 0
    return y, state, yb, sb


def delta_bwd(x, cu, G, how, h0=None, dfinal=None):
    """dict of gradients for sum(dy y) + sum(dfinal final_state), and of their bounds."""
    r = rows(x, G, how)
    T, H, P = r["v"].shape
    N, nseq = r["q"].shape[2], len(cu) - 1
    dq, dk, dv = np.zeros((T, H, N)), np.zeros((T, H, N)), np.zeros((T, H, P))
    bq, bk, bv = np.zeros((T, H, 1)), np.zeros((T, H, 1)), np.zeros((T, H, P))
    dg, db, bg = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    dh0, bh = np.zeros((nseq, H, P, N)), np.zeros((nseq, H, P, 1))
    dy = x["dy"].reshape(T, H, P)
    for s in range(nseq):
        lo, hi = cu[s], cu[s + 1]
        S0 = np.zeros((H, P, N)) if h0 is None else h0[s]
        before, us, end, c = _walk(r, lo, hi, S0)
        states = before[1:] + [end]
        d = np.zeros((H, P, N)) if dfinal is None else dfinal[s].copy()
        gmax = np.linalg.norm(d, axis=2)
        for t in range(hi - 1, lo - 1, -1):
            i = t - lo
            k, q, old = r["k"][t], r["q"][t], before[i] * r["a"][t][:, None, None]
            d = d + dy[t][:, :, None] * q[:, None, :]
            gmax = np.maximum(gmax, np.maximum(np.linalg.norm(d, axis=2), np.abs(dy[t]) * np.linalg.norm(q, axis=1)[:, None]))
            dq[t] = np.matmul(dy[t][:, None, :], states[i])[:, 0]
            du = np.matmul(d, k[:, :, None])[..., 0]
            db[t] = (du * (r["v"][t] - np.matmul(old, k[:, :, None])[..., 0])).sum(1)
            dv[t] = r["b"][t][:, None] * du
            dk[t] = np.matmul(us[i][:, None, :], d)[:, 0] - np.matmul(dv[t][:, None, :], old)[:, 0]
            d = d - dv[t][:, :, None] * k[:, None, :]
            dg[t] = (d * old).sum((1, 2))
            d = d * r["a"][t][:, None, None]
            gmax = np.maximum(gmax, np.linalg.norm(d, axis=2))
        dh0[s], bh[s] = d, (err(lo, hi) * gmax)[..., None]
        e, both = err(lo, hi), (c * gmax).sum(1)
        bv[lo:hi] = e * gmax
        bq[lo:hi] = e * (np.abs(dy[lo:hi]) * c).sum(2)[..., None]
        bk[lo:hi] = 3 * e * both[:, None]
        bg[lo:hi] = 3 * e * both
    slope = _sig(r["raw"]) if how.softplus else 1.0
    ddt = dg * x["A"] * slope
    bdt = bg * np.abs(x["A"]) * slope
    bb = r["b"] * (1 - r["b"]) if how.sigmoid else 1.0
    g = dict(dv=dv.reshape(T, -1), ddt=ddt, dbeta=db * bb, dA=(dg * r["dt"]).sum(0), ddt_bias=ddt.sum(0), dh0=dh0)
    b = dict(dv=bv.reshape(T, -1), ddt=bdt, dbeta=bg * np.abs(bb), dA=(bg * np.abs(r["dt"])).sum(0),
             ddt_bias=bdt.sum(0), dh0=bh)
    for name, d, bound, u, length, scale in (("dq", dq, bq, r["q"] / r["scale"], r["lq"], r["scale"]),
                                             ("dk", dk, bk, r["k"], r["lk"], 1.0)):
        d, bound = (v.reshape(T, G, H // G, -1).sum(2) for v in (d, bound))
        if how.norm:
            u = u[:, ::H // G]
            # the projection takes off what the gradient has along the row: rounded where it is formed
            size = np.linalg.norm(d, axis=2, keepdims=True)
            d = (d - u * (u * d).sum(2, keepdims=True)) / length
            bound = (2 * bound + BLOCK * size) / length
        g[name] = (d * scale).reshape(T, -1)
        b[name] = np.broadcast_to(bound * abs(scale), d.shape).reshape(T, -1)
    return g, b


# ---------------------------------------------------------------- norm with the residual's addition

# float32 sums over at most 32768 channels in a tree of 8 per thread and 12 levels (20
# 2^-24 < 2^-19), the reciprocal root and the products 2^-21: 2^-18 of the terms' absolute
# values; the backward has another such sum, 2^-17.  Sums over rows: 2^-24 sqrt(rows)
# of the absolute terms, four times that taken.
NORM, NORM_BWD = 2.0 ** -18, 2.0 ** -17


def add_norm(r, w, eps=1e-5):
    """y of the stored stream r."""
    return r / np.sqrt((r * r).mean(1, keepdims=True) + eps) * (1 if w is None else w)


def add_norm_bwd(dy, r, w, dr=None, eps=1e-5):
    """(dx, dweight, and the sums of their absolute terms)."""
    w = np.ones(r.shape[1]) if w is None else w
    i = 1 / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    n, u = r * i, dy * w
    d = (u - n * (u * n).mean(1, keepdims=True)) * i
    dabs = (np.abs(u) + np.abs(n) * np.abs(u * n).mean(1, keepdims=True)) * i
    if dr is not None:
        d, dabs = d + dr, dabs + np.abs(dr)
    return d, (dy * n).sum(0), dabs, np.abs(dy * n).sum(0)
