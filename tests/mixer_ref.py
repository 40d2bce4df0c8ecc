"""The Mamba-2 mixer's operators in float64: packed prompts as one oracle run a
sequence, the group norm and its gradient in numpy; inputs; and the bounds the
GPU results are held to."""
import numpy as np

import oracle

# Bounds, per element.  An output stored in bf16 is rounded once (at most half
# a step, 2^-8 of the value).  Behind it:
#  - scan, bf16 inputs: six operands of the block products rounded to 11
#    bits on the way to y (C, the state, C.B^T, the mixing matrix, x and its
#    skip) would be 2^-11 each of the sum of the terms' absolute values: 6 2^-11.
#    They hold 22 bits, and tests/test_mixer_rows_gpu.py holds them to it;
#  - scan, float32 inputs, and the state for both: operands of two 11-bit
#    pieces, 2^-21 each for four of them, the float32 sums over at most 64
#    steps and 256 states (bounded by 2^-24 sqrt(n) over random roundings,
#    four times that taken: 4 16 2^-24 = 2^-18) and exponentials and logarithms
#    of arguments up to 100, 2^-24 100 < 2^-17: 2^-16 in all;
#  - the convolution in float32: five terms, silu: 2^-20 of the terms' absolute
#    values, which the scan then spreads.
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
INNER = {"bf16": 6 * 2.0 ** -11, "f32": 2.0 ** -16}
STATE = 2.0 ** -16
CONV = 2.0 ** -20
#  - norm: float32 sums over at most 32768 channels in a tree of 8 per thread
#    and 12 levels (20 2^-24 < 2^-19), the reciprocal root, silu and the affine
#    step 2^-21 each: 2^-18 of the terms' absolute values; its backward has two
#    more such sums: 2^-17.  Sums over rows: n rows in strips, 2^-24 sqrt(n) of
#    the absolute terms, four times that taken.
NORM, NORM_BWD = 2.0 ** -18, 2.0 ** -17


def bf16(a):
    """float32 -> the nearest bf16, as float64 values."""
    b = np.ascontiguousarray(a, dtype=np.float32).view(np.uint32)
    b = (b + 0x7FFF + ((b >> 16) & 1)) & np.uint32(0xFFFF0000)
    return b.view(np.float32).astype(np.float64)


def mix_inputs(rng, tokens, nseq, H, P, G, N, W, dtype, nslots, gate=True, bias=True, state=True):
    ch = H * P + 2 * G * N
    q = bf16 if dtype == "bf16" else lambda a: a.astype(np.float32).astype(np.float64)
    f = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    x = dict(xbc=q(rng.standard_normal((tokens, ch))), dt=q(rng.standard_normal((tokens, H))),
             z=q(rng.standard_normal((tokens, H * P))) if gate else None,
             conv_weight=f(rng.uniform(-1, 1, (ch, W)) / np.sqrt(W)),
             conv_bias=f(rng.uniform(-0.5, 0.5, ch)) if bias else None,
             A=f(-rng.uniform(1, 16, H)), D=f(rng.standard_normal(H)) if bias else None,
             dt_bias=f(np.log(np.expm1(rng.uniform(1e-3, 1e-1, H)))) if bias else None)
    if state:
        x["conv_state"] = f(rng.standard_normal((nslots, ch, W - 1)))
        x["ssm_state"] = f(rng.standard_normal((nslots, H, P, N)) * 0.3)
    return x


def _split(c, H, P, G, N):
    """[channels, L] of the convolution -> x, B, C as the oracle takes them."""
    return c[None, :H * P], c[None, H * P:H * P + G * N], c[None, H * P + G * N:]


def mix(x, cu, G, slots=None, has=None, softplus=True):
    """y, conv_state, ssm_state of the packed call, and the bounds' sums: for y
    and ssm_state the sum of the terms' absolute values with the convolution's
    values (first) and with its terms' absolute values (second)."""
    tokens, ch = x["xbc"].shape
    W, H = x["conv_weight"].shape[1], len(x["A"])
    state = "ssm_state" in x
    inner = x["z"].shape[1] if x["z"] is not None else x["inner"]
    P, N = inner // H, (ch - inner) // (2 * G)
    y = np.full((tokens, inner), np.nan)
    ya, yc = np.zeros_like(y), np.zeros_like(y)
    cs = x["conv_state"].copy() if state else None
    hs = x["ssm_state"].copy() if state else None
    ha, hc = (np.zeros_like(hs), np.zeros_like(hs)) if state else (None, None)
    ab = lambda v: None if v is None else np.abs(v)  # noqa: E731
    for s in range(len(cu) - 1):
        a, b = cu[s], cu[s + 1]
        slot = s if slots is None else slots[s]
        if state and not 0 <= slot < len(hs):
            continue
        resume = state and has is not None and has[s]
        c0 = x["conv_state"][slot][None] if resume else np.zeros((1, ch, W - 1))
        h0 = x["ssm_state"][slot][None] if resume else np.zeros((1, H, P, N))
        if b > a:
            xin = np.ascontiguousarray(x["xbc"][a:b].T)[None]
            c, c1 = oracle.conv1d(xin, x["conv_weight"], bias=x["conv_bias"], state_in=c0)
            cabs, _ = oracle.conv1d(np.abs(xin), ab(x["conv_weight"]), bias=ab(x["conv_bias"]),
                                    state_in=np.abs(c0), silu=False)
            dt = np.ascontiguousarray(x["dt"][a:b].T)[None]
            zt = np.ones((1, inner, b - a))
            if x["z"] is not None:
                zt = np.ascontiguousarray(x["z"][a:b].T)[None]
                zt = zt / (1 + np.exp(-zt))

            def scan(c, D, h0):
                xs, B, C = _split(c, H, P, G, N)
                yy, h = oracle.ssd(np.ascontiguousarray(xs), dt, x["A"], np.ascontiguousarray(B),
                                   np.ascontiguousarray(C), H, G, D=D, dt_bias=x["dt_bias"],
                                   dt_softplus=softplus, h0=h0)
                return yy, h

            # The terms of y_t are decay dt_s x_s B_s C_t, the decays positive: with |B|, |C| and
            # x = |x| sign(dt) each is its absolute value, also where a step is negative; D x apart.
            raw = dt[0] + (0 if x["dt_bias"] is None else x["dt_bias"][:, None])
            sign = np.ones_like(raw) if softplus else np.where(raw < 0, -1.0, 1.0)

            def absolute(c):
                s = c.copy()
                s[:inner] *= np.repeat(sign, P, 0)
                yy, h = scan(s, None, np.abs(h0))
                if x["D"] is not None:
                    yy = yy + np.repeat(ab(x["D"]), P)[None, :, None] * c[None, :inner]
                return yy, h

            v, h1 = scan(c[0], x["D"], h0)
            y[a:b] = (v * zt)[0].T
            v, h1a = absolute(np.abs(c[0]))
            ya[a:b] = (v * np.abs(zt))[0].T
            v, h1c = absolute(cabs[0])
            yc[a:b] = (v * np.abs(zt))[0].T
        else:
            c1, h1, h1a, h1c = c0, h0, np.abs(h0), np.abs(h0)
        if state:
            cs[slot], hs[slot], ha[slot], hc[slot] = c1[0], h1[0], h1a[0], h1c[0]
    return y, cs, hs, (ya, yc), (ha, hc)


def mix_excess(got, ref, sums, dtype):
    """Largest |got - ref| over its bound, for y (dtype of the rows) or the state."""
    inner = STATE if dtype == "state" else INNER[dtype]
    tol = HALF.get(dtype, 2.0 ** -24) * np.abs(ref) + inner * sums[0] + CONV * sums[1] + 1e-30
    return float(np.max(np.abs(got - ref) / tol)) if ref.size else 0.0


# ---------------------------------------------------------------- group norm

def _sig(v):
    return 1 / (1 + np.exp(-v))


def norm_parts(x, w, G, b, z, eps, center, act, gate):
    rows, C = x.shape
    v = x * z * _sig(z) if gate == "before" else x
    vg = v.reshape(rows, G, -1)
    m = vg.mean(2, keepdims=True) if center else np.zeros((rows, G, 1))
    r = 1 / np.sqrt(((vg - m) ** 2).mean(2, keepdims=True) + eps)
    n = ((vg - m) * r).reshape(rows, C)
    nabs = ((np.abs(vg) + np.abs(m)) * r).reshape(rows, C)
    a = n * w + b
    return n, nabs, r, a


def norm(x, w, G, b, z, eps=1e-5, center=False, act="none", gate="none"):
    """(y, sum of the absolute terms); w, b, z may be None."""
    w = np.ones(x.shape[1]) if w is None else w
    b = np.zeros(x.shape[1]) if b is None else b
    n, nabs, r, a = norm_parts(x, w, G, b, z, eps, center, act, gate)
    bound = nabs * np.abs(w) + np.abs(b)
    y = a * _sig(a) if act == "silu" else a
    if gate == "after":
        y, bound = y * z * _sig(z), bound * np.abs(z) * _sig(z)
    return y, bound


def norm_bwd(dy, x, w, G, b, z, eps=1e-5, center=False, act="none", gate="none"):
    """dict of gradients, and the same dict of the sums of their absolute terms."""
    rows, C = x.shape
    w = np.ones(C) if w is None else w
    b = np.zeros(C) if b is None else b
    n, nabs, r, a = norm_parts(x, w, G, b, z, eps, center, act, gate)
    g, t = {}, {}
    aabs = nabs * np.abs(w) + np.abs(b)
    up, upabs = dy, np.abs(dy)
    if gate == "after":
        s = _sig(z)
        o = a * _sig(a) if act == "silu" else a
        g["dz"] = dy * o * s * (1 + z * (1 - s))
        t["dz"] = np.abs(dy) * aabs * s * (1 + np.abs(z) * (1 - s))
        up, upabs = up * z * s, upabs * np.abs(z) * s
    if act == "silu":
        s = _sig(a)
        # |second derivative| of silu is at most 1/2: an error of a moves it by half of that
        upabs = upabs * (s * (1 + np.abs(a) * (1 - s)) + 0.5 * aabs)
        up = up * s * (1 + a * (1 - s))
    g["dweight"], t["dweight"] = (up * n).sum(0), (upabs * nabs).sum(0)
    g["dbias"], t["dbias"] = up.sum(0), upabs.sum(0)
    grp = lambda v: v.reshape(rows, G, -1)  # noqa: E731
    u, uabs = grp(up * w), grp(upabs * np.abs(w))
    ng, nag = grp(n), grp(nabs)
    d = u - ng * (u * ng).mean(2, keepdims=True)
    dabs = uabs + nag * (uabs * nag).mean(2, keepdims=True)
    if center:
        d, dabs = d - u.mean(2, keepdims=True), dabs + uabs.mean(2, keepdims=True)
    d, dabs = (d * r).reshape(rows, C), (dabs * r).reshape(rows, C)
    if gate == "before":
        s = _sig(z)
        g["dz"], t["dz"] = d * x * s * (1 + z * (1 - s)), dabs * np.abs(x) * s * (1 + np.abs(z) * (1 - s))
        d, dabs = d * z * s, dabs * np.abs(z) * s
    g["dx"], t["dx"] = d, dabs
    return g, t
