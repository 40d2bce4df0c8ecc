"""Measured calls of the Mamba-2 mixer's operators: the causal convolution and
scan over packed prompts, the same for one token a sequence, and the group norm
with its gate or activation, forward and backward.

`run` computes each in elementary torch operations (`own` false) or through the
library (`own` true); `exact` computes the definition in float64, step by step.

Shapes: the Mamba-2 2.7B layer of the benchmark's workloads (80 heads of 64
channels, 128 states, one group, convolution of width 4), the 1536-channel
width of its 130M workload (24 heads of 64), and generic smaller ones.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64  # tokens per block of the plain scan
BIG = 32768 * 80 * 64 * 128  # scan elements of the largest listed prompt case
WIDE = 32768 * 5120  # elements of the largest listed norm case


def listed():
    def prompts(name, tokens, nseq, heads, headdim, groups, dstate, dtype, gate, resume, ragged):
        return dict(name=name, op="prompts", tokens=tokens, nseq=nseq, heads=heads, headdim=headdim,
                    groups=groups, dstate=dstate, width=4, dtype=dtype, gate=gate, resume=resume,
                    ragged=ragged)

    def step(name, batch, heads, headdim, groups, dstate, dtype, gate, pad):
        return dict(name=name, op="step", batch=batch, heads=heads, headdim=headdim, groups=groups,
                    dstate=dstate, width=4, dtype=dtype, gate=gate, pad=pad)

    def norm(name, op, rows, channels, groups, dtype, center, act, gate, bias):
        return dict(name=name, op=op, rows=rows, channels=channels, groups=groups, dtype=dtype,
                    center=center, act=act, gate=gate, bias=bias)

    return [
        # one short question on a small model: latency
        prompts("prompt_37", 37, 1, 24, 64, 1, 128, "bf16", False, False, False),
        # a serving batch of mixed prompts, some continuing from their cache
        prompts("prompts_ragged", 8111, 16, 80, 64, 1, 128, "bf16", False, True, True),
        # the benchmark's Mamba-2 layer: four prompts of 8192 tokens, gate in the scan
        prompts("prompts_4x8192", 32768, 4, 80, 64, 1, 128, "bf16", True, False, False),
        # one long document on a small model: few heads, a long axis
        prompts("prompt_32768", 32768, 1, 24, 64, 1, 128, "bf16", False, False, False),
        # float32 activations, several groups, odd lengths
        prompts("prompts_f32", 2999, 5, 16, 32, 4, 64, "f32", True, True, True),
        # a single user's next token: latency
        step("step_1", 1, 80, 64, 1, 128, "bf16", False, 0),
        # the benchmark's decode batch, a few entries of it padding
        step("step_256", 256, 80, 64, 1, 128, "bf16", False, 3),
        # float32, wide heads, large states
        step("step_f32", 19, 16, 128, 2, 256, "f32", True, 1),
        # a single user's token between scan and projection
        norm("norm_1", "norm", 1, 5120, 1, "bf16", False, "none", "before", False),
        # a long prompt's gated norm, one group
        norm("norm_32768", "norm", 32768, 5120, 1, "bf16", False, "none", "before", False),
        # training step of the same with eight groups
        norm("norm_bwd_16384", "norm_bwd", 16384, 5120, 8, "bf16", False, "none", "before", False),
        # centred norm with silu, odd row count and group size, float32
        norm("norm_bwd_odd", "norm_bwd", 1237, 1000, 5, "f32", True, "silu", "none", True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompts", "step", "norm", "norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("prompts", "step"):
        groups = rng.choice([1, 1, 2, 4])
        heads = groups * _log(rng, 1, 80 // groups)
        headdim = rng.choice([16, 32, 48, 64, 64, 64, 80, 128])
        dstate = rng.choice([16, 32, 64, 96, 128, 128, 256])
        c = dict(op=op, heads=heads, headdim=headdim, groups=groups, dstate=dstate,
                 width=rng.choice([2, 3, 4, 4]), dtype=dtype, gate=rng.random() < 0.5)
        if op == "prompts":
            nseq = _log(rng, 1, 64)
            top = max(nseq, min(32768, BIG // (heads * headdim * dstate)) - CHUNK * nseq)
            c.update(tokens=_log(rng, nseq, top), nseq=nseq, resume=rng.random() < 0.5,
                     ragged=rng.random() < 0.7)
        else:
            c.update(batch=_log(rng, 1, 256), pad=rng.choice([0, 0, 1, 2]))
        return c
    groups = rng.choice([1, 1, 2, 5, 8, 24])
    per = _log(rng, 16, 8192 // groups)
    channels = groups * per
    return dict(op=op, rows=_log(rng, 1, min(65536, WIDE // (2 * channels))), channels=channels,
                groups=groups, dtype=dtype, center=rng.random() < 0.4,
                act=rng.choice(["none", "none", "silu"]),
                gate=rng.choice(["none", "before", "before", "after"]), bias=rng.random() < 0.4)


# ---------------------------------------------------------------- inputs

_IO = {"bf16": torch.bfloat16, "f32": torch.float32}


def _cu(c):
    """Starts of the packed sequences (host)."""
    if not c["ragged"]:
        at = [c["tokens"] * s // c["nseq"] for s in range(c["nseq"] + 1)]
    else:
        r = np.random.RandomState(c["tokens"] * 7 + c["nseq"])
        at = [0, *sorted(r.randint(0, c["tokens"] + 1, c["nseq"] - 1)), c["tokens"]]
    return [int(v) for v in at]


def prepare(case, seed):
    c = case
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=dev) * std

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device=dev) * (hi - lo) + lo

    io = _IO[c["dtype"]]
    s = dict(case=c)
    if c["op"] in ("prompts", "step"):
        H, P, G, N, W = c["heads"], c["headdim"], c["groups"], c["dstate"], c["width"]
        inner, conv = H * P, H * P + 2 * G * N
        rows = c["tokens"] if c["op"] == "prompts" else c["batch"]
        # one row of the input projection holds z, the convolution's channels and dt
        proj = normal(rows, inner + conv + H).to(io)
        s.update(z=proj[:, :inner] if c["gate"] else None, xbc=proj[:, inner:inner + conv],
                 dt=proj[:, inner + conv:], conv_weight=uniform(conv, W, lo=-W ** -0.5, hi=W ** -0.5),
                 conv_bias=uniform(conv, lo=-0.5, hi=0.5), A=-uniform(H, lo=1.0, hi=16.0),
                 D=normal(H), dt_bias=torch.log(torch.expm1(uniform(H, lo=1e-3, hi=1e-1))))
        nseq = c["nseq"] if c["op"] == "prompts" else c["batch"]
        nslots = nseq + 3
        slots = torch.randperm(nslots, generator=g, device=dev)[:nseq].to(torch.int32)
        s.update(conv_state=normal(nslots, conv, W - 1), ssm_state=normal(nslots, H, P, N, std=0.1))
        s["y"] = torch.zeros(rows, inner, dtype=io, device=dev)
        if c["op"] == "prompts":
            cu = _cu(c)
            s["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device=dev)
            s["has_state"] = (torch.arange(nseq, device=dev) % 2 == 0).to(torch.uint8) if c["resume"] else None
        else:
            slots[nseq - min(c["pad"], nseq - 1):] = -1  # entries that a padded batch leaves empty
        s["slots"] = slots
        return s
    rows, C = c["rows"], c["channels"]
    s["x"] = normal(rows, C).to(io)
    s["z"] = normal(rows, 2 * C + 16).to(io)[:, :C] if c["gate"] != "none" else None  # a slice of the projection
    s["weight"] = 1 + normal(C, std=0.2)
    s["bias"] = normal(C, std=0.2) if c["bias"] else None
    if c["op"] == "norm":
        s["y"] = torch.empty(rows, C, dtype=io, device=dev)
    else:
        s["dy"] = normal(rows, C).to(io)
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return (_own if own else _plain)[state["case"]["op"]](state)


def _workspace(s, nbytes):
    """The workspace that a program keeps between its calls, made on the first."""
    if "workspace" not in s:
        s["workspace"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_prompts(s):
    import selective_state_space_43_amd as ssm
    c = s["case"]
    need = ssm.ssm_conv_ssd_workspace_size(c["tokens"], c["nseq"], c["heads"], c["headdim"],
                                           c["groups"], c["dstate"], s["xbc"].dtype)
    ssm.ssm_conv_ssd_fwd(s["xbc"], s["dt"], s["conv_weight"], s["A"], s["cu_seqlens"], c["headdim"],
                         c["groups"], conv_bias=s["conv_bias"], D=s["D"], z=s["z"],
                         dt_bias=s["dt_bias"], slots=s["slots"], has_state=s["has_state"],
                         conv_state=s["conv_state"], ssm_state=s["ssm_state"], y=s["y"],
                         workspace=_workspace(s, need))
    return s["y"], s["conv_state"], s["ssm_state"]


def _own_step(s):
    import selective_state_space_43_amd as ssm
    ssm.ssm_conv_ssd_update(s["xbc"], s["dt"], s["conv_state"], s["ssm_state"], s["conv_weight"],
                            s["A"], s["case"]["groups"], conv_bias=s["conv_bias"], D=s["D"], z=s["z"],
                            dt_bias=s["dt_bias"], slots=s["slots"], y=s["y"])
    return s["y"], s["conv_state"], s["ssm_state"]


def _own_norm(s):
    import selective_state_space_43_amd as ssm
    c = s["case"]
    return ssm.ssm_group_norm_fwd(s["x"], s["weight"], c["groups"], bias=s["bias"], z=s["z"],
                                  center=c["center"], activation=c["act"], gate=c["gate"], y=s["y"])


def _own_norm_bwd(s):
    import selective_state_space_43_amd as ssm
    c = s["case"]
    need = ssm.ssm_group_norm_bwd_workspace_size(c["rows"], c["channels"], c["groups"])
    g = ssm.ssm_group_norm_bwd(s["dy"], s["x"], s["weight"], c["groups"], bias=s["bias"], z=s["z"],
                               center=c["center"], activation=c["act"], gate=c["gate"],
                               workspace=_workspace(s, need))
    return {k: v for k, v in g.items() if v is not None}


_own = dict(prompts=_own_prompts, step=_own_step, norm=_own_norm, norm_bwd=_own_norm_bwd)


def _silu(v):
    return v / (1 + torch.exp(-v))


def _softplus(v):
    return torch.where(v > 20, v, torch.log1p(torch.exp(torch.clamp(v, max=20))))


def _plain_prompts(s):
    c = s["case"]
    H, P, G, N, W = c["heads"], c["headdim"], c["groups"], c["dstate"], c["width"]
    T, S, inner = c["tokens"], c["nseq"], H * P
    dev, cu, slots = s["xbc"].device, s["cu_seqlens"].long(), s["slots"].long()
    lens = cu[1:] - cu[:-1]
    keep = torch.zeros(S, device=dev) if s["has_state"] is None else s["has_state"].float()
    cs0 = s["conv_state"][slots] * keep[:, None, None]
    h0 = s["ssm_state"][slots] * keep[:, None, None, None]
    # causal convolution and silu; inputs before a sequence come from its cache
    x32 = s["xbc"].float()
    tok = torch.arange(T, device=dev)
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True).clamp(max=S - 1)
    pos = tok - cu[seq]
    start = torch.cat([cs0.transpose(1, 2), torch.zeros(S, W - 1, cs0.shape[1], device=dev)], 1)

    def at(back):  # the input `back` tokens before each token
        old = start[seq, (W - 1 + pos - back).clamp(0, 2 * W - 3)]
        return torch.where((pos >= back)[:, None], x32[(tok - back).clamp(min=0)], old)

    pre = s["conv_bias"] + sum(s["conv_weight"][:, k] * at(W - 1 - k) for k in range(W))
    act = _silu(pre)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    # the tokens in blocks of one sequence each, padded with steps of zero
    blocks = (lens + CHUNK - 1) // CHUNK
    ends = torch.cumsum(blocks, 0)
    nc = T // CHUNK + S
    blk = torch.arange(nc, device=dev)
    bseq = torch.searchsorted(ends, blk, right=True)
    live = bseq < S
    bseq = bseq.clamp(max=S - 1)
    first = (cu[:-1] - (ends - blocks) * CHUNK)[bseq] + blk * CHUNK
    idx = first[:, None] + torch.arange(CHUNK, device=dev)
    ok = live[:, None] & (idx < cu[1:][bseq][:, None])
    idx = idx.clamp(0, T - 1)
    xb = act[:, :inner][idx].view(nc, CHUNK, H, P).transpose(1, 2)
    per = H // G
    Bb = act[:, inner:inner + G * N][idx].view(nc, CHUNK, G, N).transpose(1, 2)
    Cb = act[:, inner + G * N:][idx].view(nc, CHUNK, G, N).transpose(1, 2)
    del pre
    dtb = torch.where(ok[..., None], dt[idx], torch.zeros((), device=dev)).transpose(1, 2)
    cum = torch.cumsum(dtb.double() * s["A"].double()[:, None], -1)
    total = cum[..., -1]
    CB = torch.matmul(Cb, Bb.transpose(-1, -2).contiguous())
    lower = torch.ones(CHUNK, CHUNK, device=dev, dtype=torch.bool).tril()
    mix = torch.exp((cum[..., :, None] - cum[..., None, :]).masked_fill(~lower, -math.inf)).float()
    mix = mix * CB.repeat_interleave(per, 1) * dtb[..., None, :]
    y = torch.matmul(mix, xb)
    del mix
    tail = torch.exp(total[..., None] - cum).float() * dtb
    local = torch.matmul((xb * tail[..., None]).transpose(-1, -2).contiguous(),
                         Bb.repeat_interleave(per, 1))
    # the state entering each block: the blocks before it in its sequence, and the cache
    E = torch.cumsum(total, 0).transpose(0, 1)
    before = E - total.transpose(0, 1)
    link = (bseq[:, None] == bseq[None, :]) & (blk[:, None] > blk[None, :])
    reach = torch.exp((before[:, :, None] - E[:, None, :]).masked_fill(~link, -math.inf)).float()
    hin = torch.matmul(reach, local.transpose(0, 1).reshape(H, nc, P * N))
    at0 = (ends - blocks)[bseq].clamp(max=nc - 1)
    since = torch.exp(before - before[:, at0]).float()
    hin = hin.view(H, nc, P, N).transpose(0, 1) + since.transpose(0, 1)[..., None, None] * h0[bseq]
    y = y + torch.exp(cum).float()[..., None] * torch.matmul(
        Cb.repeat_interleave(per, 1), hin.transpose(-1, -2).contiguous())
    y = y + s["D"][:, None, None] * xb
    hout = torch.exp(total).float()[..., None, None] * hin + local
    last = (ends - 1).clamp(min=0)
    final = torch.where((lens > 0)[:, None, None, None], hout[last], h0)
    # every token lies in one block: back to rows
    row = (ends - blocks)[seq] * CHUNK + pos
    y = y.transpose(1, 2).reshape(nc * CHUNK, inner)[row]
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["y"].copy_(y)
    back = torch.arange(W - 1, device=dev) - (W - 1)  # the last W-1 inputs, oldest first
    rel = lens[:, None] + back
    new = torch.where((rel >= 0)[..., None], x32[(cu[:-1, None] + rel).clamp(0, T - 1)],
                      start[torch.arange(S, device=dev)[:, None], (rel + W - 1).clamp(0, W - 2)])
    s["conv_state"][slots] = new.transpose(1, 2)
    s["ssm_state"][slots] = final
    return s["y"], s["conv_state"], s["ssm_state"]


def _plain_step(s):
    c = s["case"]
    H, P, G, N, W = c["heads"], c["headdim"], c["groups"], c["dstate"], c["width"]
    n, inner = c["batch"] - min(c["pad"], c["batch"] - 1), H * P  # the entries in use come first
    slots = s["slots"][:n].long()
    x32 = s["xbc"][:n].float()
    win = torch.cat([s["conv_state"][slots], x32[:, :, None]], 2)
    act = _silu((win * s["conv_weight"]).sum(2) + s["conv_bias"])
    dt = _softplus(s["dt"][:n].float() + s["dt_bias"])
    x = act[:, :inner].view(n, H, P)
    B = act[:, inner:inner + G * N].view(n, G, N).repeat_interleave(H // G, 1)
    C = act[:, inner + G * N:].view(n, G, N).repeat_interleave(H // G, 1)
    h = s["ssm_state"][slots] * torch.exp(dt * s["A"])[..., None, None]
    h = h + (dt[..., None] * x)[..., None] * B[:, :, None, :]
    y = (h * C[:, :, None, :]).sum(-1) + s["D"][:, None] * x
    y = y.reshape(n, inner)
    if s["z"] is not None:
        y = y * _silu(s["z"][:n].float())
    s["y"][:n] = y.to(s["y"].dtype)
    s["conv_state"][slots] = win[:, :, 1:]
    s["ssm_state"][slots] = h
    return s["y"], s["conv_state"], s["ssm_state"]


def _normed(s, v, wide):
    """(centred and scaled, 1 / deviation) of each group, and the affine result."""
    c = s["case"]
    rows, G = c["rows"], c["groups"]
    v = v.view(rows, G, -1)
    if c["center"]:
        v = v - v.mean(-1, keepdim=True)
    r = torch.rsqrt((v * v).mean(-1, keepdim=True) + 1e-5)
    n = v * r
    a = n.view(rows, -1) * s["weight"].to(wide)
    return n, r, a if s["bias"] is None else a + s["bias"].to(wide)


def _plain_norm(s):
    c = s["case"]
    x, z = s["x"].float(), None if s["z"] is None else s["z"].float()
    _, _, a = _normed(s, x * _silu(z) if c["gate"] == "before" else x, torch.float32)
    if c["act"] == "silu":
        a = _silu(a)
    if c["gate"] == "after":
        a = a * _silu(z)
    s["y"].copy_(a)
    return s["y"]


def _plain_norm_bwd(s):
    c = s["case"]
    rows, G = c["rows"], c["groups"]
    x, g, io = s["x"].float(), s["dy"].float(), s["x"].dtype
    out = {}
    if s["z"] is not None:
        z = s["z"].float()
        sg = 1 / (1 + torch.exp(-z))
        slope = sg * (1 + z * (1 - sg))
    n, r, a = _normed(s, x * (z * sg) if c["gate"] == "before" else x, torch.float32)
    if c["gate"] == "after":
        out["dz"] = (g * (_silu(a) if c["act"] == "silu" else a) * slope).to(io)
        g = g * (z * sg)
    if c["act"] == "silu":
        sa = 1 / (1 + torch.exp(-a))
        g = g * (sa * (1 + a * (1 - sa)))
    out["dweight"] = (g * n.view(rows, -1)).sum(0)
    if s["bias"] is not None:
        out["dbias"] = g.sum(0)
    u = (g * s["weight"]).view(rows, G, -1)
    d = u - n * (u * n).mean(-1, keepdim=True)
    if c["center"]:
        d = d - u.mean(-1, keepdim=True)
    d = (d * r).view(rows, -1)
    if c["gate"] == "before":
        out["dz"] = (d * x * slope).to(io)
        d = d * (z * sg)
    out["dx"] = d.to(io)
    return out


_plain = dict(prompts=_plain_prompts, step=_plain_step, norm=_plain_norm, norm_bwd=_plain_norm_bwd)


# ---------------------------------------------------------------- bytes and operations

def work(case):
    """Each input read once and each output written once; the recurrence's own
    operations (decay, input, readout: five per state and step)."""
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] in ("prompts", "step"):
        H, P, G, N, W = c["heads"], c["headdim"], c["groups"], c["dstate"], c["width"]
        inner, conv = H * P, H * P + 2 * G * N
        if c["op"] == "prompts":
            rows, wr = c["tokens"], c["nseq"]
            rd = (c["nseq"] + 1) // 2 if c["resume"] else 0
        else:
            rows = rd = wr = c["batch"] - min(c["pad"], c["batch"] - 1)
        state = 4 * (H * P * N + conv * (W - 1))
        par = 4 * (conv * (W + 1) + 3 * H)
        return dict(bytes=rows * e * (conv + H + inner * (2 if c["gate"] else 1)) + (rd + wr) * state + par,
                    flops=rows * (5 * H * P * N + conv * (2 * W + 4)))
    rows, C = c["rows"], c["channels"]
    gate, back = c["gate"] != "none", c["op"] == "norm_bwd"
    tensors = (3 + 2 * gate) if back else (2 + gate)
    par = 4 * C * (1 + c["bias"]) * (2 if back else 1)
    return dict(bytes=rows * C * e * tensors + par, flops=rows * C * ((16 if back else 6) + (8 if gate else 0)))


# ---------------------------------------------------------------- the definition in float64

def _exact_conv(s, hist):
    """silu of the convolution at one token a sequence: hist [sequences, width, channels]."""
    pre = (hist * s["conv_weight"].double().t()).sum(1) + s["conv_bias"].double()
    return pre * torch.sigmoid(pre)


def _exact_scan(c, s, h, act, dt, z):
    """One step of the recurrence for a batch of sequences, all in float64."""
    H, P, G, N = c["heads"], c["headdim"], c["groups"], c["dstate"]
    n, inner = act.shape[0], H * P
    x = act[:, :inner].reshape(n, G, H // G, P)
    B = act[:, inner:inner + G * N].reshape(n, G, 1, 1, N)
    C = act[:, inner + G * N:].reshape(n, G, 1, N, 1)
    dtg = dt.reshape(n, G, H // G)
    h = h.reshape(n, G, H // G, P, N)
    h = torch.exp(dtg * s["A"].double().view(G, H // G))[..., None, None] * h + (
        (dtg[..., None] * x)[..., None] * B)
    y = torch.matmul(h, C).squeeze(-1) + s["D"].double().view(G, H // G, 1) * x
    y = y.reshape(n, inner)
    if z is not None:
        y = y * (z * torch.sigmoid(z))
    return h.reshape(n, H, P, N), y


def exact(case, seed):
    c = case
    if c["op"] == "prompts":
        cu = _cu(c)
        longest = max(b - a for a, b in zip(cu, cu[1:]))
        state = c["nseq"] * c["heads"] * c["headdim"] * c["dstate"]
        if longest * (200e-6 + state * 8 * 8 / 3e12) > 18:
            return None
    s = prepare(c, seed)
    f = torch.nn.functional
    if c["op"] == "step":
        n = c["batch"] - min(c["pad"], c["batch"] - 1)
        slots = s["slots"][:n].long()
        hist = torch.cat([s["conv_state"][slots].double(), s["xbc"][:n].double()[..., None]], 2)
        dt = f.softplus(s["dt"][:n].double() + s["dt_bias"].double(), threshold=700)
        h, y = _exact_scan(c, s, s["ssm_state"][slots].double(), _exact_conv(s, hist.transpose(1, 2)),
                           dt, None if s["z"] is None else s["z"][:n].double())
        out, cs, hs = (s[k].double() for k in ("y", "conv_state", "ssm_state"))
        out[:n], cs[slots], hs[slots] = y, hist[..., 1:], h
        return out, cs, hs
    if c["op"] == "prompts":
        S, W = c["nseq"], c["width"]
        at = torch.tensor(cu[:-1], device=s["xbc"].device)
        end = torch.tensor(cu[1:], device=at.device)
        slots = s["slots"].long()
        cs, hs = s["conv_state"].double(), s["ssm_state"].double()
        hist, h = cs[slots].transpose(1, 2).contiguous(), hs[slots].clone()
        if s["has_state"] is None:
            hist.zero_(), h.zero_()
        else:
            hist[s["has_state"] == 0] = 0
            h[s["has_state"] == 0] = 0
        y = torch.zeros(c["tokens"], c["heads"] * c["headdim"], dtype=torch.float64, device=at.device)
        bias = s["dt_bias"].double()
        order = sorted(range(S), key=lambda i: cu[i] - cu[i + 1])  # the longest first
        om = torch.tensor(order, device=at.device)
        at, end, slots, hist, h = at[om], end[om], slots[om], hist[om], h[om]
        ls = [cu[i + 1] - cu[i] for i in order]
        hist = torch.cat([torch.zeros_like(hist[:, :1]), hist], 1)
        n = S
        for t in range(longest):
            while n and ls[n - 1] <= t:
                n -= 1
            rows = at[:n] + t
            hist[:n] = torch.cat([hist[:n, 1:], s["xbc"][rows].double()[:, None]], 1)
            dt = f.softplus(s["dt"][rows].double() + bias, threshold=700)
            z = None if s["z"] is None else s["z"][rows].double()
            new, yt = _exact_scan(c, s, h[:n], _exact_conv(s, hist[:n]), dt, z)
            if n == h.shape[0]:
                h = new
            else:
                h[:n] = new
            y[rows] = yt
        cs[slots], hs[slots] = hist[:, 1:].transpose(1, 2), h
        return y, cs, hs
    x = s["x"].double().requires_grad_()
    z = None if s["z"] is None else s["z"].double().requires_grad_()
    w = s["weight"].double().requires_grad_()
    b = None if s["bias"] is None else s["bias"].double().requires_grad_()
    with torch.set_grad_enabled(c["op"] == "norm_bwd"):
        v = (x * f.silu(z) if c["gate"] == "before" else x).unflatten(1, (c["groups"], -1))
        mean = v.mean(2, keepdim=True) if c["center"] else 0.0
        var = ((v - mean) ** 2).mean(2, keepdim=True)
        a = ((v - mean) / torch.sqrt(var + 1e-5)).flatten(1) * w
        a = a if b is None else a + b
        a = f.silu(a) if c["act"] == "silu" else a
        a = a * f.silu(z) if c["gate"] == "after" else a
    if c["op"] == "norm":
        return a
    leaves = {"dx": x, "dweight": w, **({"dz": z} if z is not None else {}),
              **({"dbias": b} if b is not None else {})}
    return dict(zip(leaves, torch.autograd.grad(a, list(leaves.values()), s["dy"].double())))
