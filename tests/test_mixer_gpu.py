"""The Mamba-2 mixer's operators on the GPU against float64: the convolution and
scan over packed prompts and for single tokens, the group norm and its
gradients, and a run of them as a server makes it.  Bounds: tests/mixer_ref.py."""
import numpy as np
import pytest

import mixer_ref as ref

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def ssm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import selective_state_space_43_amd as m
    m.lib()
    return m


@pytest.fixture(scope="module")
def dev(ssm):
    return torch.device("cuda:0")


def f64(t):
    return t.detach().double().cpu().numpy()


def up(a, dev, dtype=torch.float32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to(dev).to(dtype)


def rows_of(parts, dev, dtype, lead=0, tail=0):
    """The arrays as slices of one buffer's rows, with unused columns around them."""
    n = parts[0].shape[0]
    wide = torch.full((n, lead + tail + sum(p.shape[1] for p in parts)), float("nan"), device=dev).to(IO[dtype])
    out, at = [], lead
    for p in parts:
        wide[:, at:at + p.shape[1]] = up(p, dev, IO[dtype])
        out.append(wide[:, at:at + p.shape[1]])
        at += p.shape[1]
    return out


class Mix:
    """One packed problem: float64 arrays, device tensors, the reference."""

    def __init__(self, dev, lens, H, P, G, N, W, dtype, seed, gate=True, bias=True, state=True,
                 behind=0, spare=2, skip=(), lead=0, tail=0, has=None, softplus=True):
        rng = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(lens)])
        tokens, nseq = int(self.cu[-1]) + behind, len(lens)
        nslots = nseq + spare
        self.x = x = ref.mix_inputs(rng, tokens, nseq, H, P, G, N, W, dtype, nslots, gate, bias, state)
        x["inner"] = H * P
        if not softplus:  # raw steps used as they are: keep them positive
            x["dt_bias"] = np.full(H, 0.0)
            x["dt"] = ref.bf16(np.abs(x["dt"]) * 0.05) if dtype == "bf16" else np.abs(x["dt"]).astype(np.float32) * np.float32(0.05)
            x["dt"] = np.asarray(x["dt"], dtype=np.float64)
        slots = rng.permutation(nslots)[:nseq]
        for i, v in skip:
            slots[i] = v
        self.slots = slots if state else None
        self.has = (rng.random(nseq) < 0.5 if has is None else np.full(nseq, has)) if state else None
        self.G, self.P, self.dtype, self.softplus, self.dev = G, P, dtype, softplus, dev
        self.dims = (tokens, nseq, H, P, G, N, W)
        self.load(lead, tail)

    def load(self, lead=0, tail=0):
        x, dev = self.x, self.dev
        parts = [x["xbc"], x["dt"]] + ([x["z"]] if x["z"] is not None else [])
        t = rows_of(parts, dev, self.dtype, lead, tail)
        self.xbc, self.dt, self.z = t[0], t[1], t[2] if x["z"] is not None else None
        self.par = {k: up(x[k], dev) for k in ("conv_weight", "conv_bias", "A", "D", "dt_bias")}
        self.cs, self.hs = (up(x.get(k), dev) for k in ("conv_state", "ssm_state"))
        self.y = torch.full((self.dims[0], x["inner"]), 7.0, device=dev, dtype=IO[self.dtype])
        self.cu_t = torch.tensor(self.cu, dtype=torch.int32, device=dev)
        self.slots_t = None if self.slots is None else torch.tensor(self.slots, dtype=torch.int32, device=dev)
        self.has_t = None if self.has is None else torch.tensor(self.has, device=dev)

    def opts(self):
        return dict(conv_bias=self.par["conv_bias"], D=self.par["D"], z=self.z,
                    dt_bias=self.par["dt_bias"], dt_softplus=self.softplus)

    def run(self, ssm, **kw):
        a = dict(slots=self.slots_t, has_state=self.has_t, conv_state=self.cs, ssm_state=self.hs,
                 y=self.y, **self.opts())
        a.update(kw)
        return ssm.ssm_conv_ssd_fwd(self.xbc, self.dt, self.par["conv_weight"], self.par["A"], self.cu_t,
                                    self.P, self.G, **a)

    def step(self, ssm, **kw):
        a = dict(slots=self.slots_t, y=self.y, **self.opts())
        a.update(kw)
        return ssm.ssm_conv_ssd_update(self.xbc, self.dt, self.cs, self.hs, self.par["conv_weight"],
                                       self.par["A"], self.G, **a)

    def check(self, what=""):
        y, cs, hs, ysum, hsum = ref.mix(self.x, self.cu, self.G, self.slots, self.has, self.softplus)
        got = f64(self.y)
        mine = ~np.isnan(y[:, 0])
        assert (got[~mine] == 7.0).all(), "rows of no sequence were written"
        ey = ref.mix_excess(got[mine], y[mine], [v[mine] for v in ysum], self.dtype)
        eh = 0.0
        if hs is not None:
            eh = ref.mix_excess(f64(self.hs), hs, hsum, "state")
            assert np.array_equal(f64(self.cs), cs), "conv_state differs"
        print(f"{what}: y {ey:.3f}, state {eh:.3f} of the bound", flush=True)
        assert ey <= 1 and eh <= 1, (ey, eh)


PROMPTS = [  # lens, H, P, G, N, W, dtype, options
    ((1,), 1, 64, 1, 128, 4, "bf16", {}),
    ((64,), 2, 64, 1, 128, 4, "bf16", dict(gate=False)),
    ((65, 63, 1, 0, 2, 128), 4, 64, 2, 128, 4, "bf16", dict(behind=5)),
    ((0, 0, 37), 3, 64, 1, 64, 4, "bf16", dict(lead=3, tail=2)),
    ((200, 7), 2, 64, 1, 256, 4, "bf16", {}),
    ((130, 70), 6, 32, 3, 32, 3, "bf16", dict(lead=8)),
    ((77,), 5, 48, 1, 96, 2, "bf16", dict(gate=False, bias=False)),
    ((90, 33), 2, 80, 2, 16, 1, "bf16", {}),
    ((100,), 2, 129, 1, 20, 4, "bf16", dict(lead=1)),
    ((70, 3), 1, 256, 1, 100, 4, "bf16", {}),
    ((50, 20), 3, 1, 1, 1, 4, "bf16", {}),
    ((66,), 4, 17, 4, 9, 2, "bf16", dict(lead=1, tail=1)),
    ((64, 129, 1), 2, 64, 1, 128, 4, "f32", {}),
    ((33, 0, 95), 4, 32, 2, 64, 4, "f32", dict(behind=3, lead=1)),
    ((150,), 2, 128, 1, 256, 3, "f32", dict(gate=False)),
    ((40, 41), 3, 5, 1, 33, 4, "f32", dict(bias=False)),
    ((70, 90), 2, 64, 1, 128, 4, "bf16", dict(state=False)),
    ((70, 90), 2, 64, 1, 128, 4, "f32", dict(state=False)),
    ((70, 30, 20), 2, 64, 1, 128, 4, "bf16", dict(skip=((1, -1), (2, 99)))),
    ((70, 30), 2, 64, 1, 64, 4, "bf16", dict(has=True)),
    ((3, 2, 1), 2, 64, 1, 64, 4, "f32", dict(has=True)),
    ((300,), 2, 64, 1, 128, 4, "bf16", dict(softplus=False)),
    ((1,) * 40, 2, 64, 1, 128, 4, "bf16", {}),
    ((2500, 1, 700), 2, 64, 1, 128, 4, "bf16", dict(has=True)),  # a long axis: split and joined
    ((4100,), 1, 64, 1, 64, 4, "f32", dict(has=True)),
    ((3000, 2000), 10, 64, 5, 128, 4, "bf16", {}),
    ((2100,), 3, 40, 1, 256, 2, "bf16", dict(has=True, lead=1)),
    # three blocks are not cut, four are; nine leave a whole round of the joining
    ((192,), 2, 64, 1, 128, 4, "bf16", dict(has=True)),
    ((193,), 2, 64, 1, 128, 4, "bf16", dict(has=True)),
    ((576,), 2, 64, 1, 128, 4, "bf16", dict(has=True)),
    ((513,), 2, 64, 1, 128, 4, "f32", dict(has=True)),
    # segments of three blocks, their first pass in three pieces, in two, and in one
    ((1700, 100, 1, 300), 80, 64, 1, 16, 4, "bf16", dict(has=True)),
    ((1700, 100, 1, 300), 80, 64, 1, 16, 4, "f32", dict(has=True)),
    ((1500,) + (3,) * 13, 80, 64, 1, 16, 4, "bf16", {}),
    ((900, 40), 80, 64, 1, 16, 4, "bf16", {}),
]


@pytest.mark.parametrize("case", range(len(PROMPTS)))
def test_prompts(ssm, dev, case):
    lens, H, P, G, N, W, dtype, opt = PROMPTS[case]
    m = Mix(dev, lens, H, P, G, N, W, dtype, 900 + case, **opt)
    m.run(ssm)
    torch.cuda.synchronize()
    m.check(str(PROMPTS[case]))


STEPS = [  # batch, H, P, G, N, W, dtype, options
    (1, 80, 64, 1, 128, 4, "bf16", {}),
    (5, 4, 64, 2, 128, 4, "bf16", dict(skip=((1, -1), (4, 7)))),
    (3, 3, 64, 1, 64, 4, "bf16", dict(gate=False, lead=3)),
    (2, 2, 128, 1, 256, 3, "f32", {}),
    (7, 5, 48, 5, 96, 2, "bf16", dict(bias=False)),
    (4, 2, 80, 1, 16, 1, "bf16", {}),
    (3, 2, 129, 1, 20, 4, "f32", dict(lead=1)),
    (2, 3, 1, 3, 1, 4, "bf16", {}),
    (2, 1, 256, 1, 100, 4, "bf16", {}),
    (6, 4, 17, 4, 9, 2, "f32", dict(lead=1, tail=1)),
    (33, 8, 64, 1, 128, 4, "bf16", {}),
    (3, 4, 32, 2, 32, 4, "f32", dict(softplus=False)),
]


@pytest.mark.parametrize("case", range(len(STEPS)))
def test_step(ssm, dev, case):
    batch, H, P, G, N, W, dtype, opt = STEPS[case]
    m = Mix(dev, (1,) * batch, H, P, G, N, W, dtype, 700 + case, has=True, **opt)
    m.step(ssm)
    torch.cuda.synchronize()
    m.check(str(STEPS[case]))


def test_step_without_slots(ssm, dev):
    m = Mix(dev, (1,) * 6, 2, 64, 1, 128, 4, "bf16", 31, has=True)
    m.slots = np.arange(6)
    m.step(ssm, slots=None)
    torch.cuda.synchronize()
    m.check("no slots")


def test_prompt_in_pieces_and_tokens(ssm, dev):
    """A prompt cut into calls (an odd place, one token at a time at the end)
    gives what one call gives: the states carry everything."""
    lens = (333,)
    m = Mix(dev, lens, 4, 64, 2, 128, 4, "f32", 41, has=False, gate=False)
    whole = Mix(dev, lens, 4, 64, 2, 128, 4, "f32", 41, has=False, gate=False)
    whole.run(ssm)
    one = torch.ones(1, dtype=torch.bool, device=dev)
    for a, b in ((0, 1), (1, 3), (3, 130), (130, 330)):
        cu = torch.tensor([a, b], dtype=torch.int32, device=dev)
        ssm.ssm_conv_ssd_fwd(m.xbc, m.dt, m.par["conv_weight"], m.par["A"], cu, m.P, m.G, **m.opts(),
                             slots=m.slots_t, has_state=one if a else ~one, conv_state=m.cs,
                             ssm_state=m.hs, y=m.y)
    for t in range(330, 333):
        m.y[t:t + 1] = ssm.ssm_conv_ssd_update(m.xbc[t:t + 1], m.dt[t:t + 1], m.cs, m.hs,
                                               m.par["conv_weight"], m.par["A"], m.G,
                                               slots=m.slots_t, **m.opts())
    torch.cuda.synchronize()
    m.check("pieces")
    whole.check("whole")


def test_repeatable(ssm, dev):
    got = []
    for _ in range(2):
        m = Mix(dev, (2500, 40, 1), 4, 64, 1, 128, 4, "bf16", 51)
        m.run(ssm)
        m.has = np.ones(3, dtype=bool)
        torch.cuda.synchronize()
        got.append((m.y.clone(), m.cs.clone(), m.hs.clone()))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_wrong_offsets_stay_inside(ssm, dev):
    """Offsets outside the rows or out of order are clamped: the sequence in
    order between them is right, nothing outside y is touched."""
    m = Mix(dev, (20, 30, 10), 2, 64, 1, 64, 4, "bf16", 61, has=False)
    m.cu_t = torch.tensor([-5, 20, 50, 1 << 30], dtype=torch.int32, device=dev)
    m.run(ssm)
    torch.cuda.synchronize()
    m.check("clamped offsets")
    m = Mix(dev, (20, 30, 10), 2, 64, 1, 64, 4, "bf16", 61, has=False)
    m.cu_t = torch.tensor([0, 20, 10, 60], dtype=torch.int32, device=dev)  # the second one is empty
    m.run(ssm)
    torch.cuda.synchronize()
    assert torch.isfinite(m.y.float()).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["x", "B", "C", "dt", "z"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_input(ssm, dev, dtype, where, bad):
    """A non-finite input at one token: earlier tokens, other sequences and the
    channels that do not depend on it keep their values."""
    H, P, G, N, t = 2, 64, 1, 64, 70
    def make(poison):
        m = Mix(dev, (40, 150, 30), H, P, G, N, 4, dtype, 71, has=False)
        if poison:
            row = 40 + t
            if where == "dt":
                m.dt[row, 0] = bad
            elif where == "z":
                m.z[row, 5] = bad
            else:
                m.xbc[row, {"x": 5, "B": H * P + 3, "C": H * P + N + 3}[where]] = bad
        m.run(ssm)
        torch.cuda.synchronize()
        return m
    a, b = make(False), make(True)
    ya, yb = f64(a.y), f64(b.y)
    hit = np.zeros(ya.shape, dtype=bool)  # what may change
    if where == "x":
        hit[40 + t:190, 5] = True
    elif where == "B":
        hit[40 + t:190] = True
    elif where == "C":
        hit[40 + t:40 + t + 4] = True
    elif where == "dt":
        hit[40 + t:190, :P] = True
    else:
        hit[40 + t, 5] = True
    # elsewhere: the same to the operands' scales, which go by a block's largest finite value
    tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -14
    near = np.abs(ya - yb) <= tol * (1 + np.abs(ya))
    assert near[~hit].all(), np.argwhere(~near & ~hit)[:5]
    if where in ("x", "B", "z") and np.isnan(bad):
        assert np.isnan(yb[40 + t][hit[40 + t]]).all()
    ha, hb = f64(a.hs), f64(b.hs)
    other = [s for s in range(ha.shape[0]) if s != a.slots[1]]
    assert (np.abs(ha - hb)[other] <= 2.0 ** -14 * (1 + np.abs(ha[other]))).all()


def test_extreme_steps(ssm, dev):
    """A step so large that the state is forgotten, and one so small that it is
    kept, inside one block; large and tiny inputs next to each other."""
    for dtype in ("bf16", "f32"):
        m = Mix(dev, (150, 40), 2, 64, 1, 64, 4, dtype, 81, has=True, gate=False)
        dt = m.x["dt"]
        dt[30], dt[31], dt[100:110] = 60.0, -40.0, -60.0
        m.x["xbc"][60, :] *= 2.0 ** 10
        m.x["xbc"][155, :] *= 2.0 ** -20
        m.load()
        m.run(ssm)
        torch.cuda.synchronize()
        m.check("extreme " + dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["A", "dt"])
def test_growing_state(ssm, dev, dtype, how):
    """A positive A, or raw steps below zero used as they are: the weights of a
    block pass the largest step."""
    m = Mix(dev, (150, 40), 2, 64, 1, 64, 4, dtype, 83, has=True, softplus=False)
    if how == "A":
        m.x["A"] = np.array([0.5, 0.02])
    else:
        m.x["dt"][60:90] *= -1
        m.x["A"] = np.array([-3.0, -0.1])
    m.load()
    m.run(ssm)
    torch.cuda.synchronize()
    m.check(f"growing {how} {dtype}")


def test_states_without_slots(ssm, dev):
    """slots None: sequence s has slot s; has_state None: none continues."""
    m = Mix(dev, (70, 0, 5), 2, 64, 1, 64, 4, "bf16", 84, has=False)
    m.slots = np.arange(3)
    m.run(ssm, slots=None, has_state=None)
    torch.cuda.synchronize()
    m.check("no slots")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_state(ssm, dev, dtype):
    """A NaN and an infinity in the state that a prompt continues from reach their
    own channel's y and state only."""
    m = Mix(dev, (90, 30), 2, 64, 1, 64, 4, dtype, 85, has=True)
    clean = Mix(dev, (90, 30), 2, 64, 1, 64, 4, dtype, 85, has=True)
    slot = int(m.slots[0])
    m.hs[slot, 0, 5, 7], m.hs[slot, 1, 9, 3] = float("nan"), float("inf")
    m.run(ssm)
    clean.run(ssm)
    torch.cuda.synchronize()
    ya, yb = f64(clean.y), f64(m.y)
    hit = np.zeros(ya.shape, dtype=bool)
    hit[:90, 5] = hit[:90, 64 + 9] = True
    tol = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -14
    assert (np.abs(ya - yb) <= tol * (1 + np.abs(ya)))[~hit].all()
    assert np.isnan(yb[:90, 5]).all()
    ha, hb = f64(clean.hs)[slot], f64(m.hs)[slot]
    keep = np.ones(ha.shape, dtype=bool)
    keep[0, 5, 7] = keep[1, 9, 3] = False
    assert (np.abs(ha - hb) <= 2.0 ** -14 * (1 + np.abs(ha)))[keep].all() and np.isnan(hb[0, 5, 7])


def test_many_short_sequences(ssm, dev):
    """More sequences than the plan takes in one turn, every third one padding."""
    lens = tuple((i * 7) % 4 for i in range(2300))
    skip = tuple((i, -1) for i in range(0, 2300, 3))
    m = Mix(dev, lens, 1, 16, 1, 16, 4, "bf16", 86, skip=skip, behind=2)
    m.run(ssm)
    torch.cuda.synchronize()
    m.check("2300 sequences")


def test_far_rows_and_slots(ssm, dev):
    """Rows and slots whose byte offsets pass 32 bits."""
    H, P, G, N, W = 2, 64, 1, 128, 4
    ch = H * P + 2 * G * N
    m = Mix(dev, (1, 70), H, P, G, N, W, "bf16", 91, has=True)
    stride = 40_000_000
    wide = torch.zeros(71 * stride, dtype=torch.bfloat16, device=dev)  # 5.7 GB
    far = wide.as_strided((71, ch), (stride, 1))
    far.copy_(m.xbc)
    m.xbc = far
    nslots = 80_000  # 5.2 GB of states
    hs = torch.zeros(nslots, H, P, N, device=dev)
    cs = torch.zeros(nslots, ch, W - 1, device=dev)
    at = torch.tensor([nslots - 1, nslots - 2], device=dev)
    hs[at], cs[at] = m.hs[m.slots_t.long()], m.cs[m.slots_t.long()]
    m.run(ssm, slots=at.int(), conv_state=cs, ssm_state=hs)
    torch.cuda.synchronize()
    m.hs[m.slots_t.long()], m.cs[m.slots_t.long()] = hs[at], cs[at]
    m.check("far")
    assert not hs[:nslots - 2].any()


# ---------------------------------------------------------------- group norm

NORMS = [  # rows, channels, groups, dtype, center, act, gate, options
    (1, 5120, 1, "bf16", False, "none", "before", {}),
    (3, 5120, 8, "bf16", False, "none", "before", {}),
    (7, 1000, 5, "f32", True, "silu", "none", {}),
    (65, 64, 64, "bf16", True, "none", "after", {}),
    (5, 7, 1, "f32", True, "none", "before", dict(lead=1)),
    (4, 30, 10, "bf16", True, "silu", "after", dict(lead=1)),
    (300, 96, 3, "f32", False, "silu", "before", {}),
    (2, 32768, 1, "bf16", True, "none", "none", {}),
    (9, 2049, 1, "f32", False, "none", "after", {}),
    (1025, 128, 2, "bf16", False, "silu", "after", dict(lead=2)),
    (33, 640, 1, "bf16", True, "none", "before", dict(weight=False)),
    (2, 40000, 2, "f32", False, "none", "before", {}),
    (17, 4096, 1, "f32", True, "silu", "before", {}),
    (600, 260, 13, "bf16", True, "none", "none", dict(lead=3)),
    (130, 12000, 1, "bf16", False, "none", "before", {}),
    # both sides of every change of team
    (40, 192, 3, "bf16", False, "none", "before", dict(bias=False)),
    (21, 72, 1, "bf16", False, "none", "before", dict(bias=False)),
    (21, 512, 2, "bf16", False, "none", "before", dict(bias=False)),
    (9, 264, 1, "bf16", True, "silu", "after", {}),
    (6, 768, 1, "bf16", False, "none", "before", dict(bias=False)),
    (6, 776, 1, "bf16", False, "none", "before", dict(bias=False)),
    (6, 1024, 1, "bf16", True, "silu", "after", {}),
    (6, 1032, 1, "bf16", True, "none", "none", {}),
    (5, 1536, 1, "bf16", False, "none", "before", dict(bias=False)),
    (5, 2048, 1, "bf16", False, "silu", "before", {}),
    (5, 2056, 1, "bf16", True, "none", "after", {}),
    (9, 6144, 1, "bf16", False, "none", "before", dict(bias=False)),
    (9, 6152, 1, "bf16", False, "none", "before", dict(bias=False)),
    (2100, 8192, 1, "bf16", False, "none", "before", dict(bias=False)),
    (9, 8192, 1, "bf16", True, "silu", "after", {}),
    (9, 8200, 1, "bf16", False, "none", "before", dict(bias=False)),
    (7, 4100, 1, "f32", False, "none", "before", dict(bias=False)),
]


def norm_problem(dev, case, seed):
    rows, C, G, dtype, center, act, gate, opt = case
    rng = np.random.default_rng(seed)
    q = ref.bf16 if dtype == "bf16" else lambda a: a.astype(np.float32).astype(np.float64)
    f = lambda a: a.astype(np.float32).astype(np.float64)  # noqa: E731
    x = dict(x=q(rng.standard_normal((rows, C)) + 0.5), dy=q(rng.standard_normal((rows, C))),
             z=q(rng.standard_normal((rows, C))) if gate != "none" else None,
             w=f(1 + 0.3 * rng.standard_normal(C)) if opt.get("weight", True) else None,
             b=f(0.3 * rng.standard_normal(C)) if opt.get("bias", opt.get("weight", True)) else None)
    parts = [v for v in (x["x"], x["dy"], x["z"]) if v is not None]
    t = rows_of(parts, dev, dtype, opt.get("lead", 0))
    t = dict(x=t[0], dy=t[1], z=t[2] if len(t) > 2 else None, w=up(x["w"], dev), b=up(x["b"], dev))
    return x, t, dict(center=center, act=act, gate=gate)


@pytest.mark.parametrize("case", range(len(NORMS)))
def test_norm(ssm, dev, case):
    rows, C, G, dtype, center, act, gate, _ = NORMS[case]
    x, t, how = norm_problem(dev, NORMS[case], 300 + case)
    y = ssm.ssm_group_norm_fwd(t["x"], t["w"], G, bias=t["b"], z=t["z"], center=center, activation=act,
                               gate=gate)
    g = ssm.ssm_group_norm_bwd(t["dy"], t["x"], t["w"], G, bias=t["b"], z=t["z"], center=center,
                               activation=act, gate=gate)
    torch.cuda.synchronize()
    want, bound = ref.norm(x["x"], x["w"], G, x["b"], x["z"], **how)
    tol = ref.HALF[dtype] * np.abs(want) + ref.NORM * bound + 1e-30
    worst = {"y": np.max(np.abs(f64(y) - want) / tol)}
    want, bound = ref.norm_bwd(x["dy"], x["x"], x["w"], G, x["b"], x["z"], **how)
    assert (g["dz"] is None) == (gate == "none")
    for k, v in g.items():
        if v is None:
            continue
        rel = ref.NORM_BWD + (4 * 2.0 ** -24 * np.sqrt(rows) if k in ("dweight", "dbias") else 0)
        half = 2.0 ** -24 if k in ("dweight", "dbias") else ref.HALF[dtype]
        worst[k] = np.max(np.abs(f64(v) - want[k]) / (half * np.abs(want[k]) + rel * bound[k] + 1e-30))
    print(NORMS[case], {k: f"{v:.3f}" for k, v in worst.items()}, flush=True)
    assert max(worst.values()) <= 1, worst


def test_norm_autograd(ssm, dev):
    x, t, how = norm_problem(dev, (6, 40, 4, "f32", True, "silu", "before", {}), 500)
    leaves = [t[k].clone().contiguous().requires_grad_() for k in ("x", "w", "b", "z")]
    y = ssm.group_norm_fn(leaves[0], leaves[1], 4, bias=leaves[2], z=leaves[3], center=True,
                          activation="silu", gate="before")
    y.backward(t["dy"])
    want, bound = ref.norm_bwd(x["dy"], x["x"], x["w"], 4, x["b"], x["z"], **how)
    for leaf, k in zip(leaves, ("dx", "dweight", "dbias", "dz")):
        assert np.all(np.abs(f64(leaf.grad) - want[k]) <= 2 * ref.NORM_BWD * bound[k] + 1e-30), k


def test_norm_autograd_is_once_differentiable(ssm, dev):
    x = torch.randn(5, 40, device=dev, requires_grad=True)
    with pytest.raises(RuntimeError, match="gradients of its gradients"):
        torch.autograd.grad(ssm.group_norm_fn(x, None, 4).sum(), x, create_graph=True)


def test_norm_special_rows(ssm, dev):
    """Constant and zero rows (a variance of zero), a NaN and an infinity in one
    row: the other rows, and the other group of that row, keep their values."""
    x, t, how = norm_problem(dev, (6, 64, 2, "f32", True, "none", "none", {}), 510)
    x["x"][1], x["x"][2] = 0.0, 3.0
    t["x"][1], t["x"][2] = 0.0, 3.0
    t["x"][3, 5], t["x"][4, 40] = float("nan"), float("inf")
    y = ssm.ssm_group_norm_fwd(t["x"], t["w"], 2, bias=t["b"], center=True)
    g = ssm.ssm_group_norm_bwd(t["dy"], t["x"], t["w"], 2, bias=t["b"], center=True)
    torch.cuda.synchronize()
    want, bound = ref.norm(x["x"], x["w"], 2, x["b"], None, center=True)
    gw, gb = ref.norm_bwd(x["dy"], x["x"], x["w"], 2, x["b"], None, center=True)
    keep = np.ones((6, 64), dtype=bool)
    keep[3, :32] = keep[4, 32:] = False
    assert (np.abs(f64(y) - want) <= (2.0 ** -24 + ref.NORM) * bound + 1e-30)[keep].all()
    assert (np.abs(f64(g["dx"]) - gw["dx"]) <= ref.NORM_BWD * gb["dx"] + 1e-30)[keep].all()
    assert np.isnan(f64(y)[~keep]).all()


def test_norm_repeatable_and_far_rows(ssm, dev):
    case = (700, 256, 4, "bf16", False, "none", "before", {})
    x, t, how = norm_problem(dev, case, 520)
    a = ssm.ssm_group_norm_bwd(t["dy"], t["x"], t["w"], 4, bias=t["b"], z=t["z"], gate="before")
    stride = 5_000_000
    far = torch.zeros(700 * stride, dtype=torch.bfloat16, device=dev).as_strided((700, 256), (stride, 1))
    far.copy_(t["x"])  # 7 GB
    b = ssm.ssm_group_norm_bwd(t["dy"], far, t["w"], 4, bias=t["b"], z=t["z"], gate="before")
    assert all(torch.equal(a[k], b[k]) for k in a)


# ---------------------------------------------------------------- as a server runs them

def test_prompts_norm_steps_together(ssm, dev):
    """Two prompts through convolution, scan and gated norm, then three tokens
    each, the projection's rows as they come: against the reference's run."""
    H, P, G, N, W = 4, 64, 2, 128, 4
    inner = H * P
    m = Mix(dev, (70, 45), H, P, G, N, W, "f32", 600, gate=True, has=False)
    z, m.z = m.z, None
    zr, m.x["z"] = m.x["z"], None
    w = up(1 + 0.1 * np.random.default_rng(1).standard_normal(inner), dev)
    m.run(ssm)
    out = ssm.ssm_group_norm_fwd(m.y, w, G, z=z, gate="before")
    y, cs, hs, ysum, hsum = ref.mix(m.x, m.cu, G, m.slots, m.has)
    want, bound = ref.norm(y, f64(w), G, None, zr, gate="before")
    # y's own bound moves the norm by at most its share of the group's root mean square, twice
    ytol = (2.0 ** -24 + ref.INNER["f32"]) * ysum[0] + ref.CONV * ysum[1]
    v = (np.abs(y * zr) / (1 + np.exp(-zr))).reshape(len(y), G, -1)
    rms = np.sqrt((v ** 2).mean(2, keepdims=True) + 1e-5)
    dv = (ytol * np.abs(zr) / (1 + np.exp(-zr))).reshape(len(y), G, -1)
    move = (dv + v / rms * np.sqrt((dv ** 2).mean(2, keepdims=True))) / rms
    tol = ref.NORM * bound + move.reshape(len(y), -1) * np.abs(f64(w)) + 1e-30
    assert (np.abs(f64(out) - want) <= tol).all()
    # three tokens for each sequence, the second slot first
    rng = np.random.default_rng(2)
    m.x["conv_state"], m.x["ssm_state"] = cs, hs
    for _ in range(3):
        m.slots = m.slots[::-1].copy()
        new = ref.mix_inputs(rng, 2, 2, H, P, G, N, W, "f32", 4, gate=False, state=False)
        m.x["xbc"], m.x["dt"] = new["xbc"], new["dt"]
        m.xbc, m.dt = rows_of([new["xbc"], new["dt"]], dev, "f32", 2)
        m.slots_t = torch.tensor(m.slots, dtype=torch.int32, device=dev)
        m.cu, m.has = np.arange(3), np.ones(2, dtype=bool)
        m.y = torch.full((2, inner), 7.0, device=dev)
        m.step(ssm)
        torch.cuda.synchronize()
        m.check("token")
        # the GPU's own states go on, and the reference starts the next token from them
        m.x["conv_state"], m.x["ssm_state"] = f64(m.cs), f64(m.hs)


def test_same_as_the_dense_operators(ssm, dev):
    """One prompt of 256 tokens through ssm_causal_conv1d_fwd and ssm_ssd_fwd, time
    innermost, gives the packed call's result within both operators' bounds."""
    H, P, G, N = 4, 64, 2, 128
    m = Mix(dev, (256,), H, P, G, N, 4, "bf16", 610, has=False)
    m.run(ssm)
    xt = m.xbc.t().contiguous()[None]
    c, cs = ssm.ssm_causal_conv1d_fwd(xt, m.par["conv_weight"], m.par["conv_bias"], want_state_out=True)
    i = H * P
    y, hs = ssm.ssm_ssd_fwd(c[:, :i].contiguous(), m.dt.t().contiguous()[None], m.par["A"],
                            c[:, i:i + G * N].contiguous(), c[:, i + G * N:].contiguous(), H, G,
                            D=m.par["D"], z=m.z.t().contiguous()[None], dt_bias=m.par["dt_bias"])
    torch.cuda.synchronize()
    slot = int(m.slots[0])
    assert torch.equal(m.cs[slot], cs[0])
    a, b = f64(m.y), f64(y[0].t())
    assert (np.abs(a - b) <= 2e-2 * (1 + np.abs(b))).all()
    a, b = f64(m.hs[slot]), f64(hs[0])
    assert (np.abs(a - b) <= 2e-2 * (1 + np.abs(b))).all()


def test_graph_replays_and_streams(ssm, dev):
    """The prompts, a token and the norm captured into a graph with their
    workspace, replayed with eager calls of the same program in between: every
    replay equals the eager run on another stream."""
    H, P, G, N = 4, 64, 1, 128
    def fresh(seed):
        return Mix(dev, (1300, 70), H, P, G, N, 4, "bf16", seed, gate=False, has=True)
    m, tok, e, etok = fresh(620), fresh(621), fresh(620), fresh(621)
    w = torch.ones(H * P, device=dev)
    rows = m.dims[0]
    ws = torch.empty(ssm.ssm_conv_ssd_workspace_size(rows, 2, H, P, G, N), dtype=torch.uint8, device=dev)
    ws2 = torch.empty_like(ws)
    def program(m, tok, ws, out):
        m.run(ssm, workspace=ws)
        ssm.ssm_conv_ssd_update(tok.xbc[:2], tok.dt[:2], m.cs, m.hs, m.par["conv_weight"], m.par["A"], G,
                                slots=m.slots_t, y=out[:2], **{**m.opts(), "z": None})
        ssm.ssm_group_norm_fwd(m.y, w, G, y=out[2:])
        # a training program's step beside it: its gradients into the same tensors
        g = ssm.ssm_group_norm_bwd(out[2:], m.y, w, 2, bias=w, center=True)
        out[2:].copy_(g["dx"] + g["dweight"].bfloat16() + g["dbias"].bfloat16())
    out, eout = (torch.zeros(rows + 2, H * P, dtype=torch.bfloat16, device=dev) for _ in range(2))
    keep = m.cs.clone(), m.hs.clone()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        program(m, tok, ws, out)
    torch.cuda.current_stream(dev).wait_stream(side)
    torch.cuda.synchronize()
    m.cs.copy_(keep[0]), m.hs.copy_(keep[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        program(m, tok, ws, out)
    for _ in range(4):
        graph.replay()
        with torch.cuda.stream(side):
            program(e, etok, ws2, eout)
        torch.cuda.synchronize()
        assert torch.equal(out, eout) and torch.equal(m.cs, e.cs) and torch.equal(m.hs, e.hs)
