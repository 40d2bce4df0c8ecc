"""The Mamba-2 mixer's operators on the GPU where tests/test_mixer_gpu.py does not
reach: rows on 16 bytes, as a model's projection has them, in every size of the
kernels for whole vectors; the general kernels on cut prompts; prompts cut into
segments beside other work on the card.  Problems, references and bounds as
there."""
import numpy as np
import pytest

import mixer_ref as ref
import test_mixer_gpu as base
from test_mixer_gpu import IO, Mix, dev, rows_of, ssm, up  # noqa: F401  (fixtures)

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


class Aligned(Mix):
    """Rows in the projection's order, z, xbc, dt, every one of them on 16 bytes."""

    def load(self, lead=0, tail=0):
        super().load()
        x = self.x
        parts = [v for v in (x["z"], x["xbc"], x["dt"]) if v is not None]
        whole = 16 // IO[self.dtype].itemsize
        *z, self.xbc, self.dt = rows_of(parts, self.dev, self.dtype, 0, -sum(p.shape[1] for p in parts) % whole)
        self.z = z[0] if z else None
        for t in (*z, self.xbc):
            assert t.data_ptr() % 16 == 0 and t.stride(0) * t.element_size() % 16 == 0


CASES = [  # layout, lens, H, P, G, N, W, dtype, options
    # bf16: 64, 128 and 256 states; heads of whole and of broken tiles; cut from four blocks on
    (Aligned, (65, 63, 1, 0, 2, 128), 4, 64, 2, 128, 4, "bf16", dict(behind=5)),
    (Aligned, (192,), 2, 64, 1, 128, 4, "bf16", dict(has=True)),
    (Aligned, (193,), 2, 64, 1, 128, 4, "bf16", dict(has=True)),
    (Aligned, (576, 1), 2, 64, 1, 128, 4, "bf16", dict(has=True, gate=False)),
    (Aligned, (2500, 1, 700), 2, 64, 1, 128, 4, "bf16", dict(has=True)),
    (Aligned, (3000, 2000), 10, 64, 5, 128, 4, "bf16", {}),
    (Aligned, (1500, 3, 90), 24, 64, 1, 128, 4, "bf16", dict(has=True, gate=False)),
    (Aligned, (37,), 24, 64, 1, 128, 4, "bf16", dict(gate=False, state=False)),
    (Aligned, (90, 33), 8, 48, 2, 128, 4, "bf16", dict(has=True)),
    (Aligned, (300, 70), 3, 48, 1, 96, 3, "bf16", dict(gate=False, has=True)),
    (Aligned, (70, 130), 3, 80, 1, 128, 4, "bf16", dict(has=True)),
    (Aligned, (500,), 2, 80, 2, 64, 4, "bf16", dict(has=True, gate=False)),
    (Aligned, (100, 64, 30), 5, 64, 1, 64, 4, "bf16", {}),
    (Aligned, (700, 20), 5, 64, 1, 64, 2, "bf16", dict(has=True, gate=False)),
    (Aligned, (200, 7), 2, 64, 1, 256, 4, "bf16", {}),
    (Aligned, (600, 64), 3, 64, 1, 256, 4, "bf16", dict(has=True)),
    (Aligned, (900,), 4, 48, 2, 256, 4, "bf16", dict(has=True, gate=False)),
    (Aligned, (77, 300), 3, 24, 1, 200, 3, "bf16", dict(has=True)),
    (Aligned, (90, 300), 3, 8, 1, 128, 4, "bf16", dict(has=True)),
    (Aligned, (80,), 2, 256, 1, 128, 1, "bf16", dict(has=True)),
    (Aligned, (150, 9), 2, 40, 1, 20, 4, "bf16", dict(has=True)),
    # columns behind x: 32 let whole tiles be read past the last head, 24 do not
    (Aligned, (150, 9), 3, 48, 1, 16, 4, "bf16", dict(has=True)),
    (Aligned, (150, 9), 3, 48, 1, 12, 4, "bf16", dict(has=True)),
    # float32: whole and general, cut and not, up to 256 states
    (Aligned, (600, 70), 4, 64, 1, 128, 4, "f32", dict(has=True)),
    (Aligned, (64, 129, 1), 16, 64, 2, 128, 4, "f32", dict(gate=False)),
    (Aligned, (150, 40), 2, 64, 1, 256, 4, "f32", dict(has=True)),
    (Aligned, (700,), 3, 48, 1, 256, 4, "f32", dict(has=True, gate=False)),
    (Aligned, (500, 30), 3, 40, 1, 64, 4, "f32", dict(has=True)),
    (Aligned, (400,), 2, 24, 2, 32, 2, "f32", dict(has=True)),
    (Mix, (600, 70), 3, 64, 1, 128, 4, "f32", dict(has=True, lead=1)),
    (Mix, (500,), 2, 50, 1, 250, 4, "f32", dict(has=True, lead=1)),
    (Mix, (500,), 3, 33, 1, 30, 3, "f32", dict(has=True)),
    (Mix, (600, 70), 3, 64, 1, 128, 4, "bf16", dict(has=True, lead=1)),
    (Mix, (500,), 2, 50, 1, 250, 4, "bf16", dict(has=True, lead=1)),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_prompts(ssm, dev, case):  # noqa: F811
    layout, lens, H, P, G, N, W, dtype, opt = CASES[case]
    m = layout(dev, lens, H, P, G, N, W, dtype, 1100 + case, **opt)
    m.run(ssm)
    torch.cuda.synchronize()
    m.check(str(CASES[case][1:]))


@pytest.fixture
def aligned(monkeypatch):
    monkeypatch.setattr(base, "Mix", Aligned)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("where", ["x", "B", "C", "dt", "z"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_input(aligned, ssm, dev, dtype, where, bad):  # noqa: F811
    base.test_non_finite_input(ssm, dev, dtype, where, bad)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_non_finite_state(aligned, ssm, dev, dtype):  # noqa: F811
    base.test_non_finite_state(ssm, dev, dtype)


def test_extreme_steps(aligned, ssm, dev):  # noqa: F811
    base.test_extreme_steps(ssm, dev)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["A", "dt"])
def test_growing_state(aligned, ssm, dev, dtype, how):  # noqa: F811
    base.test_growing_state(ssm, dev, dtype, how)


def test_far_rows_and_slots(aligned, ssm, dev):  # noqa: F811
    base.test_far_rows_and_slots(ssm, dev)


def test_same_as_the_dense_operators(aligned, ssm, dev):  # noqa: F811
    base.test_same_as_the_dense_operators(ssm, dev)


def test_repeatable(aligned, ssm, dev):  # noqa: F811
    base.test_repeatable(ssm, dev)


def test_graph_replays_and_streams(aligned, ssm, dev):  # noqa: F811
    base.test_graph_replays_and_streams(ssm, dev)


def test_cut_prompts_beside_other_work(ssm, dev):  # noqa: F811
    """Prompts of four segments that continue from their slots, with products on
    another stream holding parts of the card: the last segment of a sequence
    may end before its first one starts, and writes the slot that the sequence
    started from.  Every call gives the quiet call's bits."""
    def fresh():
        return Mix(dev, (256, 200), 24, 64, 1, 128, 4, "bf16", 1000, gate=False, has=True)
    quiet = fresh()
    quiet.run(ssm)
    torch.cuda.synchronize()
    quiet.check("quiet")
    m = fresh()
    keep = m.cs.clone(), m.hs.clone()
    a = torch.randn(4096, 4096, device=dev).bfloat16()
    out = torch.empty_like(a)
    side = torch.cuda.Stream(dev)
    for _ in range(20):
        m.cs.copy_(keep[0]), m.hs.copy_(keep[1])
        side.wait_stream(torch.cuda.current_stream(dev))
        with torch.cuda.stream(side):
            for _ in range(3):
                torch.mm(a, a, out=out)
        m.run(ssm)
        torch.cuda.synchronize()
        assert torch.equal(m.y, quiet.y) and torch.equal(m.hs, quiet.hs) and torch.equal(m.cs, quiet.cs)


# ---------------------------------------------------------------- the bits that bf16 rows keep

def check_to_the_last_bit(m, what):
    """y of bf16 rows as float32's operators would store it: behind the one rounding
    (half a step of the stored value, 2^-9 to 2^-8 of it) no more than
    float32 rows may be off."""
    y, _, hs, (terms, conv), hsum = ref.mix(m.x, m.cu, m.G, m.slots, m.has, m.softplus)
    mine = ~np.isnan(y[:, 0])
    err = ref.INNER["f32"] * terms[mine] + ref.CONV * conv[mine] + 1e-30
    half = 2.0 ** (np.floor(np.log2(np.abs(y[mine]) + err)) - 8)
    worst = np.max(np.abs(base.f64(m.y)[mine] - y[mine]) / (half + err))
    print(f"{what}: {worst:.4f} of the bound", flush=True)
    assert worst <= 1, worst
    if hs is not None:
        assert ref.mix_excess(base.f64(m.hs), hs, hsum, "state") <= 1


BITS = [  # layout, lens, H, P, G, N, W, options
    (Aligned, (130, 64, 3), 8, 64, 1, 128, 4, dict(has=True)),
    (Aligned, (130, 64, 3), 8, 64, 1, 128, 4, dict(gate=False, state=False, bias=False)),
    (Aligned, (700,), 8, 64, 2, 64, 4, dict(has=True)),
    (Aligned, (90,), 6, 48, 1, 16, 3, dict(gate=False)),
    (Aligned, (200, 30), 4, 64, 1, 256, 4, dict(has=True)),
    (Mix, (130, 64, 3), 3, 64, 1, 128, 4, dict(has=True, lead=1)),
    (Mix, (300,), 3, 40, 1, 250, 4, dict(has=True, lead=1)),
    (Mix, (100,), 5, 33, 1, 40, 2, dict(gate=False)),
]


@pytest.mark.parametrize("case", range(len(BITS)))
def test_bf16_rows_keep_float32s_bits(ssm, dev, case):  # noqa: F811
    layout, lens, H, P, G, N, W, opt = BITS[case]
    m = layout(dev, lens, H, P, G, N, W, "bf16", 1200 + case, **opt)
    m.run(ssm)
    torch.cuda.synchronize()
    check_to_the_last_bit(m, str(BITS[case][1:]))


# ---------------------------------------------------------------- sizes far apart

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_skip_beside_tiny_B_and_C(ssm, dev, dtype):  # noqa: F811
    """B and C near 2^-62 beside a skip of 300: y is D x, and finite."""
    m = Aligned(dev, (100, 30), 2, 64, 1, 64, 4, dtype, 1300, gate=False, has=False)
    m.x["xbc"][:, 128:] *= 2.0 ** -60
    m.x["conv_bias"][128:] = 0.0
    m.x["D"][:] = (300.0, -500.0)
    m.load()
    m.run(ssm)
    torch.cuda.synchronize()
    m.check("tiny B and C")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("how", ["channel", "token", "step", "state"])
def test_sizes_far_apart(ssm, dev, dtype, how):  # noqa: F811
    """Large values beside small ones: channels of x and of the state 2^60 and 2^80
    apart, tokens 2^28, steps of 2e-9 beside one of 64 with neither skip nor state.
    Every value is held to the bound of its own terms."""
    m = Aligned(dev, (150, 40), 2, 64, 1, 64, 4, dtype, 1310, gate=False, has=how != "step")
    x = m.x
    if how == "channel":
        for c, f in ((5, 2.0 ** 30), (6, 2.0 ** -30), (70, 2.0 ** 30), (101, 2.0 ** -30)):
            x["conv_weight"][c] *= f
            x["conv_bias"][c] *= f
            x["ssm_state"][:, c // 64, c % 64] *= f
    elif how == "token":
        x["xbc"][60, :128] *= 2.0 ** 14
        x["xbc"][62, :128] *= 2.0 ** -14
    elif how == "step":
        x["dt"][:], x["dt_bias"][:], x["D"][:] = -20.0, 0.0, 0.0
        x["dt"][[10, 100]] = 64.0
    else:
        x["ssm_state"][:, 0, 5] *= 2.0 ** 40
        x["ssm_state"][:, 0, 6] *= 2.0 ** -40
    m.load()
    m.run(ssm)
    torch.cuda.synchronize()
    if dtype == "bf16":
        check_to_the_last_bit(m, how)
    else:
        m.check(how)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("P", [24, 48, 80])
def test_a_head_does_not_depend_on_its_neighbour(ssm, dev, dtype, P):  # noqa: F811
    """The tiles of a head that end inside one hold the next head's channels (or B's)
    beside its own: larger and infinite ones leave its bits as they are."""
    def run(change):
        m = Aligned(dev, (150, 40), 2, P, 1, 64, 4, dtype, 1320, gate=False, has=True)
        if change:
            m.x["xbc"][:, P:2 * P] *= 2.0 ** 40
            m.load()
            if change > 1:
                m.xbc[20, P:2 * P] = float("inf")
        m.run(ssm)
        torch.cuda.synchronize()
        return m.y[:, :P], m.hs[:, 0]
    clean = run(0)
    assert torch.isfinite(clean[0].float()).all()
    for change in (1, 2):
        assert all(torch.equal(a, b) for a, b in zip(clean, run(change)))


def test_offsets_out_of_order_and_guards(ssm, dev):  # noqa: F811
    """Offsets that run back or past the rows are read as their running maximum
    inside them; y, the states and the guards around them are what those
    offsets give."""
    for wrong, right in (((0, 20, 10, 60), (0, 20, 20, 60)), ((-5, 30, 20, 1 << 30), (0, 30, 30, 60)),
                         ((70, 10, 20, 30), (60, 60, 60, 60)), ((10, 5, 50, 40), (10, 10, 50, 50))):
        m = Mix(dev, (20, 30, 10), 2, 64, 1, 64, 4, "bf16", 1330, has=True)
        wide = torch.full((64, 160), 7.0, device=dev).bfloat16()
        m.y = wide[2:62, 16:144]
        m.cu_t = torch.tensor(wrong, dtype=torch.int32, device=dev)
        m.run(ssm)
        torch.cuda.synchronize()
        m.cu = np.array(right)
        m.check(f"{wrong}")
        wide[2:62, 16:144] = 7.0
        assert (wide == 7.0).all()


def test_two_calls_at_once(ssm, dev):  # noqa: F811
    """Two programs on streams of their own, with states and workspaces of their own:
    both get the bits that they get alone."""
    def fresh(i):
        return Aligned(dev, (700, 64, 300), 24, 64, 1, 128, 4, "bf16", 1340 + i, gate=False, has=True)
    alone = [fresh(0), fresh(1)]
    for m in alone:
        m.run(ssm)
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    for _ in range(5):
        both = [fresh(0), fresh(1)]
        torch.cuda.synchronize()
        for m, s in zip(both, streams):
            with torch.cuda.stream(s):
                m.run(ssm)
        torch.cuda.synchronize()
        for a, b in zip(alone, both):
            assert torch.equal(a.y, b.y) and torch.equal(a.hs, b.hs) and torch.equal(a.cs, b.cs)
