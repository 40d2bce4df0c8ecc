"""The Mamba-2 mixer's operators on the host: what their C entry points refuse
before anything is enqueued, the binding's checks, and the float64 references
of the GPU tests against differences and against each other."""
import ctypes

import numpy as np
import pytest

import mixer_ref as ref
import oracle

P = 1 << 24  # fake addresses, 16-byte aligned, far apart


@pytest.fixture(scope="module")
def lib():
    import selective_state_space_43_amd as ssm
    return ssm.lib()


FWD = ("xbc", "xs", "dt", "ds", "z", "zs", "cw", "cb", "A", "D", "db", "softplus", "cu", "slots",
       "has", "cs", "hs", "y", "ys", "ws", "ws_bytes", "tokens", "nseq", "nslots", "H", "P", "G", "N",
       "W", "io", "stream")


def fwd_args(**over):
    a = dict(xbc=1 * P, xs=400, dt=2 * P, ds=4, z=None, zs=0, cw=3 * P, cb=None, A=4 * P, D=None,
             db=None, softplus=1, cu=5 * P, slots=None, has=None, cs=6 * P, hs=7 * P, y=8 * P, ys=256,
             ws=9 * P, ws_bytes=P, tokens=10, nseq=2, nslots=2, H=4, P=64, G=1, N=64, W=4, io=1,
             stream=None)
    a.update(over)
    return [a[k] for k in FWD]


FWD_BAD = [
    (dict(xbc=None), 1), (dict(dt=None), 1), (dict(cw=None), 1), (dict(A=None), 1),
    (dict(cu=None), 1), (dict(y=None), 1), (dict(ws=None), 1), (dict(cs=None), 1),
    (dict(hs=None), 1), (dict(hs=None, cs=None, slots=10 * P), 1),
    (dict(hs=None, cs=None, has=10 * P), 1),
    (dict(tokens=0), 2), (dict(nseq=0), 2), (dict(H=-1), 2), (dict(P=0), 2), (dict(N=0), 2),
    (dict(G=3), 2), (dict(nslots=0), 2), (dict(nslots=1), 2), (dict(xs=383), 2), (dict(ds=3), 2),
    (dict(ys=255), 2), (dict(z=10 * P, zs=100), 2), (dict(ws_bytes=15), 2), (dict(tokens=1 << 31), 2),
    (dict(nseq=1 << 20, nslots=1 << 20), 2), (dict(xs=1 << 50), 2),
    (dict(io=2), 3), (dict(io=-1), 3),
    (dict(xbc=1 * P + 1), 4), (dict(y=8 * P + 1), 4), (dict(ws=9 * P + 8), 4), (dict(hs=7 * P + 2), 4),
    (dict(cs=6 * P + 1), 4),
    (dict(y=1 * P), 5), (dict(y=7 * P + 64), 5), (dict(ws=8 * P), 5), (dict(hs=6 * P), 5),
    (dict(cs=3 * P), 5), (dict(ws=1 * P), 5),
    (dict(xbc=1 * P, xs=1000, y=1 * P + 2 * 300, ys=1000), 5),  # columns 300.. of xbc's 384
    (dict(P=257), 6), (dict(N=257, xs=1000), 6), (dict(W=0), 6), (dict(W=5), 6),
]


@pytest.mark.parametrize("over,status", FWD_BAD, ids=lambda v: str(v) if isinstance(v, int) else "-".join(v))
def test_conv_ssd_fwd_refusals(lib, over, status):
    import selective_state_space_43_amd as ssm
    assert lib.ssm_conv_ssd_fwd(*fwd_args(**over)) == status
    assert ssm.ssm_last_error() != ""


STEP = ("xbc", "xs", "dt", "ds", "z", "zs", "cw", "cb", "A", "D", "db", "softplus", "slots", "cs",
        "hs", "y", "ys", "batch", "nslots", "H", "P", "G", "N", "W", "io", "stream")


def step_args(**over):
    a = dict(xbc=1 * P, xs=400, dt=2 * P, ds=4, z=None, zs=0, cw=3 * P, cb=None, A=4 * P, D=None,
             db=None, softplus=1, slots=None, cs=6 * P, hs=7 * P, y=8 * P, ys=256, batch=10, nslots=10,
             H=4, P=64, G=1, N=64, W=4, io=1, stream=None)
    a.update(over)
    return [a[k] for k in STEP]


@pytest.mark.parametrize("over,status", [
    (dict(xbc=None), 1), (dict(hs=None), 1), (dict(cs=None), 1), (dict(y=None), 1), (dict(A=None), 1),
    (dict(batch=0), 2), (dict(nslots=9), 2), (dict(G=8), 2), (dict(xs=1), 2), (dict(ys=255), 2),
    (dict(io=7), 3), (dict(xbc=P + 1), 4), (dict(hs=7 * P + 1), 4),
    (dict(y=1 * P), 5), (dict(hs=1 * P), 5), (dict(cs=7 * P), 5), (dict(y=6 * P + 4), 5),
    (dict(P=300), 6), (dict(N=300, xs=2000), 6), (dict(W=9), 6),
], ids=lambda v: str(v) if isinstance(v, int) else "-".join(v))
def test_conv_ssd_update_refusals(lib, over, status):
    assert lib.ssm_conv_ssd_update(*step_args(**over)) == status


def test_conv_ssd_workspace_size(lib):
    f = lib.ssm_conv_ssd_workspace_size
    assert f(10, 2, 4, 64, 1, 64, 1) > 0 and f(10, 2, 4, 64, 1, 64, 1) % 16 == 0
    for bad in ((0, 2, 4, 64, 1, 64, 1), (10, 0, 4, 64, 1, 64, 1), (10, 2, 4, 64, 3, 64, 1),
                (10, 2, 4, 300, 1, 64, 1), (10, 2, 4, 64, 1, 64, 5)):
        assert f(*bad) == -1
    assert f(100000, 2, 4, 64, 1, 64, 1) >= f(10, 2, 4, 64, 1, 64, 1)


NORM = ("x", "xs", "z", "zs", "w", "b", "eps", "center", "act", "gate", "y", "ys", "rows", "C", "G",
        "io", "stream")


def norm_args(**over):
    a = dict(x=1 * P, xs=100, z=None, zs=0, w=2 * P, b=None, eps=1e-5, center=0, act=0, gate=0, y=3 * P,
             ys=100, rows=7, C=100, G=5, io=1, stream=None)
    a.update(over)
    return [ctypes.c_float(a[k]) if k == "eps" else a[k] for k in NORM]


NORM_BAD = [
    (dict(x=None), 1), (dict(gate=1), 1), (dict(z=4 * P, zs=100), 1),
    (dict(rows=0), 2), (dict(C=0), 2), (dict(G=7), 2), (dict(G=0), 2), (dict(xs=99), 2),
    (dict(eps=-1.0), 2), (dict(eps=float("nan")), 2), (dict(eps=float("inf")), 2),
    (dict(io=3), 3), (dict(act=2), 3), (dict(gate=3), 3), (dict(act=-1), 3),
    (dict(x=P + 1), 4),
    (dict(C=40000, G=1, xs=40000, ys=40000), 6),
]


@pytest.mark.parametrize("over,status", NORM_BAD + [(dict(y=None), 1), (dict(y=1 * P), 5),
                                                    (dict(y=2 * P), 5), (dict(ys=99), 2)],
                         ids=lambda v: str(v) if isinstance(v, int) else "-".join(v))
def test_group_norm_fwd_refusals(lib, over, status):
    assert lib.ssm_group_norm_fwd(*norm_args(**over)) == status


NORMB = ("dy", "gs", "x", "xs", "z", "zs", "w", "b", "eps", "center", "act", "gate", "dx", "dxs", "dz",
         "dzs", "dw", "db", "ws", "ws_bytes", "rows", "C", "G", "io", "stream")


@pytest.mark.parametrize("over,status", NORM_BAD + [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(ws=None), 1), (dict(dz=9 * P, dzs=100), 1),
    (dict(z=4 * P, zs=100, gate=1), 1),
    (dict(gs=1), 2), (dict(ws_bytes=8), 2), (dict(ws=6 * P + 8), 4),
    (dict(dx=1 * P), 5), (dict(dw=2 * P), 5), (dict(db=6 * P), 5), (dict(dw=8 * P, db=8 * P + 64), 5),
    (dict(ws=5 * P), 5),
], ids=lambda v: str(v) if isinstance(v, int) else "-".join(v))
def test_group_norm_bwd_refusals(lib, over, status):
    a = dict(dy=5 * P, gs=100, x=1 * P, xs=100, z=None, zs=0, w=2 * P, b=None, eps=1e-5, center=0, act=0,
             gate=0, dx=3 * P, dxs=100, dz=None, dzs=0, dw=None, db=None, ws=6 * P, ws_bytes=P,
             rows=7, C=100, G=5, io=1, stream=None)
    a.update(over)
    if over.get("C") == 40000:
        a.update(gs=40000, dxs=40000)
    a = [ctypes.c_float(a[k]) if k == "eps" else a[k] for k in NORMB]
    assert lib.ssm_group_norm_bwd(*a) == status


def test_group_norm_bwd_workspace_size(lib):
    f = lib.ssm_group_norm_bwd_workspace_size
    assert f(0, 10, 1) == -1 and f(10, 0, 1) == -1 and f(10, 10, 0) == -1
    assert f(10, 10, 1) > 0 and f(10, 10, 1) % 16 == 0


def test_interleaved_slices_are_no_overlap(lib):
    """Slices of one buffer's rows with disjoint columns pass the overlap check:
    the refusal that follows is about the last argument checked after it."""
    import selective_state_space_43_amd as ssm
    # y in columns 384.. of the rows that hold xbc in columns 0..383; the workspace is too small
    args = fwd_args(xs=1000, y=1 * P + 2 * 384, ys=1000, ws_bytes=15)
    assert lib.ssm_conv_ssd_fwd(*args) == 2 and "workspace" in ssm.ssm_last_error()
    # rows behind the last column wrap into the next row's first
    args = fwd_args(xs=1000, y=1 * P + 2 * 745, ys=1000, ws_bytes=15)
    assert lib.ssm_conv_ssd_fwd(*args) == 5


def test_binding_refuses(lib):
    torch = pytest.importorskip("torch")
    import selective_state_space_43_amd as ssm
    x = torch.zeros(3, 384)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssm.ssm_conv_ssd_fwd(x, x, x, torch.zeros(4), torch.zeros(2, dtype=torch.int32), 64, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssm.ssm_conv_ssd_update(x, x, x, x, x, x, 1)
    with pytest.raises(ValueError, match="GPU tensor"):
        ssm.ssm_group_norm_fwd(x, None, 1)
    with pytest.raises(ValueError, match="out of range"):
        ssm.ssm_conv_ssd_workspace_size(0, 1, 1, 64, 1, 64)
    with pytest.raises(ValueError, match="out of range"):
        ssm.ssm_group_norm_bwd_workspace_size(0, 1, 1)


# ---------------------------------------------------------------- the references

@pytest.mark.parametrize("center", [False, True])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("gate", ["none", "before", "after"])
def test_norm_reference_gradients_against_differences(center, act, gate):
    """Central differences (step 1e-6) of the float64 forward; their own error is
    about 1e-10 of the values here."""
    rng = np.random.default_rng(7)
    rows, C, G = 3, 12, 3
    x, z, dy = (rng.standard_normal((rows, C)) for _ in range(3))
    w, b = rng.standard_normal(C), rng.standard_normal(C)
    z = z if gate != "none" else None
    how = dict(center=center, act=act, gate=gate)
    g, t = ref.norm_bwd(dy, x, w, G, b, z, **how)
    for name, leaf in (("dx", x), ("dweight", w), ("dbias", b), ("dz", z)):
        if leaf is None:
            assert name not in g
            continue
        d = np.zeros_like(leaf)
        for i in np.ndindex(leaf.shape):
            keep, both = leaf[i], []
            for e in (1e-6, -1e-6):
                leaf[i] = keep + e
                both.append((dy * ref.norm(x, w, G, b, z, **how)[0]).sum())
            leaf[i] = keep
            d[i] = (both[0] - both[1]) / 2e-6
        np.testing.assert_allclose(g[name], d, rtol=1e-6, atol=1e-7)
        assert np.all(t[name] >= np.abs(g[name]) * (1 - 1e-12))


def test_packed_reference_is_step_by_step():
    """The packed reference with its states carried equals the recurrence written
    out one token at a time in numpy."""
    rng = np.random.default_rng(8)
    H, Pd, G, N, W = 4, 3, 2, 5, 3
    x = ref.mix_inputs(rng, 9, 3, H, Pd, G, N, W, "f32", 5)
    cu, slots, has = [0, 4, 4, 8], [3, 0, 1], [True, True, False]
    y, cs, hs, _, _ = ref.mix(x, cu, G, slots, has)
    assert np.isnan(y[8]).all() and not np.isnan(y[:8]).any()
    np.testing.assert_array_equal(hs[0], x["ssm_state"][0])  # an empty sequence keeps its state
    np.testing.assert_array_equal(hs[2], x["ssm_state"][2])  # nobody's slot
    sig = lambda v: v / (1 + np.exp(-v))  # noqa: E731
    for s in (0, 2):
        hist = x["conv_state"][slots[s]].copy() if has[s] else np.zeros((x["xbc"].shape[1], W - 1))
        h = x["ssm_state"][slots[s]].copy() if has[s] else np.zeros((H, Pd, N))
        for t in range(cu[s], cu[s + 1]):
            win = np.concatenate([hist, x["xbc"][t][:, None]], 1)
            c = sig((win * x["conv_weight"]).sum(1) + x["conv_bias"])
            hist = win[:, 1:]
            xs, B, C = c[:H * Pd].reshape(H, Pd), c[H * Pd:H * Pd + G * N].reshape(G, N), c[H * Pd + G * N:].reshape(G, N)
            for i in range(H):
                d = np.log1p(np.exp(x["dt"][t, i] + x["dt_bias"][i]))
                h[i] = np.exp(d * x["A"][i]) * h[i] + d * np.outer(xs[i], B[i // 2])
                o = (h[i] @ C[i // 2] + x["D"][i] * xs[i]) * sig(x["z"][t, i * Pd:(i + 1) * Pd])
                np.testing.assert_allclose(y[t, i * Pd:(i + 1) * Pd], o, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(hs[slots[s]], h, rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(cs[slots[s]], hist, rtol=0, atol=0)


def test_bounds_hold_the_terms_absolute_values():
    """The bounds' sums against the recurrence on absolute values written out, with
    steps below zero: each term once, with its magnitude."""
    rng = np.random.default_rng(0)
    x = ref.mix_inputs(rng, 5, 1, 1, 1, 1, 2, 1, "f32", 1, gate=False)
    x["inner"], x["dt"], x["dt_bias"] = 1, -np.abs(x["dt"]) * 0.1, np.zeros(1)
    _, _, _, (ya, _), (ha, _) = ref.mix(x, [0, 5], 1, None, [True], softplus=False)
    c = x["xbc"] * x["conv_weight"][:, 0] + x["conv_bias"]
    c = c / (1 + np.exp(-c))
    h = np.abs(x["ssm_state"][0, 0, 0])
    for t in range(5):
        h = np.exp(x["dt"][t, 0] * x["A"][0]) * h + abs(x["dt"][t, 0] * c[t, 0]) * np.abs(c[t, 1:3])
        np.testing.assert_allclose(ya[t, 0], (h * np.abs(c[t, 3:])).sum() + abs(x["D"][0] * c[t, 0]))
    np.testing.assert_allclose(ha[0, 0, 0], h)


def test_bf16_helper():
    v = np.array([1.0, 1.00390625, 1.01171875, -3.1415927, 1e-20], dtype=np.float32)
    torch = pytest.importorskip("torch")
    np.testing.assert_array_equal(ref.bf16(v), torch.from_numpy(v).bfloat16().double().numpy())
    assert oracle is not None


# A launch has less than 2^32 threads: calls past that are refused before anything is enqueued
# (pointers far enough apart that nothing overlaps).

FAR = 1 << 44


def test_launches_too_large_are_refused(lib):
    import selective_state_space_43_amd as ssm
    # a workgroup of 1024 threads for every block of 64 tokens
    assert lib.ssm_conv_ssd_workspace_size(1 << 28, 1, 4, 64, 1, 64, 1) == -1
    assert "tokens / 64" in ssm.ssm_last_error()
    assert lib.ssm_conv_ssd_workspace_size((1 << 28) - 128, 1, 4, 64, 1, 64, 1) > 0
    assert lib.ssm_conv_ssd_fwd(*fwd_args(tokens=1 << 28)) == 2
    # 2^20 sequences x 64 workgroups of 256 threads
    n = (1 << 20) - 1
    far = dict(xbc=1 * FAR, dt=2 * FAR, y=3 * FAR, cs=4 * FAR, hs=5 * FAR)
    big = dict(nslots=n, H=256, P=64, G=1, N=8, xs=256 * 64 + 16, ds=256, ys=256 * 64, **far)
    need = lib.ssm_conv_ssd_workspace_size(1 << 20, n, 256, 64, 1, 8, 1)
    assert lib.ssm_conv_ssd_fwd(*fwd_args(tokens=1 << 20, nseq=n, cu=6 * FAR, ws=7 * FAR, ws_bytes=need, **big)) == 2
    assert "one call" in ssm.ssm_last_error()
    assert lib.ssm_conv_ssd_update(*step_args(batch=n, **big)) == 2
    assert "one call" in ssm.ssm_last_error()
    # 2^27 rows of a group of 512, a wave each
    assert lib.ssm_group_norm_fwd(*norm_args(x=1 * FAR, y=2 * FAR, xs=512, ys=512, rows=1 << 27, C=512, G=1)) == 2
    assert "one call" in ssm.ssm_last_error()
