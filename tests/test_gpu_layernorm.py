"""GPU layer norm against its definition in 64 bits.

Tolerances.  A 16-bit output is off by at most half a step of its type
relative to its value; the fp32 arithmetic before it is a mean over the row, a
centred square mean and a handful of products: each correct to 2^-24 of the
largest value they take in, sums of n terms in a tree of at most 64 serial
steps a thread, so INNER = 64 * 2^-24 * 4 = 1.6e-5 of the largest value.  The
weight gradients are sums over the rows, at most rows / 304 + 16 serial steps
long; their bar is (rows / 304 + 64) 2^-24 of the largest column's sum of the
terms' sizes."""

import numpy as np
import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu

INNER = 1.6e-5
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def cs():
    from complex_valued_state_gb300 import build as cbuild
    from complex_valued_state_gb300 import cssd

    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for gpu tests")
    cbuild.build()
    cssd.load()
    return cssd


def close(got, want, what, top=None, inner=INNER):
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    got = got.detach().cpu().double().numpy()
    top = np.max(np.abs(want)) if top is None else top
    err, bar = np.abs(got - want), half * np.abs(want) + inner * max(float(top), 1e-30)
    assert (err <= bar).all(), f"{what}: worst {np.nanmax(err / bar):.3g} of the bar"


def make(seed, rows, width, dtype, wdtype, affine=True):
    r = np.random.default_rng(seed)
    t = lambda x, dt: torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[dt])  # noqa: E731
    x = t(r.standard_normal((rows, width)) * np.exp(r.standard_normal((rows, 1))) + r.standard_normal((rows, 1)), dtype)
    w = t(1 + 0.3 * r.standard_normal(width), wdtype) if affine else None
    b = t(0.3 * r.standard_normal(width), wdtype) if affine else None
    return x, w, b, t(r.standard_normal((rows, width)), dtype)


def f64(t):
    return None if t is None else t.double().numpy()


def dev(t):
    return None if t is None else t.cuda()


# one lane's worth, one warp, one vector past a warp, odd widths, each register form, the streaming forms
WIDTHS = [1, 7, 8, 64, 255, 264, 768, 1000, 1536, 2056, 4096, 5001, 8192, 16384, 33000]


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("width", WIDTHS)
def test_forward_and_backward(cs, width, dtype, wdtype):
    rows = 37 if width < 9000 else 5
    x, w, b, dy = make(width, rows, width, dtype, wdtype)
    y, mean, rstd = cs.layernorm(x.cuda(), dev(w), dev(b), eps=1e-5)
    want, m, r = ref.layernorm(f64(x), f64(w), f64(b), 1e-5)
    top = np.max(np.abs(f64(x)), axis=1)
    close(mean, m, "mean", top=top.max())
    if width > 1:
        close(rstd / torch.from_numpy(r).cuda().float(), np.ones_like(r), "rstd", inner=8 * INNER)
        close(y, want, "y", inner=4 * INNER)
    else:  # every row is its own mean
        close(y, want, "y")
    g = cs.layernorm_backward(dy.cuda(), x.cuda(), dev(w), mean, rstd)
    gx, gw, gb = ref.layernorm_backward(f64(dy), f64(x), f64(w), 1e-5)
    xh = (f64(x) - m[:, None]) * r[:, None]
    steps = (rows / 304 + 64) * 2.0 ** -24
    if width > 1:
        close(g["gx"], gx, "gx", inner=8 * INNER)
        close(g["gweight"], gw, "gweight", top=np.max(np.sum(np.abs(f64(dy) * xh), 0)), inner=steps + 4 * INNER)
    close(g["gbias"], gb, "gbias", top=np.max(np.sum(np.abs(f64(dy)), 0)), inner=steps)


@pytest.mark.parametrize("rows", [1, 3, 4, 5, 303, 1217, 5000])
def test_row_counts(cs, rows):
    for width in (64, 50):
        x, w, b, dy = make(rows, rows, width, "fp32", "fp32")
        y, mean, rstd = cs.layernorm(x.cuda(), dev(w), dev(b))
        want, m, r = ref.layernorm(f64(x), f64(w), f64(b), 1e-5)
        close(y, want, "y", inner=4 * INNER)
        g = cs.layernorm_backward(dy.cuda(), x.cuda(), dev(w), mean, rstd)
        gx, gw, gb = ref.layernorm_backward(f64(dy), f64(x), f64(w), 1e-5)
        xh = (f64(x) - m[:, None]) * r[:, None]
        steps = (rows / 304 + 64) * 2.0 ** -24
        close(g["gx"], gx, "gx", inner=8 * INNER)
        close(g["gweight"], gw, "gweight", top=np.max(np.sum(np.abs(f64(dy) * xh), 0)), inner=steps + 4 * INNER)
        close(g["gbias"], gb, "gbias", top=np.max(np.sum(np.abs(f64(dy)), 0)), inner=steps)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,width", [(1, 4096), (2, 6144), (3, 8192), (7, 12296), (5, 16001)])
def test_few_wide_rows(cs, rows, width, dtype):
    """Fewer rows than groups that sum them; rows of other widths between a
    thread's registers, a ring's stages and the streamed sums."""
    x, w, b, dy = make(rows + width, rows, width, dtype, "fp32")
    y, mean, rstd = cs.layernorm(x.cuda(), dev(w), dev(b))
    want, m, r = ref.layernorm(f64(x), f64(w), f64(b), 1e-5)
    close(y, want, "y", inner=4 * INNER)
    ws = torch.empty(cs.layernorm_backward_workspace_bytes(rows, width), dtype=torch.uint8, device="cuda")
    g = cs.layernorm_backward(dy.cuda(), x.cuda(), dev(w), mean, rstd, workspace=ws)
    gx, gw, gb = ref.layernorm_backward(f64(dy), f64(x), f64(w), 1e-5)
    xh = (f64(x) - m[:, None]) * r[:, None]
    steps = (rows / 304 + 64) * 2.0 ** -24
    close(g["gx"], gx, "gx", inner=8 * INNER)
    close(g["gweight"], gw, "gweight", top=np.max(np.sum(np.abs(f64(dy) * xh), 0)), inner=steps + 4 * INNER)
    close(g["gbias"], gb, "gbias", top=np.max(np.sum(np.abs(f64(dy)), 0)), inner=steps)
    assert cs.device_status() == 0


@pytest.mark.parametrize("width", [96, 101])
def test_without_affine_and_partial_gradients(cs, width):
    x, _, _, dy = make(3, 20, width, "fp16", "fp16", affine=False)
    y, mean, rstd = cs.layernorm(x.cuda())
    want, m, r = ref.layernorm(f64(x), None, None, 1e-5)
    close(y, want, "y", inner=4 * INNER)
    gx, gw, gb = ref.layernorm_backward(f64(dy), f64(x), None, 1e-5)
    g = cs.layernorm_backward(dy.cuda(), x.cuda(), None, mean, rstd, want_weight=False, want_bias=False)
    assert set(g) == {"gx"}
    close(g["gx"], gx, "gx", inner=8 * INNER)
    g = cs.layernorm_backward(dy.cuda(), x.cuda(), None, mean, rstd, want_weight=False)
    assert set(g) == {"gx", "gbias"}
    close(g["gbias"], gb, "gbias", top=np.max(np.sum(np.abs(f64(dy)), 0)), inner=64 * 2.0 ** -24)


def test_large_offset_rows(cs):
    """Rows far from zero (mean 1000 deviations): the centred variance keeps its digits."""
    r = np.random.default_rng(4)
    x = torch.from_numpy((1000.0 + r.standard_normal((9, 512))).astype(np.float32))
    y, mean, rstd = cs.layernorm(x.cuda())
    want, m, rs = ref.layernorm(f64(x), None, None, 1e-5)
    # the mean is off by at most INNER 1000, which shifts every y by that many deviations
    close(y, want, "y", top=1000.0)
    close(rstd, rs, "rstd", inner=8 * INNER)


def test_constant_rows_and_nonfinite_rows(cs):
    """A constant row has y = bias; a row with a NaN or an infinity does not touch its neighbours."""
    x = torch.randn(8, 256, generator=torch.Generator().manual_seed(5))
    x[2] = 3.0
    x[4, 7] = float("nan")
    x[6, 9] = float("inf")
    y, mean, rstd = cs.layernorm(x.cuda(), torch.ones(256).cuda(), torch.full((256,), 0.5).cuda())
    want, _, _ = ref.layernorm(f64(x), np.ones(256), np.full(256, 0.5), 1e-5)
    assert (y[2] == 0.5).all()
    assert torch.isnan(y[4]).all() and torch.isnan(y[6]).any()
    keep = [0, 1, 3, 5, 7]
    close(y[keep], want[keep], "y", inner=4 * INNER)


def test_in_place_stream_and_graph(cs):
    x, w, b, dy = make(6, 300, 768, "bf16", "bf16")
    xd, wd, bd, dyd = x.cuda(), dev(w), dev(b), dy.cuda()
    y, mean, rstd = cs.layernorm(xd, wd, bd)
    inplace = xd.clone()
    cs.layernorm(inplace, wd, bd, y=inplace)
    assert torch.equal(inplace, y)
    g = cs.layernorm_backward(dyd, xd, wd, mean, rstd)
    for over in ("dy", "x"):
        a, c = dyd.clone(), xd.clone()
        g2 = cs.layernorm_backward(a, c, wd, mean, rstd, grads={"gx": a if over == "dy" else c})
        for n in g:
            assert torch.equal(g[n], g2[n])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    y2, _, _ = cs.layernorm(xd, wd, bd, stream=s)
    g3 = cs.layernorm_backward(dyd, xd, wd, mean, rstd, stream=s)
    s.synchronize()
    assert torch.equal(y, y2) and all(torch.equal(g[n], g3[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y4, m4, r4 = cs.layernorm(xd, wd, bd)
        g4 = cs.layernorm_backward(dyd, xd, wd, m4, r4)
    xd.copy_(x.flip(0))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y4, y.flip(0))
    want = cs.layernorm_backward(dyd, xd, wd, m4, r4)
    for n in g4:
        assert torch.equal(g4[n], want[n])


@pytest.mark.parametrize("width", [8192, 8190])
def test_offsets_past_32_bits(cs, width):
    rows = (1 << 31) // width + 40
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    r = np.random.default_rng(7)
    last = torch.from_numpy(r.standard_normal((8, width)).astype(np.float32)).to(torch.bfloat16)
    x[-8:] = last.cuda()
    y, mean, rstd = cs.layernorm(x)
    want, m, rs = ref.layernorm(f64(last), None, None, 1e-5)
    close(y[-8:], want, "y", inner=4 * INNER)
    dy = x.clone()
    g = cs.layernorm_backward(dy, x, None, mean, rstd)
    gx, gw, gb = ref.layernorm_backward(f64(last), f64(last), None, 1e-5)
    close(g["gx"][-8:], gx, "gx", top=np.max(rs), inner=8 * INNER)
    close(g["gbias"], gb, "gbias", top=np.max(np.sum(np.abs(f64(last)), 0)))


@pytest.mark.parametrize("width", [96, 101, 8200])
def test_float_bias_without_weight(cs, width):
    """A float32 bias of a bfloat16 x: its gradient keeps float32's digits (the
    sums of 300 rows in bfloat16 would be off by up to 2^-9 of themselves)."""
    x, _, _, dy = make(8, 300, width, "bf16", "fp32", affine=False)
    b = torch.linspace(-1, 1, width)
    y, mean, rstd = cs.layernorm(x.cuda(), None, b.cuda())
    want, m, r = ref.layernorm(f64(x), None, f64(b), 1e-5)
    close(y, want, "y", inner=4 * INNER)
    g = cs.layernorm_backward(dy.cuda(), x.cuda(), None, mean, rstd, want_weight=False, wdtype=torch.float32)
    assert g["gbias"].dtype is torch.float32
    _, _, gb = ref.layernorm_backward(f64(dy), f64(x), None, 1e-5)
    close(g["gbias"], gb, "gbias", top=np.max(np.sum(np.abs(f64(dy)), 0)), inner=(300 / 304 + 64) * 2.0 ** -24)


@pytest.mark.parametrize("dtype,width", [("fp32", 512), ("fp32", 1028), ("fp32", 4096), ("fp32", 513), ("fp16", 512)])
def test_gradients_of_rows_far_from_zero(cs, dtype, width):
    """Rows 10000 deviations from zero (100 in fp16): with the mean as it is given,
    x - mean is off by 2^-24 of itself, so x^ and each term of the weight gradient
    by 3 x 2^-24, whatever the offset."""
    r = np.random.default_rng(9)
    x = torch.from_numpy(((100.0 if dtype == "fp16" else 1e4) + r.standard_normal((9, width))).astype(np.float32)).to(TYPES[dtype])
    dy = torch.from_numpy(r.standard_normal((9, width)).astype(np.float32)).to(TYPES[dtype])
    w = torch.from_numpy((1 + 0.3 * r.standard_normal(width)).astype(np.float32))
    _, mean, rstd = cs.layernorm(x.cuda(), w.cuda())
    g = cs.layernorm_backward(dy.cuda(), x.cuda(), w.cuda(), mean, rstd)
    rs = f64(rstd.cpu())[:, None]
    xh = (f64(x) - f64(mean.cpu())[:, None]) * rs
    a = f64(dy) * f64(w)
    gx = rs * (a - a.mean(1, keepdims=True) - xh * (a * xh).mean(1, keepdims=True))
    close(g["gx"], gx, "gx")
    terms = np.max(np.sum(np.abs(f64(dy) * xh), 0))
    close(g["gweight"], (f64(dy) * xh).sum(0), "gweight", top=terms, inner=(9 / 304 + 64 + 3) * 2.0 ** -24)
