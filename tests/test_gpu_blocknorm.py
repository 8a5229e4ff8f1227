"""GPU norms before and after a block against their definitions in 64 bits.

Tolerances.  A 16-bit output is off by at most half a step of its type relative
to its value (the largest value's, where the largest sizes bound the errors).
The fp32 arithmetic before it is a mean over the row, a centred square mean and
a handful of products: each correct to 2^-24 of the largest value they take in,
sums of n terms in a tree of at most 64 serial steps a thread, so INNER = 64 *
2^-24 * 4 = 1.6e-5 of the row's largest value.  The exponential of the gate adds 2
steps of fp32 and 2^-24 |z|.  s is rounded to its type before the norm reads
it: where the two sides round differently (a tie or nearly one) the value moves
by a step of s's type, which y follows, so y is checked against the norm of the
s that came back.  Sums over the rows are at most rows / 304 + 64 serial
steps; their bar is (rows / 304 + 64) 2^-24 of the column's sum of the terms'
sizes plus INNER of the largest one's, and half a step of their type."""

import block_reference as ref
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

INNER = 1.6e-5
EPS = 1e-5
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
    """`top`: the size that the fp32 arithmetic's errors are relative to (by rows: [R, 1])."""
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = 2.0 ** -25 if got.dtype == torch.float16 else 0.0
    got = got.detach().cpu().double().numpy()
    if top is None:
        top = np.max(np.abs(want), axis=-1, keepdims=True)
    err, bar = np.abs(got - want), half * np.abs(want) + inner * top + tiny + 1e-30
    assert (err <= bar).all(), f"{what}: worst {np.nanmax(err / bar):.3g} of the bar, {(~(err <= bar)).sum()} of {err.size}"


def columns(got, want, terms, rows, what):
    close(got, want, what, top=terms * ((rows / 304 + 64) * 2.0 ** -24) + INNER * terms.max(), inner=1.0)


def t(x, dt):
    return torch.from_numpy(np.asarray(x, np.float32)).to(TYPES[dt])


def f64(x):
    return None if x is None else x.double().numpy()


def dev(x):
    return None if x is None else x.cuda()


def vectors(r, D, dt, bias, n=3):
    v = [t(1 + 0.3 * r.standard_normal(D), dt), t(0.3 * r.standard_normal(D), dt) if bias else None, t(0.5 + 0.2 * r.standard_normal(D), dt)]
    return v[:n]


WIDTHS = [1, 5, 8, 40, 64, 256, 333, 512, 1001, 1024, 1536, 2048, 2056, 4096, 6144, 8200]
ROWS = {1: 700, 64: 1000, 1536: 700, 6144: 9, 8200: 4}


@pytest.mark.parametrize("types", [("bf16", "fp32", "bf16"), ("bf16", "bf16", "fp32"), ("fp16", "fp16", "fp16"), ("fp16", "fp32", "fp32"),
                                   ("fp32", "fp32", "fp32")])
@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_add_norm(cs, D, kind, types):
    xt, rt, wt = types
    R, layer = ROWS.get(D, 37), kind == "layer"
    full = (D + len(xt)) % 2 == 0  # with scale and bias
    r = np.random.default_rng(D)
    w, b, sc = vectors(r, D, wt, full)
    sc = sc if full else None
    x, res, dy, ds = (t(r.standard_normal((R, D)) * np.exp(r.standard_normal((R, 1))) + r.standard_normal((R, 1)), k) for k in (xt, rt, xt, rt))
    y, s, mean, rstd = cs.add_norm(dev(x), dev(res), dev(w), dev(b), kind=kind, alpha=0.7, scale=dev(sc), eps=EPS)
    _, ws, _, _ = ref.add_norm(f64(x), f64(res), f64(w), f64(b), layer, 0.7, f64(sc), EPS)
    close(s, ws, "s", top=np.abs(f64(res)) + np.abs(f64(x)), inner=2.0 ** -22)
    kept = f64(s.cpu())
    wy, _, wm, wr = ref.add_norm(0 * kept, kept, f64(w), f64(b), layer, 0.0, None, EPS)
    amp = np.abs(kept).max(1, keepdims=True) * wr[:, None]  # of norm(s), before the mean is taken off
    close(y, wy, "y", top=amp * 2 + np.abs(wy).max(1, keepdims=True))
    close(rstd, wr, "rstd", top=wr, inner=INNER * (1 + (np.abs(wm) * wr) ** 2) if layer else INNER)
    if layer:
        close(mean, wm, "mean", top=np.abs(kept).max(1))
    else:
        assert mean is None
    want = ref.add_norm_backward(f64(dy), f64(ds), f64(x), kept, f64(w), layer, 0.7, f64(sc), EPS)
    g = cs.add_norm_backward(dev(dy), dev(ds), dev(x), s, dev(w), mean, rstd, alpha=0.7, scale=dev(sc), want_bias=full)
    assert ("gbias" in g) == full and ("gscale" in g) == full
    size = wr[:, None] * np.abs(f64(dy)).max(1, keepdims=True) * np.abs(f64(w)).max() * (1 + amp) + np.abs(f64(ds)).max(1, keepdims=True)
    close(g["gresidual"], want["gresidual"], "gresidual", top=size)
    close(g["gx"], want["gx"], "gx", top=size)
    for n in ("gweight", "gbias", "gscale"):
        if n in g:
            columns(g[n], want[n], want[n + "_terms"], R, n)


GROUPS = [(1, 1), (5, 5), (64, 64), (64, 16), (96, 32), (256, 64), (333, 333), (512, 128), (960, 80), (1001, 143), (1536, 64), (1536, 1536),
          (2048, 256), (2048, 512), (2056, 2056), (4096, 4096), (4096, 128), (6144, 2048), (8200, 8200)]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("widths", GROUPS)
@pytest.mark.parametrize("form", [("rms", False), ("rms", True), ("layer", False), ("layer", True)])
def test_gated_norm(cs, widths, form, types):
    (D, group), (kind, first), (xt, wt) = widths, form, types
    R, layer = ROWS.get(D, 37), kind == "layer"
    bias = (D + len(xt) + first) % 2 == 0
    r = np.random.default_rng(D + group)
    w, b = vectors(r, D, wt, bias, 2)
    x, z, dy = (t(r.standard_normal((R, D)) * np.exp(r.standard_normal((R, 1))) + m * r.standard_normal((R, 1)), xt) for m in (1, 1, 0))
    y, mean, rstd = cs.gated_norm(dev(x), dev(z), dev(w), dev(b), kind=kind, group=group, gate_first=first, eps=EPS)
    assert rstd.shape == (R, D // group) and (mean is not None) == layer
    X, Z, DY, W, B = (f64(v) for v in (x, z, dy, w, b))
    wy, wm, wr = ref.gated_norm(X, Z, W, B, layer, group, first, EPS)
    gate = np.abs(ref.silu(Z))
    h = (X * ref.silu(Z) if first else X).reshape(R, -1, group)
    wide = lambda v: np.repeat(v, group, axis=1)  # noqa: E731
    peak = np.abs(h).max(2)
    amp = wide(peak * wr)  # of norm(h), before the mean is taken off
    out = (2 * amp * (1 + np.abs(W)) + (0 if B is None else np.abs(B))) * (1 if first else gate)
    zed = 1 + np.abs(Z).max() / 64
    close(y, wy, "y", top=out, inner=INNER * zed)
    close(rstd, wr, "rstd", top=wr, inner=INNER * zed * (1 + (np.abs(wm) * wr).max() ** 2))
    if layer:
        close(mean, wm, "mean", top=peak, inner=INNER * zed)
    want = ref.gated_norm_backward(DY, X, Z, W, B, layer, group, first, EPS)
    g = cs.gated_norm_backward(dev(dy), dev(x), dev(z), dev(w), dev(b), mean, rstd, group=group, gate_first=first, want_bias=bias)
    assert ("gbias" in g) == bias
    du = np.abs(DY) * (1 if first else gate)
    dh = wide(wr * (du * np.abs(W)).reshape(R, -1, group).max(2)) * (2 + 2 * amp * wide(peak * wr))
    slope = 1.2
    top = {"gx": dh * (gate if first else 1), "gz": slope * (dh * np.abs(X) if first else np.abs(DY) * out / np.maximum(gate, 1e-30))}
    for n in ("gx", "gz"):
        close(g[n], want[n], n, top=top[n], inner=INNER * zed)
    for n in ("gweight", "gbias"):
        if n in g:
            columns(g[n], want[n], want[n + "_terms"] + INNER * 0, R, n)


def test_vectors_left_out(cs):
    """No weight, no bias, no scale, nothing else that reaches s, and gradients of the vectors by their named type."""
    r = np.random.default_rng(3)
    x, res, dy = (t(r.standard_normal((50, 192)), "bf16") for _ in range(3))
    y, s, mean, rstd = cs.add_norm(dev(x), dev(res), kind="layer")
    kept = f64(s.cpu())
    close(y, ref.norm(kept, True, 1e-5)[0], "y", top=np.abs(kept).max())
    want = ref.add_norm_backward(f64(dy), None, f64(x), kept, None, True, 1.0, None, 1e-5)
    g = cs.add_norm_backward(dev(dy), None, dev(x), s, None, mean, rstd, want_scale=True, wdtype=torch.float32)
    for n in ("gresidual", "gx"):
        close(g[n], want[n], n, top=4 * np.abs(f64(dy)).max())
    for n in ("gweight", "gbias", "gscale"):
        assert g[n].dtype is torch.float32
        columns(g[n], want[n], want[n + "_terms"], 50, n)
    g2 = cs.add_norm_backward(dev(dy), None, None, s, None, mean, rstd, want_weight=False, want_bias=False)
    assert set(g2) == {"gx", "gresidual"} and torch.equal(g2["gx"], g["gx"])
    y, _, rstd = cs.gated_norm(dev(x), dev(res))
    close(y, ref.gated_norm(f64(x), f64(res), None, None, False, 192, False, 1e-5)[0], "gated y", top=8 * np.abs(f64(res)).max())
    g = cs.gated_norm_backward(dev(dy), dev(x), dev(res), None, None, None, rstd)
    want = ref.gated_norm_backward(f64(dy), f64(x), f64(res), None, None, False, 192, False, 1e-5)
    for n in ("gx", "gz"):
        close(g[n], want[n], n, top=8 * np.abs(f64(dy)).max() * np.abs(f64(res)).max())
    columns(g["gweight"], want["gweight"], want["gweight_terms"], 50, "gweight")


@pytest.mark.parametrize("D", [512, 1536, 333])
def test_in_place(cs, D):
    """Results over the tensors that the documentation allows."""
    r = np.random.default_rng(4)
    x, res, z, dy, ds = (t(r.standard_normal((300, D)), "bf16").cuda() for _ in range(5))
    w = t(1 + 0.3 * r.standard_normal(D), "bf16").cuda()
    y, s, _, rstd = cs.add_norm(x, res, w)
    x2, r2 = x.clone(), res.clone()
    cs.add_norm(x2, r2, w, s=r2, y=x2)
    assert torch.equal(x2, y) and torch.equal(r2, s)
    g = cs.add_norm_backward(dy, ds, x, s, w, None, rstd, want_scale=True)
    for over in (("dy", "ds"), ("x", "s")):
        t_ = {"dy": dy.clone(), "ds": ds.clone(), "x": x.clone(), "s": s.clone()}
        h = cs.add_norm_backward(t_["dy"], t_["ds"], t_["x"], t_["s"], w, None, rstd, want_scale=True,
                                 grads={"gx": t_[over[0]], "gresidual": t_[over[1]]})
        for n in g:
            assert torch.equal(g[n], h[n]), (over, n)
    y, _, rstd = cs.gated_norm(x, z, w)
    for k in (0, 1):
        t_ = [x.clone(), z.clone()]
        cs.gated_norm(*t_, w, y=t_[k])
        assert torch.equal(t_[k], y)
    g = cs.gated_norm_backward(dy, x, z, w, None, None, rstd)
    for a, b in ((0, 1), (1, 2), (2, 0), (0, 2)):
        t_ = [dy.clone(), x.clone(), z.clone()]
        h = cs.gated_norm_backward(*t_, w, None, None, rstd, grads={"gx": t_[a], "gz": t_[b]})
        for n in g:
            assert torch.equal(g[n], h[n]), (a, b, n)


def test_gates_at_their_ends(cs):
    """Gates far from zero on both sides, and zero: silu(z) is z, 0 or 0, its slope 1, 0 or 1/2."""
    z = torch.tensor([0.0, 1e4, -1e4, 60.0, -60.0, 120.0, -120.0, 1.0] * 8).repeat(3, 1)
    x = torch.linspace(-2, 3, 64).repeat(3, 1)
    for first in (False, True):
        y, _, rstd = cs.gated_norm(x.cuda(), z.cuda(), gate_first=first)
        wy, _, _ = ref.gated_norm(f64(x), f64(z), None, None, False, 64, first, 1e-5)
        close(y, wy, "y", top=np.abs(wy) + (0 if first else 1e-3))
        g = cs.gated_norm_backward(torch.ones(3, 64).cuda(), x.cuda(), z.cuda(), None, None, None, rstd, gate_first=first)
        want = ref.gated_norm_backward(np.ones((3, 64)), f64(x), f64(z), None, None, False, 64, first, 1e-5)
        for n in ("gx", "gz"):
            assert torch.isfinite(g[n]).all()
            close(g[n], want[n], n, top=np.abs(want[n]).max())


def test_rows_far_from_zero(cs):
    """Rows 1000 deviations from zero: the mean is taken off before rstd is multiplied on."""
    r = np.random.default_rng(5)
    x = t(1000 + r.standard_normal((64, 512)), "fp32")
    dy = t(r.standard_normal((64, 512)), "fp32")
    zero = torch.zeros_like(x).cuda()
    y, s, mean, rstd = cs.add_norm(zero, x.cuda(), kind="layer")
    hh, m, rs = ref.norm(f64(x), True, 1e-5)
    # the mean is right to 64 2^-24 of 1000: 4e-3 deviations at most, and half of a step of the values themselves
    close(y, hh, "y", top=1000 * rs[:, None], inner=2.0 ** -22)
    g = cs.add_norm_backward(dy.cuda(), None, zero, s, None, mean, rstd)
    want = ref.add_norm_backward(f64(dy), None, 0 * f64(x), f64(x), None, True, 1.0, None, 1e-5)
    close(g["gweight"], want["gweight"], "gweight", top=np.abs(f64(dy)).sum(0) * 1000 * 2.0 ** -22, inner=1.0)


@pytest.mark.parametrize("D", [1536, 333])
def test_other_stream_and_graph(cs, D):
    r = np.random.default_rng(6)
    x, res, z, dy, ds = (t(r.standard_normal((900, D)), "bf16").cuda() for _ in range(5))
    w = t(1 + 0.3 * r.standard_normal(D), "bf16").cuda()

    def both(stream=None):
        y, s, _, rstd = cs.add_norm(x, res, w, scale=w, stream=stream)
        out = [y, s, *cs.add_norm_backward(dy, ds, x, s, w, None, rstd, scale=w, stream=stream).values()]
        y, _, rstd = cs.gated_norm(x, z, w, stream=stream)
        return out + [y, *cs.gated_norm_backward(dy, x, z, w, None, None, rstd, stream=stream).values()]

    want = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = both()
    x.copy_(dy * 2)
    z.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(both(), got))


def test_many_rows(cs):
    """More rows than blocks, and tensors of more than 2^31 elements: the last rows are right."""
    R, D = (1 << 31) // 512 + 5, 512
    x = torch.empty(R, D, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    z = torch.ones_like(x)
    for y, last in ((cs.gated_norm(x, z, group=64)[0][-3:], ref.gated_norm(f64(x[-3:].cpu()), np.ones((3, D)), None, None, False, 64, False, EPS)[0]),
                    (cs.add_norm(x, z)[0][-3:], None)):
        if last is None:
            last = ref.norm(f64((x[-3:].float() + 1).bfloat16().cpu()), False, EPS)[0]
        close(y, last, "y", top=8.0)


def test_a_layer(cs):
    """The operators as a layer runs them: the norm with the residual sum, the
    attention over a prompt and then token by token, the gated norm of the
    heads; a prompt and its steps give what the whole sequence gives."""
    B, T, H, P, D = 2, 70, 4, 64, 256
    gen = torch.Generator().manual_seed(7)
    rnd = lambda *s: torch.randn(*s, generator=gen).cuda()  # noqa: E731
    x, res, z = (rnd(B, T, D) for _ in range(3))
    W = rnd(3, D, H * P) * D ** -0.5
    w, g = 1 + 0.2 * rnd(D), -torch.rand(H, generator=gen).cuda()

    def layer(x, res, z, mix):
        y, s, _, _ = cs.add_norm(x, res, w, alpha=0.5)
        q, k, v = (torch.matmul(y, W[i]).unflatten(-1, (H, P)) for i in range(3))
        o = mix(q, k * P ** -0.5, v)
        return cs.gated_norm(o.flatten(-2), z, w, group=P)[0], s

    state = {}

    def prompt(q, k, v):
        o, state["h"] = cs.linattn_forward(q, k, v, g)
        return o

    whole, s = layer(x, res, z, prompt)
    first, s1 = layer(*(t_[:, :50].contiguous() for t_ in (x, res, z)), prompt)
    rest = [layer(*(t_[:, i].contiguous() for t_ in (x, res, z)), lambda q, k, v: cs.linattn_step(state["h"], q, k, v, g)) for i in range(50, T)]
    got, kept = torch.cat([first] + [a[:, None] for a, _ in rest], 1), torch.cat([s1] + [b[:, None] for _, b in rest], 1)
    assert torch.equal(kept, s)
    # (the products in front are a library's, whose sums of 256 terms may go another way: 256 2^-24 of their sizes, before a norm)
    close(got, f64(whole.cpu()), "layer", top=np.abs(f64(whole.cpu())).max(), inner=2e-4)


@pytest.mark.parametrize("group", [64, 50, 1500])
def test_float32_gates_are_float32(cs, group):
    """Every element of float32 results, with gates from -80 to 20.  With the rstd that came back the norm is one
    product.  Steps of 2^-24: the gate's exponential 2, the sum 1, the quick quotient 4, its product with z 1, the norm 1
    and its product with the gate 1: 10 of y.  gz is the norm times the slope s (1 + z (1 - s)): s 7, 1 - s and the bracket
    (below z = -3 of size |z| - 1 or more) 1 each and 1.5 times more for the 1 beside z, what s moves in it 0.5, the two products
    and the norm 3: below 14 of gz."""
    z = torch.linspace(-80, 20, 300 * group).reshape(300, group).flip(0).contiguous()
    x = torch.rand(z.shape, generator=torch.Generator().manual_seed(8)) + 0.5
    y, _, rstd = cs.gated_norm(x.cuda(), z.cuda())
    hh = f64(x) * f64(rstd.cpu())
    close(y, hh * ref.silu(f64(z)), "y", top=np.abs(hh * ref.silu(f64(z))), inner=10 * 2.0 ** -24)
    g = cs.gated_norm_backward(torch.ones_like(x).cuda(), x.cuda(), z.cuda(), None, None, None, rstd)
    s = 1 / (1 + np.exp(-f64(z)))
    want, low = hh * s * (1 + f64(z) * (1 - s)), f64(z) < -3
    err = np.abs(f64(g["gz"].cpu()) - want)[low] / np.abs(want)[low]
    assert (err <= 14 * 2.0 ** -24).all(), err.max() * 2 ** 24


@pytest.mark.parametrize("widths", [(7296, 24), (14592, 48), (960, 80), (7296, 912)])
def test_sums_over_many_rows_of_many_groups(cs, widths):
    """Equal rows, whose sums are known: the gradients of the weights over 20000 of them are within (rows / 304 + 64)
    2^-24 of the sums, as everywhere, however many groups share the blocks, and 10 2^-24 for a row's own products."""
    (D, group), R = widths, 20000
    r = np.random.default_rng(9)
    x, z, dy = (t(np.abs(r.standard_normal(D)) + 0.1, "bf16") for _ in range(3))
    X, Z, DY = (v.cuda().expand(R, D).contiguous() for v in (x, z, dy))
    rstd = cs.gated_norm(X, Z, group=group)[2]
    assert (rstd == rstd[0]).all()
    g = cs.gated_norm_backward(DY, X, Z, None, None, None, rstd, group=group, wdtype=torch.float32)
    du = f64(dy) * ref.silu(f64(z))
    hh = f64(x) * np.repeat(f64(rstd[0].cpu()), group)
    for n, want in (("gbias", R * du), ("gweight", R * du * hh)):
        off = np.abs(f64(g[n].cpu()) / want - 1).max() * 2 ** 24
        assert off <= R / 304 + 64 + 10, (n, off)


def check_add(cs, R, D, kind, types, bias=True, scale=True, ds=True, wants=True):
    """One call and its gradients; ds: something else reaches s; wants: the vectors' gradients are asked for (x is not read without)."""
    (xt, rt, wt), layer = types, kind == "layer"
    r = np.random.default_rng(R + D)
    w, b, sc = vectors(r, D, wt, bias)
    sc = sc if scale else None
    x, res, dy, ds_ = (t(r.standard_normal((R, D)) * np.exp(r.standard_normal((R, 1))) + r.standard_normal((R, 1)), k) for k in (xt, rt, xt, rt))
    ds_ = ds_ if ds else None
    y, s, mean, rstd = cs.add_norm(dev(x), dev(res), dev(w), dev(b), kind=kind, alpha=0.7, scale=dev(sc), eps=EPS)
    kept = f64(s.cpu())
    # (alpha in fp32: 2^-25 of the term; the products and the sum 2^-24 each)
    close(s, f64(res) + 0.7 * f64(x) * (1 if sc is None else f64(sc)), "s", top=np.abs(f64(res)) + np.abs(f64(x)) * (1 if sc is None else np.abs(f64(sc))),
          inner=2.0 ** -22)
    wy, _, wm, wr = ref.add_norm(0 * kept, kept, f64(w), f64(b), layer, 0.0, None, EPS)
    amp = np.abs(kept).max(1, keepdims=True) * wr[:, None]
    close(y, wy, "y", top=amp * 2 + np.abs(wy).max(1, keepdims=True))
    close(rstd, wr, "rstd", top=wr, inner=INNER * (1 + (np.abs(wm) * wr) ** 2) if layer else INNER)
    if layer:
        close(mean, wm, "mean", top=np.abs(kept).max(1))
    want = ref.add_norm_backward(f64(dy), f64(ds_), f64(x), kept, f64(w), layer, 0.7, f64(sc), EPS)
    g = cs.add_norm_backward(dev(dy), dev(ds_), dev(x) if wants else None, s, dev(w), mean, rstd, alpha=0.7, scale=dev(sc), want_weight=wants,
                             want_bias=bias and wants, want_scale=scale and wants)
    assert set(g) == {"gx", "gresidual"} | ({"gweight"} if wants else set()) | ({"gbias"} if bias and wants else set()) | ({"gscale"} if scale and wants else set())
    size = wr[:, None] * np.abs(f64(dy)).max(1, keepdims=True) * np.abs(f64(w)).max() * (1 + amp)
    size = size + (np.abs(f64(ds_)).max(1, keepdims=True) if ds else 0)
    close(g["gresidual"], want["gresidual"], "gresidual", top=size)
    close(g["gx"], want["gx"], "gx", top=size)
    for n in set(g) - {"gx", "gresidual"}:
        columns(g[n], want[n], want[n + "_terms"], R, n)


def check_gated(cs, R, D, group, kind, first, types, bias=True):
    (xt, wt), layer = types, kind == "layer"
    r = np.random.default_rng(R + D + group)
    w, b = vectors(r, D, wt, bias, 2)
    x, z, dy = (t(r.standard_normal((R, D)) * np.exp(r.standard_normal((R, 1))) + m * r.standard_normal((R, 1)), xt) for m in (1, 1, 0))
    y, mean, rstd = cs.gated_norm(dev(x), dev(z), dev(w), dev(b), kind=kind, group=group, gate_first=first, eps=EPS)
    X, Z, DY, W, B = (f64(v) for v in (x, z, dy, w, b))
    wy, wm, wr = ref.gated_norm(X, Z, W, B, layer, group, first, EPS)
    gate = np.abs(ref.silu(Z))
    peak = np.abs((X * ref.silu(Z) if first else X).reshape(R, -1, group)).max(2)
    wide = lambda v: np.repeat(v, group, axis=1)  # noqa: E731
    amp = wide(peak * wr)
    out = (2 * amp * (1 + np.abs(W)) + (0 if B is None else np.abs(B))) * (1 if first else gate)
    zed = 1 + np.abs(Z).max() / 64
    close(y, wy, "y", top=out, inner=INNER * zed)
    close(rstd, wr, "rstd", top=wr, inner=INNER * zed * (1 + (np.abs(wm) * wr).max() ** 2))
    if layer:
        close(mean, wm, "mean", top=peak, inner=INNER * zed)
    want = ref.gated_norm_backward(DY, X, Z, W, B, layer, group, first, EPS)
    g = cs.gated_norm_backward(dev(dy), dev(x), dev(z), dev(w), dev(b), mean, rstd, group=group, gate_first=first, want_bias=bias)
    assert set(g) == {"gx", "gz", "gweight"} | ({"gbias"} if bias else set())
    du = np.abs(DY) * (1 if first else gate)
    dh = wide(wr * (du * np.abs(W)).reshape(R, -1, group).max(2)) * (2 + 2 * amp * wide(peak * wr))
    top = {"gx": dh * (gate if first else 1), "gz": 1.2 * (dh * np.abs(X) if first else np.abs(DY) * out / np.maximum(gate, 1e-30))}
    for n in ("gx", "gz"):
        close(g[n], want[n], n, top=top[n], inner=INNER * zed)
    for n in set(g) - {"gx", "gz"}:
        columns(g[n], want[n], want[n + "_terms"], R, n)


# Rows enough that every group of warps takes five or six one after another: each buffer of the ring is filled again, in
# both of its barrier's phases, and the last round is ragged.
@pytest.mark.parametrize("case", [
    (12163, 64, "rms", ("bf16", "fp32", "bf16")), (12163, 512, "layer", ("bf16", "bf16", "fp32")), (6083, 1000, "rms", ("fp16", "fp16", "fp16")),
    (3043, 1536, "layer", ("bf16", "fp32", "fp32")), (6083, 1536, "rms", ("bf16", "bf16", "bf16")), (1523, 4096, "rms", ("bf16", "fp32", "bf16")),
    (3043, 1536, "rms", ("fp32", "fp32", "fp32")), (12163, 128, "layer", ("fp32", "fp32", "fp32")), (6083, 333, "layer", ("bf16", "fp32", "bf16"))])
@pytest.mark.parametrize("given", [(True, True), (False, True), (True, False), (False, False)])
def test_add_norm_over_many_rows(cs, case, given):
    R, D, kind, types = case
    check_add(cs, R, D, kind, types, ds=given[0], wants=given[1])


@pytest.mark.parametrize("case", [
    (12163, 256, 64, ("bf16", "bf16")), (6083, 1536, 64, ("bf16", "fp32")), (1523, 4096, 128, ("bf16", "bf16")), (3043, 1536, 64, ("fp32", "fp32")),
    (6083, 1536, 1536, ("bf16", "fp32")), (1523, 4096, 4096, ("fp16", "fp16")), (3043, 2048, 512, ("bf16", "bf16")), (1003, 960, 80, ("bf16", "fp32")),
    (3043, 960, 96, ("fp32", "fp32")), (12163, 64, 64, ("fp16", "fp32")), (3043, 960, 24, ("bf16", "bf16")), (6083, 333, 111, ("bf16", "bf16"))])
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("first", [False, True])
def test_gated_norm_over_many_rows(cs, case, kind, first):
    R, D, group, types = case
    check_gated(cs, R, D, group, kind, first, types)


# Each vector there or not, on every path: rows in registers and rings, streamed rows, narrow and wide ones.
@pytest.mark.parametrize("types", [("bf16", "fp32", "bf16"), ("fp16", "fp16", "fp32"), ("fp32", "fp32", "fp32")])
@pytest.mark.parametrize("D", [5, 8, 333, 1001, 1536, 2048, 2056, 8200])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("scale", [False, True])
def test_add_norm_vectors(cs, D, types, bias, scale):
    check_add(cs, 41, D, "layer" if D % 16 else "rms", types, bias=bias, scale=scale)


@pytest.mark.parametrize("types", [("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32")])
@pytest.mark.parametrize("widths", [(5, 5), (64, 16), (333, 333), (960, 80), (960, 24), (1001, 143), (1536, 64), (1536, 1536), (2048, 512), (2056, 2056)])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("first", [False, True])
def test_gated_norm_vectors(cs, widths, types, bias, first):
    check_gated(cs, 41, *widths, "layer" if widths[1] % 16 else "rms", first, types, bias)


@pytest.mark.parametrize("types", [("bf16", "bf16", "bf16"), ("bf16", "fp32", "bf16"), ("fp16", "fp16", "fp16"), ("fp32", "fp32", "fp32")])
@pytest.mark.parametrize("D", [512, 333, 4096])
@pytest.mark.parametrize("scale", [False, True])
def test_residual_sum_to_the_bit(cs, D, types, scale):
    """s is the formula's operations rounded one by one to fp32, then to its type: ties of a decimal alpha go as they should."""
    xt, rt, wt = types
    gen = torch.Generator().manual_seed(12)
    x, res, sc = torch.randn(600, D, generator=gen).to(TYPES[xt]), (2 * torch.randn(600, D, generator=gen)).to(TYPES[rt]), None
    want = x.float()
    if scale:
        sc = (0.5 + 0.2 * torch.randn(D, generator=gen)).to(TYPES[wt])
        want = sc.float() * want
    want = want * torch.tensor(0.7)
    want = (res.float() + want).to(TYPES[rt])
    s = cs.add_norm(dev(x), dev(res), None, None, alpha=0.7, scale=dev(sc))[1]
    assert torch.equal(s.cpu(), want), (s.cpu() != want).sum()
