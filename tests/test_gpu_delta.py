"""GPU kernels of the gated delta rule against the 64-bit recurrence.

Tolerances.  An output of a 16-bit type is off by at most half a step of that
type relative to its value; before that rounding, and for float32 outputs, a
value is a chain of three sums of at most 128, 64 and 64 products (the answer
of the state, the triangular solve, the write), each product and addition
correct to 2^-24 relative, so (128 + 64 + 64) 2^-24 = 1.5e-5 of the largest
value bounds it; INNER = 2e-5 is used for every tensor, of its largest value.
dL/dg is a difference of inner products with the state, so its bar is INNER of
the largest sum of the terms' sizes.  A value past its type's range is infinite."""

import numpy as np
import pytest
import torch

import delta_reference as ref

pytestmark = pytest.mark.gpu

INNER = 2e-5
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


def make(seed, B, T, H, KH, N, P, dtype="fp32", state=False, ragged=None, rate=1.0):
    """CPU tensors of one call, rounded to their type."""
    r = np.random.default_rng(seed)

    def t(x, dt=torch.float32):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dt)

    def unit(*s):
        x = r.standard_normal(s)
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    dt = TYPES[dtype]
    d = {"q": t(unit(B, T, KH, N), dt), "k": t(unit(B, T, KH, N), dt), "v": t(r.standard_normal((B, T, H, P)), dt),
         "g": t(-rate * r.uniform(0, 1, (B, T, H)) * np.exp(r.uniform(-5, 0, H))), "beta": t(r.uniform(0, 1, (B, T, H)))}
    opt = {"h0": t(r.standard_normal((B, H, N, P))) if state else None,
           "lens": torch.tensor(ragged, dtype=torch.int32) if ragged is not None else None}
    back = {"do": t(r.standard_normal((B, T, H, P)), dt), "dh_final": t(r.standard_normal((B, H, N, P))) if state else None}
    return d, opt, back


def on(d, dev="cuda"):
    return {k: None if v is None else v.to(dev) for k, v in d.items()}


def np64(d):
    return {k: None if v is None else v.double().numpy() if v.is_floating_point() else v.numpy() for k, v in d.items()}


def close(got, want, what, scale=None, inner=INNER):
    dt = got.dtype
    half = 0.0 if dt == torch.float32 else torch.finfo(dt).eps / 2
    got = got.detach().cpu().double().numpy()
    top = float(np.max(np.abs(want))) if scale is None else float(np.max(scale))
    bar = half * np.abs(want) + inner * max(top, 1e-30)
    over = np.abs(want) - bar > torch.finfo(dt).max  # rounds to infinity in this type
    assert (got[over] == np.sign(want[over]) * np.inf).all(), f"{what}: values past the type's range"
    near = np.abs(want) + bar > torch.finfo(dt).max  # may round to it
    with np.errstate(invalid="ignore"):
        err = np.where(over | (near & np.isinf(got)), 0.0, np.abs(got - want))
    bad = ~(err <= bar)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / bar):.3g} of the bar (top {top:.3g})"


def check_forward(cs, d, opt, scale=0.25):
    o, h = cs.delta_forward(**on(d), **on(opt), scale=scale)
    n, m = np64(d), np64(opt)
    want_o, want_h, _ = ref.delta_forward(*(n[k] for k in ("q", "k", "v", "g", "beta")), scale, m["h0"], m["lens"])
    close(o, want_o, "o")
    close(h, want_h, "h_final")


def check_backward(cs, d, opt, back, scale=0.25):
    r = cs.delta_backward(**on(d), **on(back), **on(opt), scale=scale)
    n, m, b = np64(d), np64(opt), np64(back)
    w = ref.delta_backward(*(n[k] for k in ("q", "k", "v", "g", "beta")), scale, b["do"], m["h0"], b["dh_final"], m["lens"])
    for name in ("gq", "gk", "gv", "gbeta", "gh0"):
        close(r[name], w[name], name)
    close(r["gg"], w["gg"], "gg", scale=w["gg_terms"])


SHAPES = [  # B, T, H, KH, N, P
    (1, 1, 1, 1, 16, 16), (2, 1, 2, 1, 64, 64), (1, 2, 3, 3, 128, 128), (1, 63, 2, 2, 64, 64), (2, 64, 2, 1, 64, 64),
    (1, 65, 4, 2, 128, 64), (2, 129, 2, 2, 64, 128), (1, 200, 3, 1, 128, 128), (1, 130, 2, 2, 96, 80),
    (1, 100, 2, 2, 32, 48), (1, 70, 1, 1, 48, 112), (3, 257, 2, 1, 16, 32)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(cs, shape, dtype):
    d, opt, _ = make(sum(shape), *shape, dtype=dtype, state=shape[1] % 2 == 1)
    check_forward(cs, d, opt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(cs, shape, dtype):
    d, opt, back = make(sum(shape) + 1, *shape, dtype=dtype, state=shape[1] % 2 == 1)
    check_backward(cs, d, opt, back)


# State widths that end inside a warp's 32 rows, on both sides of the head count
# at which the fp32 scan takes narrower slices (batch x heads x headdim / 16 = 76).
UNEVEN = [(1, 200, 2, 1, 80, 64), (2, 130, 3, 3, 112, 48), (1, 64, 1, 1, 112, 128), (2, 150, 10, 5, 80, 64),
          (1, 129, 20, 20, 112, 80)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("shape", UNEVEN)
def test_uneven_state_widths(cs, shape, ragged, dtype):
    lens = [shape[1] - 70, 65][:shape[0]] if ragged else None
    d, opt, back = make(sum(shape) + 3, *shape, dtype=dtype, state=True, ragged=lens)
    check_forward(cs, d, opt)
    check_backward(cs, d, opt, back)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128), (48, 80)])
def test_ragged_rows(cs, NP, dtype):
    """Rows of 0, 1, a chunk, a chunk and one, and all tokens (a length past
    the end counts as all, a negative one as none); what lies behind is NaN and
    must not be read, and outputs and gradients there are zero."""
    lens = [0, 1, 64, 65, 150, 1000, -3]
    d, opt, back = make(5, len(lens), 150, 4, 2, *NP, dtype=dtype, state=True, ragged=lens)
    for b, n in enumerate(lens):
        n = min(max(n, 0), 150)
        for t in (d["q"], d["k"], d["v"], d["g"], d["beta"], back["do"]):
            t[b, n:] = float("nan")
    o, h = cs.delta_forward(**on(d), **on(opt))
    r = cs.delta_backward(**on(d), **on(back), **on(opt))
    clean = {k: torch.nan_to_num(v) for k, v in d.items()}
    back = {k: torch.nan_to_num(v) for k, v in back.items()}
    n, m, w = np64(clean), np64(opt), np64(back)
    args = [n[k] for k in ("q", "k", "v", "g", "beta")]
    want_o, want_h, _ = ref.delta_forward(*args, NP[0] ** -0.5, m["h0"], m["lens"])
    close(o, want_o, "o")
    close(h, want_h, "h_final")
    want = ref.delta_backward(*args, NP[0] ** -0.5, w["do"], m["h0"], w["dh_final"], m["lens"])
    for name in ("gq", "gk", "gv", "gbeta", "gh0"):
        close(r[name], want[name], name)
    close(r["gg"], want["gg"], "gg", scale=want["gg_terms"])
    for b, ln in enumerate(lens):
        ln = min(max(ln, 0), 150)
        for t in (o, r["gq"], r["gk"], r["gv"], r["gg"], r["gbeta"]):
            assert (t[b, ln:] == 0).all()
    assert torch.equal(h[0].cpu(), opt["h0"][0]) and torch.equal(r["gh0"][0].cpu(), back["dh_final"][0])


@pytest.mark.parametrize("NP", [(64, 64), (128, 128)])
def test_gates_at_their_ends(cs, NP):
    """beta 0 (nothing written), beta 1, no decay at all, decays that underflow
    inside a chunk, a full reset (-inf), and all of them in one sequence."""
    d, opt, back = make(6, 1, 140, 6, 6, *NP, dtype="bf16", state=True)
    d["beta"][:, :, 0] = 0.0
    d["beta"][:, :, 1] = 1.0
    d["g"][:, :, 1] = 0.0
    d["g"][:, :, 2] = -30.0
    d["g"][:, :, 3] = 0.0
    d["g"][:, 70, 3] = -float("inf")
    d["g"][:, ::5, 4] = -200.0
    d["beta"][:, 1::2, 5] = 0.0
    check_forward(cs, d, opt)
    check_backward(cs, d, opt, back)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_magnitudes(cs, dtype):
    """Keys, values and states of very different sizes, in one head and between
    heads: the bar is of each head's largest value."""
    d, opt, back = make(7, 1, 190, 4, 4, 64, 64, dtype=dtype, state=True)
    for h, (sv, ss) in enumerate([(1e-3, 1e3), (1e3, 1e-3), (1.0, 0.0), (1e-2, 1e2)]):
        d["v"][:, :, h] = (d["v"][:, :, h].float() * sv).to(d["v"].dtype)
        opt["h0"][:, h] *= ss
    d["q"][:, :, 1] = (d["q"][:, :, 1].float() * 16).to(d["q"].dtype)
    o, hf = cs.delta_forward(**on(d), **on(opt), scale=1.0)
    r = cs.delta_backward(**on(d), **on(back), **on(opt), scale=1.0)
    n, m, b = np64(d), np64(opt), np64(back)
    args = [n[k] for k in ("q", "k", "v", "g", "beta")]
    want_o, want_h, _ = ref.delta_forward(*args, 1.0, m["h0"])
    w = ref.delta_backward(*args, 1.0, b["do"], m["h0"], b["dh_final"])
    for h in range(4):
        close(o[:, :, h], want_o[:, :, h], f"o {h}")
        close(hf[:, h], want_h[:, h], f"h {h}")
        for name in ("gv", "gbeta"):
            close(r[name][:, :, h], w[name][:, :, h], f"{name} {h}")
        for name in ("gq", "gk"):
            close(r[name][:, :, h], w[name][:, :, h], f"{name} {h}")
        close(r["gg"][:, :, h], w["gg"][:, :, h], f"gg {h}", scale=w["gg_terms"][:, :, h])


def test_equal_keys(cs):
    """All keys the same unit vector at beta 1 and no decay: the triangular
    system is as full as it gets, and every token replaces the stored value."""
    d, opt, _ = make(8, 1, 200, 1, 1, 64, 64)
    d["k"][:] = d["k"][:, :1]
    d["k"] /= d["k"].norm(dim=-1, keepdim=True)
    d["q"].copy_(d["k"])
    d["g"].zero_()
    d["beta"].fill_(1.0)
    o, h = cs.delta_forward(**on(d), scale=1.0)
    close(o, d["v"].double().numpy(), "o")


def test_split_sequence_and_steps_agree(cs):
    """A sequence in one call, in two calls joined by the state, and token by
    token through delta_step."""
    d, opt, _ = make(9, 2, 150, 4, 2, 128, 64, state=True)
    g, h0 = on(d), opt["h0"].cuda()
    o, h = cs.delta_forward(**g, h0=h0)
    state = h0.clone()
    first = {k: v[:, :77].contiguous() for k, v in g.items()}
    second = {k: v[:, 77:].contiguous() for k, v in g.items()}
    o1, _ = cs.delta_forward(**first, h0=state, h_final=state)  # the state in place
    o2, _ = cs.delta_forward(**second, h0=state, h_final=state)
    want = o.double().cpu().numpy()
    close(torch.cat([o1, o2], 1), want, "two calls", inner=2 * INNER)
    close(state, h.double().cpu().numpy(), "state of two calls", inner=2 * INNER)
    state = h0.clone()
    steps = torch.stack([cs.delta_step(state, *(g[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")))
                         for t in range(150)], 1)
    close(steps, want, "steps", inner=2 * INNER)
    close(state, h.double().cpu().numpy(), "state of the steps", inner=2 * INNER)


def test_gradients_match_differences(cs):
    """<gradient, direction> against a central difference of the GPU's own
    forward in fp32: step 1e-2 leaves the third-order term (about 1e-4) and the
    forward's 1e-5 over the step."""
    d, opt, back = make(10, 1, 100, 2, 1, 64, 64, state=True)
    r = cs.delta_backward(**on(d), **on(back), **on(opt), scale=0.5)
    do, dh = back["do"].double(), back["dh_final"].double()
    gen = torch.Generator().manual_seed(3)

    def loss(x, h0):
        o, h = cs.delta_forward(**on(x), h0=h0.cuda(), scale=0.5)
        return float((o.cpu().double() * do).sum() + (h.cpu().double() * dh).sum())

    for name in ("q", "k", "v", "g", "beta", "h0"):
        src = opt["h0"] if name == "h0" else d[name]
        way = torch.randn(src.shape, generator=gen)
        way *= 1e-2 / way.abs().max()
        vals = []
        for s in (1.0, -1.0):
            x = dict(d)
            h0 = opt["h0"]
            if name == "h0":
                h0 = h0 + s * way
            else:
                x[name] = x[name] + s * way
            vals.append(loss(x, h0))
        diff = (vals[0] - vals[1]) / 2
        got = float((r["g" + name].cpu().double() * way.double()).sum())
        size = float((r["g" + name].cpu().double().abs() * way.double().abs()).sum())
        assert abs(diff - got) < 2e-3 * size, (name, diff, got, size)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (3, 4, 2, 64, 64), (2, 8, 2, 128, 128), (5, 3, 3, 96, 80),
                                   (2, 2, 1, 112, 48), (37, 12, 12, 64, 64)])
def test_step(cs, shape, dtype):
    B, H, KH, N, P = shape
    d, opt, _ = make(sum(shape) + 2, B, 1, H, KH, N, P, dtype=dtype, state=True)
    one = {k: v[:, 0].contiguous() for k, v in d.items()}
    h = opt["h0"].cuda()
    o = cs.delta_step(h, **on(one), scale=0.3)
    n = np64(one)
    rep = lambda x: np.repeat(x, H // KH, axis=1)  # noqa: E731
    S, want, _ = ref.token(opt["h0"].double().numpy(), rep(n["q"]), rep(n["k"]), n["v"], n["g"], n["beta"])
    close(o, 0.3 * want, "o")
    close(h, S, "h")


def test_step_slots(cs):
    """Rows name their states in any order; a slot outside the pool writes
    nothing and answers zero; states no row names are left alone."""
    B, H, N, P, pool = 6, 4, 64, 80, 9
    d, _, _ = make(11, B, 1, H, 2, N, P, dtype="bf16")
    one = {k: v[:, 0].contiguous() for k, v in d.items()}
    h0 = torch.randn(pool, H, N, P, generator=torch.Generator().manual_seed(1))
    slots = [7, -1, 0, 9, 3, 1 << 30]
    h = h0.cuda()
    o = cs.delta_step(h, **on(one), slots=torch.tensor(slots, dtype=torch.int32).cuda())
    n = np64(one)
    want_h = h0.double().numpy()
    for b, s in enumerate(slots):
        if not 0 <= s < pool:
            assert (o[b] == 0).all()
            continue
        S, ob, _ = ref.token(h0[s].double().numpy(), np.repeat(n["q"][b], 2, 0), np.repeat(n["k"][b], 2, 0), n["v"][b],
                             n["g"][b], n["beta"][b])
        close(o[b], N ** -0.5 * ob, "o")
        want_h[s] = S
    close(h, want_h, "h")
    for s in (1, 2, 4, 5, 6, 8):
        assert torch.equal(h[s].cpu(), h0[s])


def test_step_offsets_past_32_bits(cs):
    """A pool of states of more than 2^31 elements: the last one is the one used."""
    N = P = 128
    pool = (1 << 31) // (N * P) + 3
    d, opt, _ = make(12, 1, 1, 1, 1, N, P, dtype="bf16", state=True)
    one = {k: v[:, 0].contiguous() for k, v in d.items()}
    h = torch.empty(pool, 1, N, P, device="cuda")
    h[-1] = opt["h0"][0].cuda()
    o = cs.delta_step(h, **on(one), slots=torch.tensor([pool - 1], dtype=torch.int32).cuda(), scale=1.0)
    n = np64(one)
    S, want, _ = ref.token(opt["h0"].double().numpy(), n["q"], n["k"], n["v"], n["g"], n["beta"])
    close(o, want, "o")
    close(h[-1:], S, "h")


def test_other_stream_and_graph(cs):
    """On a stream of the caller's, and captured into a graph whose replays
    redo the work on new contents of the same buffers."""
    d, opt, back = make(13, 2, 130, 4, 2, 64, 64, dtype="bf16", state=True)
    g, o_, b_ = on(d), on(opt), on(back)
    want = cs.delta_forward(**g, **o_) + tuple(cs.delta_backward(**g, **b_, **o_).values())
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = cs.delta_forward(**g, **o_, stream=s) + tuple(cs.delta_backward(**g, **b_, **o_, stream=s).values())
    s.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cs.delta_forward(**g, **o_) + tuple(cs.delta_backward(**g, **b_, **o_).values())
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    d2, _, _ = make(14, 2, 130, 4, 2, 64, 64, dtype="bf16", state=True)
    for n in g:
        g[n].copy_(d2[n])
    graph.replay()
    want = cs.delta_forward(**g, **o_) + tuple(cs.delta_backward(**g, **b_, **o_).values())
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)


def test_same_call_same_bits(cs):
    d, opt, back = make(15, 2, 333, 8, 2, 128, 128, dtype="bf16", state=True)
    runs = [cs.delta_forward(**on(d), **on(opt)) + tuple(cs.delta_backward(**on(d), **on(back), **on(opt)).values())
            for _ in range(2)]
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    assert cs.device_status() == 0


def test_given_buffers_and_workspace(cs):
    d, opt, back = make(16, 1, 90, 2, 2, 64, 64, dtype="fp16", state=True)
    g, o_, b_ = on(d), on(opt), on(back)
    ws = torch.empty(cs.delta_workspace_bytes(1, 90, 2, 2, 64, 64, torch.float16), dtype=torch.uint8, device="cuda")
    o = torch.empty_like(g["v"])
    out, h = cs.delta_forward(**g, **o_, o=o, want_state=False, workspace=ws)
    assert out is o and h is None
    assert torch.equal(o, cs.delta_forward(**g, **o_)[0])
    need = cs.delta_backward_workspace_bytes(1, 90, 2, 2, 64, 64, torch.float16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    r = cs.delta_backward(**g, **b_, **o_, workspace=ws)
    dh = b_["dh_final"].clone()  # gh0 over dh_final
    r2 = cs.delta_backward(**g, do=b_["do"], dh_final=dh, **o_, grads={"gh0": dh}, workspace=ws)
    for n in r:
        assert torch.equal(r[n], r2[n])
    with pytest.raises(cs.CssdError):
        cs.delta_backward(**g, **b_, **o_, workspace=ws[:-16])
    with pytest.raises(cs.CssdError):
        cs.delta_forward(g["q"][..., :8].contiguous(), g["k"][..., :8].contiguous(), g["v"], g["g"], g["beta"])


def test_long_sequence(cs):
    """2000 tokens of slow decays, 16-bit, sampled against the recurrence."""
    d, opt, _ = make(17, 1, 2000, 3, 1, 128, 128, dtype="bf16", state=True, rate=0.02)
    check_forward(cs, d, opt)


@pytest.mark.parametrize("shape", [(6, 2085, 2, 1, 64, 64), (6, 2048, 1, 1, 128, 128), (6, 3300, 2, 2, 48, 80)])
def test_long_ragged_rows(cs, shape):
    """Few heads of many chunks: rows that end in the first chunks, at and just
    past the middle, and at the last token; the state is written over h0."""
    T = shape[1]
    lens = [0, 1, 700, 1024, 1025, T]
    d, opt, _ = make(18, *shape, dtype="bf16", state=True, ragged=lens, rate=0.05)
    for b, n in enumerate(lens):
        for t in d.values():
            t[b, n:] = float("nan")
    n, m = np64({k: torch.nan_to_num(v) for k, v in d.items()}), np64(opt)
    want_o, want_h, _ = ref.delta_forward(*(n[k] for k in ("q", "k", "v", "g", "beta")), 0.25, m["h0"], m["lens"])
    g, o_ = on(d), on(opt)
    o, h = cs.delta_forward(**g, h0=o_["h0"], lens=o_["lens"], h_final=o_["h0"], scale=0.25)
    assert h is o_["h0"]
    close(o, want_o, "o")
    close(h, want_h, "h_final")
    for b, ln in enumerate(lens):
        assert (o[b, ln:] == 0).all()
    assert torch.equal(h[0].cpu(), opt["h0"][0])
    alone, none = cs.delta_forward(**g, **on(opt), scale=0.25, want_state=False)
    assert none is None and torch.equal(alone, o)


def test_long_sequence_stream_and_graph(cs):
    """The same over several launches: another stream, back to back calls on
    one workspace, a captured graph replayed twice on other contents."""
    shape = (1, 4200, 3, 3, 64, 64)
    d, opt, _ = make(19, *shape, dtype="fp16", state=True, rate=0.05)
    d2, opt2, _ = make(20, *shape, dtype="fp16", state=True, rate=0.05)
    ws = torch.empty(cs.delta_workspace_bytes(*shape, torch.float16), dtype=torch.uint8, device="cuda")
    g, o_, g2, o2 = on(d), on(opt), on(d2), on(opt2)
    check_forward(cs, d, opt)
    want, want2 = cs.delta_forward(**g, **o_), cs.delta_forward(**g2, **o2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = [cs.delta_forward(**a, **b, workspace=ws, stream=s) for a, b in ((g, o_), (g2, o2)) * 3]
    s.synchronize()
    for i, (o, h) in enumerate(got):
        w = (want, want2)[i % 2]
        assert torch.equal(o, w[0]) and torch.equal(h, w[1]), i
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, h = cs.delta_forward(**g, **o_)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(h, want[1])
    for a, b in ((g, g2), (o_, o2)):
        for n in a:
            if a[n] is not None:
                a[n].copy_(b[n])
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want2[0]) and torch.equal(h, want2[1])
    assert cs.device_status() == 0


@pytest.mark.parametrize("shape", [(10, 700, 17, 17, 64, 64), (3, 650, 90, 90, 32, 32), (2, 333, 100, 50, 128, 128)])
def test_more_heads_than_sms(cs, shape):
    """More chains than SMs, whose scans are cut into pieces: rows that end in
    each piece, with a state and gradients of it, twice the same bits."""
    B, T = shape[:2]
    lens = [0, 1, T // 3, T // 2 + 1, T - 1, T, 64, 65, 128, 300][-B:]
    d, opt, back = make(21, *shape, dtype="bf16", state=True, ragged=lens, rate=0.2)
    check_forward(cs, d, opt)
    check_backward(cs, d, opt, back)
    runs = [cs.delta_forward(**on(d), **on(opt)) + tuple(cs.delta_backward(**on(d), **on(back), **on(opt)).values())
            for _ in range(2)]
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    assert cs.device_status() == 0


def unit(x):
    return x / np.linalg.norm(x, axis=-1, keepdims=True)


def repeats(d):
    """The largest sum of sizes in a row of (I + A)^-1 over the chunks: how often
    an error of R counts in U (key heads not shared, no decay)."""
    n = np64(d)
    most = 1.0
    for b in range(n["k"].shape[0]):
        for h in range(n["k"].shape[2]):
            for c in range(0, n["k"].shape[1], 64):
                k, beta = n["k"][b, c:c + 64, h], n["beta"][b, c:c + 64, h]
                t = np.linalg.inv(np.eye(len(k)) + np.tril(beta[:, None] * (k @ k.T), -1))
                most = max(most, np.abs(t).sum(1).max())
    return most


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("beta,alike", [((1.0, 1.9), 0.0), ((2.0, 2.0), 0.0), ((0.9, 1.0), 0.9), ((1.0, 1.9), 0.9)])
@pytest.mark.parametrize("NP", [(64, 64), (16, 32), (128, 128)])
def test_strong_writes(cs, NP, beta, alike, dtype):
    """Writes that overshoot (beta above 1) and keys that are much alike, without
    decay: the triangular system sums terms larger than its solution, so the bar
    counts them."""
    N, P = NP
    d, opt, back = make(22, 1, 330, 2, 2, N, P, state=True)
    r = np.random.default_rng(23)
    k = unit((1 - alike) * r.standard_normal(d["k"].shape) + 3 * alike * r.standard_normal((1, 1, 2, N)))
    d["k"] = torch.from_numpy(k).float()
    for n in ("q", "k", "v"):
        d[n] = d[n].to(TYPES[dtype])
    back["do"] = back["do"].to(TYPES[dtype])
    d["g"].zero_()
    d["beta"] = torch.from_numpy(r.uniform(*beta, d["beta"].shape)).float()
    inner = INNER * repeats(d)
    o, h = cs.delta_forward(**on(d), **on(opt), scale=0.25)
    g = cs.delta_backward(**on(d), **on(back), **on(opt), scale=0.25)
    n, m, b = np64(d), np64(opt), np64(back)
    args = [n[x] for x in ("q", "k", "v", "g", "beta")]
    want_o, want_h, _ = ref.delta_forward(*args, 0.25, m["h0"])
    w = ref.delta_backward(*args, 0.25, b["do"], m["h0"], b["dh_final"])
    close(o, want_o, "o", inner=inner)
    close(h, want_h, "h_final", inner=inner)
    for name in ("gq", "gk", "gv", "gbeta", "gh0"):
        close(g[name], w[name], name, inner=inner)
    close(g["gg"], w["gg"], "gg", scale=w["gg_terms"], inner=inner)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("where", ["v", "do"])
@pytest.mark.parametrize("size", [1e3, 1e4])
@pytest.mark.parametrize("beta,known", [((0.0, 1.0), False), ((1.0, 1.9), False), ((0.9, 1.0), True)])
@pytest.mark.parametrize("NP", [(16, 32), (64, 64), (128, 128)])
def test_one_large_token(cs, NP, beta, known, size, where, dtype):
    """One value, or one output's gradient, thousands of times the others, which
    the state has forgotten by the end (few keys, no decay): the float32 results
    against what the fp32 kernels make of the same 16-bit inputs.  An operand of
    the 16-bit kernels is held to 2^-24 of its row's largest value while its scale
    is at most 2^16 off, to 2^-22 at 2^18, 4 times an fp32 rounding, and a
    product has two such operands at most: 8 times the fp32 kernels' error, and
    the 1e-6 that every result may be off by."""
    N, P = NP
    T, H = 512, 2
    r = np.random.default_rng(24)
    k, q, v, do = unit(r.standard_normal((1, T, H, N))), unit(r.standard_normal((1, T, H, N))), \
        r.standard_normal((1, T, H, P)), r.standard_normal((1, T, H, P))
    if known:  # the state comes to answer every value
        v = np.einsum("bthn,hnp->bthp", k, r.standard_normal((H, N, P)))
    (v if where == "v" else do)[:, 266] *= size
    q, k, v, do = (torch.from_numpy(x).float().to(TYPES[dtype]) for x in (q, k, v, do))
    g, b = torch.zeros(1, T, H), torch.from_numpy(r.uniform(*beta, (1, T, H))).float()
    n = [x.double().numpy() for x in (q, k, v, g, b)]
    want = {"h": ref.delta_forward(*n, 1.0)[1], **ref.delta_backward(*n, 1.0, do.double().numpy())}
    got, plain = [], []
    for to, into in ((lambda x: x.cuda(), got), (lambda x: x.float().cuda(), plain)):
        a = [to(q), to(k), to(v), g.cuda(), b.cuda()]
        back = cs.delta_backward(*a, to(do), scale=1.0)
        into += [cs.delta_forward(*a, scale=1.0)[1], back["gh0"], back["gbeta"]]
    for x, y, name in zip(got, plain, ("h", "gh0", "gbeta")):
        top = np.abs(want[name]).max()
        err, fp32 = (np.abs(t.cpu().double().numpy() - want[name]).max() / top for t in (x, y))
        assert err <= 8 * fp32 + 1e-6, f"{name}: {err:.2g} of its largest value, the fp32 kernels {fp32:.2g}"
