"""GPU kernels of linear attention with a decay for each head against the
64-bit recurrence.

Tolerances.  An output of a 16-bit type is off by at most half a step of that
type relative to its value.  Before that rounding every result is a sum of
products (with the sizes of those products, the "terms", summed alike by the
reference), in which
  - scores and states are held as two bfloat16 planes for 16-bit results: what
    two roundings leave is 2^-9 2^-9 = 2^-18 of each term (three planes, 2^-27,
    for float32 ones);
  - a decay is up to three exponentials of sums right to 2^-24: 2^-21 of each
    term;
  - a matrix instruction adds 16 products to its sum and may drop what lies
    below the sum's last bit, 2^-23 of the terms: a chunk has at most 8 of them
    for a score, 8 for the state and 8 for the tokens, six plane pairs each, of
    which one has terms larger than 2^-8 of the sum, and a long row adds a
    rounding (2^-24) a chunk: 32 2^-23 + 5 2^-24 + ... < 2^-17.9.
Together below 2^-18 + 2^-21 + 2^-17.9 < 2^-17; INNER = 2^-17 of the terms.  A
value past its type's range is infinite."""

import block_reference as ref
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

INNER = 2.0 ** -17
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


def make(seed, B, T, H, KH, N, P, dtype="fp32", state=False, ragged=None, rate=1.0, head=False):
    """CPU tensors of one call, rounded to their type."""
    r = np.random.default_rng(seed)

    def t(x, dt=torch.float32):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).to(dt)

    dt = TYPES[dtype]
    rates = np.exp(r.uniform(-5, 0, H))
    d = {"q": t(r.standard_normal((B, T, KH, N)), dt), "k": t(r.standard_normal((B, T, KH, N)) * N ** -0.5, dt),
         "v": t(r.standard_normal((B, T, H, P)), dt), "g": t(-rate * (rates if head else r.uniform(0, 1, (B, T, H)) * rates))}
    opt = {"h0": t(r.standard_normal((B, H, N, P))) if state else None,
           "lens": torch.tensor(ragged, dtype=torch.int32) if ragged is not None else None}
    back = {"do": t(r.standard_normal((B, T, H, P)), dt), "dh_final": t(r.standard_normal((B, H, N, P))) if state else None}
    return d, opt, back


def on(d, dev="cuda"):
    return {k: None if v is None else v.to(dev) for k, v in d.items()}


def np64(d):
    return {k: None if v is None else v.double().numpy() if v.is_floating_point() else v.numpy() for k, v in d.items()}


def close(got, want, terms, what, inner=INNER):
    half = 0.0 if got.dtype == torch.float32 else torch.finfo(got.dtype).eps / 2
    tiny = 0.0 if got.dtype != torch.float16 else 2.0 ** -25  # half a step of its smallest numbers
    most = torch.finfo(got.dtype).max
    got = got.detach().cpu().double().numpy()
    bar = half * np.abs(want) + inner * terms + tiny + 1e-37
    over = np.abs(want) - bar > most  # rounds to infinity in this type
    assert (got[over] == np.sign(want[over]) * np.inf).all(), f"{what}: values past the type's range"
    may = (np.abs(want) + bar > most) & np.isinf(got)  # may round to it
    with np.errstate(invalid="ignore"):
        err = np.where(over | may, 0.0, np.abs(got - want))
    bad = ~(err <= bar)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(err / bar):.3g} of the bar"


def check_forward(cs, d, opt, scale=0.25, inner=INNER, **kw):
    o, h = cs.linattn_forward(**on(d), **on(opt), scale=scale, **kw)
    n, m = np64(d), np64(opt)
    wo, wh, w = ref.linattn_forward(n["q"], n["k"], n["v"], n["g"], scale, m["h0"], m["lens"])
    close(o, wo, w["o_terms"], "o", inner)
    close(h, wh, w["h_terms"], "h_final", inner)
    return o, h


def check_backward(cs, d, opt, back, scale=0.25, inner=INNER, **kw):
    r = cs.linattn_backward(**on(d), **on(back), **on(opt), scale=scale, **kw)
    n, m, b = np64(d), np64(opt), np64(back)
    w = ref.linattn_backward(n["q"], n["k"], n["v"], n["g"], scale, b["do"], m["h0"], b["dh_final"], m["lens"])
    for name in ("gq", "gk", "gv", "gh0", "gg"):
        close(r[name], w[name], w[name + "_terms"], name, inner)
    return r


SHAPES = [  # B, T, H, KH, N, P
    (1, 1, 1, 1, 16, 16), (2, 1, 2, 1, 64, 64), (1, 2, 3, 3, 128, 128), (1, 31, 2, 2, 64, 64), (2, 64, 2, 1, 64, 64),
    (1, 65, 4, 2, 128, 64), (2, 129, 2, 2, 64, 128), (1, 200, 3, 1, 128, 128), (1, 130, 2, 2, 96, 80), (1, 128, 2, 1, 80, 96),
    (1, 100, 2, 2, 32, 48), (1, 70, 1, 1, 48, 112), (3, 257, 2, 1, 16, 32), (1, 300, 2, 2, 64, 64), (1, 33, 2, 1, 112, 16)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward(cs, shape, dtype):
    d, opt, _ = make(sum(shape), *shape, dtype=dtype, state=shape[1] % 2 == 1, head=shape[2] % 2 == 1)
    check_forward(cs, d, opt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", SHAPES)
def test_backward(cs, shape, dtype):
    d, opt, back = make(sum(shape) + 1, *shape, dtype=dtype, state=shape[1] % 2 == 1, head=shape[2] % 2 == 1)
    check_backward(cs, d, opt, back)


# Enough heads that a row's chunks are walked by one block, and fewer heads than chunks.
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(8, 270, 40, 20, 16, 32), (5, 140, 40, 40, 32, 80), (1, 1500, 1, 1, 64, 64)])
@pytest.mark.parametrize("state", [False, True])
def test_walks_and_segments(cs, shape, state, dtype):
    B, T = shape[:2]
    lens = [T - 61 * b for b in range(B)] if B > 1 else None
    lens = None if lens is None else [max(0, x) for x in lens]
    d, opt, back = make(sum(shape) + 2, *shape, dtype=dtype, state=state, ragged=lens, head=state)
    check_forward(cs, d, opt)
    check_backward(cs, d, opt, back)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128), (48, 80)])
def test_ragged_rows(cs, NP, dtype):
    """Rows of 0, 1, a chunk, a chunk and one, and all tokens (a length past
    the end counts as all, a negative one as none); what lies behind is NaN and
    must not be read, and outputs and gradients there are zero."""
    lens = [0, 1, 64, 65, 128, 129, 150, 1000, -3]
    d, opt, back = make(5, len(lens), 150, 4, 2, *NP, dtype=dtype, state=True, ragged=lens)
    clean, cback = {k: v.clone() for k, v in d.items()}, {k: v.clone() for k, v in back.items()}
    for b, n in enumerate(lens):
        n = min(max(n, 0), 150)
        for t, c in ((d["q"], clean["q"]), (d["k"], clean["k"]), (d["v"], clean["v"]), (d["g"], clean["g"]), (back["do"], cback["do"])):
            t[b, n:] = float("nan")
            c[b, n:] = 0
    o, h = cs.linattn_forward(**on(d), **on(opt))
    r = cs.linattn_backward(**on(d), **on(back), **on(opt))
    n, m, w = np64(clean), np64(opt), np64(cback)
    args = [n[k] for k in ("q", "k", "v", "g")]
    wo, wh, wt = ref.linattn_forward(*args, NP[0] ** -0.5, m["h0"], m["lens"])
    close(o, wo, wt["o_terms"], "o")
    close(h, wh, wt["h_terms"], "h_final")
    want = ref.linattn_backward(*args, NP[0] ** -0.5, w["do"], m["h0"], w["dh_final"], m["lens"])
    for name in ("gq", "gk", "gv", "gh0", "gg"):
        close(r[name], want[name], want[name + "_terms"], name)
    for b, ln in enumerate(lens):
        ln = min(max(ln, 0), 150)
        for t in (o, r["gq"], r["gk"], r["gv"], r["gg"]):
            assert (t[b, ln:] == 0).all()
    assert torch.equal(h[0].cpu(), opt["h0"][0]) and torch.equal(r["gh0"][0].cpu(), back["dh_final"][0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128)])
def test_decays_at_their_ends(cs, NP, dtype):
    """No decay at all, decays that underflow inside a chunk, full resets (-inf)
    alone and side by side, growth, and all of them in one sequence."""
    d, opt, back = make(6, 1, 290, 6, 6, *NP, dtype=dtype, state=True)
    d["g"][:, :, 0] = 0.0
    d["g"][:, :, 1] = -30.0
    d["g"][:, :, 2] = 0.0
    d["g"][:, 70, 2] = -float("inf")
    d["g"][:, 128:131, 2] = -float("inf")
    d["g"][:, ::5, 3] = -200.0
    d["g"][:, :, 4] = 0.01
    check_forward(cs, d, opt)
    check_backward(cs, d, opt, back)


def test_one_decay_a_head_at_its_ends(cs):
    d, opt, back = make(16, 2, 200, 4, 4, 64, 64, dtype="bf16", state=True, head=True)
    d["g"][:] = torch.tensor([0.0, -1e-6, -40.0, -float("inf")])
    check_forward(cs, d, opt)
    check_backward(cs, d, opt, back)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_magnitudes(cs, dtype):
    """Values, keys and states of very different sizes, between heads and tokens."""
    d, opt, back = make(7, 1, 190, 4, 4, 64, 64, dtype=dtype, state=True)
    for h, (sv, ss) in enumerate([(1e-3, 1e3), (1e3, 1e-3), (1.0, 0.0), (1e-2, 1e2)]):
        d["v"][:, :, h] = (d["v"][:, :, h].float() * sv).to(d["v"].dtype)
        opt["h0"][:, h] *= ss
    d["q"][:, :, 1] = (d["q"][:, :, 1].float() * 16).to(d["q"].dtype)
    d["v"][:, 90] = (d["v"][:, 90].float() * 16).to(d["v"].dtype)
    check_forward(cs, d, opt, scale=1.0)
    check_backward(cs, d, opt, back, scale=1.0)


def test_large_values_stay_in_range(cs):
    """float16 tensors near the ends of their range: the planes have float32's exponents."""
    d, opt, _ = make(17, 1, 140, 2, 2, 64, 64, dtype="fp16", state=False)
    d["v"] = (d["v"].float() * 10000).clamp(-60000, 60000).half()
    d["k"] = (d["k"].float() * 1000).half()
    check_forward(cs, d, opt, scale=1e-6)


def test_split_sequence_and_steps_agree(cs):
    """A sequence in one call, in two calls joined by the state in place, and
    token by token through linattn_step."""
    d, opt, _ = make(9, 2, 150, 4, 2, 128, 64, state=True)
    g, h0 = on(d), opt["h0"].cuda()
    n, m = np64(d), np64(opt)
    wo, wh, w = ref.linattn_forward(n["q"], n["k"], n["v"], n["g"], 128 ** -0.5, m["h0"])
    state = h0.clone()
    first = {k: v[:, :77].contiguous() for k, v in g.items()}
    second = {k: v[:, 77:].contiguous() for k, v in g.items()}
    o1, _ = cs.linattn_forward(**first, h0=state, h_final=state)
    o2, _ = cs.linattn_forward(**second, h0=state, h_final=state)
    close(torch.cat([o1, o2], 1), wo, w["o_terms"], "two calls")
    close(state, wh, w["h_terms"], "state of two calls")
    state = h0.clone()
    steps = torch.stack([cs.linattn_step(state, *(g[n][:, t].contiguous() for n in ("q", "k", "v", "g"))) for t in range(150)], 1)
    close(steps, wo, w["o_terms"], "steps")
    close(state, wh, w["h_terms"], "state of the steps")


def test_gradients_match_differences(cs):
    """<gradient, direction> against a central difference of the GPU's own
    forward in fp32 (step 1e-2: a third-order term of 1e-4, and the forward's
    1e-5 over the step).  One decay for all T = 100 tokens of a head enters as
    exp(T step): its third-order term is (T step)^2 / 6 of the first, 0.17 at 1e-2,
    so its step is 1e-2 / T, which leaves the same 2e-5."""
    for head in (False, True):
        d, opt, back = make(10, 1, 100, 2, 1, 64, 64, state=True, head=head)
        r = cs.linattn_backward(**on(d), **on(back), **on(opt), scale=0.5)
        do, dh = back["do"].double(), back["dh_final"].double()
        gen = torch.Generator().manual_seed(3)

        def loss(x, h0):
            o, h = cs.linattn_forward(**on(x), h0=h0.cuda(), scale=0.5)
            return float((o.cpu().double() * do).sum() + (h.cpu().double() * dh).sum())

        for name in ("q", "k", "v", "g", "h0"):
            src = opt["h0"] if name == "h0" else d[name]
            way = torch.randn(src.shape, generator=gen)
            way *= (1e-4 if head and name == "g" else 1e-2) / way.abs().max()
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


def test_what_is_not_wanted(cs):
    """No last state, no gradient of g, outputs and workspaces given by the caller."""
    d, opt, back = make(14, 2, 140, 2, 2, 64, 64, dtype="bf16", state=True)
    g, o_, b = on(d), on(opt), on(back)
    o, h = cs.linattn_forward(**g, **o_)
    r = cs.linattn_backward(**g, **b, **o_)
    out = torch.empty_like(o)
    ws = torch.empty(cs.linattn_workspace_bytes(2, 140, 2, 2, 64, 64, torch.bfloat16), dtype=torch.uint8, device="cuda")
    o2, none = cs.linattn_forward(**g, **o_, want_state=False, o=out, workspace=ws)
    assert none is None and o2 is out and torch.equal(o, o2)
    ws = torch.empty(cs.linattn_backward_workspace_bytes(2, 140, 2, 2, 64, 64, torch.bfloat16), dtype=torch.uint8, device="cuda")
    b["dh_final"] = b["dh_final"].clone()
    r2 = cs.linattn_backward(**g, **b, **o_, want_g=False, grads={"gh0": b["dh_final"]}, workspace=ws)  # gh0 over dh_final
    assert "gg" not in r2 and r2["gh0"] is b["dh_final"]
    for n in ("gq", "gk", "gv", "gh0"):
        assert torch.equal(r[n], r2[n]), n
    with pytest.raises(cs.CssdError, match="WORKSPACE"):
        cs.linattn_forward(**g, **o_, workspace=ws[:64])


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 1, 1, 16, 16), (3, 4, 2, 64, 64), (2, 8, 2, 128, 128), (5, 3, 3, 96, 80),
                                   (2, 2, 1, 112, 48), (37, 12, 12, 64, 64)])
@pytest.mark.parametrize("head", [False, True])
def test_step(cs, shape, head, dtype):
    B, H, KH, N, P = shape
    d, opt, _ = make(sum(shape) + 2, B, 1, H, KH, N, P, dtype=dtype, state=True, head=head)
    one = {k: v if v.dim() == 1 else v[:, 0].contiguous() for k, v in d.items()}
    h = opt["h0"].cuda()
    o = cs.linattn_step(h, **on(one), scale=0.3)
    n, m = np64(d), np64(opt)
    wo, wh, w = ref.linattn_forward(n["q"], n["k"], n["v"], n["g"], 0.3, m["h0"])
    close(o, wo[:, 0], w["o_terms"][:, 0], "o")
    close(h, wh, w["h_terms"], "h")


def test_step_slots(cs):
    """Rows name their states in any order; a slot outside the pool writes
    nothing and answers zero; states no row names are left alone."""
    B, H, N, P, pool = 6, 4, 64, 80, 9
    d, _, _ = make(11, B, 1, H, 2, N, P, dtype="bf16")
    one = {k: v[:, 0].contiguous() for k, v in d.items()}
    h0 = torch.randn(pool, H, N, P, generator=torch.Generator().manual_seed(1))
    slots = [7, -1, 0, 9, 3, 1 << 30]
    h = h0.cuda()
    o = cs.linattn_step(h, **on(one), slots=torch.tensor(slots, dtype=torch.int32).cuda())
    n = np64(d)
    for b, s in enumerate(slots):
        if not 0 <= s < pool:
            assert (o[b] == 0).all()
            continue
        wo, wh, w = ref.linattn_forward(*(n[k][b:b + 1] for k in ("q", "k", "v", "g")), N ** -0.5, h0[s:s + 1].double().numpy())
        close(o[b], wo[0, 0], w["o_terms"][0, 0], "o")
        close(h[s], wh[0], w["h_terms"][0], "h")
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
    o = cs.linattn_step(h, **on(one), slots=torch.tensor([pool - 1], dtype=torch.int32).cuda(), scale=1.0)
    n, m = np64(d), np64(opt)
    wo, wh, w = ref.linattn_forward(n["q"], n["k"], n["v"], n["g"], 1.0, m["h0"])
    close(o, wo[:, 0], w["o_terms"][:, 0], "o")
    close(h[-1:], wh, w["h_terms"], "h")


def test_tensors_past_32_bits(cs):
    """More than 2^31 elements of v, most of them of rows without tokens: the
    last row's tokens are found, and the empty rows' outputs are zeros."""
    B, T, H, P = 260, 1024, 64, 128
    q = torch.zeros(B, T, 1, 16, dtype=torch.bfloat16, device="cuda")
    v = torch.empty(B, T, H, P, dtype=torch.bfloat16, device="cuda")
    assert v.numel() > 1 << 31
    d, _, _ = make(13, 1, T, H, 1, 16, P, dtype="bf16", head=True)
    k = q.clone()
    q[-1], k[-1], v[-1] = (d[n][0].cuda() for n in ("q", "k", "v"))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = 130
    o, h = cs.linattn_forward(q, k, v, d["g"].cuda(), scale=0.25, lens=lens)
    n = np64(d)
    wo, wh, w = ref.linattn_forward(n["q"][:, :130], n["k"][:, :130], n["v"][:, :130], n["g"], 0.25)
    close(o[-1:, :130], wo, w["o_terms"], "o")
    close(h[-1:], wh, w["h_terms"], "h")
    assert not o[:-1].any() and not o[-1, 130:].any() and not h[:-1].any()


def test_other_stream_and_graph(cs):
    """On a stream of the caller's, and captured into a graph whose replays
    redo the work on new contents of the same buffers; equal calls, equal bits."""
    d, opt, back = make(15, 2, 300, 4, 2, 64, 64, dtype="bf16", state=True)
    other, _, _ = make(25, 2, 300, 4, 2, 64, 64, dtype="bf16")
    g, o_, b = on(d), on(opt), on(back)
    want = cs.linattn_forward(**g, **o_), cs.linattn_backward(**g, **b, **o_)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o, h = cs.linattn_forward(**g, **o_, stream=side)
    r = cs.linattn_backward(**g, **b, **o_, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, want[0][0]) and torch.equal(h, want[0][1])
    for n in r:
        assert torch.equal(r[n], want[1][n]), n
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, h = cs.linattn_forward(**g, **o_)
        r = cs.linattn_backward(**g, **b, **o_)
        step = cs.linattn_step(h, *(g[n][:, 0].contiguous() for n in ("q", "k", "v", "g")))
    for n in ("q", "k", "v", "g"):
        g[n].copy_(other[n])
    graph.replay()
    torch.cuda.synchronize()
    wo, wh = cs.linattn_forward(**g, **o_)
    wr = cs.linattn_backward(**g, **b, **o_)
    assert torch.equal(o, wo)
    for n in r:
        assert torch.equal(r[n], wr[n]), n
    ws = cs.linattn_step(wh, *(g[n][:, 0].contiguous() for n in ("q", "k", "v", "g")))
    assert torch.equal(step, ws) and torch.equal(h, wh)


def test_errors_are_roundings(cs):
    """A layer's call in bfloat16: the last state, gh0 and gg (float32) are
    within 1e-6 of the 64-bit result in the 2-norm (32 chunks' sums of 2^-24
    each, adding up like a random walk, and the exponentials' 2^-22), the
    16-bit outputs within their own rounding (2^-9 at most, relative)."""
    d, opt, back = make(18, 1, 1100, 2, 2, 64, 64, dtype="bf16", state=True)
    o, h = cs.linattn_forward(**on(d), **on(opt))
    r = cs.linattn_backward(**on(d), **on(back), **on(opt))
    n, m, b = np64(d), np64(opt), np64(back)
    wo, wh, _ = ref.linattn_forward(n["q"], n["k"], n["v"], n["g"], 0.125, m["h0"])
    w = ref.linattn_backward(n["q"], n["k"], n["v"], n["g"], 0.125, b["do"], m["h0"], b["dh_final"])

    def off(x, y):
        return np.linalg.norm(x.cpu().double().numpy() - y) / np.linalg.norm(y)

    assert off(h, wh) < 1e-6 and off(r["gh0"], w["gh0"]) < 1e-6 and off(r["gg"], w["gg"]) < 1e-6
    for x, y in ((o, wo), (r["gq"], w["gq"]), (r["gk"], w["gk"]), (r["gv"], w["gv"])):
        assert off(x, y) < 2.0 ** -9


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128), (96, 80)])
def test_states_in_place(cs, NP, dtype):
    """The last state over the first one, and gh0 over dh_final, where a row's walk is cut into segments (few
    heads, many chunks) that all read the first one."""
    d, opt, back = make(19, 1, 1100, 1, 1, *NP, dtype=dtype, state=True)
    g, b, h0 = on(d), on(back), opt["h0"].cuda()
    o, h = cs.linattn_forward(**g, h0=h0)
    r = cs.linattn_backward(**g, **b, h0=h0)
    for _ in range(20):
        state, dh = h0.clone(), b["dh_final"].clone()
        o2, _ = cs.linattn_forward(**g, h0=state, h_final=state)
        cs.linattn_backward(**g, do=b["do"], dh_final=dh, h0=h0, grads={"gh0": dh})
        assert torch.equal(o, o2) and torch.equal(h, state) and torch.equal(r["gh0"], dh)


@pytest.mark.parametrize("NP", [(128, 128), (128, 64), (64, 128), (112, 80)])
def test_wide_gradients_side_by_side(cs, NP):
    """The wide bfloat16 gradients (products on the tensor cores' own memory): many blocks at once and two streams
    at once give the bits of one call after another, and no wait inside a kernel gives up."""
    d, opt, back = make(20, 2, 900, 12, 6, *NP, dtype="bf16", state=True, ragged=[900, 517])
    g, o_, b = on(d), on(opt), on(back)
    want = cs.linattn_backward(**g, **b, **o_)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [cs.linattn_backward(**g, **b, **o_, stream=streams[i % 2]) for i in range(6)]
    torch.cuda.synchronize()
    for r in got:
        for n in want:
            assert torch.equal(r[n], want[n]), n
    assert cs.device_status() == 0


@pytest.mark.parametrize("dtype", ["fp16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128), (128, 64), (16, 32)])
def test_float32_results_are_float32(cs, NP, dtype):
    """Every float32 result (all of float32 tensors; states and their gradients, and g's, of float16 ones) is within
    1e-6 of the 64-bit one in the 2-norm: a sum of up to 128 products (a random walk of 2^-24 each, 7e-7) twice over
    is 1e-6, and most sums are shorter."""
    d, opt, back = make(21, 1, 400, 2, 1, *NP, dtype=dtype, state=True)
    o, h = cs.linattn_forward(**on(d), **on(opt))
    r = cs.linattn_backward(**on(d), **on(back), **on(opt))
    n, m, b = np64(d), np64(opt), np64(back)
    wo, wh, _ = ref.linattn_forward(n["q"], n["k"], n["v"], n["g"], NP[0] ** -0.5, m["h0"])
    w = ref.linattn_backward(n["q"], n["k"], n["v"], n["g"], NP[0] ** -0.5, b["do"], m["h0"], b["dh_final"])
    for name, x, y in [("o", o, wo), ("h", h, wh)] + [(k, r[k], w[k]) for k in ("gq", "gk", "gv", "gg", "gh0")]:
        if x.dtype == torch.float32:
            off = np.linalg.norm(x.cpu().double().numpy() - y) / np.linalg.norm(y)
            assert off < 1e-6, (name, off)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128), (128, 32), (96, 80)])
@pytest.mark.parametrize("head", [False, True])
def test_no_decay_no_gradient(cs, NP, head, dtype):
    """Rows of at most one token without a state before it: nothing decays, so the gradient of g is zero, to the bit."""
    for B, T, lens in ((3, 1, None), (4, 2, [0, 1, 1, 0]), (3, 300, [1, 0, 1])):
        d, opt, back = make(22, B, T, 4, 2, *NP, dtype=dtype, ragged=lens, head=head)
        r = cs.linattn_backward(**on(d), **on(back), **on(opt))
        assert r["gg"].shape == d["g"].shape and not r["gg"].any()
        assert r["gq"].any() and r["gk"].any() and r["gv"].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128)])
@pytest.mark.parametrize("head", [False, True])
def test_decay_gradients_of_heads_that_forget_fast(cs, NP, head, dtype):
    """The gradient of g where a token keeps e^-5 or e^-10 of the state: of the size of what is kept, and right to
    float32 there.  A token's spanning pairs carry the quick exponential's error ((2 + 1.2 |g|) 2^-23 at most, 1.7e-6 at -10),
    their scores' (a random walk of at most 128 products, 7e-7) and, of the running sums over the chunk's 128 tokens,
    a random walk of 2^-24 of those pairs' sizes, 7e-7 again: below 4e-6 of the gradient's 2-norm over the tokens, and (one
    decay a head: the tokens' sum) of the tokens' sizes summed up."""
    d, opt, back = make(23, 1, 300, 4, 4, *NP, dtype=dtype, state=True, head=head)
    d["g"][:] = torch.tensor([-3.0, -5.0, -10.0, -14.0])
    r = cs.linattn_backward(**on(d), **on(back), **on(opt), scale=0.25)
    n, m, b = np64(d), np64(opt), np64(back)
    w = ref.linattn_backward(n["q"], n["k"], n["v"], np.broadcast_to(n["g"], (1, 300, 4)), 0.25, b["do"], m["h0"], b["dh_final"])["gg"]
    got = r["gg"].cpu().double().numpy()
    for h in range(4):
        if head:
            assert abs(got[h] - w[..., h].sum()) < 4e-6 * np.abs(w[..., h]).sum(), h
        else:
            assert np.linalg.norm(got[..., h] - w[..., h]) < 4e-6 * np.linalg.norm(w[..., h]), h


RATES = [3e-4, 3.7e-4, 4.9e-4, 6.1e-4, 8.3e-4, 1.1e-3]


def off(x, y):
    return float((x.double() - y).norm() / y.norm())


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("NP", [(64, 64), (128, 128)])
@pytest.mark.parametrize("B", [1, 70])
def test_states_of_slow_heads(cs, NP, dtype, B):
    """One decay a head, heads that remember thousands of tokens, rows walked whole and cut: the last state and gh0 of each head are
    within 1e-6 of the 64-bit recurrence in the 2-norm.  Of a state's size, at random: a chunk's rounding (2^-23 / sqrt(12), at
    most 7 of them as chunks of 32 tokens are forgotten: 2.5e-7), its products' sums in two or more steps that drop up to 2^-23 (2.4e-7),
    the tokens' decays to the chunk's end 1.2e-7: 4e-7; what is the same in every chunk, its decay's error, is below 2^-24 of what is forgotten."""
    T, H, (N, P) = 5000, len(RATES), NP
    gen = torch.Generator(device="cuda").manual_seed(5)
    q, k, v, do = (torch.randn(T, H, w, generator=gen, device="cuda").to(TYPES[dtype]) for w in (N, N, P, P))
    g = -torch.tensor(RATES, device="cuda")
    h0, dh = (torch.randn(1, H, N, P, generator=gen, device="cuda") for _ in range(2))
    S, D, a = h0[0].double(), dh[0].double(), torch.exp(g.double())[:, None, None]
    for t in range(T):
        S = torch.baddbmm(a * S, k[t].double()[:, :, None], v[t].double()[:, None])
        u = T - 1 - t
        D = a * torch.baddbmm(D, q[u].double()[:, :, None], 0.25 * do[u].double()[:, None])
    many = lambda x: x[None].expand(B, *x.shape).contiguous()  # noqa: E731
    h0, dh = (x.expand(B, -1, -1, -1).contiguous() for x in (h0, dh))
    _, h = cs.linattn_forward(many(q), many(k), many(v), g, scale=0.25, h0=h0)
    r = cs.linattn_backward(many(q), many(k), many(v), g, many(do), scale=0.25, h0=h0, dh_final=dh)
    for e in range(H):
        assert off(h[0, e], S[e]) < 1e-6 and off(r["gh0"][0, e], D[e]) < 1e-6, (e, off(h[0, e], S[e]), off(r["gh0"][0, e], D[e]))


def test_steps_of_slow_heads(cs):
    """4000 tokens one by one where a head remembers up to 3300 of them: a token rounds a state twice (2^-23 / sqrt(12) at most, at random),
    41 times that as it forgets: 1.4e-6, and its decay's error, the same for every token, is below 2^-24 of what is forgotten."""
    T, H, N, P = 4000, len(RATES), 64, 64
    gen = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(T, 1, H, w, generator=gen, device="cuda") for w in (N, P))
    g = -torch.tensor(RATES, device="cuda")
    h = torch.randn(1, H, N, P, generator=gen, device="cuda")
    S, a = h[0].double(), torch.exp(g.double())[:, None, None]
    for t in range(T):
        cs.linattn_step(h, k[t], k[t], v[t], g)
        S = torch.baddbmm(a * S, k[t, 0].double()[:, :, None], v[t, 0].double()[:, None])
    for e in range(H):
        assert off(h[0, e], S[e]) < 2e-6, (e, off(h[0, e], S[e]))


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("NP", [(128, 128), (64, 128)])
def test_decay_gradients_keep_float32(cs, NP, dtype):
    """The gradient of g within 5e-7 of the 64-bit one in the 2-norm, whatever the planes of the tensors: a pair's two scores
    are sums in at most 8 steps that drop half of 2^-23 on average, at random, 2.4e-7 for both; as much for the states' terms in it,
    and 1e-7 for the exponentials: the three together, as independent errors, below 3.6e-7."""
    for seed in (30, 31, 32):
        d, opt, back = make(seed, 4, 172, 2, 2, *NP, dtype=dtype, state=False)
        r = cs.linattn_backward(**on(d), **on(back), **on(opt))
        n, b = np64(d), np64(back)
        w = torch.from_numpy(ref.linattn_backward(n["q"], n["k"], n["v"], n["g"], NP[0] ** -0.5, b["do"])["gg"])
        assert off(r["gg"].cpu(), w) < 5e-7, (seed, off(r["gg"].cpu(), w))
