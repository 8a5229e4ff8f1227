"""The gated delta rule and layer norm on the host: the 64-bit references
against differences and closed forms, and the entry points' refusals (no GPU
needed, nothing launched)."""

import ctypes

import numpy as np
import pytest
import torch

import delta_reference as ref
from complex_valued_state_gb300 import build as cbuild
from complex_valued_state_gb300 import cssd


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cssd.load()


def case(seed, B=2, T=7, H=4, KH=2, N=5, P=3):
    r = np.random.default_rng(seed)
    d = dict(q=r.standard_normal((B, T, KH, N)), k=r.standard_normal((B, T, KH, N)) / np.sqrt(N),
             v=r.standard_normal((B, T, H, P)), g=-r.uniform(0, 1, (B, T, H)), beta=r.uniform(0, 1, (B, T, H)))
    return d, r


def test_reference_gradients_match_differences():
    d, r = case(0)
    h0, dh = r.standard_normal((2, 4, 5, 3)), r.standard_normal((2, 4, 5, 3))
    do = r.standard_normal((2, 7, 4, 3))
    lens = np.array([7, 4])

    def loss(x):
        o, h, _ = ref.delta_forward(x["q"], x["k"], x["v"], x["g"], x["beta"], 0.7, x["h0"], lens)
        return float(np.sum(o * do) + np.sum(h * dh))

    x = dict(d, h0=h0)
    g = ref.delta_backward(d["q"], d["k"], d["v"], d["g"], d["beta"], 0.7, do, h0, dh, lens)
    for name in ("q", "k", "v", "g", "beta", "h0"):
        step = 1e-6
        for at in r.choice(x[name].size, 12, replace=False):
            up, down = dict(x), dict(x)
            up[name], down[name] = x[name].copy(), x[name].copy()
            up[name].flat[at] += step
            down[name].flat[at] -= step
            diff = (loss(up) - loss(down)) / (2 * step)
            assert abs(diff - g["g" + name].flat[at]) < 1e-7 * max(1.0, abs(diff)), name


def test_reference_closed_forms():
    """Orthonormal keys at beta 1 and g 0 store and return their values; a key
    written twice keeps the second value; g = -inf forgets."""
    N, P = 4, 3
    r = np.random.default_rng(1)
    k = np.eye(N)[None, :, None, :]
    v = r.standard_normal((1, N, 1, P))
    one, zero = np.ones((1, N, 1)), np.zeros((1, N, 1))
    o, h, _ = ref.delta_forward(k, k, v, zero, one, 1.0)
    assert np.allclose(o, v) and np.allclose(h[0, 0], v[0, :, 0])
    k2 = np.concatenate([k[:, :1], k[:, :1]], 1)
    _, h, _ = ref.delta_forward(k2, k2, v[:, :2], zero[:, :2], one[:, :2], 1.0)
    assert np.allclose(h[0, 0, 0], v[0, 1, 0])
    _, h, _ = ref.delta_forward(k2, k2, v[:, :2], np.array([[[0.0], [-np.inf]]]), one[:, :2], 1.0,
                                h0=r.standard_normal((1, 1, N, P)))
    assert np.allclose(h[0, 0], np.outer(k2[0, 1, 0], v[0, 1, 0]))


def test_reference_norm_gradients_match_differences():
    r = np.random.default_rng(2)
    x, w, b, dy = r.standard_normal((3, 6)), r.standard_normal(6), r.standard_normal(6), r.standard_normal((3, 6))
    gx, gw, gb = ref.layernorm_backward(dy, x, w, 1e-3)
    for a, ga in ((x, gx), (w, gw), (b, gb)):
        for at in range(a.size):
            keep = a.flat[at]
            vals = []
            for s in (1e-6, -1e-6):
                a.flat[at] = keep + s
                vals.append(np.sum(ref.layernorm(x, w, b, 1e-3)[0] * dy))
            a.flat[at] = keep
            assert abs((vals[0] - vals[1]) / 2e-6 - ga.flat[at]) < 1e-7


def ptrs(n):
    return [ctypes.c_void_p(0x10000 + 0x1000 * i) for i in range(n)]


def dims(*v):
    return ctypes.byref(cssd.DeltaDims(*v))


OK = (2, 100, 4, 2, 64, 64)


def forward(lib, d=OK, dtype=0, ws=0x900000, ws_bytes=1 << 40, **kw):
    names = ("q", "k", "v", "g", "beta", "h0", "lens", "o", "h_final")
    p = dict(zip(names, ptrs(9)))
    p.update({k: ctypes.c_void_p(v) if v else None for k, v in kw.items()})
    return lib.cssd_delta_forward(None if d is None else dims(*d), dtype, p["q"], p["k"], p["v"], p["g"], p["beta"],
                                  ctypes.c_float(1.0), p["h0"], p["lens"], p["o"], p["h_final"], ctypes.c_void_p(ws),
                                  ws_bytes, None)


def test_forward_refusals(lib):
    assert forward(lib, None) == -1
    for bad in ((0, 100, 4, 2, 64, 64), (2, 0, 4, 2, 64, 64), (2, 100, 4, 0, 64, 64), (2, 100, 4, 3, 64, 64),
                (2, 100, 2, 4, 64, 64), (2, -1, 4, 2, 64, 64), (1 << 20, 1 << 20, 1 << 9, 1, 64, 64),
                (1 << 40, 1, 1, 1, 64, 64), (1, 1 << 40, 1, 1, 64, 64)):
        assert forward(lib, bad) == -2, bad
    for bad in ((2, 100, 4, 2, 8, 64), (2, 100, 4, 2, 64, 20), (2, 100, 4, 2, 144, 64), (2, 100, 4, 2, 64, 256)):
        assert forward(lib, bad) == -3, bad
    assert forward(lib, dtype=3) == -3 and forward(lib, dtype=-1) == -3
    for n in ("q", "k", "v", "g", "beta", "o"):
        assert forward(lib, **{n: 0}) == -1, n
    for n in ("q", "k", "v", "h0", "o", "h_final"):
        assert forward(lib, **{n: 0x10008}) == -4, n
    for n in ("g", "beta", "lens"):
        assert forward(lib, **{n: 0x10002}) == -4, n
    assert forward(lib, ws=0x900008) == -4
    assert forward(lib, ws_bytes=16) == -5
    assert lib.cssd_delta_workspace_bytes(dims(*OK), 0) > 0
    assert lib.cssd_delta_workspace_bytes(dims(2, 100, 4, 3, 64, 64), 0) == 0
    assert lib.cssd_delta_workspace_bytes(dims(*OK), 7) == 0


def test_sizes_past_the_grid(lib):
    """A sequence in fp32 takes a block per head and 16 columns, the gradients two:
    sizes whose count of blocks would not fit 31 bits are refused."""
    heads = (1 << 31) // 16
    for dtype in (0, 2):
        for n, P in ((heads, 128), (1 << 28, 64), (1 << 29, 16), (1 << 29, 32)):
            for b, h in ((n, 1), (1, n), (1 << 10, n >> 10)):
                d = (b, 1, h, 1, 16, P)
                assert lib.cssd_delta_workspace_bytes(dims(*d), dtype) == 0, d
                assert lib.cssd_delta_backward_workspace_bytes(dims(*d), dtype) == 0, d
                assert forward(lib, d, dtype) == -2, d
        for n, P in ((heads - 1, 128), ((1 << 28) - 1, 64), ((1 << 29) - 1, 32), ((1 << 29) - 1, 16)):
            assert lib.cssd_delta_workspace_bytes(dims(1, 1, n, 1, 16, P), dtype) > 0, (n, P)
            assert lib.cssd_delta_backward_workspace_bytes(dims(n, 1, 1, 1, 16, P), dtype) > 0, (n, P)


def test_backward_refusals(lib):
    need = lib.cssd_delta_backward_workspace_bytes(dims(*OK), 2)
    assert need >= 2 * 4 * 2 * 4 * 2 * 64 * 64  # two fp32 states a head and chunk
    names = ("q", "k", "v", "g", "beta", "h0", "lens", "do", "dh", "gq", "gk", "gv", "gg", "gbeta", "gh0")

    def call(d=OK, dtype=2, ws_bytes=1 << 40, **kw):
        p = dict(zip(names, ptrs(15)))
        p.update({k: ctypes.c_void_p(v) if v else None for k, v in kw.items()})
        v = list(p.values())
        return lib.cssd_delta_backward(None if d is None else dims(*d), dtype, *v[:5], ctypes.c_float(1.0), *v[5:],
                                       ctypes.c_void_p(0x900000), ws_bytes, None)

    assert call(None) == -1
    assert call((2, 100, 4, 3, 64, 64)) == -2
    assert call((2, 100, 4, 2, 64, 72)) == -3
    assert call(dtype=9) == -3
    for n in ("q", "k", "v", "g", "beta", "do", "gq", "gk", "gv", "gg", "gbeta"):
        assert call(**{n: 0}) == -1, n
    for n in ("do", "dh", "gq", "gk", "gv", "gh0", "h0"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(gg=0x10002) == -4 and call(gbeta=0x10001) == -4 and call(lens=0x10002) == -4
    assert call(ws_bytes=need - 1) == -5


def test_step_refusals(lib):
    def call(d=OK, dtype=1, nslots=5, **kw):
        p = dict(zip(("h", "slots", "q", "k", "v", "g", "beta", "o"), ptrs(8)))
        p.update({k: ctypes.c_void_p(v) if v else None for k, v in kw.items()})
        v = list(p.values())
        return lib.cssd_delta_step(None if d is None else dims(*d), dtype, v[0], nslots, *v[1:7], ctypes.c_float(1.0),
                                   v[7], None)

    assert call(None) == -1
    assert call((0, 1, 4, 2, 64, 64)) == -2 and call((2, 1, 4, 3, 64, 64)) == -2
    assert call((2, 1, 4, 2, 63, 64)) == -3 and call(dtype=5) == -3
    assert call(nslots=0) == -2 and call(nslots=1, slots=0) == -2  # fewer states than rows, and no slots
    for n in ("h", "q", "k", "v", "g", "beta", "o"):
        assert call(**{n: 0}) == -1, n
    for n in ("h", "q", "k", "v", "o"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(slots=0x10002) == -4 and call(g=0x10001) == -4


def test_norm_refusals(lib):
    def call(rows=4, width=8, xt=0, wt=2, eps=1e-5, **kw):
        p = dict(zip(("x", "w", "b", "y", "mean", "rstd"), ptrs(6)))
        p.update({k: ctypes.c_void_p(v) if v else None for k, v in kw.items()})
        return lib.cssd_layernorm(rows, width, xt, wt, p["x"], p["w"], p["b"], ctypes.c_float(eps), p["y"], p["mean"],
                                  p["rstd"], None)

    assert call(rows=0) == -2 and call(width=0) == -2 and call(width=1 << 25) == -2 and call(rows=1 << 32) == -2
    assert call(xt=3) == -3 and call(xt=0, wt=1) == -3 and call(xt=2, wt=0) == -3
    assert call(eps=-1.0) == -2 and call(eps=float("nan")) == -2
    assert call(x=0) == -1 and call(y=0) == -1
    for n in ("x", "w", "b", "y"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(mean=0x10002) == -4

    def back(rows=4, width=8, xt=0, wt=2, ws_bytes=1 << 40, **kw):
        p = dict(zip(("dy", "x", "w", "mean", "rstd", "gx", "gw", "gb"), ptrs(8)))
        p.update({k: ctypes.c_void_p(v) if v else None for k, v in kw.items()})
        return lib.cssd_layernorm_backward(rows, width, xt, wt, *p.values(), ctypes.c_void_p(0x900000), ws_bytes, None)

    assert back(rows=-1) == -2 and back(wt=1) == -3
    for n in ("dy", "x", "mean", "rstd", "gx"):
        assert back(**{n: 0}) == -1, n
    assert back(gw=0x10004) == -4 and back(rstd=0x10002) == -4
    assert back(ws_bytes=8) == -5
    assert lib.cssd_layernorm_backward_workspace_bytes(0, 8) == 0


def test_binding_rejects_wrong_tensors():
    q = torch.zeros(1, 8, 2, 16)
    v = torch.zeros(1, 8, 2, 16)
    g = torch.zeros(1, 8, 2)
    with pytest.raises(TypeError):
        cssd.delta_forward(q.double(), q.double(), v.double(), g, g)
    with pytest.raises(TypeError):
        cssd.delta_forward(q, q.half(), v, g, g)
    with pytest.raises(TypeError):
        cssd.delta_forward(q, q, v, g.half(), g)
    with pytest.raises(ValueError):
        cssd.delta_forward(q, q[:, :4], v, g, g)
    with pytest.raises(ValueError):
        cssd.delta_forward(q, q, v.transpose(1, 2).contiguous().transpose(1, 2), g, g)
    with pytest.raises(ValueError):
        cssd.delta_forward(q, q, v, g, g, h0=torch.zeros(1, 2, 16, 15))
    with pytest.raises(TypeError):
        cssd.delta_forward(q, q, v, g, g, lens=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        cssd.delta_backward(q, q, v, g, g, v[:, :4])
    with pytest.raises(ValueError):
        cssd.delta_step(torch.zeros(1, 2, 16, 8), q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0])
    with pytest.raises(ValueError):
        cssd.delta_step(torch.zeros(2, 16, 16), q[:, 0], q[:, 0], v[:, 0], g[:, 0], g[:, 0])
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError):
        cssd.layernorm(x.double())
    with pytest.raises(TypeError):
        cssd.layernorm(x, torch.zeros(8, dtype=torch.float16))
    with pytest.raises(TypeError):
        cssd.layernorm(x.half(), torch.zeros(8), torch.zeros(8, dtype=torch.float16))
    with pytest.raises(ValueError):
        cssd.layernorm(x, torch.zeros(7))
    with pytest.raises(ValueError):
        cssd.layernorm(x.t())
    with pytest.raises(ValueError):
        cssd.layernorm_backward(x, x, None, torch.zeros(3), torch.zeros(4))


def test_binding_types_of_norm_gradients():
    """Without a weight `wdtype` names the bias's type: its gradient is taken in
    that type (past the checks, tensors off the GPU are refused)."""
    x, stat = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4)
    f32, half = torch.zeros(8), torch.zeros(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        cssd.layernorm_backward(x, x, None, stat, stat, want_weight=False, wdtype=torch.float32, grads={"gbias": f32})
    with pytest.raises(ValueError, match="CUDA device"):
        cssd.layernorm_backward(x, x, f32, stat, stat, wdtype=torch.float32, grads={"gweight": f32, "gbias": f32})
    with pytest.raises(TypeError, match="gbias"):
        cssd.layernorm_backward(x, x, None, stat, stat, wdtype=torch.float32, grads={"gbias": half})
    with pytest.raises(TypeError, match="gbias"):
        cssd.layernorm_backward(x, x, None, stat, stat, grads={"gbias": f32})
    with pytest.raises(TypeError, match="wdtype"):
        cssd.layernorm_backward(x, x, None, stat, stat, wdtype=torch.float16)
    with pytest.raises(TypeError, match="wdtype"):
        cssd.layernorm_backward(x, x, f32, stat, stat, wdtype=torch.bfloat16)
