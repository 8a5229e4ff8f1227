"""Linear attention and the norms of a block, without a GPU: the 64-bit
reference against differences, and what the entry points refuse."""

import ctypes

import block_reference as ref
import numpy as np
import pytest
import torch

from complex_valued_state_gb300 import build as cbuild
from complex_valued_state_gb300 import cssd


@pytest.fixture(scope="module")
def lib():
    cbuild.build()
    return cssd.load()


@pytest.mark.parametrize("per_head", [False, True])
def test_reference_linattn_gradients_match_differences(per_head):
    r = np.random.default_rng(1)
    B, T, H, KH, N, P = 2, 5, 4, 2, 3, 2
    d = {"q": r.standard_normal((B, T, KH, N)), "k": r.standard_normal((B, T, KH, N)), "v": r.standard_normal((B, T, H, P)),
         "g": -r.uniform(0, 1, H if per_head else (B, T, H)), "h0": r.standard_normal((B, H, N, P))}
    do, dh, lens = r.standard_normal((B, T, H, P)), r.standard_normal((B, H, N, P)), np.array([5, 3])

    def loss():
        o, h, _ = ref.linattn_forward(d["q"], d["k"], d["v"], d["g"], 0.7, d["h0"], lens)
        return (o * do).sum() + (h * dh).sum()

    got = ref.linattn_backward(d["q"], d["k"], d["v"], d["g"], 0.7, do, d["h0"], dh, lens)
    for n, x in d.items():
        for at in range(x.size):
            keep, vals = x.flat[at], []
            for s in (1e-6, -1e-6):
                x.flat[at] = keep + s
                vals.append(loss())
            x.flat[at] = keep
            assert abs((vals[0] - vals[1]) / 2e-6 - got["g" + n].flat[at]) < 1e-6, n


@pytest.mark.parametrize("layer", [False, True])
def test_reference_norm_gradients_match_differences(layer):
    r = np.random.default_rng(2)
    R, D, eps = 3, 6, 1e-3
    x, res, z, dy, ds = (r.standard_normal((R, D)) for _ in range(5))
    w, b, sc = (r.standard_normal(D) for _ in range(3))

    def check(loss, pairs):
        for a, ga in pairs:
            for at in range(a.size):
                keep, vals = a.flat[at], []
                for s in (1e-6, -1e-6):
                    a.flat[at] = keep + s
                    vals.append(loss())
                a.flat[at] = keep
                assert abs((vals[0] - vals[1]) / 2e-6 - ga.flat[at]) < 1e-6

    def add():
        y, s, _, _ = ref.add_norm(x, res, w, b, layer, 0.7, sc, eps)
        return (y * dy).sum() + (s * ds).sum()

    s = ref.add_norm(x, res, w, b, layer, 0.7, sc, eps)[1]
    g = ref.add_norm_backward(dy, ds, x, s, w, layer, 0.7, sc, eps)
    check(add, ((x, g["gx"]), (res, g["gresidual"]), (w, g["gweight"]), (b, g["gbias"]), (sc, g["gscale"])))
    for first in (False, True):
        for group in (3, 6):
            g = ref.gated_norm_backward(dy, x, z, w, b, layer, group, first, eps)
            check(lambda: (ref.gated_norm(x, z, w, b, layer, group, first, eps)[0] * dy).sum(),
                  ((x, g["gx"]), (z, g["gz"]), (w, g["gweight"]), (b, g["gbias"])))


def ptrs(n):
    return [ctypes.c_void_p(0x10000 + 0x1000 * i) for i in range(n)]


def dims(*v):
    return ctypes.byref(cssd.DeltaDims(*v))


OK = (2, 100, 4, 2, 64, 64)


def given(names, kw):
    p = dict(zip(names, ptrs(len(names))))
    p.update({k: ctypes.c_void_p(v) if v else None for k, v in kw.items()})
    return list(p.values())


def test_linattn_forward_refusals(lib):
    def call(d=OK, dtype=0, ws=0x900000, ws_bytes=1 << 40, **kw):
        p = given(("q", "k", "v", "g", "h0", "lens", "o", "h_final"), kw)
        return lib.cssd_linattn_forward(None if d is None else dims(*d), dtype, *p[:4], 1, ctypes.c_float(1.0), *p[4:],
                                        ctypes.c_void_p(ws), ws_bytes, None)

    assert call(None) == -1
    for bad in ((0, 100, 4, 2, 64, 64), (2, 0, 4, 2, 64, 64), (2, 100, 4, 3, 64, 64), (2, 100, 2, 4, 64, 64), (2, -1, 4, 2, 64, 64),
                (1 << 40, 1, 1, 1, 64, 64), (1, 1 << 40, 1, 1, 64, 64), (1 << 10, 1 << 26, 1, 1, 64, 64)):
        assert call(bad) == -2, bad
        assert lib.cssd_linattn_workspace_bytes(dims(*bad), 0) == 0 and lib.cssd_linattn_backward_workspace_bytes(dims(*bad), 0) == 0
    for bad in ((2, 100, 4, 2, 8, 64), (2, 100, 4, 2, 64, 20), (2, 100, 4, 2, 144, 64), (2, 100, 4, 2, 64, 256)):
        assert call(bad) == -3, bad
    assert call(dtype=3) == -3 and call(dtype=-1) == -3
    for n in ("q", "k", "v", "g", "o"):
        assert call(**{n: 0}) == -1, n
    for n in ("q", "k", "v", "h0", "o", "h_final"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(g=0x10002) == -4 and call(lens=0x10002) == -4 and call(ws=0x900008) == -4
    need = lib.cssd_linattn_workspace_bytes(dims(*OK), 0)
    assert need >= 2 * 4 * 64 * 64 * 4  # a state a chunk of 128 tokens and head
    assert call(ws_bytes=need - 1) == -5


def test_linattn_backward_refusals(lib):
    def call(d=OK, dtype=0, ws_bytes=1 << 40, **kw):
        p = given(("q", "k", "v", "g", "h0", "lens", "do", "dh", "gq", "gk", "gv", "gg", "gh0"), kw)
        return lib.cssd_linattn_backward(None if d is None else dims(*d), dtype, *p[:4], 0, ctypes.c_float(1.0), *p[4:],
                                         ctypes.c_void_p(0x900000), ws_bytes, None)

    assert call(None) == -1 and call((2, 100, 4, 3, 64, 64)) == -2 and call((2, 100, 4, 2, 64, 72)) == -3 and call(dtype=9) == -3
    for n in ("q", "k", "v", "g", "do", "gq", "gk", "gv"):
        assert call(**{n: 0}) == -1, n
    for n in ("do", "dh", "gq", "gk", "gv", "gh0", "h0"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(gg=0x10002) == -4 and call(lens=0x10002) == -4
    need = lib.cssd_linattn_backward_workspace_bytes(dims(*OK), 0)
    assert need >= 2 * 2 * 4 * 64 * 64 * 4 + 2 * 2 * 100 * 4 * 64 * 4  # two states, and the parts of shared key heads
    assert call(ws_bytes=need - 1) == -5


def test_linattn_step_refusals(lib):
    def call(d=OK, dtype=1, nslots=5, **kw):
        p = given(("h", "slots", "q", "k", "v", "g", "o"), kw)
        return lib.cssd_linattn_step(None if d is None else dims(*d), dtype, p[0], nslots, *p[1:6], 1, ctypes.c_float(1.0), p[6], None)

    assert call(None) == -1 and call((0, 1, 4, 2, 64, 64)) == -2 and call((2, 1, 4, 3, 64, 64)) == -2
    assert call((2, 1, 4, 2, 63, 64)) == -3 and call(dtype=5) == -3
    assert call(nslots=0) == -2 and call(nslots=1, slots=0) == -2
    for n in ("h", "q", "k", "v", "g", "o"):
        assert call(**{n: 0}) == -1, n
    for n in ("h", "q", "k", "v", "o"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(slots=0x10002) == -4 and call(g=0x10001) == -4


def test_add_norm_refusals(lib):
    def call(rows=4, width=8, xt=0, rt=2, wt=2, kind=1, eps=1e-5, **kw):
        p = given(("x", "res", "scale", "w", "b", "s", "y", "mean", "rstd"), kw)
        return lib.cssd_add_norm(rows, width, xt, rt, wt, kind, *p[:3], ctypes.c_float(1.0), *p[3:5], ctypes.c_float(eps), *p[5:], None)

    assert call(rows=0) == -2 and call(width=0) == -2 and call(width=1 << 25) == -2 and call(rows=1 << 32) == -2
    assert call(xt=3) == -3 and call(wt=1) == -3 and call(rt=1) == -3 and call(xt=2, rt=0) == -3 and call(kind=2) == -3 and call(kind=-1) == -3
    assert call(eps=-1.0) == -2 and call(eps=float("nan")) == -2
    for n in ("x", "res", "s", "y"):
        assert call(**{n: 0}) == -1, n
    for n in ("x", "res", "scale", "w", "b", "s", "y"):
        assert call(**{n: 0x10008}) == -4, n
    assert call(mean=0x10002) == -4 and call(rstd=0x10002) == -4

    def back(rows=4, width=8, xt=0, rt=0, wt=2, kind=1, ws_bytes=1 << 40, **kw):
        p = given(("dy", "ds", "x", "s", "scale", "w", "mean", "rstd", "gx", "gres", "gscale", "gw", "gb"), kw)
        return lib.cssd_add_norm_backward(rows, width, xt, rt, wt, kind, *p[:5], ctypes.c_float(1.0), *p[5:],
                                          ctypes.c_void_p(0x900000), ws_bytes, None)

    assert back(rows=-1) == -2 and back(wt=1) == -3 and back(rt=1) == -3 and back(kind=7) == -3
    for n in ("dy", "s", "mean", "rstd", "gx", "gres", "x"):
        assert back(**{n: 0}) == -1, n
    assert back(mean=0, kind=0, ws_bytes=8) == -5 and back(x=0, gscale=0, ws_bytes=8) == -5  # not needed there
    for n in ("dy", "ds", "x", "s", "scale", "w", "gx", "gres", "gscale", "gw", "gb"):
        assert back(**{n: 0x10008}) == -4, n
    assert back(rstd=0x10002) == -4 and back(ws_bytes=8) == -5
    assert lib.cssd_add_norm_backward_workspace_bytes(0, 8) == 0


def test_gated_norm_refusals(lib):
    def call(rows=4, width=8, group=4, xt=0, wt=2, kind=1, eps=1e-5, **kw):
        p = given(("x", "z", "w", "b", "y", "mean", "rstd"), kw)
        return lib.cssd_gated_norm(rows, width, group, xt, wt, kind, 0, *p[:4], ctypes.c_float(eps), *p[4:], None)

    assert call(rows=0) == -2 and call(width=0) == -2 and call(group=0) == -2 and call(group=3) == -2 and call(group=16) == -2
    assert call(group=-4) == -2 and call(rows=1 << 30, width=16, group=1) == -2
    assert call(xt=3) == -3 and call(wt=1) == -3 and call(kind=2) == -3 and call(eps=-1.0) == -2
    for n in ("x", "z", "y"):
        assert call(**{n: 0}) == -1, n
    for n in ("x", "z", "w", "b", "y"):
        assert call(**{n: 0x10008}) == -4, n

    def back(rows=4, width=8, group=8, xt=0, wt=2, kind=0, ws_bytes=1 << 40, **kw):
        p = given(("dy", "x", "z", "w", "b", "mean", "rstd", "gx", "gz", "gw", "gb"), kw)
        return lib.cssd_gated_norm_backward(rows, width, group, xt, wt, kind, 1, *p, ctypes.c_void_p(0x900000), ws_bytes, None)

    assert back(group=5) == -2 and back(wt=1) == -3 and back(kind=3) == -3
    for n in ("dy", "x", "z", "rstd", "gx", "gz"):
        assert back(**{n: 0}) == -1, n
    assert back(mean=0, kind=1) == -1
    for n in ("dy", "x", "z", "w", "b", "gx", "gz", "gw", "gb"):
        assert back(**{n: 0x10008}) == -4, n
    assert back(ws_bytes=8) == -5
    assert lib.cssd_gated_norm_backward_workspace_bytes(4, 8, 3) == 0


def test_binding_rejects_wrong_tensors():
    q, g = torch.zeros(1, 8, 2, 16), torch.zeros(1, 8, 2)
    for bad in ((q.double(), q.double(), q.double(), g), (q, q.half(), q, g), (q, q, q, g.half()), (q, q, q, None)):
        with pytest.raises(TypeError):
            cssd.linattn_forward(*bad)
    for bad in ((q, q[:, :4], q, g), (q, q, q.transpose(1, 2).contiguous().transpose(1, 2), g), (q, q, q, torch.zeros(3)),
                (q, q, q, torch.zeros(8, 2)), (q[0], q[0], q, g)):
        with pytest.raises(ValueError):
            cssd.linattn_forward(*bad)
    with pytest.raises(ValueError):
        cssd.linattn_forward(q, q, q, g, h0=torch.zeros(1, 2, 16, 15))
    with pytest.raises(TypeError):
        cssd.linattn_forward(q, q, q, g, lens=torch.zeros(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        cssd.linattn_backward(q, q, q, g, q[:, :4])
    with pytest.raises(ValueError):
        cssd.linattn_step(torch.zeros(1, 2, 16, 8), q[:, 0], q[:, 0], q[:, 0], g[:, 0])
    with pytest.raises(ValueError):
        cssd.linattn_step(torch.zeros(1, 2, 16, 16), q[:, 0], q[:, 0], q[:, 0], torch.zeros(3))
    x, h = torch.zeros(4, 8), torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(TypeError):
        cssd.add_norm(x, h)
    with pytest.raises(TypeError):
        cssd.add_norm(h, h, torch.zeros(8), torch.zeros(8, dtype=torch.float16))
    with pytest.raises(TypeError):
        cssd.add_norm(h, h, torch.zeros(8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="kind"):
        cssd.add_norm(x, x, kind="batch")
    with pytest.raises(ValueError):
        cssd.add_norm(x, x[:2])
    with pytest.raises(ValueError):
        cssd.add_norm(x, x, scale=torch.zeros(7))
    with pytest.raises(ValueError, match="gscale"):
        cssd.add_norm_backward(x, None, None, x, None, None, torch.zeros(4), scale=torch.zeros(8))
    with pytest.raises(ValueError):
        cssd.add_norm_backward(x, None, x, x, None, torch.zeros(3), torch.zeros(4))
    with pytest.raises(ValueError, match="group"):
        cssd.gated_norm(x, x, group=3)
    with pytest.raises(TypeError):
        cssd.gated_norm(x, h)
    with pytest.raises(ValueError):
        cssd.gated_norm_backward(x, x, x, None, None, None, torch.zeros(4), group=4)
    with pytest.raises(ValueError, match="CUDA device"):
        cssd.gated_norm(x, x, group=4)
    with pytest.raises(ValueError, match="CUDA device"):
        cssd.add_norm_backward(h, None, None, h, None, None, torch.zeros(4), wdtype=torch.float32)
    with pytest.raises(TypeError):
        cssd.add_norm_backward(h, None, None, h, None, None, torch.zeros(4), wdtype=torch.bfloat16)


def test_linattn_longest_sequences(lib):
    """A length that rounded up to chunks of 128 tokens leaves 32 bits is refused, by both calls and their sizes."""
    for dtype in (0, 1, 2):
        for T, ok in (((1 << 31) - 128, True), ((1 << 31) - 127, False), ((1 << 31) - 65, False)):
            d = dims(1, T, 1, 1, 16, 16)
            assert (lib.cssd_linattn_workspace_bytes(d, dtype) > 0) == ok and (lib.cssd_linattn_backward_workspace_bytes(d, dtype) > 0) == ok
            if not ok:
                p = ptrs(13)
                assert lib.cssd_linattn_forward(d, dtype, *p[:4], 1, ctypes.c_float(1.0), *p[4:8], None, 0, None) == -2
                assert lib.cssd_linattn_backward(d, dtype, *p[:4], 1, ctypes.c_float(1.0), *p[4:], None, 0, None) == -2
