"""Memory of the results of a call on a stream of the caller's (`stream=`).

A result dropped while that stream still writes it must not become another
tensor of the current stream, and a result that the current stream still reads
must not be written again by the next call on the caller's stream."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cs():
    from complex_valued_state_gb300 import build as cbuild
    from complex_valued_state_gb300 import cssd

    if not torch.cuda.is_available():
        pytest.fail("CUDA device required for gpu tests")
    cbuild.build()
    cssd.load()
    return cssd


def calls(cs):
    """Name -> a call that takes `stream` and returns its results."""
    B, T, H, N, P = 1, 70, 2, 64, 64
    half = [torch.randn(B, T, H, n, device="cuda", dtype=torch.bfloat16) * 0.1 for n in (N, N, P, P)]
    q, k, v, do = half
    g, beta = -torch.rand(B, T, H, device="cuda"), torch.rand(B, T, H, device="cuda")
    state = torch.zeros(B, H, N, P, device="cuda")
    token = [t[:, 0].contiguous() for t in (q, k, v, g, beta)]
    x = torch.randn(300, 256, device="cuda")
    y, mean, rstd = cs.layernorm(x)
    c = [torch.randn(B, T, H, n, device="cuda", dtype=torch.complex64) for n in (P, N, N)]
    A, D, dt = torch.full((H,), -1 + 1j, device="cuda", dtype=torch.complex64), torch.ones(H, device="cuda"), 0.1 * torch.rand(B, T, H, device="cuda")
    ssd = (c[0], dt, A, c[1], c[2], D)
    one = (c[0][:, 0].contiguous(), dt[:, 0].contiguous(), A, c[1][:, 0].contiguous(), c[2][:, 0].contiguous(), D)
    cstate = torch.zeros(B, H, N, P, device="cuda", dtype=torch.complex64)
    angle = torch.rand(B, T, H, N, device="cuda")
    attn = [torch.randn(B, T, H, 16, device="cuda", dtype=torch.complex64) for _ in range(3)]
    return {
        "delta_forward": lambda s: cs.delta_forward(q, k, v, g, beta, stream=s),
        "delta_backward": lambda s: tuple(cs.delta_backward(q, k, v, g, beta, do, stream=s).values()),
        "delta_step": lambda s: (cs.delta_step(state, *token, stream=s),),
        "layernorm": lambda s: cs.layernorm(x, stream=s),
        "layernorm_backward": lambda s: tuple(cs.layernorm_backward(x, x, None, mean, rstd, stream=s).values()),
        "chunked_forward": lambda s: cs.chunked_forward(*ssd, stream=s),
        "chunked_forward_noalloc": lambda s: cs.chunked_forward_noalloc(*ssd, stream=s),
        "chunked_backward": lambda s: tuple(cs.chunked_backward(*ssd, c[0], stream=s).values()),
        "step": lambda s: (cs.step(cstate, *one, stream=s),),
        "step_n": lambda s: (cs.step_n(cstate, *one, 3, stream=s),),
        "step_infinite": lambda s: (cs.step_infinite(*one, stream=s),),
        "cayley_scan": lambda s: cs.cayley_scan(angle, angle, c[1], c[2], stream=s),
        "born_attention": lambda s: (cs.born_attention(*attn, stream=s),),
    }


NAMES = ["delta_forward", "delta_backward", "delta_step", "layernorm", "layernorm_backward", "chunked_forward",
         "chunked_forward_noalloc", "chunked_backward", "step", "step_n", "step_infinite", "cayley_scan", "born_attention"]


@pytest.mark.parametrize("name", NAMES)
def test_dropped_results_stay_with_their_stream(cs, name):
    call = calls(cs)[name]
    call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results = call(side)
    like = [(t.shape, t.dtype, t.data_ptr()) for t in results]
    del results
    others = [[torch.empty(shape, dtype=dtype, device="cuda") for _ in range(4)] for shape, dtype, _ in like]
    ours = {p for _, _, p in like}
    assert not any(t.data_ptr() in ours for group in others for t in group), name
    side.synchronize()


@pytest.mark.parametrize("name", NAMES)
def test_results_being_read_are_not_written(cs, name):
    call = calls(cs)[name]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results = call(side)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(400_000_000)  # (a fifth of a second) the current stream is busy, then reads them
    kept = [t.clone() for t in results]
    ours = {t.data_ptr() for t in results}
    del results
    again = call(side)
    assert not any(t.data_ptr() in ours for t in again), name
    torch.cuda.synchronize()
    assert len(kept) == len(again)


@pytest.mark.parametrize("name", ["delta_forward", "delta_backward", "layernorm", "layernorm_backward", "chunked_forward"])
def test_side_stream_in_a_captured_graph(cs, name):
    call = calls(cs)[name]
    want = call(None)
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        got = call(side)
        torch.cuda.current_stream().wait_stream(side)
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b), name
