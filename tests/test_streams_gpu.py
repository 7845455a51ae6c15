"""Calls on another stream than the current one, with work queued on both and
nothing in between (needs a GPU).  The calls of the two streams have inputs of
their own, so that memory which both use at once shows: every result is
compared, bit for bit, with the same call's made alone."""
import pytest
import torch

import rmsnorm_backward_gb300 as gbn

pytestmark = pytest.mark.gpu

M, N, EPS = 8192, 4096, 1e-6
BUSY = 20_000_000  # clock cycles of a kernel that does nothing else: about 10 ms


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {k: torch.randn(M, N, generator=g, device="cuda").to(torch.bfloat16) for k in ("x", "residual", "dy", "dh")}
    t["gamma"] = (1 + 0.1 * torch.randn(N, generator=g, device="cuda")).to(torch.bfloat16)
    t["beta"] = (0.1 * torch.randn(N, generator=g, device="cuda")).to(torch.bfloat16)
    t["y"], t["h"], t["rstd"] = gbn.rms_add_fwd(t["x"], t["residual"], t["gamma"], EPS)
    _, t["mean"], t["rstd_ln"] = gbn.ln_fwd(t["x"], t["gamma"], t["beta"], EPS)
    return t


def tensors(out):
    return out if isinstance(out, tuple) else (out,)


CALLS = {
    "rms_fwd": lambda t, **k: gbn.rms_fwd(t["x"], t["gamma"], EPS, **k),
    "ln_fwd": lambda t, **k: gbn.ln_fwd(t["x"], t["gamma"], t["beta"], EPS, **k),
    "rms_bwd": lambda t, **k: gbn.rms_bwd(t["dy"], t["h"], t["gamma"], t["rstd"], **k),
    "rms_bwd accumulate": lambda t, **k: gbn.rms_bwd(t["dy"], t["h"], t["gamma"], t["rstd"], accumulate=True, **k),
    "ln_bwd": lambda t, **k: gbn.ln_bwd(t["dy"], t["x"], t["gamma"], t["mean"], t["rstd_ln"], **k),
    "rms_add_fwd": lambda t, **k: gbn.rms_add_fwd(t["x"], t["residual"], t["gamma"], EPS, **k),
    "rms_add_fwd_q8": lambda t, **k: tuple(a.view(torch.uint8) if a.element_size() == 1 else a for a in gbn.rms_add_fwd_q8(
        t["x"], t["residual"], t["gamma"], EPS, group=128, **k)),
    "rms_add_bwd": lambda t, **k: gbn.rms_add_bwd(t["dy"], t["dh"], t["h"], t["gamma"], t["rstd"], **k),
    "rms_add_bwd accumulate": lambda t, **k: gbn.rms_add_bwd(t["dy"], t["dh"], t["h"], t["gamma"], t["rstd"],
                                                             accumulate=True, **k),
    "grad_norm": lambda t, **k: gbn.grad_norm([t["dy"], t["dh"], t["gamma"]], **k),
    "grad_clip": lambda t, **k: gbn.grad_clip([t["dy"], t["dh"]], 1e9, **k),
}


@pytest.fixture(scope="module")
def two():
    pair = inputs(1), inputs(2)
    torch.cuda.synchronize()
    return pair


@pytest.mark.parametrize("name", CALLS)
def test_a_call_on_each_stream(name, two):
    """A call on the current stream, whose workspace is let go at once, then the other inputs' on a side stream."""
    call, (a, b) = CALLS[name], two
    want_a, want_b = ([o.clone() for o in tensors(call(t))] for t in (a, b))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        torch.cuda._sleep(BUSY // 20)  # the first call waits on its stream while the second is queued
        got_a = tensors(call(a))
        del got_a
        got_a = tensors(call(a))
        got_b = tensors(call(b, stream=side))
        got_c = tensors(call(b, stream=side.cuda_stream))
        torch.cuda.synchronize()
        for got, want in ((got_a, want_a), (got_b, want_b), (got_c, want_b)):
            assert all(torch.equal(x, y) for x, y in zip(got, want))


@pytest.mark.parametrize("name", [n for n in CALLS if "accumulate" in n])
def test_accumulated_from_nothing_beside_a_busy_stream(name, two):
    """No dgamma given: it starts at zero on the call's own stream, whatever the current one still has to do."""
    call, (a, _) = CALLS[name], two
    want = [o.clone() for o in tensors(call(a))]
    filled = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # memory to come by is not zeros
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    del filled
    torch.cuda._sleep(BUSY)
    got = tensors(call(a, stream=side))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_results_that_are_let_go_while_the_current_stream_reads_them(two):
    """A side stream's result, read on the current stream and dropped, is not given out again before that read."""
    a, b = two
    side = torch.cuda.Stream()
    want = CALLS["rms_add_fwd"](a)[0].clone()
    for _ in range(3):
        torch.cuda.synchronize()
        y, h, rstd = gbn.rms_add_fwd(a["x"], a["residual"], a["gamma"], EPS, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(BUSY // 4)
        copy = y.clone()
        del y, h, rstd
        for _ in range(2):  # of the same sizes, at once on the side stream
            gbn.rms_add_fwd(b["x"], b["residual"], b["gamma"], EPS, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(copy, want)


def test_a_side_stream_of_a_capture(two):
    a, b = two
    side = torch.cuda.Stream()
    t = {k: v.clone() for k, v in a.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        side.wait_stream(torch.cuda.current_stream())
        on_side = gbn.rms_add_bwd(t["dy"], t["dh"], t["h"], t["gamma"], t["rstd"], accumulate=True, stream=side)
        here = gbn.rms_add_fwd(t["x"], t["residual"], t["gamma"], EPS)
        norm = gbn.grad_norm([t["dy"]], stream=side)
        torch.cuda.current_stream().wait_stream(side)
    for k in t:
        t[k].copy_(b[k])
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for got, want in ((on_side, CALLS["rms_add_bwd"](b)), (here, CALLS["rms_add_fwd"](b)),
                      ((norm,), (gbn.grad_norm([b["dy"]]),))):
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_the_default_streams_handle_while_another_is_current(two):
    a, _ = two
    want = [o.clone() for o in CALLS["rms_add_bwd"](a)]
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = CALLS["rms_add_bwd"](a, stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
