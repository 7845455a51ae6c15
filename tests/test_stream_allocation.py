"""What a call with stream= allocates or fills belongs to that stream (no GPU
needed: CPU tensors that say they are on a GPU, streams and a library that
only record)."""
import contextlib

import pytest
import torch

import rmsnorm_backward_gb300 as gbn

DEVICE = torch.device("cuda", 0)
_empty, _zeros, _empty_like = torch.empty, torch.zeros, torch.empty_like


class Here(torch.Tensor):
    """A CPU tensor that says it is on DEVICE."""

    is_cuda = property(lambda self: True)
    device = property(lambda self: DEVICE)

    def get_device(self):
        return 0

    def record_stream(self, stream):
        self.in_use = getattr(self, "in_use", []) + [stream]


class Stream:
    def __init__(self, cuda_stream):
        self.cuda_stream = cuda_stream


class Recorder:
    """Streams, allocations and library calls."""

    def __init__(self):
        self.current = self.default = Stream(0)
        self.made = []   # (tensor, stream current at the time)
        self.calls = []  # (function, stream handle)

    def make(self, what):
        def call(*args, device=None, pin_memory=False, **kw):
            t = what(*args, **kw)
            if device is not None or what is _empty_like:
                t = t.as_subclass(Here)
                self.made.append((t, self.current))
            return t
        return call

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s
        yield
        self.current = before

    def __getattr__(self, name):  # the library's functions
        def call(*args):
            if name.endswith("workspace_bytes") or name.endswith("workspace_bytes_ex"):
                return 96
            if name != "gbn_grad_check":
                self.calls.append((name, args[-1]))
            return 0
        return call


@pytest.fixture
def rec(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(torch, "empty", r.make(_empty))
    monkeypatch.setattr(torch, "zeros", r.make(_zeros))
    monkeypatch.setattr(torch, "empty_like", r.make(_empty_like))
    monkeypatch.setattr(torch.cuda, "stream", r.stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: r.current)
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: r.default)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: Stream(handle))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", lambda d: contextlib.nullcontext())
    monkeypatch.setattr(gbn, "_raw_stream", lambda index: r.current.cuda_stream)
    monkeypatch.setattr(gbn, "_lib", r)
    return r


M, N = 4, 64


def rows():
    return torch.ones(M, N).as_subclass(Here)


def vec(n=N):
    return torch.ones(n).as_subclass(Here)


def host(n=M):
    return torch.ones(n, N)


CALLS = {
    "ln_fwd": lambda s: gbn.ln_fwd(rows(), vec(), vec(), 1e-6, stream=s),
    "rms_fwd": lambda s: gbn.rms_fwd(rows(), vec(), 1e-6, stream=s),
    "ln_bwd": lambda s: gbn.ln_bwd(rows(), rows(), vec(), vec(M), vec(M), stream=s),
    "ln_bwd accumulate": lambda s: gbn.ln_bwd(rows(), rows(), vec(), vec(M), vec(M), accumulate=True, stream=s),
    "rms_bwd": lambda s: gbn.rms_bwd(rows(), rows(), vec(), vec(M), stream=s),
    "rms_bwd accumulate": lambda s: gbn.rms_bwd(rows(), rows(), vec(), vec(M), accumulate=True, stream=s),
    "ln_bwd_rows": lambda s: gbn.ln_bwd_rows(rows(), rows(), vec(), vec(M), vec(M), workspace=vec(), stream=s),
    "rms_bwd_rows": lambda s: gbn.rms_bwd_rows(rows(), rows(), vec(), vec(M), workspace=vec(), stream=s),
    "silu_bwd": lambda s: gbn.silu_bwd(rows(), rows(), stream=s),
    "gelu_bwd": lambda s: gbn.gelu_bwd(rows(), rows(), stream=s),
    "rms_add_fwd": lambda s: gbn.rms_add_fwd(rows(), rows(), vec(), 1e-6, stream=s),
    "rms_fwd_q8": lambda s: gbn.rms_fwd_q8(rows(), vec(), 1e-6, stream=s),
    "rms_add_fwd_q8": lambda s: gbn.rms_add_fwd_q8(rows(), rows(), vec(), 1e-6, group=128, stream=s),
    "rms_add_bwd": lambda s: gbn.rms_add_bwd(rows(), rows(), rows(), vec(), vec(M), stream=s),
    "rms_add_bwd accumulate": lambda s: gbn.rms_add_bwd(rows(), rows(), rows(), vec(), vec(M), accumulate=True, stream=s),
    "grad_norm": lambda s: gbn.grad_norm([rows(), vec()], stream=s),
    "grad_clip": lambda s: gbn.grad_clip([rows(), vec()], 1.0, stream=s),
    "ln_bwd_host": lambda s: gbn.ln_bwd_host(host(), host(), host()[0], host()[:, 0].contiguous(),
                                             host()[:, 0].contiguous(), device=DEVICE, stream=s),
    "rms_bwd_host": lambda s: gbn.rms_bwd_host(host(), host(), host()[0], host()[:, 0].contiguous(), device=DEVICE,
                                               stream=s),
    "silu_bwd_host": lambda s: gbn.silu_bwd_host(host(), host(), device=DEVICE, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("kind", ["stream", "handle", "default", "none"])
def test_what_a_call_allocates_is_its_streams(rec, name, kind):
    outer = rec.current = Stream(0x1000)
    given = {"stream": Stream(0x2000), "handle": 0x3000, "default": 0, "none": None}[kind]
    want = {"stream": 0x2000, "handle": 0x3000, "default": 0, "none": 0x1000}[kind]
    CALLS[name](given)
    assert rec.current is outer
    assert [h for _, h in rec.calls] == [want]
    assert rec.made, "nothing was allocated"
    for t, s in rec.made:
        assert s.cuda_stream == want, f"{tuple(t.shape)} was allocated on another stream than the call's"
        # and the caller's stream, which goes on with it, keeps it from being given out again too early
        assert kind == "none" or outer in getattr(t, "in_use", [])
