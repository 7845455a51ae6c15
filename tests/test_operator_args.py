"""Refusals of the residual / 8-bit RMSNorm, its backward, the gradient norm
and the clip: bad arguments are errors on the host, before anything is
enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

import rmsnorm_backward_gb300 as gbn

OK, EINVAL, EDTYPE = 0, 1, 2
BF16, E4M3, INT8 = 2, 16, 17


@pytest.fixture(scope="module")
def lib():
    from rmsnorm_backward_gb300 import build
    build.build()
    return gbn.lib()


def at(address):
    """A device address that is only compared, never read."""
    return ctypes.c_void_p(address)


X, R, G, Y, H, S, C = (at(0x100000 * i) for i in range(1, 8))


def add_fwd(lib, x=X, r=R, g=G, y=Y, h=H, rstd=S, eps=1e-6, M=4, N=8, dtype=BF16, ld=(0, 0, 0, 0), kernel=0):
    return lib.rms_add_fwd(x, r, g, y, h, rstd, eps, M, N, dtype, *ld, kernel, None)


def add_q8(lib, x=X, r=R, g=G, q=Y, scale=C, h=H, rstd=S, eps=1e-6, M=4, N=8, dtype=BF16, q_dtype=E4M3, group=0,
           ld=(0, 0, 0, 0), kernel=0):
    return lib.rms_add_fwd_q8(x, r, g, q, scale, h, rstd, eps, M, N, dtype, q_dtype, group, *ld, kernel, None)


def q8(lib, x=X, g=G, q=Y, scale=C, rstd=S, eps=1e-6, M=4, N=8, dtype=BF16, q_dtype=E4M3, group=0, ld=(0, 0), kernel=0):
    return lib.rms_fwd_q8(x, g, q, scale, rstd, eps, M, N, dtype, q_dtype, group, *ld, kernel, None)


@pytest.mark.parametrize("call", [add_fwd, add_q8, q8])
def test_forward_arguments(lib, call):
    assert call(lib, M=0) == OK  # nothing to do, no device needed
    assert call(lib, M=-1) == EINVAL
    assert call(lib, N=0) == EINVAL
    assert call(lib, N=(1 << 24) + 1) == EINVAL
    assert call(lib, dtype=3) == EDTYPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(lib, eps=eps) == EINVAL
    for kernel in (1, 3, -1):
        assert call(lib, kernel=kernel) == EINVAL
    assert call(lib, x=None) == EINVAL
    assert call(lib, g=None) == EINVAL
    assert call(lib, rstd=None) == EINVAL
    strides = 2 if call is q8 else 4
    for i in range(strides):
        assert call(lib, ld=tuple(7 if j == i else 0 for j in range(strides))) == EINVAL


@pytest.mark.parametrize("call", [add_fwd, add_q8, q8])
def test_addresses_and_reach(lib, call):
    for k in ("x", "g", "rstd"):
        assert call(lib, **{k: at(0x100001)}) == EINVAL  # between two elements
    far = (1 << 60, 0) if call is q8 else (1 << 60, 0, 0, 0)
    assert call(lib, ld=far) == EINVAL  # rows beyond 64 bits


@pytest.mark.parametrize("call", [add_q8, q8])
def test_quantization_arguments(lib, call):
    assert call(lib, q_dtype=BF16) == EDTYPE
    assert call(lib, group=64) == EINVAL
    assert call(lib, group=-1) == EINVAL
    assert call(lib, scale=None) == EINVAL
    assert call(lib, q=None) == EINVAL


def test_forward_overlaps(lib):
    assert add_fwd(lib, h=Y) == EINVAL                         # y and h in one place
    assert add_fwd(lib, y=at(X.value + 16)) == EINVAL          # y one row into x
    assert add_fwd(lib, h=R, ld=(0, 16, 0, 0)) == EINVAL       # h on residual, other stride
    assert add_fwd(lib, h=at(R.value - 2)) == EINVAL           # one element into residual's first
    assert add_fwd(lib, y=X, h=X) == EINVAL
    assert add_q8(lib, q=X) == EINVAL                          # codes are narrower than x's rows
    assert add_q8(lib, q=H) == EINVAL
    assert q8(lib, q=at(X.value + 63)) == EINVAL               # the last byte of x
    # rows that interleave in one wider buffer, and reach into one another
    ld16 = (16, 0, 16, 0)
    assert add_fwd(lib, y=at(X.value + 14), ld=ld16, M=4) == EINVAL
    assert add_fwd(lib, y=at(X.value + 18), ld=ld16, M=4) == EINVAL


def add_bwd(lib, dy=X, dh=R, h=H, g=G, rstd=S, dx=Y, dg=C, M=4, N=8, dtype=BF16, ws=at(0x10000000), wsb=1 << 30,
            ld_dh=0, **opt):
    o = gbn.GbnOptions()
    for k, v in opt.items():
        setattr(o, k, v)
    return lib.rms_add_bwd(dy, dh, h, g, rstd, dx, dg, M, N, dtype, ws, wsb, ld_dh, ctypes.byref(o), None)


def test_backward_arguments(lib):
    for name in ("dy", "dh", "h", "g", "rstd", "dx", "dg", "ws"):
        assert add_bwd(lib, **{name: None}) == EINVAL
    assert add_bwd(lib, M=-1) == EINVAL
    assert add_bwd(lib, N=0) == EINVAL
    assert add_bwd(lib, dtype=9) == EDTYPE
    assert add_bwd(lib, ld_dh=7) == EINVAL
    assert add_bwd(lib, ld_x=7) == EINVAL
    assert add_bwd(lib, accumulate=2) == EINVAL
    assert add_bwd(lib, grad_dtype=1) == EDTYPE
    assert add_bwd(lib, reduce_mode=1) == EINVAL
    assert add_bwd(lib, kernel=1) == EINVAL
    assert add_bwd(lib, host_chunk=8) == EINVAL
    assert add_bwd(lib, dx=at(X.value + 2)) == EINVAL
    assert add_bwd(lib, dx=at(R.value + 16)) == EINVAL
    assert add_bwd(lib, dx=H, ld_out=9) == EINVAL
    assert add_bwd(lib, dy=at(0x100001)) == EINVAL
    assert add_bwd(lib, dg=at(0x700002)) == EINVAL
    assert add_bwd(lib, ld_dh=1 << 60) == EINVAL


def table(*entries):
    t = (gbn._GbnTensor * max(1, len(entries)))()
    for e, (p, n, d) in zip(t, entries):
        e.data, e.n, e.dtype = p, n, d
    return t


def test_gradient_arguments(lib):
    good = table((0x1000, 16, 0), (0x2000, 5, 2))
    norm, ws = at(0x100), at(0x10000)
    for call in (lambda t, n, **k: lib.gbn_grad_norm(t, n, k.get("norm", norm), k.get("ws", ws), 1 << 20, None),
                 lambda t, n, **k: lib.gbn_grad_clip(t, None, n, 1.0, 0.0, k.get("norm", norm), k.get("ws", ws),
                                                     1 << 20, None)):
        assert call(good, -1) == EINVAL
        assert call(None, 2) == EINVAL
        assert call(good, 2, norm=None) == EINVAL
        assert call(good, 2, ws=None) == EINVAL
        assert call(good, 2, norm=at(0x102)) == EINVAL
        assert call(table((0x1002, 4, 0)), 1) == EINVAL      # not aligned to its element
        assert call(table((0x1001, 4, 1)), 1) == EINVAL
        assert call(table((0, 4, 1)), 1) == EINVAL           # no address
        assert call(table((0x1000, -4, 1)), 1) == EINVAL
        assert call(table((0x1000, 4, 16)), 1) == EINVAL     # not a gradient's type
    for limit, eps in ((-1.0, 0.0), (float("nan"), 0.0), (1.0, -1.0), (1.0, float("nan"))):
        assert lib.gbn_grad_clip(good, None, 2, limit, eps, norm, ws, 1 << 20, None) == EINVAL
    for out in (table((0x9000, 16, 0), (0xa000, 4, 2)), table((0x9000, 16, 1), (0xa000, 5, 2))):
        assert lib.gbn_grad_clip(good, out, 2, 1.0, 0.0, norm, ws, 1 << 20, None) == EINVAL


def test_gradient_overlaps(lib):
    assert lib.gbn_grad_check(None, 0) == OK
    assert lib.gbn_grad_check(table((0x1000, 16, 0), (0x1040, 5, 2), (0x1000, 0, 0)), 3) == OK
    assert lib.gbn_grad_check(table((0x1040, 5, 2), (0x1000, 17, 0)), 2) == EINVAL
    assert lib.gbn_grad_check(table((0x1000, 16, 0), (0x1000, 16, 0)), 2) == EINVAL


def test_python_refuses_cpu_tensors_and_unknown_choices():
    x, g = torch.randn(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        gbn.rms_add_fwd(x, x, g, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        gbn.rms_fwd_q8(x, g, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        gbn.rms_add_fwd_q8(x, x, g, 1e-6)
    with pytest.raises(ValueError, match="CUDA"):
        gbn.rms_add_bwd(x, x, x, g, torch.ones(4))
    with pytest.raises(ValueError, match="CUDA"):
        gbn.GradList([x])
    with pytest.raises(ValueError, match="CUDA"):
        gbn.grad_norm([x, g])
    with pytest.raises(ValueError, match="CUDA"):
        gbn.grad_clip([x], 1.0)


def test_dense_layouts():
    t = torch.empty(4, 6, 8)
    assert gbn._dense(t) and gbn._dense(t.transpose(0, 2)) and gbn._dense(t[1:3]) and gbn._dense(t[:, :1, 0:8][0])
    assert gbn._dense(torch.empty(0, 5)) and gbn._dense(torch.empty(()))
    assert not gbn._dense(t[:, ::2]) and not gbn._dense(t[:, :3]) and not gbn._dense(torch.empty(3).expand(2, 3))
