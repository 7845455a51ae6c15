"""8-bit output of rows of zeros with eps = 0, and of rows that hold a NaN or an
infinity: every scale and code of such a row, on every kernel (needs a GPU).

The codes of ordinary rows and groups are compared with the same float32
operations in torch, bit for bit: no order of a sum changes them."""
import pytest
import torch

import rmsnorm_backward_gb300 as gbn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
# short rows of vectors and of elements, one and several groups; ring rows of
# all vectors, of fewer, and across 16-byte boundaries
WIDTHS = [(64, "auto"), (100, "auto"), (256, "auto"), (391, "auto"), (1024, "auto"), (4096, "auto"), (4808, "auto"),
          (4099, "auto"), (1024, "plain"), (517, "plain")]


def codes(v, q_dtype, group):
    """(codes, maxima) of float32 v, for rows (groups) of finite values."""
    top = 448.0 if q_dtype == torch.float8_e4m3fn else 127.0
    M, N = v.shape
    parts = torch.nn.functional.pad(v, (0, -N % (group or N))).view(M, -1, group or N)
    a = parts.abs().amax(-1)
    factor = torch.where(a == 0, torch.zeros_like(a), torch.full_like(a, top) / a)
    code = (parts * factor[..., None]).view(M, -1)[:, :N]
    return (code.to(q_dtype) if q_dtype == torch.float8_e4m3fn else code.round().to(q_dtype)), a


def call(x, gamma, eps, res, **kw):
    if res:  # 3/4 and 1/4 of x: exact in every type here
        q, scale, h, rstd = gbn.rms_add_fwd_q8(x * 0.75, x * 0.25, gamma, eps, **kw)
    else:
        q, scale, rstd = gbn.rms_fwd_q8(x, gamma, eps, **kw)
    return q.cpu(), scale.cpu(), rstd.cpu()


def values(M, N, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randint(-20, 21, (M, N), generator=g).float() * 4).to(DT[dtype])  # quarters are exact
    gamma = (1 + 0.1 * torch.randn(N, generator=g)).to(DT[dtype])
    return x, gamma


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("q_dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,kernel", WIDTHS)
def test_rows_of_zeros_without_eps(N, kernel, dtype, q_dtype, group, res):
    x, gamma = values(9, N, dtype, N)
    x[2] = 0
    x[5, : N // 2] = 0   # a group of zeros, where there are several
    x[8] = 0
    q, scale, rstd = call(x.cuda(), gamma.cuda(), 0.0, res, q_dtype=q_dtype, group=group, kernel=kernel)
    want, a = codes(gamma.float() * x.float(), q_dtype, group)
    assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
    assert torch.isinf(rstd[[2, 8]]).all()
    scale = scale.view(9, -1)
    assert (scale[[2, 8]] == 0).all() and (scale[a == 0] == 0).all()
    assert (scale[a > 0] > 0).all() and torch.isfinite(scale).all()


@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("q_dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N,kernel", WIDTHS)
def test_rows_that_hold_a_nan_or_an_infinity(N, kernel, dtype, q_dtype, group, res):
    e4m3 = q_dtype == torch.float8_e4m3fn
    x, gamma = values(7, N, dtype, N + 1)
    clean = x.clone()
    spots = {1: (N // 2, float("nan")), 2: (0, float("inf")), 4: (N - 1, -float("inf")), 5: (N // 3, float("nan"))}
    x[5, N - N // 4:] = 0  # zeros beside a NaN
    clean[5, N - N // 4:] = 0
    for r, (c, bad) in spots.items():
        x[r, c] = bad
    q, scale, rstd = call(x.cuda(), gamma.cuda(), 1e-6, res, q_dtype=q_dtype, group=group, kernel=kernel)
    scale = scale.view(7, -1)
    width = group or N
    plain, _ = codes(gamma.float() * clean.float(), q_dtype, group)
    value, bits, plain = q.float(), q.view(torch.uint8), plain.view(torch.uint8)
    for r in range(7):
        if r not in spots:
            assert torch.equal(bits[r], plain[r])
            assert torch.isfinite(scale[r]).all()
            continue
        c, bad = spots[r]
        at = c // width                                   # the group that holds it
        own = slice(at * width, min(N, (at + 1) * width))
        others = torch.ones(N, dtype=torch.bool)
        others[own] = False
        assert torch.equal(bits[r][others], plain[r][others])
        rest = torch.arange(scale.shape[1]) != at
        if bad != bad:
            assert torch.isnan(rstd[r]) and torch.isnan(scale[r]).all()
            assert torch.isnan(value[r, own]).all() if e4m3 else (value[r, own] == 0).all()
        else:
            assert rstd[r] == 0 and torch.isnan(scale[r, at]) and (scale[r, rest] == 0).all()
            assert torch.isnan(value[r, c]) if e4m3 else value[r, c] == 0
            finite = [i for i in range(own.start, own.stop) if i != c]
            assert (value[r, finite] == 0).all()


@pytest.mark.parametrize("N", [64, 1024, 4099])
def test_squares_above_float32(N):
    """Finite values whose squares' sum is not a float32: rstd and scales are 0."""
    x, gamma = values(3, N, "f32", 3)
    x[1] *= 1e30
    for group in (0, 128):
        q, scale, rstd = call(x.cuda(), gamma.cuda(), 1e-6, False, group=group)
        assert rstd[1] == 0 and (scale.view(3, -1)[1] == 0).all()
        want, _ = codes(gamma.float() * x.float(), q.dtype, group)
        assert torch.equal(q.view(torch.uint8), want.view(torch.uint8))
