"""Statistics, scales and weights over the rows that a call writes or reads, or
over one another, are refused on the host, as the header says (no GPU needed);
beside them, between two rows too, they are taken (needs a GPU)."""
import ctypes

import pytest
import torch

import rmsnorm_backward_gb300 as gbn
from test_operator_args import BF16, EINVAL, C, G, H, R, S, X, Y, add_bwd, add_fwd, add_q8, at, lib, q8  # noqa: F401

M, N = 4, 8           # rows of 16 bytes, rstd and a row's scales of 16 bytes
ROWS = M * N * 2


@pytest.mark.parametrize("call,name", [(add_fwd, n) for n in ("x", "r", "y", "h")] +
                         [(add_q8, n) for n in ("x", "r", "q", "h")] + [(q8, n) for n in ("x", "q")])
def test_statistics_over_rows(lib, call, name):
    base = {"x": X, "r": R, "y": Y, "q": Y, "h": H}[name].value
    end = base + (M * N if name == "q" else ROWS)
    spots = (base, base + 16, base - 12, end - 4)
    for spot in spots:
        assert call(lib, rstd=at(spot)) == EINVAL, hex(spot)
        if call is not add_fwd:
            assert call(lib, scale=at(spot)) == EINVAL, hex(spot)


@pytest.mark.parametrize("call", [add_fwd, add_q8, q8])
def test_weights_under_outputs(lib, call):
    for spot in (G.value, G.value + 12, G.value - 12):
        assert call(lib, rstd=at(spot)) == EINVAL
    outs = {add_fwd: ("y", "h"), add_q8: ("q", "h"), q8: ("q",)}[call]
    for name in outs:
        assert call(lib, **{name: G}) == EINVAL
    if call is not add_fwd:
        assert call(lib, scale=G) == EINVAL
        assert call(lib, scale=S) == EINVAL
        assert call(lib, scale=at(S.value + 12)) == EINVAL


def test_scales_by_group(lib):
    """300 columns have three scales a row."""
    for call in (add_q8, q8):
        assert call(lib, N=300, group=128, scale=at(S.value - 4 * 3 * M + 4)) == EINVAL
        assert call(lib, N=300, group=128, scale=at(X.value - 4 * 3 * M + 4)) == EINVAL


def test_rows_with_a_stride(lib):
    """Rows of 16 bytes 64 apart: into the next row, or longer than the gap."""
    ld = (32, 0, 0, 0)
    for spot in (16 + 36, 64, 64 + 12, 3 * 64 + 12):
        assert add_fwd(lib, ld=ld, rstd=at(X.value + spot)) == EINVAL, spot
    assert add_fwd(lib, M=16, ld=ld, rstd=at(X.value + 16)) == EINVAL  # 64 bytes in a gap of 48


def test_backward(lib):
    for spot in (Y.value, Y.value + ROWS - 4, Y.value - 12):
        assert add_bwd(lib, g=at(spot)) == EINVAL
        assert add_bwd(lib, rstd=at(spot)) == EINVAL
        assert add_bwd(lib, dg=at(spot)) == EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_beside_and_between_rows(dtype):
    """Statistics in the gap between two rows, scales right behind the last one: the results of calls with tensors apart."""
    g = torch.Generator().manual_seed(1)
    M, N, ld = 3, 256, 512
    buf = torch.randn(M * ld, generator=g).to(dtype).cuda()
    x = buf.as_strided((M, N), (ld, 1))
    es = buf.element_size()
    r, gamma = torch.randn(M, N, generator=g).to(dtype).cuda(), torch.randn(N, generator=g).to(dtype).cuda()
    want = gbn.rms_add_fwd(x, r, gamma, 1e-6)
    want8 = gbn.rms_fwd_q8(x, gamma, 1e-6, group=128)
    gap = buf.view(torch.uint8)[N * es:ld * es]            # between rows 0 and 1
    tail = buf.view(torch.uint8)[((M - 1) * ld + N) * es:]  # behind the last row
    rstd = gap[:4 * M].view(torch.float32)
    got = gbn.rms_add_fwd(x, r, gamma, 1e-6, rstd=rstd)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    got = gbn.rms_fwd_q8(x, gamma, 1e-6, group=128, rstd=gap[(ld - N) * es - 4 * M:].view(torch.float32),
                         scale=tail[:8 * M].view(torch.float32).view(M, 2))
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want8))
    # dgamma and rstd between dx's rows
    dy, dh = torch.randn(M, N, generator=g).to(dtype).cuda(), torch.randn(M, N, generator=g).to(dtype).cuda()
    want = gbn.rms_add_bwd(dy, dh, want[1], gamma, want[2])
    h = gbn.rms_add_fwd(x, r, gamma, 1e-6)[1]
    wide = torch.zeros(M, 2 * N, dtype=torch.float32, device="cuda")
    dx = wide.view(dtype)[:, :N]
    between = wide.view(-1).view(torch.uint8)[N * es:]
    dg = between[:4 * N].view(torch.float32)  # fills the gap of float32 rows
    got = gbn.rms_add_bwd(dy, dh, h, gamma, rstd, dx=dx, dgamma=dg)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
