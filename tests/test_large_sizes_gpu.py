"""More than 2^31 elements in one tensor: rows to the last one, and gradients
(needs a GPU with 60 GB to spare).

The rows at both ends and around the 2^31st element are compared in float64
with the tolerances of test_rms_add_gpu.py; dgamma is compared with the same
sum in float64."""
import pytest
import torch

import rmsnorm_backward_gb300 as gbn
from test_rms_add_gpu import EPS, check_backward, check_forward, check_q8, u

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of device memory")
    yield
    torch.cuda.empty_cache()


def drawn(M, N, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    for at in range(0, M, 1 << 19):
        rows = t[at:at + (1 << 19)]
        rows.copy_(torch.randn(rows.shape, generator=g, device="cuda").mul_(scale))
    return t


@pytest.mark.parametrize("M,N", [(2_150_001, 1000), (17_000_003, 128), (1_080_011, 2001), (530_003, 4096)])
def test_rows_beyond_2_31_elements(M, N):
    assert M * N > 1 << 31
    x, r = drawn(M, N, 1), drawn(M, N, 2)
    gamma = drawn(1, N, 3)[0]
    middle = (1 << 31) // N
    spots = torch.cat([torch.arange(0, 40), torch.arange(middle - 20, middle + 20), torch.arange(M - 40, M)]).cuda()

    def some(t):
        return t[spots].cpu()

    y, h, rstd = gbn.rms_add_fwd(x, r, gamma, EPS)
    t = {"x": some(x), "residual": some(r), "gamma": gamma.cpu()}
    check_forward(t, some(y), some(h), some(rstd))
    for group in (0, 128):
        q, scale, rstd8 = gbn.rms_fwd_q8(h, gamma, EPS, group=group)
        check_q8(some(h), t["gamma"], some(q.view(torch.uint8)).view(q.dtype), some(scale), some(rstd8), group)
        del q, scale, rstd8
    dx, dg = gbn.rms_add_bwd(y, r, h, gamma, rstd, dx=x)
    t.update(dy=some(y), dh=some(r))
    # dx of the rows looked at (for dgamma, checked below as a whole, their own sum is handed in)
    part = (t["dy"].double() * some(h).double() * some(rstd).double()[:, None]).sum(0).float()
    check_backward(t, some(h), some(rstd), some(dx), part)
    want, size = torch.zeros(N, dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    for at in range(0, M, 1 << 18):
        rows = slice(at, at + (1 << 18))
        terms = y[rows].double() * h[rows].double() * rstd[rows].double()[:, None]
        want += terms.sum(0)
        size += terms.abs().sum(0)
    # the longest chain of additions: a CTA's rows, its slots and warps, and the CTAs' partial rows
    longest = -(-M // 100) + 400
    assert ((dg.double() - want).abs() <= u * (longest + 2) * size).all()
    assert gbn.device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_gradient_beyond_2_31_elements(dtype):
    n = (1 << 31) + 4097
    t = torch.full((n + 1,), 2.0 ** -10, dtype=dtype, device="cuda")[1:]
    t[-1] = 3.0
    t[(1 << 31) + 1] = -5.0
    want = ((n - 2) * 2.0 ** -20 + 34) ** 0.5
    assert abs(float(gbn.grad_norm([t])) - want) <= 6 * u * want
    gbn.grad_clip([t], 2 * want, eps=0.0)  # below the limit: as it was
    assert float(t[-1]) == 3.0
    norm = gbn.grad_clip([t], want / 4, eps=0.0)
    assert abs(float(norm) - want) <= 6 * u * want
    tol = torch.finfo(dtype).eps / 2 + 10 * u
    for at, value in ((0, 2.0 ** -12), (n // 2, 2.0 ** -12), ((1 << 31) + 1, -1.25), (n - 2, 2.0 ** -12), (n - 1, 0.75)):
        assert abs(float(t[at]) - value) <= abs(value) * tol
    assert int((t == 0).sum()) == 0
