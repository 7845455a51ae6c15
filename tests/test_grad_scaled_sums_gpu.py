"""The gradient norm where every batch's squares are scaled first: many batches
a thread (needs a GPU).

The bound is the ordinary one: a batch of at most 32 squares is off by 10 u of
its sum, u = 2^-24, 5 u of the root; the sums of batches are pairs, which lose
nothing next to that, and the float32 norm is one rounding more: 6 u.  Scaling
by a power of two is exact.  The two values are those of 4000 drawn ones at
which 108 equal batches, added in float32 one by one, drift farthest: 28 u of
the sum."""
import pytest
import torch

import rmsnorm_backward_gb300 as gbn

pytestmark = pytest.mark.gpu

u = 2.0 ** -24


def off(norm, want):
    return abs(float(norm) - want) / (u * want)


@pytest.mark.parametrize("value", [1.5076081930163326e-14, 1727967920128.0])
def test_equal_values(value):
    n = 1 << 28  # 1 GiB: 107 or 108 batches of 16 a thread on 152 SMs
    t = torch.full((n,), value, device="cuda")
    want = float(t[0].double()) * n ** 0.5
    assert off(gbn.grad_norm([t]), want) <= 6
    out = torch.empty_like(t)
    assert off(gbn.grad_clip([t], want / 2, eps=0.0, out=[out]), want) <= 6
    # the norm's 6 u, the roundings of max_norm, of norm + eps, of the quotient and of the product
    assert (out.double() - value / 2).abs().max() <= 10 * u * value / 2


@pytest.mark.parametrize("scale", [1e-14, 1e-25, 1e-37, 1e13, 1e25])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_drawn_values(scale, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    t = torch.randn(60_000_001, generator=g, device="cuda").mul_(scale).to(dtype)
    parts = list(t[1:].split([40_000_000, 19_999_997, 3]))
    want = float(torch.linalg.vector_norm(t[1:].double().div_(scale))) * scale
    assert off(gbn.grad_norm(parts), want) <= 6
    # beside ordinary ones, whose batches are gathered apart
    more = torch.randn(1_000_000, generator=g, device="cuda")
    both = float(more.double().square().sum() + want ** 2) ** 0.5
    assert off(gbn.grad_norm(parts + [more]), both) <= 6


@pytest.mark.parametrize("count", [1, 97, 2100])
def test_lists_of_several_tables(count):
    """Sums that go from one launch to the next through memory."""
    g = torch.Generator(device="cuda").manual_seed(4)
    small = [torch.randn(4001, generator=g, device="cuda") * 1e-20 for _ in range(count)]
    large = [torch.randn(4001, generator=g, device="cuda") * 1e20 for _ in range(count)]
    for tensors, scale in ((small, 1e-20), (large, 1e20)):
        want = float(torch.stack([(t.double() / scale).square().sum() for t in tensors]).sum()) ** 0.5 * scale
        assert off(gbn.grad_norm(tensors), want) <= 6
    assert off(gbn.grad_norm(small + large), want) <= 6


@pytest.mark.parametrize("n", [7, 100_000, 30_000_000])
def test_infinities_and_nan_among_scaled_batches(n):
    for scale in (1e-20, 1e20, 1.0):
        t = torch.full((n,), scale, device="cuda")
        t[n // 2] = float("inf")
        t[0] = -float("inf")
        assert float(gbn.grad_norm([t])) == float("inf")
        t[n - 1] = float("nan")
        assert torch.isnan(gbn.grad_norm([t]))
    t = torch.full((n,), 3e38, device="cuda")  # the norm of n of them is no float32
    assert float(gbn.grad_norm([t])) == float("inf")


@pytest.mark.parametrize("max_norm", [0.0, 1.0, float("inf")])
def test_an_infinite_norm(max_norm):
    """Finite elements become zero, but where max_norm is infinite too: inf / inf is NaN, and so is every output."""
    t = torch.ones(1000, device="cuda")
    t[10] = float("inf")
    assert float(gbn.grad_clip([t], max_norm)) == float("inf")
    assert torch.isnan(t[10])
    rest = torch.cat([t[:10], t[11:]])
    assert torch.isnan(rest).all() if max_norm == float("inf") else (rest == 0).all()
