"""The global gradient norm and the clip against float64 (needs a GPU).

Tolerances, u = 2^-24: a batch of at most 32 squares is a float32 sum of
positive terms: one rounding for each square and at most nine additions after
one another, so 10 u of the sum at most, 5 u of its root; the sums of batches
keep what their roundings lose and add nothing next to that; the float32 norm
is one rounding more: 6 u.  A clipped value has the norm's error, the
roundings of norm + eps, of the quotient, of the product, and the one to the
storage type: 9 u + eps / 2 (half a quantum below the smallest normal value)."""
import pytest
import torch

import guards
import rmsnorm_backward_gb300 as gbn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
u = 2.0 ** -24
EPS = 1e-6


def make(sizes, dtypes, seed=0, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(scale * torch.randn(n, generator=g)).to(DT[dtypes[i % len(dtypes)]]) for i, n in enumerate(sizes)]


def norm_of(grads):
    return torch.stack([g.double().square().sum() for g in grads]).sum().sqrt() if grads else torch.zeros(())


def check_norm(got, grads):
    ref = float(norm_of(grads))
    assert got.dtype == torch.float32 and got.dim() == 0
    if ref > torch.finfo(torch.float32).max:  # sqrt(5020) * 1e37 = 7.1e38 > 3.4e38: no float32
        assert float(got) == float("inf")
    else:
        assert abs(float(got) - ref) <= 6 * u * ref, (float(got), ref)
    return ref


def check_clipped(got, grads, max_norm):
    ref = float(norm_of(grads))
    coef = min(1.0, max_norm / (ref + EPS))
    for i, (o, g) in enumerate(zip(got, grads)):
        f = torch.finfo(g.dtype)
        want = g.double() * coef
        tol = want.abs() * (f.eps / 2 + 9 * u) * (1 + 2.0 ** -8) + f.tiny * f.eps / 2
        bad = ~((o.double().cpu() - want).abs() <= tol)
        assert not bad.any(), f"gradient {i}: {int(bad.sum())} of {bad.numel()} values off"


LISTS = [[], [0], [1], [1, 0, 3], [4096], [7, 8, 9, 15, 16, 17], [100003, 1, 5, 65536], [4097] * 95, [33] * 97,
         [5, 1000] * 520, [3] * 2100, [1 << 20, 12345, 1 << 18]]


@pytest.mark.parametrize("dtypes", [("f32",), ("bf16",), ("f16",), ("bf16", "f32", "f16")])
@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0] if s else 0}")
def test_norm_and_clip(sizes, dtypes):
    cpu = make(sizes, dtypes)
    g = guards.Guarded("cuda")
    dev = [g.copy_in(t, f"g{i}") if t.numel() else t.cuda() for i, t in enumerate(cpu)]
    ws = g.workspace(gbn.grad_workspace_bytes(), misalign=8)
    check_norm(gbn.grad_norm(dev, workspace=ws), cpu)
    ref = float(norm_of(cpu))
    grads = gbn.GradList(dev)
    for max_norm in (0.37 * ref, 3.0 * ref + 1.0):
        outs = [g.empty((t.numel(),), t.dtype, f"out{i}") if t.numel() else t.cuda() for i, t in enumerate(cpu)]
        check_norm(gbn.grad_clip(grads, max_norm, out=outs, workspace=ws), cpu)
        g.check()  # the gradients as they were, nothing beside the outputs
        check_clipped(outs, cpu, max_norm)
        same = [t.clone() for t in dev]
        check_norm(gbn.grad_clip(same, max_norm), cpu)
        check_clipped(same, cpu, max_norm)
        if max_norm > ref:
            assert all(torch.equal(a.cpu(), b) for a, b in zip(same, cpu))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift", [(1, 1), (1, 2), (0, 3), (5, 0)])
def test_unaligned(dtype, shift):
    """Gradients and outputs that start between 16-byte boundaries, alike and not alike."""
    sizes = [40000, 3, 8, 1]
    cpu = make(sizes, (dtype,), seed=1)
    src = torch.zeros(sum(sizes) + 8, dtype=DT[dtype], device="cuda")[shift[0]:][:sum(sizes)].copy_(torch.cat(cpu))
    base = torch.full((sum(sizes) + 16,), 7.0, dtype=DT[dtype], device="cuda")
    out = base[shift[1]:][:sum(sizes)]
    check_norm(gbn.grad_clip(src.split(sizes), 0.5, out=out.split(sizes)), cpu)
    check_clipped(out.split(sizes), cpu, 0.5)
    assert (base[:shift[1]] == 7).all() and (base[shift[1] + sum(sizes):] == 7).all()


def test_layouts():
    g = torch.Generator().manual_seed(5)
    a, b = torch.randn(64, 48, generator=g), torch.randn(3, 5, 7, generator=g)
    dev = [a.cuda().t(), b.cuda().permute(2, 0, 1)]
    check_norm(gbn.grad_norm(dev), [a, b])
    gbn.grad_clip(dev, 1.5)
    check_clipped([dev[0].t(), dev[1].permute(1, 2, 0)], [a, b], 1.5)
    with pytest.raises(ValueError, match="block of memory"):
        gbn.grad_norm([torch.zeros(4, 8, device="cuda")[:, :6]])


@pytest.mark.parametrize("scale", [1e-30, 1e-38, 1e18, 1e36, 1e37])
def test_norms_whose_squares_leave_float32(scale):
    cpu = make([5000, 17, 3], ("f32",), seed=2, scale=scale)
    dev = [t.cuda() for t in cpu]
    check_norm(gbn.grad_norm(dev), cpu)
    # small batches next to ordinary ones
    both = cpu + make([4096], ("f32",), seed=3)
    check_norm(gbn.grad_norm([t.cuda() for t in both]), both)


def test_zeros_and_values_that_are_not_finite():
    z = [torch.zeros(1000, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.bfloat16)]
    assert float(gbn.grad_clip(z, 1.0)) == 0.0 and all((t == 0).all() for t in z)
    for bad, at in ((float("nan"), 0), (float("inf"), 999), (-float("inf"), 500)):
        t = [torch.ones(1000, device="cuda"), torch.ones(5, device="cuda", dtype=torch.float16)]
        t[0][at] = bad
        n = gbn.grad_clip(t, 1.0)
        if bad != bad:
            assert torch.isnan(n) and all(torch.isnan(x).all() for x in t)
        else:
            assert torch.isinf(n) and torch.isnan(t[0][at]) and (t[1] == 0).all() and int((t[0] == 0).sum()) == 999
    t = [torch.full((100,), 3e38, device="cuda")]
    assert torch.isinf(gbn.grad_norm(t))  # 3e39 is not a float32
    t = [torch.ones(100, device="cuda")]
    gbn.grad_clip(t, 0.0)
    assert (t[0] == 0).all()
    t = [torch.ones(100, device="cuda")]
    gbn.grad_clip(t, float("inf"))
    assert (t[0] == 1).all()
    gbn.grad_clip(z, 0.0, eps=0.0)  # 0 / 0
    assert all((x == 0).all() for x in z)


def test_the_same_bits_from_run_to_run():
    dev = [t.cuda() for t in make([1 << 20, 77777, 5], ("bf16", "f32"), seed=4)]
    first = gbn.grad_norm(dev)
    for _ in range(5):
        assert torch.equal(first, gbn.grad_norm(dev))
        assert torch.equal(first, gbn.grad_clip(dev, 1e9))


def test_another_stream_and_captured_graphs():
    cpu, new = make([100000, 33], ("bf16", "f32"), seed=6), make([100000, 33], ("bf16", "f32"), seed=7, scale=3e-2)
    dev = [t.cuda() for t in cpu]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = [torch.empty_like(t) for t in dev]
    n = gbn.grad_clip(dev, 0.5, out=outs, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    check_norm(n, cpu)
    check_clipped(outs, cpu, 0.5)
    # two graphs of the same gradients, each with the workspace of its capture; the list is gone before the replay
    graphs, results = [], []
    for max_norm in (0.5, 1.5):
        outs = [torch.empty_like(t) for t in dev]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            n = gbn.grad_clip(dev, max_norm, out=outs)
        graphs.append(graph)
        results.append((max_norm, n, outs))
    for t, v in zip(dev, new):
        t.copy_(v)
    for graph in graphs:
        graph.replay()
    torch.cuda.synchronize()
    for max_norm, n, outs in results:
        check_norm(n, new)
        check_clipped(outs, new, max_norm)


def test_refusals():
    t = torch.ones(64, device="cuda")
    with pytest.raises(ValueError, match="share memory"):
        gbn.grad_clip([t, t], 1.0)
    with pytest.raises(ValueError, match="share memory"):
        gbn.grad_clip([t[:40], t[30:]], 1.0)
    assert float(gbn.grad_norm([t, t])) == pytest.approx(128 ** 0.5, rel=1e-6)  # read twice, counted twice
    with pytest.raises(ValueError, match="share memory"):
        gbn.grad_clip([t[:32], t[32:]], 1.0, out=[t[32:], t[:32]])
    with pytest.raises(ValueError, match="share memory"):
        gbn.grad_clip([t[:32]], 1.0, out=[t[1:33]])
    with pytest.raises(ValueError):
        gbn.grad_clip([t], 1.0, out=[t[:32]])
    with pytest.raises(ValueError):
        gbn.grad_clip([t], 1.0, out=[t, t[:1]])
    with pytest.raises(ValueError):
        gbn.grad_clip([t], 1.0, out=[t.half()])
    with pytest.raises(ValueError):
        gbn.grad_norm([t.double()])
    with pytest.raises(gbn.GbnError):
        gbn.grad_clip([t], -1.0)
    with pytest.raises(gbn.GbnError) as e:
        gbn.grad_norm([t], workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    # some of the outputs in place, the others beside
    a, b, c = torch.ones(4, device="cuda"), torch.ones(5, device="cuda"), torch.empty(5, device="cuda")
    gbn.grad_clip([a, b], 1.5, out=[a, c])
    assert torch.allclose(a, torch.full_like(a, 0.5)) and torch.allclose(c, torch.full_like(c, 0.5)) and (b == 1).all()


def test_a_training_step():
    """Three pre-norm blocks forward and backward with the residual norm, then the clip of the weights' gradients,
    against autograd in float64.  fp32 throughout: each block's float32 error is far below the last tolerance."""
    M, N, L = 200, 512, 3
    g = torch.Generator().manual_seed(8)
    x0, res = torch.randn(M, N, generator=g), torch.randn(M, N, generator=g)
    gammas = [1 + 0.1 * torch.randn(N, generator=g) for _ in range(L)]
    mix = [torch.randn(N, generator=g) for _ in range(L)]  # stands for the block: elementwise weights
    # the program
    x, r, saved = x0.cuda(), res.cuda(), []
    for gamma, m in zip(gammas, mix):
        y, r, rstd = gbn.rms_add_fwd(x, r, gamma.cuda(), EPS)
        saved.append((r, rstd))
        x = y * m.cuda()
    dx, dr = torch.ones_like(x), torch.full_like(x, 0.5)
    grads = []
    for i in reversed(range(L)):
        dx, dg = gbn.rms_add_bwd(dx * mix[i].cuda(), dr, saved[i][0], gammas[i].cuda(), saved[i][1])
        dr = dx
        grads.insert(0, dg)
    first = dx.clone()
    norm = gbn.grad_clip(grads, 10.0)
    # the same in float64
    leaf = [t.double().requires_grad_() for t in [x0, res] + gammas]
    xx, rr = leaf[0], leaf[1]
    for gamma, m in zip(leaf[2:], mix):
        rr = xx + rr
        xx = gamma * rr / torch.sqrt((rr * rr).mean(-1, keepdim=True) + EPS) * m.double()
    (xx.sum() + 0.5 * rr.sum()).backward()
    want = torch.cat([t.grad for t in leaf[2:]])
    ref = want.norm()
    # 3 blocks of at most 64 float32 operations each, errors of both signs taken as if of one
    assert abs(float(norm) - float(ref)) <= 200 * u * float(ref)
    scale = want.abs().max()
    assert ((torch.cat(grads).cpu().double() - want * (10.0 / (ref + EPS))).abs() <= 400 * u * scale).all()
    assert ((first.cpu().double() - leaf[0].grad).abs() <= 400 * u * leaf[0].grad.abs().max()).all()
