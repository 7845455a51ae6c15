"""RMSNorm with the residual's addition, its 8-bit output and its backward,
against plain float64 computations (needs a GPU).

Tolerances.  u = 2^-24 is float32's rounding, U = finfo(T).eps / 2 the storage
type's.  A sum of n positive float32 terms, added in any order whose longest
chain of additions is `chain`, is off by at most chain*u of itself (to first
order); a thread adds at most N/32 terms (one warp to a row) before the
exchanges among lanes and warps, 5 + 16 additions, so chain <= N/32 + 24.
  rstd: half the sum's error, plus eps' addition, the division by N, the root
    and the division: chain/2 + 4 u.
  y: rstd's error, two products, one rounding to T.
  codes: float32 operations on single elements, whose order nothing changes:
    the same bits as the same operations in torch; times the scale they are
    within half a step of the code of v.
  dx: with t = rstd*(|dyhat| + |xhat| mean|dyhat xhat|) + |dh| the terms'
    magnitude, eight float32 operations at t, the sum's error at its own term,
    one rounding to T.
  dgamma: the terms' magnitudes sum|dy xhat| times u for each addition of the
    longest chain (rows of a CTA, then the CTAs' partial rows) plus two.
Roundings to T below the smallest normal value are half a quantum."""
import math

import numpy as np
import pytest
import torch

import guards
import rmsnorm_backward_gb300 as gbn

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
u = 2.0 ** -24
EPS = 1e-6


def half_step(t):
    """(relative, absolute) error of one rounding to dtype t."""
    f = torch.finfo(t)
    return f.eps / 2, f.tiny * f.eps / 2


def chain(N):
    return N / 32 + 24


def inputs(M, N, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(1000 * seed + 7 * M + N)
    t = {k: torch.randn(M, N, generator=g).mul_(scale) for k in ("x", "residual", "dy", "dh")}
    t["residual"][:, :: max(1, N // 5)] *= 20.0
    t["gamma"] = 1.0 + 0.1 * torch.randn(N, generator=g)
    return {k: v.to(DT[dtype]) for k, v in t.items()}


def check(name, got, ref, tol):
    got, ref, tol = got.double().cpu(), ref.double().cpu(), torch.as_tensor(tol, dtype=torch.float64).cpu()
    bad = ~((got - ref).abs() <= tol)
    if bad.any():
        i = int(bad.reshape(-1).nonzero()[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} off, first at {i}: "
                             f"{got.reshape(-1)[i]} for {ref.reshape(-1)[i]}")


def summed(x, residual):
    """h as stored: the float32 sum, rounded."""
    return (x.float() + residual.float()).to(x.dtype)


def check_rstd(h, rstd):
    h = h.double().cpu()
    ref = 1.0 / torch.sqrt((h * h).mean(-1) + EPS)
    check("rstd", rstd, ref, ref * (chain(h.shape[-1]) / 2 + 4) * u)
    return ref


def check_forward(t, y, h, rstd):
    want = summed(t["x"], t["residual"])
    assert torch.equal(h.cpu(), want), "h is not the rounded sum"
    ref = check_rstd(want, rstd)
    ref = want.double() * ref[..., None] * t["gamma"].double()
    rel, tiny = half_step(y.dtype)
    check("y", y, ref, ref.abs() * (1 + 2.0 ** -8) * (rel + (chain(want.shape[-1]) / 2 + 6) * u) + tiny)


def codes_and_scale(h, gamma, rstd, q_dtype, group):
    """The operator's own float32 operations in torch, given rstd."""
    top = 448.0 if q_dtype == torch.float8_e4m3fn else 127.0
    N = h.shape[-1]
    v = gamma.float() * h.float()
    width = group or N
    parts = torch.nn.functional.pad(v, (0, -N % width)).view(v.shape[0], -1, width)
    a = parts.abs().amax(-1)
    pre = torch.where(a < 2.0 ** -100, 2.0 ** 100, 1.0)
    # a tensor over a tensor: torch takes a number over a tensor as a product with the reciprocal
    mul = torch.where(a == 0, torch.zeros_like(a), torch.full_like(a, top) / (a * pre))
    code = ((parts * pre[..., None]) * mul[..., None]).view(v.shape[0], -1)[:, :N]
    code = code.to(q_dtype) if q_dtype == torch.float8_e4m3fn else code.round().nan_to_num(0.0).to(q_dtype)
    scale = rstd.float()[:, None] * a * float(np.float32(1) / np.float32(top))
    return code, scale if group else scale[:, 0]


def check_q8(h, gamma, q, scale, rstd, group):
    """h: the stored rows, on the CPU."""
    check_rstd(h, rstd)
    code, want = codes_and_scale(h, gamma, rstd.cpu(), q.dtype, group)
    assert torch.equal(q.cpu().view(torch.uint8), code.view(torch.uint8)), "codes differ"
    assert torch.equal(scale.cpu(), want), "scales differ"
    # and what they stand for, in 64 bits
    s = scale.double().cpu()
    s = s.repeat_interleave(group, dim=1)[:, :h.shape[1]] if group else s[:, None]
    ref = h.double() * rstd.double().cpu()[:, None] * gamma.double()
    # half a step of the code, and six float32 roundings (v, Q/a, their product, 1/Q, two of the scale)
    if q.dtype == torch.int8:
        tol = 0.5 * s + 7 * u * 127 * s
    else:
        tol = torch.maximum(ref.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -10)
    check("code * scale", q.double().cpu() * s, ref, tol)


def add_bwd_ref(t, h, rstd):
    dy, dh, hh, g = (a.double() for a in (t["dy"], t["dh"], h, t["gamma"]))
    rs = rstd.double()[:, None]
    xhat, dyhat = hh * rs, dy * g
    mean = (dyhat * xhat).mean(-1, keepdim=True)
    dx = rs * (dyhat - xhat * mean) + dh
    dgamma = (dy * xhat).sum(0)
    size = (dyhat * xhat).abs().mean(-1, keepdim=True)
    term = rs * (dyhat.abs() + xhat.abs() * size) + dh.abs()
    return dx, dgamma, term, rs * xhat.abs() * size, (dy * xhat).abs().sum(0)


def check_backward(t, h, rstd, dx, dgamma, before=None):
    ref, dg, term, mean_term, dg_size = add_bwd_ref(t, h, rstd)
    M, N = h.shape
    rel, tiny = half_step(dx.dtype)
    check("dx", dx, ref, ref.abs() * rel * (1 + 2.0 ** -8) + tiny + u * (10 * term + (chain(N) + 4) * mean_term))
    longest = math.ceil(M / 100) + 200
    if before is not None:
        dg = dg + before.double()
        dg_size = dg_size + before.double().abs()
    rel, tiny = (0.0, 0.0) if dgamma.dtype == torch.float32 else half_step(dgamma.dtype)
    check("dgamma", dgamma, dg, u * (longest + 2) * dg_size + dg.abs() * rel * (1 + 2.0 ** -8) + tiny)


SHAPES = [(1, 1), (1, 8), (2, 7), (1, 4096), (3, 4097), (5, 256), (4, 127), (7, 1000), (33, 1024), (160, 498),
          (64, 2052), (70, 8192), (19, 8193), (9, 16384), (305, 640), (2, 40000), (1000, 72), (513, 130),
          (1700, 515), (311, 8191), (8, 12), (9, 9), (155, 4100)]


@pytest.mark.parametrize("kernel", ["auto", "plain"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_add_forward_and_backward(M, N, dtype, kernel):
    t = inputs(M, N, dtype)
    g = guards.Guarded("cuda")
    d = {k: g.copy_in(v, k) for k, v in t.items()}
    y, h, dx = (g.empty((M, N), DT[dtype], k) for k in ("y", "h", "dx"))
    rstd = g.empty((M,), torch.float32, "rstd")
    dg = g.empty((N,), torch.float32, "dgamma")
    ws = g.workspace(gbn.bwd_workspace_bytes(M, N, DT[dtype], False))
    out = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS, y=y, h=h, rstd=rstd, kernel=kernel)
    assert out[0] is y and out[1] is h and out[2] is rstd
    out = gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd, dx=dx, dgamma=dg, workspace=ws, kernel=kernel)
    assert out[0] is dx and out[1] is dg
    g.check()
    check_forward(t, y, h, rstd)
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg)
    assert gbn.device_error() == 0


@pytest.mark.parametrize("kernel", ["auto", "plain"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("q_dtype", [torch.float8_e4m3fn, torch.int8])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,N", SHAPES)
def test_q8(M, N, dtype, q_dtype, group, kernel):
    t = inputs(M, N, dtype, seed=1)
    g = guards.Guarded("cuda")
    d = {k: g.copy_in(t[k], k) for k in ("x", "residual", "gamma")}
    wide = (M, -(-N // 128)) if group else (M,)
    for add in (True, False):
        q, scale = g.empty((M, N), q_dtype, "q"), g.empty(wide, torch.float32, "scale")
        rstd = g.empty((M,), torch.float32, "rstd")
        if add:
            h = g.empty((M, N), DT[dtype], "h")
            gbn.rms_add_fwd_q8(d["x"], d["residual"], d["gamma"], EPS, group=group, q=q, scale=scale, h=h, rstd=rstd,
                               kernel=kernel)
            want = summed(t["x"], t["residual"])
            assert torch.equal(h.cpu(), want)
        else:
            gbn.rms_fwd_q8(d["x"], d["gamma"], EPS, group=group, q=q, scale=scale, rstd=rstd, kernel=kernel)
            want = t["x"]
        g.check()
        check_q8(want, t["gamma"], q, scale, rstd, group)
    assert gbn.device_error() == 0


def strided(t, extra, fill=float("nan")):
    """t in the first columns of a wider CUDA buffer; (view, buffer)."""
    buf = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=torch.float32, device="cuda").to(t.dtype)
    buf[:, :t.shape[1]] = t.cuda()
    return buf[:, :t.shape[1]], buf


@pytest.mark.parametrize("N", [1024, 1000, 515])
@pytest.mark.parametrize("extra", [(64, 64, 64, 64), (3, 3, 3, 3), (8, 16, 5, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strided_rows(N, extra, dtype):
    M = 333
    t = inputs(M, N, dtype, seed=2)
    (x, xb), (r, rb) = strided(t["x"], extra[0]), strided(t["residual"], extra[1])
    zero = torch.zeros(M, N, dtype=DT[dtype])
    (y, yb), (h, hb), (dx, dxb) = strided(zero, extra[2]), strided(zero, extra[3]), strided(zero, extra[0])
    (dy, dyb), (dh, dhb) = strided(t["dy"], extra[1]), strided(t["dh"], extra[2])
    gamma = t["gamma"].cuda()
    _, _, rstd = gbn.rms_add_fwd(x, r, gamma, EPS, y=y, h=h)
    check_forward(t, y, h, rstd)
    _, dg = gbn.rms_add_bwd(dy, dh, h, gamma, rstd, dx=dx)
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg)
    for q_dtype in gbn.Q_DTYPE_CODES:
        for group in (0, 128):
            qb = torch.full((M, N + extra[3]), 99, dtype=torch.uint8, device="cuda")
            q = qb.view(q_dtype)[:, :N]
            _, scale, h2, rstd = gbn.rms_add_fwd_q8(x, r, gamma, EPS, group=group, q=q)
            check_q8(h2.cpu(), t["gamma"], q.contiguous(), scale, rstd, group)
            assert (qb[:, N:] == 99).all()
    for b in (xb, rb, yb, hb, dxb, dyb, dhb):
        assert torch.isnan(b[:, N:]).all(), "the row padding was written"


@pytest.mark.parametrize("shift", [1, 2, 4, 5])
@pytest.mark.parametrize("N", [512, 1001])
def test_unaligned_bases(shift, N):
    """Tensors that start between 16-byte boundaries, alike and not alike."""
    M, dtype = 50, "bf16"
    t = inputs(M, N, dtype, seed=3)

    def moved(src, by):
        flat = torch.zeros(M * N + 16, dtype=DT[dtype], device="cuda")
        view = flat[by:by + M * N].view(M, N)
        if src is not None:
            view.copy_(src)
        return view

    for other in (shift, 0):
        x, r = moved(t["x"], shift), moved(t["residual"], other)
        gamma = torch.zeros(N + 8, dtype=DT[dtype], device="cuda")[shift:shift + N].copy_(t["gamma"])
        y, h, rstd = gbn.rms_add_fwd(x, r, gamma, EPS, y=moved(None, shift), h=moved(None, other))
        check_forward(t, y, h, rstd)
        dx, dg = gbn.rms_add_bwd(moved(t["dy"], shift), moved(t["dh"], other), h, gamma, rstd, dx=moved(None, shift))
        check_backward(t, h.cpu(), rstd.cpu(), dx, dg)
        for group in (0, 128):
            q = torch.zeros(M * N + 16, dtype=torch.int8, device="cuda")[shift:shift + M * N].view(M, N)
            _, scale, h2, rstd2 = gbn.rms_add_fwd_q8(x, r, gamma, EPS, q=q, group=group)
            check_q8(h2.cpu(), t["gamma"], q, scale, rstd2, group)


@pytest.mark.parametrize("N", [4096, 777])
def test_in_place(N):
    M, dtype = 300, "bf16"
    t = inputs(M, N, dtype, seed=4)
    gamma = t["gamma"].cuda()
    x, r = t["x"].cuda(), t["residual"].cuda()
    y, h, rstd = gbn.rms_add_fwd(x, r, gamma, EPS, y=x, h=r)
    check_forward(t, y, h, rstd)
    x, r = t["x"].cuda(), t["residual"].cuda()
    y, h, rstd = gbn.rms_add_fwd(x, r, gamma, EPS, y=r, h=x)
    check_forward(t, y, h, rstd)
    x, r = t["x"].cuda(), t["residual"].cuda()
    q, scale, h, rstd = gbn.rms_add_fwd_q8(x, r, gamma, EPS, h=x)
    check_q8(h.cpu(), t["gamma"], q, scale, rstd, 0)
    assert h is x and torch.equal(x.cpu(), summed(t["x"], t["residual"]))
    for over in ("dy", "dh", "h"):
        d = {k: t[k].cuda() for k in ("dy", "dh")}
        d["h"] = h.clone()
        dx, dg = gbn.rms_add_bwd(d["dy"], d["dh"], d["h"], gamma, rstd, dx=d[over])
        check_backward(t, h.cpu(), rstd.cpu(), dx, dg)
    # x and the residual as the two halves of one buffer's rows, y and h over them
    both = torch.cat([t["x"], t["residual"]], dim=1).cuda()
    y, h, rstd = gbn.rms_add_fwd(both[:, :N], both[:, N:], gamma, EPS, y=both[:, :N], h=both[:, N:])
    check_forward(t, y, h, rstd)


def test_the_same_tensor_twice():
    """x is also the residual: h = 2x."""
    t = inputs(40, 1024, "bf16", seed=5)
    t["residual"] = t["x"]
    x = t["x"].cuda()
    check_forward(t, *gbn.rms_add_fwd(x, x, t["gamma"].cuda(), EPS))


@pytest.mark.parametrize("N", [8, 4096, 4099])
def test_rows_that_are_not_finite(N):
    """NaN and infinities stay in their rows; zero and tiny rows have their values."""
    t = inputs(8, N, "f32", seed=6)
    x, r = t["x"], t["residual"]
    x[1, N // 2] = float("nan")
    x[2, 0] = float("inf")
    r[3, N - 1] = -float("inf")
    x[4] = 0.0
    r[4] = 0.0
    x[5] = x[5] * 1e-38
    r[5] = 0.0
    fine = [0, 4, 5, 6, 7]
    d = {k: v.cuda() for k, v in t.items()}
    for kernel in ("auto", "plain"):
        y, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS, kernel=kernel)
        part = {k: v[fine] if v.dim() == 2 else v for k, v in t.items()}
        check_forward(part, y[fine], h[fine], rstd[fine])
        assert torch.isnan(y[1]).all() and torch.isnan(rstd[1])
        assert rstd[2] == 0 and torch.isnan(y[2, 0]) and (y[2, 1:] == 0).all()
        assert rstd[3] == 0 and torch.isnan(y[3, N - 1]) and (y[3, :N - 1] == 0).all()
        for q_dtype in gbn.Q_DTYPE_CODES:
            for group in (0, 128):
                q, scale, h, rstd = gbn.rms_add_fwd_q8(d["x"], d["residual"], d["gamma"], EPS, q_dtype=q_dtype,
                                                       group=group, kernel=kernel)
                check_q8(h[fine].cpu(), t["gamma"], q[fine], scale[fine], rstd[fine], group)
                assert (q[4].float() == 0).all() and (scale[4] == 0).all()
                assert q[5].float().abs().max() == (448 if q_dtype != torch.int8 else 127)
                if group == 0:
                    assert torch.isnan(scale[1:4]).all()
                    if q_dtype != torch.int8:
                        assert torch.isnan(q[1].float()).all()
                else:
                    assert torch.isnan(scale[1, (N // 2) // 128]) and torch.isnan(scale[2, 0])
                    assert torch.isnan(scale[3, (N - 1) // 128])


def test_leading_dimensions_and_no_rows():
    t = inputs(6, 264, "bf16", seed=7)
    x, r, gamma = (t[k].cuda() for k in ("x", "residual", "gamma"))
    y, h, rstd = gbn.rms_add_fwd(x.view(2, 3, 264), r.view(2, 3, 264), gamma, EPS)
    assert y.shape == (2, 3, 264) and rstd.shape == (6,)
    check_forward(t, y.view(6, 264), h.view(6, 264), rstd)
    q, scale, rstd = gbn.rms_fwd_q8(x.view(2, 3, 264), gamma, EPS, group=128)
    assert scale.shape == (2, 3, 3)
    check_q8(t["x"], t["gamma"], q.view(6, 264), scale.view(6, 3), rstd, 128)
    none = x[:0]
    y, h, rstd = gbn.rms_add_fwd(none, none, gamma, EPS)
    assert y.shape == (0, 264) and rstd.shape == (0,)
    gbn.rms_fwd_q8(none, gamma, EPS)
    dg = torch.full((264,), 3.0, device="cuda")
    gbn.rms_add_bwd(none, none, none, gamma, rstd, dgamma=dg, accumulate=True)
    assert (dg == 3).all()
    gbn.rms_add_bwd(none, none, none, gamma, rstd, dgamma=dg)
    assert (dg == 0).all()


@pytest.mark.parametrize("N", [1024, 4096, 771])
@pytest.mark.parametrize("grad_dtype", ["f32", "bf16"])
def test_accumulate_and_grad_dtype(N, grad_dtype):
    t = inputs(700, N, "bf16", seed=8)
    d = {k: v.cuda() for k, v in t.items()}
    _, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS)
    before = (50.0 * torch.randn(N, generator=torch.Generator().manual_seed(3))).to(DT[grad_dtype])
    dg = before.cuda()
    dx, got = gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd, dgamma=dg, accumulate=True,
                              grad_dtype=DT[grad_dtype])
    assert got is dg
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg, before)
    dx, dg = gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd, grad_dtype=DT[grad_dtype])
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg)


def test_backward_is_the_same_from_run_to_run():
    t = inputs(1000, 4096, "bf16", seed=9)
    d = {k: v.cuda() for k, v in t.items()}
    _, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS)
    first = [a.clone() for a in gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd)]
    for _ in range(5):
        for a, b in zip(first, gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd)):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """Central differences of the float64 forward: with f = sum(wy*y) + sum(wh*h) and a step s, the difference is off
    by s^2/6 of the third derivative, which the halved step measures; the kernel's own error is u of its terms."""
    M, N = 3, 24
    t = inputs(M, N, "f32", seed=10)
    x, r, g, wy, wh = (t[k].double() for k in ("x", "residual", "gamma", "dy", "dh"))
    d = {k: v.cuda() for k, v in t.items()}
    _, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS)
    dx, dg = gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd)

    def f(x, g):
        h = x + r
        y = g * h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS)
        return (wy * y).sum() + (wh * h).sum()

    def slope(make, s):
        return (make(s) - make(-s)) / (2 * s)

    for i in range(M):
        for j in range(0, N, 5):
            e = torch.zeros_like(x)
            e[i, j] = 1.0
            coarse, fine = (float(slope(lambda s: f(x + s * e, g), s)) for s in (2e-4, 1e-4))
            tol = abs(coarse - fine) + 1e-7 * (1 + abs(fine)) + 64 * u * (1 + abs(fine))
            assert abs(float(dx[i, j]) - fine) <= tol, (i, j, float(dx[i, j]), fine)
    for j in range(N):
        e = torch.zeros_like(g)
        e[j] = 1.0
        fine = float(slope(lambda s: f(x, g + s * e), 1e-3))  # f is linear in gamma
        assert abs(float(dg[j]) - fine) <= 1e-8 * (1 + abs(fine)) + 64 * u * (1 + abs(fine)), (j, float(dg[j]), fine)


def test_another_stream_and_a_captured_graph():
    M, N = 512, 2048
    t = inputs(M, N, "bf16", seed=11)
    new = inputs(M, N, "bf16", seed=12)
    d = {k: v.cuda() for k, v in t.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS, stream=side)
    dx, dg = gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd, stream=side)
    q, scale, h2, rstd2 = gbn.rms_add_fwd_q8(d["x"], d["residual"], d["gamma"], EPS, stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    check_forward(t, y, h, rstd)
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg)
    check_q8(h2.cpu(), t["gamma"], q, scale, rstd2, 0)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS)
        q, scale, rstd_q = gbn.rms_fwd_q8(h, d["gamma"], EPS, group=128)
        dx, dg = gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd)
    # an eager call of the same inputs between capture and replay
    gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], torch.ones_like(rstd))
    for k, v in new.items():
        d[k].copy_(v)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    check_forward(new, y, h, rstd)
    check_q8(h.cpu(), new["gamma"], q, scale, rstd_q, 128)
    check_backward(new, h.cpu(), rstd.cpu(), dx, dg)


def test_offsets_beyond_32_bits():
    """Rows 2^31 + 8 elements apart: byte and element offsets pass 32 bits."""
    M, N, ld = 3, 1000, (1 << 31) + 8
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    t = inputs(M, N, "bf16", seed=13)
    buf = torch.empty(2 * ld + 4 * N, dtype=torch.bfloat16, device="cuda")
    rows = {}
    for i, k in enumerate(("x", "residual", "dy", "dh")):
        rows[k] = buf[i * N:].as_strided((M, N), (ld, 1))
        rows[k].copy_(t[k])
    gamma = t["gamma"].cuda()
    y, h, rstd = gbn.rms_add_fwd(rows["x"], rows["residual"], gamma, EPS, h=rows["residual"])
    check_forward(t, y, h, rstd)
    dx, dg = gbn.rms_add_bwd(rows["dy"], rows["dh"], h, gamma, rstd, dx=rows["dh"])
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg)
    q, scale, rstd2 = gbn.rms_fwd_q8(h, gamma, EPS)
    check_q8(h.cpu(), t["gamma"], q, scale, rstd2, 0)


def test_refusals():
    x = torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16)
    g = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    r = torch.ones(8, device="cuda")
    for bad in (x.float(), x[:4], x.cpu(), x.t()):
        with pytest.raises(ValueError):
            gbn.rms_add_fwd(x, bad, g, EPS)
        with pytest.raises(ValueError):
            gbn.rms_add_bwd(x, bad, x, g, r)
        with pytest.raises(ValueError):
            gbn.rms_add_fwd(x, x.clone(), g, EPS, y=bad)
    with pytest.raises(ValueError):
        gbn.rms_add_fwd(x, x, g.float(), EPS)
    with pytest.raises(gbn.GbnError):
        gbn.rms_add_fwd(x, x, g, -1.0)
    with pytest.raises(gbn.GbnError):
        gbn.rms_add_fwd(x, x, g, EPS, y=x, h=x)
    with pytest.raises(KeyError):
        gbn.rms_add_fwd(x, x, g, EPS, kernel="slot")
    with pytest.raises(ValueError):
        gbn.rms_fwd_q8(x, g, EPS, q_dtype=torch.uint8)
    with pytest.raises(ValueError):
        gbn.rms_fwd_q8(x, g, EPS, group=32)
    with pytest.raises(ValueError):
        gbn.rms_fwd_q8(x, g, EPS, scale=torch.empty(9, device="cuda"))
    with pytest.raises(ValueError):
        gbn.rms_add_bwd(x, x, x, g, r.half())
    with pytest.raises(ValueError):
        gbn.rms_add_bwd(x, x, x, g, r, grad_dtype=torch.float16)
    with pytest.raises(gbn.GbnError) as e:
        gbn.rms_add_bwd(x, x.clone(), x.clone(), g, r, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4


def test_backward_wait_that_runs_out():
    """A wait limit far below a copy's latency: the kernel reports error 1 and returns, and the next call is right."""
    import ctypes

    M, N = 2000, 4096
    t = inputs(M, N, "bf16", seed=14)
    d = {k: v.cuda() for k, v in t.items()}
    _, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS)
    dx, dg = torch.empty_like(h), torch.empty(N, device="cuda")
    ws = torch.empty(gbn.bwd_workspace_bytes(M, N, h.dtype, False), dtype=torch.uint8, device="cuda")
    assert gbn.device_error() == 0
    opt = gbn.GbnOptions(0, 0, 0, 0, 0, 0, 0, 0, 1)
    s = torch.cuda.current_stream().cuda_stream
    assert gbn.lib().rms_add_bwd(d["dy"].data_ptr(), d["dh"].data_ptr(), h.data_ptr(), d["gamma"].data_ptr(),
                                 rstd.data_ptr(), dx.data_ptr(), dg.data_ptr(), M, N, 2, ws.data_ptr(), ws.numel(), 0,
                                 ctypes.byref(opt), s) == 0
    assert gbn.device_error(clear=True) == 1
    gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd, dx=dx, dgamma=dg, workspace=ws)
    assert gbn.device_error() == 0
    check_backward(t, h.cpu(), rstd.cpu(), dx, dg)


FIRST_CALL_IN_A_CAPTURE = """
import torch
import rmsnorm_backward_gb300 as gbn
x = torch.randn(64, 1536, device="cuda", dtype=torch.bfloat16)
r, dy, dh = (torch.randn_like(x) for _ in range(3))
g = torch.ones(1536, device="cuda", dtype=torch.bfloat16)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, h, rstd = gbn.rms_add_fwd(x, r, g, 1e-6)
    q, scale, _ = gbn.rms_fwd_q8(h, g, 1e-6)
    dx, dg = gbn.rms_add_bwd(dy, dh, h, g, rstd)
    norm = gbn.grad_clip([dg], 0.5)
graph.replay()
torch.cuda.synchronize()
y2, h2, rstd2 = gbn.rms_add_fwd(x, r, g, 1e-6)
dx2, dg2 = gbn.rms_add_bwd(dy, dh, h2, g, rstd2)
assert torch.equal(y, y2) and torch.equal(dx, dx2)
assert torch.equal(norm, gbn.grad_clip([dg2], 0.5)) and torch.equal(dg, dg2)
assert gbn.device_error() == 0
print("captured")
"""


def test_first_call_in_a_capture():
    """A process whose first calls are captured ones."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL_IN_A_CAPTURE], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stdout + r.stderr


def test_two_streams_at_once():
    """The same inputs on two streams, each call with buffers of its own."""
    M, N = 4000, 4096
    t = inputs(M, N, "bf16", seed=15)
    d = {k: v.cuda() for k, v in t.items()}
    _, h, rstd = gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = []
    for _ in range(3):
        for s in streams:
            out.append(gbn.rms_add_fwd(d["x"], d["residual"], d["gamma"], EPS, stream=s)
                       + gbn.rms_add_bwd(d["dy"], d["dh"], h, d["gamma"], rstd, stream=s))
    torch.cuda.synchronize()
    for o in out:
        assert all(torch.equal(a, b) for a, b in zip(o, out[0]))
    check_forward(t, *out[0][:3])
    check_backward(t, h.cpu(), rstd.cpu(), *out[0][3:])


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_codes_at_ties(dtype, group):
    """Values half way between two codes in float32, on rows of every kernel: many rows of few-bit values, whose products
    with the factor often are such."""
    g = torch.Generator().manual_seed(16)
    for N in (64, 496, 640, 1024, 4096, 4808, 8192, 1001, 4099):
        x = (torch.randint(-128, 129, (120, N), generator=g).float() / 64).to(DT[dtype])
        x[:, 0] = 127.0 / 64
        gamma = torch.ones(N, dtype=DT[dtype])
        for q_dtype in gbn.Q_DTYPE_CODES:
            q, scale, rstd = gbn.rms_fwd_q8(x.cuda(), gamma.cuda(), EPS, q_dtype=q_dtype, group=group)
            code, _ = codes_and_scale(x, gamma, rstd.cpu(), q_dtype, group)
            assert torch.equal(q.cpu().view(torch.uint8), code.view(torch.uint8)), (N, q_dtype)
            q, scale, _, rstd = gbn.rms_add_fwd_q8(x.cuda(), torch.zeros_like(x).cuda(), gamma.cuda(), EPS,
                                                   q_dtype=q_dtype, group=group)
            assert torch.equal(q.cpu().view(torch.uint8), code.view(torch.uint8)), (N, q_dtype)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("N", [517, 1030, 2049, 2055, 4099, 6474])
def test_codes_of_rows_across_boundaries(N, dtype, group):
    """The same codes from both kernels at every shift of rows and of codes, with groups of zeros, tiny, infinite and NaN
    values; bytes between the rows' codes stay as they are."""
    M = 37 if N > 2100 else 2500  # the latter: several rows to a slot
    g = torch.Generator().manual_seed(N)
    x = torch.randn(M, N, generator=g).to(DT[dtype])
    tiny = 6e-8 if dtype == "f16" else 1e-34
    x[1] = 0
    x[2, 100:300] = 0
    x[3, 100:300] = tiny
    x[4, 130] = float("inf")
    x[5, 255] = float("nan")
    x[6, N - 1] = float("-inf")
    x[7, 0] = float("nan")
    x[M // 2:M // 2 + 8] = x[:8]
    x, gamma = x.cuda(), torch.randn(N, generator=g).to(DT[dtype]).cuda()
    for more, more_q, at in ((0, 0, 0), (1, 1, 0), (2, 0, 1), (5, 3, 3), (8 - N % 8, 8 - N % 8, 0), (8 - N % 8, 8 - N % 8, 4)):
        def rows(values, start, dt, ld):
            buf = torch.full((start + M * ld + 8,), 85, dtype=dt, device="cuda")
            view = buf.as_strided((M, N), (ld, 1), start)
            if values is not None:
                view.copy_(values)
            return buf, view

        _, xs = rows(x, at, DT[dtype], N + more)
        _, rs = rows(torch.zeros_like(x), at, DT[dtype], N + more)
        for q_dtype in gbn.Q_DTYPE_CODES:
            for res in (False, True):
                got = []
                for kernel in ("auto", "plain"):
                    buf, q = rows(None, at, torch.uint8, N + more_q)
                    if res:
                        _, h = rows(None, at, DT[dtype], N + more)
                        out = gbn.rms_add_fwd_q8(xs, rs, gamma, EPS, q_dtype=q_dtype, group=group, q=q.view(q_dtype), h=h,
                                                 kernel=kernel)
                        assert torch.equal(torch.nan_to_num(h), torch.nan_to_num(x)), (more, q_dtype, kernel)
                    else:
                        out = gbn.rms_fwd_q8(xs, gamma, EPS, q_dtype=q_dtype, group=group, q=q.view(q_dtype), kernel=kernel)
                    got.append((buf, out[1]))
                assert torch.equal(got[0][0], got[1][0]), (more, more_q, at, q_dtype, res)
                # rstd's sum may differ in its last bits: (N + 8) / 2 roundings of 2^-24 at most, halved by the root
                torch.testing.assert_close(got[0][1], got[1][1], rtol=(N + 8) * 2.0**-25, atol=0, equal_nan=True)
