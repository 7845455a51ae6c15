"""Cases of the residual RMSNorm, its gradient, its 8-bit form and the gradient clip.

Where ``own`` is false, ``run`` computes an operator in elementary torch
operations; where it is true, it makes the calls of rmsnorm_backward_gb300.
"""
import random

import torch

own = False

EPS = 1e-6
CLIP_EPS = 1e-6
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
Q_DTYPES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
Q_MAX = {"e4m3": 448.0, "int8": 127.0}
GROUP = 128
# rows x columns of the largest drawn case of each kind of norm
MOST = 1 << 26


def listed():
    return [
        # one decoding step of a few sequences: the residual's addition before each norm
        {"name": "add_fwd_decode", "op": "add_fwd", "M": 4, "N": 4096, "dtype": "bf16"},
        # a training step's forward, the package's headline shape
        {"name": "add_fwd_train", "op": "add_fwd", "M": 16384, "N": 4096, "dtype": "bf16"},
        # a ragged batch of an odd width: no row but every eighth starts on 16 bytes
        {"name": "add_fwd_odd", "op": "add_fwd", "M": 1151, "N": 8193, "dtype": "f16"},
        # decoding into an 8-bit product: one scale a token
        {"name": "q8_decode", "op": "add_q8", "M": 32, "N": 8192, "dtype": "bf16", "q": "e4m3", "group": 0},
        # prefill into an 8-bit product with a scale for each 128 columns, wide rows
        {"name": "q8_prefill", "op": "add_q8", "M": 8192, "N": 16384, "dtype": "bf16", "q": "e4m3", "group": GROUP},
        # the first norm of a model (no residual yet), whole-number codes, a ragged number of tokens
        {"name": "q8_int8", "op": "q8", "M": 2047, "N": 5128, "dtype": "f16", "q": "int8", "group": 0},
        # the gradient at the smallest shape of the package's workloads
        {"name": "add_bwd_small", "op": "add_bwd", "M": 64, "N": 256, "dtype": "f32"},
        # a training step's backward, the package's headline shape
        {"name": "add_bwd_train", "op": "add_bwd", "M": 16384, "N": 4096, "dtype": "bf16"},
        # the backward of a ragged batch of an odd width
        {"name": "add_bwd_odd", "op": "add_bwd", "M": 1151, "N": 8191, "dtype": "f16"},
        # clipping the norms' own gradients, as a fine-tuning of the norms alone has them
        {"name": "clip_gammas", "op": "clip", "layers": 32, "width": 4096, "inner": 0, "odd": 0, "dtype": "f32", "over": True},
        # clipping all gradients of a model
        {"name": "clip_model", "op": "clip", "layers": 16, "width": 2048, "inner": 8192, "odd": 0, "dtype": "bf16", "over": True},
        # the ordinary step, whose norm is below the limit, on a bucket of ragged parameters
        {"name": "clip_below", "op": "clip", "layers": 24, "width": 1000, "inner": 4001, "odd": 1, "dtype": "f32", "over": False},
    ]


def _log(rng, low, high):
    return int(round(low * (high / low) ** rng.random()))


def draw(rng: random.Random):
    op = rng.choice(("add_fwd", "add_q8", "q8", "add_bwd", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "clip":
        width = _log(rng, 64, 4096)
        inner = rng.choice((0, 4 * width, 4 * width + 1, _log(rng, 64, 16384)))
        layers = _log(rng, 1, 64)
        most = (1 << 27) if dtype == "f32" else (1 << 28)
        layers = max(1, min(layers, most // (2 * width + width * (width + inner))))
        return {"op": op, "layers": layers, "width": width, "inner": inner, "odd": rng.choice((0, 1)), "dtype": dtype,
                "over": rng.choice((True, False))}
    N = _log(rng, 64, 16384)
    if rng.random() < 0.6:  # most widths are multiples of 8; the others are as they fall
        N = max(64, N // 8 * 8)
    M = min(_log(rng, 1, 32768), max(1, (MOST if dtype != "f32" else MOST // 2) // N))
    case = {"op": op, "M": M, "N": N, "dtype": dtype}
    if op in ("add_q8", "q8"):
        case["q"] = rng.choice(("e4m3", "e4m3", "int8"))
        case["group"] = rng.choice((0, GROUP))
    return case


def _sizes(case):
    """Elements of each gradient: two norm weights, a square and an inner matrix a layer; ``odd`` makes them ragged."""
    w, inner = case["width"], case["inner"]
    layer = [w, w] + ([w * w, w * inner] if inner else [])
    return [n + (i * 7 % 5 if case["odd"] else 0) for i, n in enumerate(layer * case["layers"])]


def _normal(g, shape, dtype, scale=1.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(generator=g)
    return t.mul_(scale).to(dtype)


def _stream(g, M, N, dtype):
    """A residual stream: normal, with a few columns much larger than the others."""
    t = torch.empty(M, N, dtype=torch.float32, device="cuda").normal_(generator=g)
    cols = torch.randperm(N, generator=g, device="cuda")[: max(1, N // 100)]
    t[:, cols] *= 20.0
    return t.to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] == "clip":
        sizes = _sizes(case)
        total = sum(sizes)
        # one bucket for the gradients and one for the clipped ones; below the limit the bucket is clipped in place
        bucket = _normal(g, (total,), dt, 1e-2)
        s["grads"] = list(bucket.split(sizes))
        s["bucket"] = bucket
        norm = 1e-2 * total ** 0.5
        s["max_norm"] = 0.3 * norm if case["over"] else 4.0 * norm
        s["out"] = torch.empty_like(bucket) if case["over"] else bucket
        s["outs"] = list(s["out"].split(sizes))
        s["norm"] = torch.empty((), dtype=torch.float32, device="cuda")
        if own:  # the plan of a program that keeps its gradients in place
            import rmsnorm_backward_gb300 as gbn

            s["list"] = gbn.GradList(s["grads"])
            s["out_list"] = gbn.GradList(s["outs"]) if case["over"] else None
            s["workspace"] = torch.empty(gbn.grad_workspace_bytes(), dtype=torch.uint8, device="cuda")
        return s
    M, N = case["M"], case["N"]
    s["gamma"] = (1.0 + 0.02 * _normal(g, (N,), torch.float32)).to(dt)
    s["rstd"] = torch.empty(M, dtype=torch.float32, device="cuda")
    if case["op"] == "add_bwd":
        s["h"] = _stream(g, M, N, dt)
        s["dy"] = _normal(g, (M, N), dt, 1e-2)
        s["dh"] = _normal(g, (M, N), dt, 1e-2)
        h = s["h"].float()
        s["rstd"] = torch.rsqrt((h * h).mean(-1) + EPS)
        s["dx"] = torch.empty(M, N, dtype=dt, device="cuda")
        s["dgamma"] = torch.empty(N, dtype=torch.float32, device="cuda")
        if own:
            import rmsnorm_backward_gb300 as gbn

            s["workspace"] = torch.empty(gbn.bwd_workspace_bytes(M, N, dt, False), dtype=torch.uint8, device="cuda")
        return s
    s["x"] = _normal(g, (M, N), dt)
    if case["op"] != "q8":
        s["residual"] = _stream(g, M, N, dt)
        s["h"] = torch.empty(M, N, dtype=dt, device="cuda")
    if case["op"] == "add_fwd":
        s["y"] = torch.empty(M, N, dtype=dt, device="cuda")
    else:
        s["codes"] = torch.empty(M, N, dtype=Q_DTYPES[case["q"]], device="cuda")
        s["scale"] = torch.empty((M, -(-N // GROUP)) if case["group"] else (M,), dtype=torch.float32, device="cuda")
    return s


def _own(s):
    import rmsnorm_backward_gb300 as gbn

    op = s["op"]
    if op == "add_fwd":
        return gbn.rms_add_fwd(s["x"], s["residual"], s["gamma"], EPS, y=s["y"], h=s["h"], rstd=s["rstd"])
    if op == "q8":
        return gbn.rms_fwd_q8(s["x"], s["gamma"], EPS, group=s["group"], q=s["codes"], scale=s["scale"], rstd=s["rstd"])
    if op == "add_q8":
        return gbn.rms_add_fwd_q8(s["x"], s["residual"], s["gamma"], EPS, group=s["group"], q=s["codes"], scale=s["scale"],
                                  h=s["h"], rstd=s["rstd"])
    if op == "add_bwd":
        return gbn.rms_add_bwd(s["dy"], s["dh"], s["h"], s["gamma"], s["rstd"], dx=s["dx"], dgamma=s["dgamma"],
                               workspace=s["workspace"])
    norm = gbn.grad_clip(s["list"], s["max_norm"], eps=CLIP_EPS, out=s["out_list"], norm=s["norm"], workspace=s["workspace"])
    return norm, s["out"]


def _quantized(v, rstd, q, group):
    """Codes and scales of v * rstd in float32: q = round(v * (Q / max|v|)), scale = rstd * max|v| / Q.

    Q is a tensor in the quotients: torch takes a number over a tensor as a product with the reciprocal, which is
    another float32 value."""
    M, N = v.shape
    top = Q_MAX[q]
    if group:
        width = -(-N // group) * group
        wide = torch.nn.functional.pad(v, (0, width - N)).view(M, width // group, group)
        most = wide.abs().amax(-1)
        t = (wide * (torch.full_like(most, top) / most)[..., None]).view(M, width)[:, :N]
        scale = rstd[:, None] * most / torch.full_like(most, top)
    else:
        most = v.abs().amax(-1)
        t = v * (torch.full_like(most, top) / most)[:, None]
        scale = rstd * most / torch.full_like(most, top)
    codes = t.to(torch.float8_e4m3fn) if q == "e4m3" else t.round().to(torch.int8)
    return codes.contiguous(), scale


def _plain(s):
    op = s["op"]
    if op == "clip":
        flat = torch.cat(s["grads"])
        # the sum of squares is long: in 64 bits
        norm = flat.double().square().sum().sqrt()
        coef = torch.clamp(s["max_norm"] / (norm + CLIP_EPS), max=1.0).float()
        return norm.float(), (flat.float() * coef).to(flat.dtype)
    dt = DTYPES[s["dtype"]]
    g = s["gamma"].float()
    if op == "add_bwd":
        h, dy, rs = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
        xhat, dyhat = h * rs, dy * g
        dx = rs * (dyhat - xhat * (dyhat * xhat).mean(-1, keepdim=True)) + s["dh"].float()
        return dx.to(dt), (dy * xhat).sum(0)
    if op == "q8":
        h = s["x"].float()
    else:
        stored = (s["x"].float() + s["residual"].float()).to(dt)
        h = stored.float()
    rstd = torch.rsqrt((h * h).mean(-1) + EPS)
    if op == "add_fwd":
        return (g * h * rstd[:, None]).to(dt), stored, rstd
    codes, scale = _quantized(g * h, rstd, s["q"], s["group"])
    return (codes, scale, rstd) if op == "q8" else (codes, scale, stored, rstd)


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    es = BYTES[case["dtype"]]
    if case["op"] == "clip":
        n = sum(_sizes(case))
        # below the limit nothing has to be written
        return {"bytes": n * es * (2 if case["over"] else 1) + 4, "flops": n * (3 if case["over"] else 2)}
    M, N = case["M"], case["N"]
    n = M * N
    if case["op"] == "add_fwd":
        return {"bytes": 4 * n * es + N * es + 4 * M, "flops": 5 * n}
    if case["op"] == "add_bwd":
        return {"bytes": 4 * n * es + N * es + 4 * M + 4 * N, "flops": 10 * n}
    scales = M * (-(-N // GROUP) if case["group"] else 1)
    streams = 1 if case["op"] == "q8" else 3
    return {"bytes": streams * n * es + n + N * es + 4 * scales + 4 * M, "flops": 7 * n}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        flat = s["bucket"].to(torch.float64)
        norm = torch.linalg.vector_norm(flat)
        factor = s["max_norm"] / (norm + CLIP_EPS)
        return norm, flat * factor if float(factor) < 1.0 else flat
    gamma = s["gamma"].to(torch.float64)
    N = case["N"]
    if case["op"] == "add_bwd":
        dx = torch.empty_like(s["dy"], dtype=torch.float64)
        dgamma = torch.zeros(N, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 24) // N)
        for at in range(0, case["M"], step):
            rows = slice(at, at + step)
            inv = s["rstd"][rows].to(torch.float64).unsqueeze(1)
            normed = s["h"][rows].to(torch.float64) * inv
            dy = s["dy"][rows].to(torch.float64)
            dgamma += torch.einsum("mn,mn->n", dy, normed)
            weighted = dy * gamma
            along = torch.einsum("mn,mn->m", weighted, normed).unsqueeze(1) / N
            dx[rows] = (weighted - along * normed) * inv + s["dh"][rows].to(torch.float64)
        return dx, dgamma
    dt = DTYPES[case["dtype"]]
    stored = s["x"].to(torch.float64)
    if case["op"] != "q8":
        stored = stored + s["residual"].to(torch.float64)
    # the statistics are those of the stored sum
    held = stored.to(dt).to(torch.float64)
    rstd = 1.0 / torch.sqrt(held.pow(2).sum(1) / N + EPS)
    normed = held * rstd.unsqueeze(1) * gamma
    if case["op"] == "add_fwd":
        return normed, stored, rstd
    top = Q_MAX[case["q"]]
    if case["group"]:
        parts = normed.split(GROUP, dim=1)
        scale = torch.stack([p.abs().max(1).values for p in parts], dim=1) / top
        wide = scale.repeat_interleave(GROUP, dim=1)[:, :N]
    else:
        scale = normed.abs().max(1).values / top
        wide = scale.unsqueeze(1)
    codes = (normed / wide).to(torch.float8_e4m3fn).to(torch.float64) if case["q"] == "e4m3" else None
    return (codes, scale, rstd) if case["op"] == "q8" else (codes, scale, stored, rstd)
