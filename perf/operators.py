"""The operators around the collectives, as they are timed and checked.

Three families, each with its plain form (elementary torch operations in 32
bits or more, rounded once at the end) and the library's call:

  norm    RMS norm of a residual stream: the residual's addition, the norm,
          and an output in the stream's type or in e4m3 with scales
          (api.rmsnorm)
  rsnorm  the same behind a reduce-scatter: the R partial sums of tensor
          parallel ranks are added, and each rank norms its own tokens
          (Comm.reduce_scatter_rmsnorm)
  back    the norm's backward pass: the stream's gradient, and each rank's
          gradient of the weight (api.rmsnorm_backward)
  clip    the global 2-norm over many gradient tensors, and the gradients
          scaled to a largest norm (Comm.grad_norm, Comm.grad_clip); with
          "clip": False the norm alone

`own` chooses between the two; nothing of the package is imported for the
plain forms.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "bf16": 2}
E4M3_MAX = 448.0
TINY = 2.0 ** -126  # the smallest scale: a group of zeros has this one


def listed():
    return [
        # one new token of one sequence: the call's latency is all that counts
        dict(name="norm_1x4096", op="norm", rows=1, cols=4096, dtype="bf16", out="same", group=0,
             residual=True, pad=0),
        # a batch of new tokens ahead of an 8-bit product, one scale a token
        dict(name="norm_32x8192_e4m3", op="norm", rows=32, cols=8192, dtype="bf16", out="e4m3",
             group=0, residual=True, pad=0),
        # a prompt ahead of an 8-bit product, a scale for each 128 columns
        dict(name="norm_8192x8192_e4m3", op="norm", rows=8192, cols=8192, dtype="bf16", out="e4m3",
             group=128, residual=True, pad=0),
        # odd rows that are a part of wider ones, in float32, no residual: a norm on a slice
        dict(name="norm_16384x1001_f32", op="norm", rows=16384, cols=1001, dtype="f32", out="same",
             group=0, residual=False, pad=22),
        # one token of each of 8 tensor parallel ranks
        dict(name="rsnorm_r8_1x4096", op="rsnorm", R=8, rows=1, cols=4096, dtype="bf16", out="same",
             group=0, residual=True),
        # 2048 tokens over 8 ranks, 8-bit output for the all-gather that follows
        dict(name="rsnorm_r8_256x8192_e4m3", op="rsnorm", R=8, rows=256, cols=8192, dtype="bf16",
             out="e4m3", group=128, residual=True),
        # a small model's step
        dict(name="back_64x1024_f32", op="back", R=1, rows=64, cols=1024, dtype="f32",
             residual=True),
        # odd columns, 8 ranks' tokens, no gradient from the residual's side
        dict(name="back_r8_625x2049", op="back", R=8, rows=625, cols=2049, dtype="bf16",
             residual=False),
        # a long sequence's step
        dict(name="back_8192x8192", op="back", R=1, rows=8192, cols=8192, dtype="bf16",
             residual=True),
        # one float32 gradient vector of 64 MiB, its norm alone (a step's log)
        dict(name="clip_norm_64MiB_f32", op="clip", tensors=1, total=16777216, dtype="f32",
             clip=False),
        # a model's parameters one by one: a few large matrices, many small vectors, odd sizes
        dict(name="clip_291_tensors", op="clip", tensors=291, total=40000000, dtype="bf16",
             clip=True),
        # the reduce-scattered shards of 40 gradient buckets of 25 MiB, all ranks
        dict(name="clip_40_buckets_25MiB", op="clip", tensors=40, total=40 * 13107200, dtype="bf16",
             clip=True),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cols(rng):
    if rng.random() < 0.4:  # any length: odd ones, shorter than a wave, not a multiple of a vector
        return _spread(rng, 33, 16000) | 1
    while True:
        c = rng.choice((1, 5, 7, 9)) * 2 ** rng.randint(5, 14)
        if 64 <= c <= 16384:
            return c


def draw(rng):
    op = rng.choice(("norm", "rsnorm", "back", "clip"))
    dtype = rng.choice(("bf16", "bf16", "f32"))
    if op == "clip":
        tensors = _spread(rng, 1, 700)
        total = max(_spread(rng, 20000, 200_000_000), 40 * tensors)
        return dict(op=op, tensors=tensors, total=total | rng.randint(0, 1), dtype=dtype,
                    clip=rng.random() < 0.7)
    cols = _cols(rng)
    R = 1 if op == "norm" or (op == "back" and rng.random() < 0.5) else rng.choice((2, 4, 5, 8, 16))
    most = max(1, 8192 * 8192 // (cols * R * (R if op == "rsnorm" else 1)))
    rows = _spread(rng, 1, min(most, 16384))
    if rows > 8:
        rows |= 1
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.6)
    if op != "norm":
        case["R"] = R
    if op != "back":
        case["out"] = rng.choice(("same", "e4m3"))
        case["group"] = rng.choice((0, 0, 32, 64, 128, 256)) if case["out"] == "e4m3" else 0
    if op == "norm":
        case["pad"] = rng.choice((0, 0, 3, 64))
    return case


def _generator(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1_000_003 + salt)
    return g


def _stream_values(g, rows, cols, dtype, scale):
    """A residual stream's values: a few columns are far larger than the others."""
    x = torch.randn((rows, cols), generator=g, device="cuda", dtype=torch.float32)
    wide = torch.rand((cols,), generator=g, device="cuda")
    return x.mul_(scale * torch.where(wide > 0.99, 12.0, 1.0)).to(dtype)


def _sizes(case):
    """Lengths of the tensors of a gradient list: equal buckets, or few large and many small."""
    n, total = case["tensors"], case["total"]
    if total % n == 0:
        return [total // n] * n
    rng = np.random.default_rng([case["tensors"], case["total"]])
    w = np.exp(rng.normal(0.0, 2.5, n))
    sizes = np.maximum(1, np.floor(w / w.sum() * (total - n))).astype(np.int64)
    sizes[int(np.argmax(sizes))] += total - int(sizes.sum())
    return [int(s) for s in sizes]


def prepare(case, seed):
    dt = TYPES[case["dtype"]]
    op = case["op"]
    g = _generator(seed, 17)
    s = dict(case=case)
    if own:
        from collective_communication_ring_amd import api
        s["api"] = api
    if op == "clip":
        # the tensors are views of one flat buffer, as a trainer's buckets hold them
        flat = torch.empty(case["total"], device="cuda", dtype=dt)
        for lo in range(0, case["total"], 1 << 26):
            part = flat[lo:lo + (1 << 26)]
            part.copy_(torch.randn(part.shape, generator=g, device="cuda") * 0.02)
        sizes = _sizes(case)
        s["flat"] = flat
        s["norm"] = torch.empty(1, device="cuda", dtype=torch.float32)
        # about a third of the gradients' norm, so that they are scaled
        s["max_norm"] = 0.02 * math.sqrt(case["total"]) / 3
        if case["clip"]:
            s["clipped"] = torch.empty_like(flat)
        if own:
            s["comm"] = api.Comm(2, 1, "float32")
            s["grads"] = api.TensorList(flat.split(sizes))
            if case["clip"]:
                s["out"] = api.TensorList(s["clipped"].split(sizes))
        return s
    R = case.get("R", 1)
    rows, cols = case["rows"], case["cols"]
    tokens = R * rows
    s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
    if op == "back":
        s["x"] = _stream_values(g, tokens, cols, dt, 1.5)
        s["dy"] = (torch.randn((tokens, cols), generator=g, device="cuda") * 0.02).to(dt)
        if case["residual"]:
            s["dsum"] = (torch.randn((tokens, cols), generator=g, device="cuda") * 0.02).to(dt)
        ms = s["x"].double().square().mean(dim=1)
        s["rstd"] = (1.0 / torch.sqrt(ms + EPS)).to(torch.float32)
        s["dx"] = torch.empty((tokens, cols), device="cuda", dtype=dt)
        s["dweight"] = torch.empty((R, cols), device="cuda", dtype=torch.float32)
        if own:
            s["workspace"] = api.rmsnorm_backward_workspace(R, tokens, cols)
        return s
    ydt = torch.float8_e4m3fn if case["out"] == "e4m3" else dt
    groups = -(-cols // (case["group"] or cols))
    if op == "norm":
        width = cols + case["pad"]
        s["x"] = _stream_values(g, rows, width, dt, 1.0)[:, :cols]
        shape, per_token = (rows, cols), (rows,)
    else:
        s["send"] = _stream_values(g, R, R * rows * cols, dt, 1.0 / math.sqrt(R))
        shape, per_token = (R, rows * cols), (R, rows)
        if own:
            s["comm"] = api.Comm(R, R * rows * cols, {"f32": "float32"}.get(case["dtype"], "bf16"))
    if case["residual"]:
        s["residual"] = _stream_values(g, tokens, cols, dt, 1.5).view(shape)
        s["sum"] = torch.empty(shape, device="cuda", dtype=dt)
    s["y"] = torch.empty(shape, device="cuda", dtype=ydt)
    s["rstd"] = torch.empty(per_token, device="cuda", dtype=torch.float32)
    if case["out"] == "e4m3":
        s["scale"] = torch.empty(per_token[:-1] + (per_token[-1] * groups,) if op == "rsnorm"
                                 else per_token + (groups,), device="cuda", dtype=torch.float32)
    return s


# ---- plain forms --------------------------------------------------------------

def _plain_norm(h, weight, case, shape, per_token, dt, residual):
    """y, rstd (and the new stream, and scales) of h [tokens, cols] in float32."""
    cols = case["cols"]
    out = {}
    rstd = 1.0 / torch.sqrt((h * h).sum(dim=1) / cols + EPS)
    v = h * rstd[:, None] * weight.to(torch.float32)
    out["rstd"] = rstd.view(per_token)
    if residual:
        out["sum"] = h.to(dt).view(shape)
    if case["out"] == "same":
        out["y"] = v.to(dt).view(shape)
        return out
    group = case["group"] or cols
    groups = -(-cols // group)
    padded = torch.nn.functional.pad(v, (0, groups * group - cols)).view(-1, groups, group)
    amax = padded.abs().amax(dim=2)
    scale = torch.clamp(amax / E4M3_MAX, min=TINY)
    q = (padded / scale[:, :, None]).view(-1, groups * group)[:, :cols]
    out["y"] = q.to(torch.float8_e4m3fn).reshape(shape)
    out["scale"] = scale.reshape(per_token[:-1] + (-1,) if case["op"] == "rsnorm"
                                 else per_token + (groups,))
    return out


def _plain(s):
    case = s["case"]
    dt = TYPES[case["dtype"]]
    op = case["op"]
    if op == "clip":
        norm = torch.sqrt((s["flat"].to(torch.float64) ** 2).sum()).to(torch.float32)
        if not case["clip"]:
            return {"norm": norm.view(1)}
        coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
        return {"norm": norm.view(1), "grads": (s["flat"].to(torch.float32) * coef).to(dt)}
    R, cols = case.get("R", 1), case["cols"]
    if op == "back":
        w = s["weight"].to(torch.float32)
        xhat = s["x"].to(torch.float32) * s["rstd"][:, None]
        dy = s["dy"].to(torch.float32)
        gy = dy * w
        dx = s["rstd"][:, None] * (gy - xhat * ((gy * xhat).sum(dim=1, keepdim=True) / cols))
        if case["residual"]:
            dx = dx + s["dsum"].to(torch.float32)
        return {"dx": dx.to(dt), "dweight": (dy * xhat).view(R, -1, cols).sum(dim=1)}
    if op == "norm":
        h = s["x"].to(torch.float32)
        shape, per_token = (case["rows"], cols), (case["rows"],)
    else:
        h = s["send"].to(torch.float32).sum(dim=0).view(-1, cols)
        shape, per_token = (R, case["rows"] * cols), (R, case["rows"])
    if case["residual"]:
        h = h + s["residual"].to(torch.float32).view(-1, cols)
    return _plain_norm(h, s["weight"], case, shape, per_token, dt, case["residual"])


def run(s):
    if not own:
        return _plain(s)
    case = s["case"]
    op = case["op"]
    api = s["api"]
    if op == "clip":
        s["comm"].grad_norm(s["grads"], s["norm"])
        if not case["clip"]:
            return {"norm": s["norm"]}
        s["comm"].grad_clip(s["grads"], s["norm"], s["max_norm"], out=s["out"])
        return {"norm": s["norm"], "grads": s["clipped"]}
    if op == "back":
        api.rmsnorm_backward(s["dy"], s["x"], s["weight"], s["rstd"], s["dx"], s["dweight"],
                             dsum=s.get("dsum"), workspace=s["workspace"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "norm":
        api.rmsnorm(s["x"], s["weight"], s["y"], EPS, residual=s.get("residual"), sum=s.get("sum"),
                    scale=s.get("scale"), group=case["group"], rstd=s["rstd"])
    else:
        s["comm"].reduce_scatter_rmsnorm(s["send"], s["weight"], s["y"], EPS,
                                         residual=s.get("residual"), sum=s.get("sum"),
                                         scale=s.get("scale"), group=case["group"], rstd=s["rstd"])
    return {k: s[k] for k in ("y", "rstd", "sum", "scale") if k in s}


def work(case):
    z, op = SIZE[case["dtype"]], case["op"]
    if op == "clip":
        n = case["total"]
        return {"bytes": (2 if case["clip"] else 1) * n * z + 4, "flops": (3 if case["clip"] else 2) * n}
    R, cols = case.get("R", 1), case["cols"]
    n = R * case["rows"] * cols
    if op == "back":
        return {"bytes": (4 if case["residual"] else 3) * n * z + cols * z + R * cols * 4
                + R * case["rows"] * 4, "flops": 10 * n}
    parts = R if op == "rsnorm" else 1
    b = (parts + (2 if case["residual"] else 0)) * n * z + cols * z + R * case["rows"] * 4
    if case["out"] == "e4m3":
        b += n + R * case["rows"] * -(-cols // (case["group"] or cols)) * 4
    else:
        b += n * z
    return {"bytes": b, "flops": (parts + 5) * n}


# ---- from the definitions, in 64 bits -------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        total = torch.zeros((), dtype=torch.float64, device="cuda")
        for part in s["flat"].split(1 << 26):
            d = part.double()
            total += torch.dot(d, d)
        norm = torch.sqrt(total)
        if not case["clip"]:
            return {"norm": norm.view(1)}
        coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm.view(1), "grads": s["flat"].double() * coef}
    R, cols, rows = case.get("R", 1), case["cols"], case["rows"]
    w = s["weight"].double()
    if op == "back":
        dx = torch.empty((R * rows, cols), dtype=torch.float64, device="cuda")
        dw = torch.zeros((R, cols), dtype=torch.float64, device="cuda")
        for r in range(R):
            for lo in range(r * rows, (r + 1) * rows, 2048):
                at = slice(lo, min(lo + 2048, (r + 1) * rows))
                n = s["x"][at].double() * s["rstd"][at, None].double()
                dy = s["dy"][at].double()
                along = ((dy * w) * n).mean(dim=1, keepdim=True)
                dx[at] = (dy * w - along * n) * s["rstd"][at, None].double()
                if case["residual"]:
                    dx[at] += s["dsum"][at].double()
                dw[r] += torch.linalg.vecdot(dy, n, dim=0)
        return {"dx": dx, "dweight": dw}
    if op == "norm":
        h = s["x"].double()
    else:
        h = torch.zeros((R, rows * cols), dtype=torch.float64, device="cuda")
        for q in range(R):
            h += s["send"][q].double().view(R, rows * cols)
        h = h.view(R * rows, cols)
    if case["residual"]:
        h = h + s["residual"].double().reshape(R * rows, cols)
    shape = (rows, cols) if op == "norm" else (R, rows * cols)
    inv = (h.pow(2).mean(dim=1) + EPS).pow(-0.5)
    v = h * inv[:, None] * w
    out = {"rstd": inv.view((rows,) if op == "norm" else (R, rows))}
    if case["residual"]:
        out["sum"] = h.view(shape)
    if case["out"] == "same":
        out["y"] = v.view(shape)
        return out
    group = case["group"] or cols
    groups = -(-cols // group)
    scale = torch.empty((R * rows, groups), dtype=torch.float64, device="cuda")
    for k in range(groups):
        part = v[:, k * group:(k + 1) * group]
        scale[:, k] = torch.clamp(part.abs().amax(dim=1) / E4M3_MAX, min=TINY)
        part /= scale[:, k:k + 1]
    out["y"] = v.view(shape)  # before its rounding to e4m3, as the others before theirs
    out["scale"] = scale.view((rows, groups) if op == "norm" else (R, rows * groups))
    return out
