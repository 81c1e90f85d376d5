"""The library's operators at the edges of a loss-scaled backward pass, case by case.

Four operators, each in a plain form (elementary torch operations, 32 or 64
bits) and as the calls a training program makes of the library:

    norm   global L2 norm of a gradient list, with every tensor's own norm
    clip   that norm, then the gradients scaled to a largest norm
    loss   softmax cross entropy of a head  logits = hidden @ weight.T
    grad   the same with the loss-scaled gradients of hidden and weight

Gradient lists are those of the library's workloads (one flat tensor, the
161 tensors of a convolutional network, a 24-layer transformer with a
vocabulary of 50257, a ragged list); heads have that vocabulary and the
widths of those lists.
"""
import math

import torch

own = False

TYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16, "float32": torch.float32}
IGNORE = -100


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one million gradients: a small model's step, where launches count
        {"name": "norm_flat", "op": "norm", "list": "flat", "count": 1, "size": 1048576,
         "type": "float16", "scale": 1024.0, "clip": 0.0, "overflow": False},
        # the norm alone of a 355M-parameter transformer, as logged each step
        {"name": "norm_transformer", "op": "norm", "list": "transformer", "layers": 24, "width": 1024,
         "vocab": 50257, "type": "float16", "scale": 65536.0, "clip": 1.0, "overflow": False},
        # clipping of a small bf16 model (no loss scale)
        {"name": "clip_flat", "op": "clip", "list": "flat", "count": 1, "size": 1048573,
         "type": "bfloat16", "scale": 1.0, "clip": 0.001, "unscale": False, "out": "bfloat16", "overflow": False},
        # fp16 gradients of a convolutional network unscaled, clipped and widened for an fp32 optimizer
        {"name": "clip_conv", "op": "clip", "list": "conv", "type": "float16", "scale": 128.0, "clip": 1.0,
         "unscale": True, "out": "float32", "overflow": False},
        # many tensors of all sizes, most of them tiny and at odd lengths
        {"name": "clip_ragged", "op": "clip", "list": "ragged", "count": 2000, "log2_max": 18,
         "type": "float32", "scale": 1.0, "clip": 0.5, "unscale": False, "out": "float32", "overflow": False},
        # bf16 gradients of a 355M-parameter transformer
        {"name": "clip_transformer", "op": "clip", "list": "transformer", "layers": 24, "width": 1024,
         "vocab": 50257, "type": "bfloat16", "scale": 1.0, "clip": 1.0, "unscale": False, "out": "bfloat16",
         "overflow": False},
        # the score of one token, as when answers are ranked while they are decoded
        {"name": "loss_one_token", "op": "loss", "tokens": 1, "vocab": 50257, "width": 1024,
         "type": "float16", "ignored": 0.0, "wide_rows": False},
        # evaluation of one odd-length document with a wide head
        {"name": "loss_document", "op": "loss", "tokens": 509, "vocab": 50257, "width": 2048,
         "type": "bfloat16", "ignored": 0.0, "wide_rows": True},
        # evaluation of a full batch
        {"name": "loss_batch", "op": "loss", "tokens": 8192, "vocab": 50257, "width": 1024,
         "type": "float16", "ignored": 0.05, "wide_rows": False},
        # a small classifier head: latency
        {"name": "grad_small", "op": "grad", "tokens": 77, "vocab": 1000, "width": 512, "type": "float16",
         "scale": 1024.0, "scale_on_device": False, "ignored": 0.1, "wide_rows": False},
        # a padded micro-batch of the 355M model, bf16 without a loss scale
        {"name": "grad_micro_batch", "op": "grad", "tokens": 1001, "vocab": 50257, "width": 1024,
         "type": "bfloat16", "scale": 1.0, "scale_on_device": False, "ignored": 0.3, "wide_rows": False},
        # a full batch of the 1.3B model, fp16 with the loss scale on the device
        {"name": "grad_batch", "op": "grad", "tokens": 8192, "vocab": 50257, "width": 2048, "type": "float16",
         "scale": 65536.0, "scale_on_device": True, "ignored": 0.05, "wide_rows": False},
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "clip", "loss", "grad"])
    if op in ("norm", "clip"):
        case = {"op": op, "list": rng.choice(["flat", "ragged", "ragged", "transformer"])}
        if case["list"] == "flat":
            case |= {"count": rng.choice([1, 1, 2, 7]), "size": _log_between(rng, 1000, 40_000_000)}
        elif case["list"] == "ragged":
            case |= {"count": _log_between(rng, 3, 4000), "log2_max": rng.choice([6, 12, 16, 18])}
        else:
            case |= {"layers": rng.randint(1, 24), "width": 64 * rng.randint(1, 16), "vocab": _log_between(rng, 300, 50257)}
        kind = rng.choice(sorted(TYPES))
        case |= {"type": kind, "scale": rng.choice([1.0, 128.0, 1000.0, 65536.0]) if kind == "float16" else 1.0,
                 "clip": rng.choice([0.001, 1.0, 1e9]), "overflow": rng.random() < 0.15}
        if op == "clip":
            case |= {"unscale": rng.random() < 0.5, "out": rng.choice([kind, "float32"])}
            if case["out"] == "float16":  # gradients stay scaled where they stay in 16 bits
                case |= {"unscale": False, "scale": 65536.0 if case["clip"] < 1.0 else max(128.0, case["scale"])}
        return case
    case = {"op": op, "tokens": _log_between(rng, 1, 8192), "vocab": _log_between(rng, 257, 50257),
            "width": 8 * _log_between(rng, 8, 256), "type": rng.choice(["float16", "bfloat16"]),
            "ignored": rng.choice([0.0, 0.05, 0.5]), "wide_rows": rng.random() < 0.3}
    if op == "grad":
        s = 2.0 ** (4 + max(0, int(math.log2(case["tokens"]))))
        case |= {"scale": s if case["type"] == "float16" else 1.0, "scale_on_device": rng.random() < 0.5}
    return case


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _sizes(case):
    """Element counts of a gradient list."""
    if case["list"] == "flat":
        return [case["size"]] * case["count"]
    if case["list"] == "ragged":  # log-uniform lengths, at least 1
        g = torch.Generator().manual_seed(case["count"])
        u = torch.rand(case["count"], generator=g, dtype=torch.float64)
        return [max(1, int(x)) for x in torch.exp(u * (case["log2_max"] * math.log(2.0))).tolist()]
    if case["list"] == "conv":  # the 161 tensors of a 50-layer residual network
        sizes, cin = [64 * 3 * 49, 64, 64], 64
        for blocks, w in zip([3, 4, 6, 3], [64, 128, 256, 512]):
            for b in range(blocks):
                sizes += [w * cin, w, w, w * w * 9, w, w, 4 * w * w, 4 * w, 4 * w]
                if b == 0:
                    sizes += [4 * w * cin, 4 * w, 4 * w]
                cin = 4 * w
        return sizes + [1000 * 2048, 1000]
    d = case["width"]
    layer = [d, d, 3 * d * d, 3 * d, d * d, d, d, d, 4 * d * d, 4 * d, 4 * d * d, d]
    return [case["vocab"] * d, 1024 * d] + layer * case["layers"] + [d, d]


def _prepare_list(case, gen):
    sizes, kind = _sizes(case), TYPES[case["type"]]
    starts, total = [], 0
    for n in sizes:  # every tensor at a multiple of 16 elements of one buffer, zeros between
        starts.append(total)
        total += (n + 15) // 16 * 16
    # magnitudes log-normal over many binades, as measured gradients are
    flat = torch.randn(total, generator=gen, device="cuda").mul_(3.0).add_(math.log2(case["scale"]) - 17.0).exp2_()
    flat *= torch.randint(0, 2, (total,), generator=gen, device="cuda", dtype=torch.int8).mul_(2).sub_(1)
    if kind == torch.float16:
        flat.clamp_(-60000.0, 60000.0)
    ends = torch.tensor(sizes).cumsum(0)
    pad = torch.tensor([(n + 15) // 16 * 16 for n in sizes])
    at = torch.tensor(starts)
    owner = torch.repeat_interleave(torch.arange(len(sizes)), pad)
    keep = (torch.arange(total) - at[owner]) < torch.tensor(sizes)[owner]
    flat = torch.where(keep.cuda(), flat, 0.0).to(kind)
    if case["overflow"]:
        k = int(torch.randint(0, len(sizes), (1,), generator=gen, device="cuda"))
        flat[starts[k] + sizes[k] - 1] = math.inf
    state = {"case": case, "flat": flat, "starts": at.cuda(), "pad": pad.cuda(), "total": int(ends[-1])}
    views = [flat[a:a + n] for a, n in zip(starts, sizes)]
    if case["op"] == "clip":
        state["out"] = torch.zeros(total, dtype=TYPES[case["out"]], device="cuda")
    if own:
        from loss_scaled_fp32_b200 import GradList, grad_pointers
        state["list"] = GradList(sizes, kind, out_dtypes=TYPES[case["out"]] if case["op"] == "clip" else None)
        state["grads"] = grad_pointers(views)
        if case["op"] == "clip":
            state["outs"] = grad_pointers([state["out"][a:a + n] for a, n in zip(starts, sizes)])
    return state


def _rows(values, wide):
    """The same values as rows of a wider buffer."""
    if not wide:
        return values
    n, d = values.shape
    room = torch.zeros(n, d + 64, dtype=values.dtype, device=values.device)
    room[:, :d] = values
    return room[:, :d]


def _prepare_head(case, gen):
    n, v, d, kind = case["tokens"], case["vocab"], case["width"], TYPES[case["type"]]
    weight = torch.randn(v, d, generator=gen, device="cuda").mul_(0.02)
    # token frequencies fall as one over the rank
    rank = torch.rand(n, generator=gen, device="cuda").mul_(math.log(v)).exp_().long().sub_(1).clamp_(0, v - 1)
    # normalised activations that point at their target with a strength from none to sure
    sure = torch.rand(n, 1, generator=gen, device="cuda") * 30.0
    hidden = torch.randn(n, d, generator=gen, device="cuda")
    hidden += sure * torch.nn.functional.normalize(weight[rank], dim=1)
    skip = torch.rand(n, generator=gen, device="cuda") < case["ignored"]
    targets = torch.where(skip, torch.full_like(rank, IGNORE), rank)
    state = {"case": case, "hidden": _rows(hidden.to(kind), case["wide_rows"]),
             "weight": _rows(weight.to(kind), case["wide_rows"]), "targets": targets}
    if case["op"] == "grad":
        state["scale"] = torch.full((1,), case["scale"], device="cuda") if case["scale_on_device"] else case["scale"]
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_list(case, gen) if case["op"] in ("norm", "clip") else _prepare_head(case, gen)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _plain_norms(state):
    """Norms and the clip factor in 64 bits; the factor in 32."""
    case, flat = state["case"], state["flat"]
    sq = flat.double().square().view(-1, 16).sum(1)  # no block of 16 spans two tensors
    per = torch.segment_reduce(sq, "sum", lengths=state["pad"] // 16, unsafe=True)
    bad = (~torch.isfinite(flat)).sum().reshape(1)
    found = bad > 0
    per = torch.where(torch.isfinite(per), per, math.inf)
    norm = torch.where(found, math.inf, per.sum().sqrt() / case["scale"])
    clipped = ~found & (norm > case["clip"]) if case["clip"] > 0 else torch.zeros_like(found)
    coef = torch.where(clipped, case["clip"] / norm, 1.0).float()
    return {"norm": norm, "coef": coef, "found_inf": found.int(), "n_nonfinite": bad,
            "tensor_norms": per.sqrt() / case["scale"]}


def _plain_head(state):
    case, targets = state["case"], state["targets"]
    hidden, weight = state["hidden"].float(), state["weight"].float()
    logits = hidden @ weight.t()
    valid = targets != IGNORE
    at = torch.where(valid, targets, 0)[:, None]
    picked = logits.gather(1, at)[:, 0]
    # the other logits against the target's: a sure answer's small loss keeps its digits
    rest = logits.scatter(1, at, -math.inf)
    top = rest.max(1, keepdim=True).values
    over = (rest - top).exp_().sum(1).log() + top[:, 0] - picked
    del rest
    each = over.clamp(min=0.0) + (-over.abs()).exp().log1p()
    lse = picked + each
    each = torch.where(valid, each, 0.0)
    n = valid.sum().reshape(1)
    out = {"loss": (each.double().sum() / n.clamp(min=1)).float(), "token_loss": each, "lse": lse, "n_valid": n}
    if case["op"] == "grad":
        scale = state["scale"] / n.clamp(min=1).float()
        dz = (logits - lse[:, None]).exp_()
        dz.scatter_(1, at, torch.expm1(-each)[:, None])
        dz *= torch.where(valid, 1.0, 0.0)[:, None] * scale
        out["grad_hidden"] = (dz @ weight).to(state["hidden"].dtype)
        out["grad_weight"] = (dz.t() @ hidden).to(state["weight"].dtype)
    return out


def run(state):
    case = state["case"]
    op = case["op"]
    if op == "norm":
        if own:
            return state["list"].norm(state["grads"], scale=case["scale"], clip=case["clip"], tensor_norms=True)
        return _plain_norms(state)
    if op == "clip":
        if own:
            r = state["list"].clip(state["grads"], case["clip"], out=state["outs"], scale=case["scale"],
                                   unscale=case["unscale"], tensor_norms=True)
        else:
            r = _plain_norms(state)
            x = state["flat"].float()
            x = x * (1.0 / case["scale"]) if case["unscale"] else x
            state["out"].copy_(x * r["coef"])
        return r | {"out": state["out"]}
    if own:
        from loss_scaled_fp32_b200 import xent_grad, xent_loss
        if op == "loss":
            return xent_loss(state["hidden"], state["weight"], state["targets"], ignore_index=IGNORE)._asdict()
        return xent_grad(state["hidden"], state["weight"], state["targets"], scale=state["scale"],
                         ignore_index=IGNORE)._asdict()
    return _plain_head(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] in ("norm", "clip"):
        sizes = _sizes(case)
        n, width = sum(sizes), TYPES[case["type"]].itemsize
        moved = n * width + 8 * len(sizes)
        if case["op"] == "clip":
            moved += n * TYPES[case["out"]].itemsize
        return {"bytes": moved, "flops": (2 if case["op"] == "norm" else 3) * n}
    n, v, d = case["tokens"], case["vocab"], case["width"]
    moved = 2 * (n + v) * d + 16 * n
    if case["op"] == "loss":
        return {"bytes": moved, "flops": 2 * n * v * d}
    return {"bytes": moved + 2 * (n + v) * d, "flops": 6 * n * v * d}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] in ("norm", "clip"):
        x = state["flat"].double()
        sums = torch.zeros(len(state["pad"]), dtype=torch.float64, device="cuda")
        sums.index_add_(0, torch.repeat_interleave(state["pad"]), torch.where(torch.isfinite(x), x * x, math.inf))
        size = torch.sqrt(sums.sum()).reshape(1) / case["scale"]
        wild = int((~torch.isfinite(x)).sum())
        factor = 1.0
        if case["clip"] > 0 and not wild and float(size) > case["clip"]:
            factor = case["clip"] / float(size)
        r = {"norm": size, "coef": torch.full_like(size, factor), "found_inf": None, "n_nonfinite": None,
             "tensor_norms": torch.sqrt(sums) / case["scale"]}
        if case["op"] == "clip":
            r["out"] = x * (factor / (case["scale"] if case["unscale"] else 1.0))
        return r
    n, v = case["tokens"], case["vocab"]
    h, w, t = state["hidden"].double(), state["weight"].double(), state["targets"]
    z = torch.einsum("nd,vd->nv", h, w)
    lse = torch.logsumexp(z, 1)
    live = t.ne(IGNORE)
    rows = torch.arange(n, device="cuda")[live]
    picked = torch.zeros(n, dtype=torch.float64, device="cuda")
    picked[rows] = lse[rows] - z[rows, t[rows]]  # 64 bits: off by 1e-15
    count = max(1, int(live.sum()))
    r = {"loss": picked.sum() / count, "token_loss": picked, "lse": lse, "n_valid": None}
    if case["op"] == "grad":
        q = torch.softmax(z, 1)
        q[~live] = 0.0
        q[rows, t[rows]] -= 1.0
        q *= case["scale"] / count
        r["grad_hidden"] = torch.einsum("nv,vd->nd", q, w)
        r["grad_weight"] = torch.einsum("nv,nd->vd", q, h)
    return r
