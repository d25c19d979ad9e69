"""The two ends of a language model's training step and what stands between its blocks, as a user's
program calls them: softmax cross entropy of a linear map onto a vocabulary with its gradients, the
embedding of token ids with its gradient, and the norms before and after a block with its gate and
residual scale.

Every case is a dict of plain values.  run() computes it in a plain form of elementary torch
operations, or, where `own` is true, through this repository's package.
"""
import math

import torch

own = False

IGNORED = -100
EPS = 1e-5


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # a few tokens of a small model: launches and latency
        _loss("loss_small", 37, 256, 515),
        # GPT-2 small's validation loss on two sequences: no gradients
        _loss("loss_eval", 2048, 768, 50257, grad=False, ids32=True),
        # GPT-2 small's training batch, a sixth of it padding
        _loss("loss_gpt2", 4096, 768, 50257, padded=True),
        # the 1.3B model's training batch
        _loss("loss_1p3b", 8192, 2048, 50257),
        # one token of generation
        _embed("embed_one_token", "embed", 1, 2048, 50257),
        # the 1.3B model's training batch, scaled as a table shared with the loss is
        _embed("embed_train", "embed", 8192, 2048, 50257, scale=True),
        # its gradient, every row of the vocabulary written
        _embed("embed_grad_train", "embed_grad", 8192, 2048, 50257, scale=True),
        # GPT-2 small's, added to the fp32 gradient that the loss wrote to the same table; padding left out
        _embed("embed_grad_shared", "embed_grad", 4096, 768, 50257, f32=True, add=True, padded=True, ids32=True),
        # one token of generation through a Llama-7B block's sum and norm
        _norm("norm_one_token", "norm", 1, 4096),
        # the 1.3B model's training batch: both norms of a block, a learned gate, residual scale
        _norm("norm_train", "norm", 8192, 2048, post="rms", gate="vector"),
        # a small model of odd width with LayerNorm and biases, a gate for each element, fp32 gradients
        _norm("norm_grad_odd", "norm_grad", 1003, 775, post="layer", gate="matrix", kind="layer", f32=True),
        # norm_train's gradient
        _norm("norm_grad_train", "norm_grad", 8192, 2048, post="rms", gate="vector"),
    ]


def _loss(name, rows, width, vocab, *, grad=True, padded=False, ids32=False):
    return {"name": name, "op": "loss", "rows": rows, "width": width, "vocab": vocab, "grad": grad, "padded": padded, "ids32": ids32}


def _embed(name, op, rows, width, vocab, *, scale=False, f32=False, add=False, padded=False, ids32=False):
    return {"name": name, "op": op, "rows": rows, "width": width, "vocab": vocab, "scale": scale, "f32": f32, "add": add, "padded": padded,
            "ids32": ids32}


def _norm(name, op, rows, width, *, post="none", gate="none", kind="rms", f32=False):
    return {"name": name, "op": op, "rows": rows, "width": width, "post": post, "gate": gate, "kind": kind, "f32": f32}


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width: a multiple of 64 half of the time, of 8 a quarter, any number otherwise."""
    n, unit = _log(rng, low, high), (64, 64, 8, 1)[rng.randrange(4)]
    return max(n // unit, 1) * unit


def draw(rng):
    op = ("loss", "loss", "embed", "embed_grad", "norm", "norm_grad")[rng.randrange(6)]
    if op == "loss":
        while True:
            rows, width, vocab = _log(rng, 1, 8192), _width(rng, 64, 4096), _log(rng, 2, 131072)
            if rows * width * vocab <= 8192 * 2048 * 50257:
                break
        case = _loss("", rows, width, vocab, grad=rng.random() < 0.75, padded=rng.random() < 0.4, ids32=rng.random() < 0.5)
    elif op in ("embed", "embed_grad"):
        rows, width, vocab = _log(rng, 1, 16384), _width(rng, 64, 2048), _log(rng, 2, 50257)
        back, f32 = op == "embed_grad", rng.random() < 0.5
        case = _embed("", op, rows, width, vocab, scale=rng.random() < 0.5, f32=back and f32, add=back and f32 and rng.random() < 0.6,
                      padded=back and rng.random() < 0.5, ids32=rng.random() < 0.5)
    else:
        rows, width = _log(rng, 1, 8192), _width(rng, 32, 8192)
        post, gate = ("none", "rms", "layer")[rng.randrange(3)], ("none", "vector", "matrix")[rng.randrange(3)]
        case = _norm("", op, rows, width, post=post, gate=gate, kind=("rms", "layer")[rng.randrange(2)], f32=op == "norm_grad" and rng.random() < 0.5)
    case.pop("name")
    return case


# ------------------------------------------------------------------------------ inputs

def _ids(case, gen):
    """Token ids as text has them: the k-th commonest about 1/k as often as the first."""
    u = torch.rand(case["rows"], generator=gen, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(case["vocab"] + 1)) - 1).long().clamp(0, case["vocab"] - 1)
    return ids.int() if case["ids32"] else ids


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, sigma, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)

    def padding(ids, value):  # a batch of six sequences, the last sixth of each filled up
        length = max(ids.numel() // 6, 2)
        at = torch.arange(ids.numel(), device="cuda") % length
        return torch.where(at >= length * 5 // 6, torch.full_like(ids, value), ids)

    s, m, d = {"case": case}, case["rows"], case["width"]
    if case["op"] == "loss":
        v = case["vocab"]
        s["w"] = normal((v, d), 0.02)
        t = _ids(case, gen)
        # logits of a model that has learnt something: the target's stands out by 0 to 12 at every token
        lead = torch.rand((m, 1), generator=gen, device="cuda") * 12.0
        of = s["w"][t.long()].float()
        s["x"] = (normal((m, d), 1.0) + lead * of / of.square().sum(1, keepdim=True)).to(torch.bfloat16)
        s["t"] = padding(t, IGNORED) if case["padded"] else t
        s["losses"] = torch.empty(m, dtype=torch.float32, device="cuda")
        s["total"] = torch.empty(1, dtype=torch.float32, device="cuda")
        s["dx"] = torch.empty_like(s["x"]) if case["grad"] else None
        s["dw"] = torch.empty_like(s["w"]) if case["grad"] else None
        return s
    if case["op"] in ("embed", "embed_grad"):
        v = case["vocab"]
        s["ids"] = padding(_ids(case, gen), 0) if case["padded"] else _ids(case, gen)
        s["scale"] = math.sqrt(d) if case["scale"] else 1.0
        if case["op"] == "embed":
            s["table"] = normal((v, d), 0.02)
            s["y"] = torch.empty((m, d), dtype=torch.bfloat16, device="cuda")
            return s
        s["pad"] = 0 if case["padded"] else None
        s["dy"] = normal((m, d), 1e-3)
        kind = torch.float32 if case["f32"] else torch.bfloat16
        s["dtable"] = normal((v, d), 1e-3, kind) if case["add"] else torch.empty((v, d), dtype=kind, device="cuda")
        return s

    # a residual stream has a few channels far larger than the others
    large = torch.ones(d, device="cuda")
    large[:: max(d // 5, 1)] = 20.0
    s["alpha"] = 0.25 if case["post"] != "none" else 1.0
    s["h"] = normal((m, d), 1.0)
    layer = {"post": case["post"] == "layer", "": case["kind"] == "layer"}
    s["post_weight"] = (1 + normal((d,), 0.1, torch.float32)).bfloat16() if case["post"] != "none" else None
    s["post_bias"] = normal((d,), 0.1) if layer["post"] else None
    s["weight"] = (1 + normal((d,), 0.1, torch.float32)).bfloat16()
    s["bias"] = normal((d,), 0.1) if layer[""] else None
    s["gate"] = normal((d,), 0.5) if case["gate"] == "vector" else normal((m, d), 0.5) if case["gate"] == "matrix" else None
    if case["op"] == "norm":
        s["r"] = (normal((m, d), 2.0) * large).bfloat16()
        s["s"], s["y"] = torch.empty_like(s["r"]), torch.empty_like(s["r"])
        return s
    s["s"] = (normal((m, d), 2.0) * large).bfloat16()
    s["dy"], s["ds"] = normal((m, d), 1e-3), normal((m, d), 1e-3)
    kind = torch.float32 if case["f32"] else torch.bfloat16
    s["dr"] = torch.empty_like(s["s"])
    s["dh"] = torch.empty_like(s["s"])
    s["dgate"] = None
    if case["gate"] != "none":  # a gate that a map made gets its gradient in that map's type
        s["dgate"] = torch.empty_like(s["gate"], dtype=kind if case["gate"] == "vector" else torch.bfloat16)
    for name in ("post_weight", "post_bias", "weight", "bias"):
        s["d" + name] = torch.empty(d, dtype=kind, device="cuda") if s[name] is not None else None
    return s


# -------------------------------------------------------------------------------- runs

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"loss": _plain_loss, "embed": _plain_embed, "embed_grad": _plain_embed_grad, "norm": _plain_norm,
            "norm_grad": _plain_norm_grad}[case["op"]](case, state)


def _run_own(case, s):
    import zero_partitioned_mixed_adam_gb300 as za
    if case["op"] == "loss":
        za.zero_linear_cross_entropy(s["x"], s["w"], s["t"], s["losses"], s["total"], dx=s["dx"], dw=s["dw"], ignore_index=IGNORED)
        return [s["losses"], s["total"]] + ([s["dx"], s["dw"]] if case["grad"] else [])
    if case["op"] == "embed":
        za.zero_embedding_forward(s["ids"], s["table"], s["y"], scale=s["scale"])
        return s["y"]
    if case["op"] == "embed_grad":
        za.zero_embedding_backward(s["dy"], s["ids"], s["dtable"], scale=s["scale"], padding=s["pad"], accumulate=case["add"])
        return s["dtable"]
    kinds = {"none": za.ZERO_NORM_NONE, "rms": za.ZERO_NORM_RMS, "layer": za.ZERO_NORM_LAYER}
    block = {"h": s["h"], "post": kinds[case["post"]], "post_weight": s["post_weight"], "post_bias": s["post_bias"], "gate": s["gate"],
             "alpha": s["alpha"], "kind": kinds[case["kind"]], "weight": s["weight"], "eps": EPS}
    if case["op"] == "norm":
        za.zero_block_norm_forward(s["r"], s["y"], s=s["s"], bias=s["bias"], **block)
        return [s["s"], s["y"]]
    za.zero_block_norm_backward(s["dy"], s["s"], ds=s["ds"], dr=s["dr"], dh=s["dh"], dgate=s["dgate"], dpost_weight=s["dpost_weight"],
                                dpost_bias=s["dpost_bias"], dweight=s["dweight"], dbias=s["dbias"], **block)
    return _grads(s)


def _grads(s):
    names = ("dr", "dh", "dgate", "dpost_weight", "dpost_bias", "dweight", "dbias")
    return {name: s[name] for name in names if s[name] is not None}


def _plain_loss(case, s):
    x, w, t = s["x"].float(), s["w"].float(), s["t"].long()
    keep = t != IGNORED
    at = torch.where(keep, t, 0)[:, None]
    z = x @ w.t()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    losses = torch.where(keep, (top + torch.log(total) - z.gather(1, at))[:, 0], 0.0)
    c = keep.float() / keep.sum().clamp(min=1)
    out = [losses, (losses * c).sum()[None]]
    if case["grad"]:
        dz = e.mul_(c[:, None] / total)
        dz.scatter_(1, at, dz.gather(1, at) - c[:, None])
        out += [(dz @ w).to(torch.bfloat16), (dz.t() @ x).to(torch.bfloat16)]
    return out


def _plain_embed(case, s):
    return (s["table"][s["ids"].long()].float() * s["scale"]).to(torch.bfloat16)


def _plain_embed_grad(case, s):
    ids, dy = s["ids"].long(), s["dy"].float() * s["scale"]
    if s["pad"] is not None:
        dy = dy * (ids != s["pad"])[:, None]
    sums = torch.zeros(s["dtable"].shape, dtype=torch.float32, device="cuda").index_add_(0, ids, dy)
    return s["dtable"].add_(sums) if case["add"] else sums.to(s["dtable"].dtype)


def _standard(x, kind):
    """x less its row's mean (layer), over its row's root mean square; and that root's inverse."""
    if kind == "layer":
        x = x - x.mean(1, keepdim=True)
    inverse = torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)
    return x * inverse, inverse


def _after(case, s):
    """The block's output through the norm after it."""
    if case["post"] == "none":
        return s["h"].float()
    p = _standard(s["h"].float(), case["post"])[0] * s["post_weight"].float()
    return p + s["post_bias"].float() if s["post_bias"] is not None else p


def _plain_norm(case, s):
    p = _after(case, s) * s["alpha"]
    if s["gate"] is not None:
        p = p * s["gate"].float()
    r = s["r"].float() + p
    y = _standard(r, case["kind"])[0] * s["weight"].float()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return [r.to(torch.bfloat16), y.to(torch.bfloat16)]


def _standard_grad(u, standard, inverse, kind):
    g = u - standard * (u * standard).mean(1, keepdim=True)
    if kind == "layer":
        g = g - u.mean(1, keepdim=True)
    return g * inverse


def _plain_norm_grad(case, s):
    out, dy = {}, s["dy"].float()
    standard, inverse = _standard(s["s"].float(), case["kind"])
    out["dweight"], out["dbias"] = (dy * standard).sum(0), dy.sum(0)
    ds = s["ds"].float() + _standard_grad(dy * s["weight"].float(), standard, inverse, case["kind"])
    out["dr"] = ds
    p = _after(case, s)
    dp = ds * s["alpha"]
    if s["gate"] is not None:
        out["dgate"] = dp * p if case["gate"] == "matrix" else (dp * p).sum(0)
        dp = dp * s["gate"].float()
    out["dh"] = dp
    if case["post"] != "none":
        standard, inverse = _standard(s["h"].float(), case["post"])
        out["dpost_weight"], out["dpost_bias"] = (dp * standard).sum(0), dp.sum(0)
        out["dh"] = _standard_grad(dp * s["post_weight"].float(), standard, inverse, case["post"])
    return {name: out[name].to(s[name].dtype) for name in _grads(s)}


# --------------------------------------------------------------------- cost and values

def _touched(case):
    """About how many rows of the table `rows` ids touch: k-th id with a chance of ln((k+2)/(k+1)) / ln(vocab+1)."""
    v, span = case["vocab"], math.log(case["vocab"] + 1)
    k = torch.arange(v, dtype=torch.float64)
    return float((1.0 - (1.0 - torch.log((k + 2) / (k + 1)) / span).clamp(0, 1) ** case["rows"]).sum())


def work(case):
    """What a pass cannot do without: each input read once, each output written once, and its products."""
    m, d = case["rows"], case["width"]
    if case["op"] == "loss":
        v, id_bytes = case["vocab"], 4 if case["ids32"] else 8
        grad = 2 if case["grad"] else 1
        return {"bytes": 2 * grad * (m * d + v * d) + (id_bytes + 4) * m, "flops": (6 if case["grad"] else 2) * m * d * v}
    if case["op"] in ("embed", "embed_grad"):
        id_bytes, size = 4 if case["ids32"] else 8, 4 if case["f32"] else 2
        rows = _touched(case)
        if case["op"] == "embed":
            return {"bytes": int(2 * d * (rows + m)) + id_bytes * m, "flops": m * d}
        table = 2 * size * rows * d if case["add"] else size * case["vocab"] * d
        return {"bytes": int(2 * m * d + table) + id_bytes * m, "flops": 2 * m * d}
    gate = {"none": 0, "vector": d, "matrix": m * d}[case["gate"]]
    vectors = d * (1 + (case["kind"] == "layer") + (case["post"] != "none") + (case["post"] == "layer"))
    if case["op"] == "norm":
        return {"bytes": 2 * (4 * m * d + gate + vectors), "flops": 12 * m * d}
    size = 4 if case["f32"] else 2
    gate_grad = (size if case["gate"] == "vector" else 2) * gate
    return {"bytes": 2 * (6 * m * d + gate + vectors) + gate_grad + size * vectors, "flops": 30 * m * d}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    f = {k: x.double() for k, x in s.items() if torch.is_tensor(x) and x.is_floating_point()}
    if case["op"] == "loss":
        t = s["t"].long()
        rows = torch.nonzero(t != IGNORED)[:, 0]
        n, t = rows.numel(), t[rows]
        x = f["x"][rows]
        z = torch.einsum("mk,vk->mv", x, f["w"])
        norm = torch.logsumexp(z, 1)
        loss = norm - z[torch.arange(n, device="cuda"), t]
        losses = torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
        losses[rows] = loss
        out = [losses, losses.sum()[None] / max(n, 1)]
        if case["grad"]:
            p = torch.exp(z.sub_(norm[:, None]))
            p[torch.arange(n, device="cuda"), t] -= 1.0
            p /= max(n, 1)
            dx = torch.zeros_like(f["x"])
            dx[rows] = torch.einsum("mv,vk->mk", p, f["w"])
            out += [dx, torch.einsum("mv,mk->vk", p, x)]
        return out
    if case["op"] == "embed":
        return torch.index_select(f["table"], 0, s["ids"].long()) * s["scale"]
    if case["op"] == "embed_grad":
        # the rows in the order of their ids, and differences of their running sums
        ids, order = torch.sort(s["ids"].long(), stable=True)
        if s["pad"] is not None:
            order, ids = order[ids != s["pad"]], ids[ids != s["pad"]]
        run = torch.zeros((ids.numel() + 1, case["width"]), dtype=torch.float64, device="cuda")
        run[1:] = torch.cumsum(f["dy"][order], 0)
        v = torch.arange(case["vocab"], device="cuda")
        grad = (run[torch.searchsorted(ids, v, right=True)] - run[torch.searchsorted(ids, v)]) * s["scale"]
        return grad + f["dtable"] if case["add"] else grad

    def moments(x, kind):
        mean = x.mean(1) if kind == "layer" else torch.zeros_like(x[:, 0])
        return mean[:, None], (torch.einsum("md,md->m", x, x) / x.shape[1] - mean ** 2 + EPS).sqrt()[:, None]

    weight, h, gate = f["weight"], f["h"], f.get("gate", torch.ones((), dtype=torch.float64, device="cuda"))
    after, p = torch.ones((), dtype=torch.float64, device="cuda"), h
    if case["post"] != "none":
        mean, root = moments(h, case["post"])
        after = f["post_weight"]
        p = (h - mean) / root * after + f.get("post_bias", 0.0)
    if case["op"] == "norm":
        r = f["r"] + s["alpha"] * gate * p
        mean_r, root_r = moments(r, case["kind"])
        return [r, (r - mean_r) / root_r * weight + f.get("bias", 0.0)]

    def back(x, mean, root, u, kind):
        """The gradient of (x - mean) / root for the gradient u, by the quotient's rule: d root = sum (x - mean) dx / (n root)."""
        n, c = x.shape[1], x - mean
        g = u / root - c * torch.einsum("md,md->m", u, c)[:, None] / (n * root ** 3)
        return g - g.sum(1, keepdim=True) / n if kind == "layer" else g

    mean_s, root_s = moments(f["s"], case["kind"])
    dr = f["ds"] + back(f["s"], mean_s, root_s, f["dy"] * weight, case["kind"])
    out = {"dr": dr, "dweight": torch.einsum("md,md->d", f["dy"], (f["s"] - mean_s) / root_s), "dbias": torch.einsum("md->d", f["dy"])}
    out["dgate"] = s["alpha"] * dr * p if case["gate"] == "matrix" else s["alpha"] * torch.einsum("md,md->d", dr, p)
    dp = s["alpha"] * gate * dr
    out["dh"] = dp
    if case["post"] != "none":
        out["dh"] = back(h, mean, root, dp * after, case["post"])
        out["dpost_weight"], out["dpost_bias"] = torch.einsum("md,md->d", dp, (h - mean) / root), torch.einsum("md->d", dp)
    return {name: out[name] for name in _grads(s)}
