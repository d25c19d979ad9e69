"""The operators of one training step, as a user's program calls them: a linear layer with its
epilogue, its backward pass, the gradients' global norm, and AdamW over a list of tensors.

Every case is a dict of plain values.  run() computes it in a plain form of elementary torch
operations, or, where `own` is true, through this repository's package.
"""
import math

import torch

own = False

ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
BLOCK = 256  # elements that share one scale of an 8-bit moment


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one token of generation through a Llama-7B layer's up projection: reading the weight once
        _linear("forward_one_token", "forward", 1, 4096, 11008, act="silu"),
        # a ragged batch of short sequences through GPT-2's attention projection, onto the stream
        _linear("forward_ragged", "forward", 777, 768, 2304, bias=True, residual=True),
        # a training batch through the 1.3B model's first MLP map, which keeps what gelu was given
        _linear("forward_train", "forward", 8192, 2048, 8192, bias=True, act="gelu", pre=True),
        # a small layer of odd widths, where no row starts on a 16-byte boundary
        _linear("backward_odd", "backward", 1003, 775, 2311, bias=True, act="silu"),
        # the 1.3B model's first MLP map, its activation differentiated on the way
        _linear("backward_train", "backward", 8192, 2048, 8192, bias=True, act="gelu"),
        # a Llama-7B layer's down projection: fp32 gradients added to those of earlier micro-batches,
        # and the gradient of the map before it taken through that map's activation
        _linear("backward_accumulate", "backward", 4096, 11008, 4096, act_in="silu", f32=True, add=True),
        # one small layer's gradients, where launches and the final sum are all there is
        _tensors("norm_small", "norm", 1, 256, f32=True),
        # the whole 1.3B model's bf16 gradients
        _tensors("norm_1p3b", "norm", 24, 2048, 50257, 2048),
        # one small layer of odd width: latency
        _tensors("adamw_small", "adamw", 1, 131, f32=True),
        # the 1.3B model, gradients clipped, moments in 32 bits
        _tensors("adamw_1p3b", "adamw", 24, 2048, 50257, 2048, clip=True),
        # GPT-2 small, moments in 8 bits
        _tensors("adamw8_gpt2", "adamw", 12, 768, 50257, 1024, eight=True),
        # the 1.3B model, moments in 8 bits
        _tensors("adamw8_1p3b", "adamw", 24, 2048, 50257, 2048, eight=True),
    ]


def _linear(name, kind, rows, width_in, width_out, *, bias=False, act="none", residual=False, pre=False, act_in="none", f32=False,
            add=False):
    return {"name": name, "kind": kind, "rows": rows, "in": width_in, "out": width_out, "bias": bias, "act": act, "residual": residual,
            "pre": pre, "act_in": act_in, "f32": f32, "add": add}


def _tensors(name, kind, layers, width, vocab=0, context=0, *, f32=False, clip=False, eight=False):
    return {"name": name, "kind": kind, "layers": layers, "width": width, "vocab": vocab, "context": context, "f32": f32, "clip": clip,
            "eight": eight}


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width: a multiple of 64 half of the time, of 8 a quarter, any number otherwise."""
    n, unit = _log(rng, low, high), (64, 64, 8, 1)[rng.randrange(4)]
    return n // unit * unit


def draw(rng):
    kind = ("forward", "forward", "backward", "backward", "norm", "adamw", "adamw")[rng.randrange(7)]
    if kind in ("forward", "backward"):
        while True:
            rows, a, b = _log(rng, 1 if kind == "forward" else 16, 8192), _width(rng, 256, 11008), _width(rng, 256, 11008)
            if rows * a * b <= 8192 * 2048 * 8192 and 3072 not in (rows, a, b):
                break
        act = ("none", "relu", "gelu", "silu")[rng.randrange(4)]
        if kind == "forward":
            return {k: v for k, v in _linear("", kind, rows, a, b, bias=rng.random() < 0.5, act=act, residual=rng.random() < 0.3,
                                             pre=act != "none" and rng.random() < 0.5).items() if k != "name"}
        f32 = rng.random() < 0.3  # gradients in 32 bits are asked for where there is no activation to differentiate
        return {k: v for k, v in _linear("", kind, rows, a, b, bias=rng.random() < 0.5, act="none" if f32 else act,
                                         act_in=("none", "gelu", "silu")[rng.randrange(3)], f32=f32,
                                         add=f32 and rng.random() < 0.5).items() if k != "name"}
    while True:
        layers, width, vocab = _log(rng, 1, 24), _width(rng, 128, 1900), rng.choice((0, 0, 8191, 50257))
        context = _log(rng, 64, 2048) if vocab else 0
        if 3072 not in (width, 3 * width, 4 * width):
            break
    eight = kind == "adamw" and rng.random() < 0.5
    return {k: v for k, v in _tensors("", kind, layers, width, vocab, context, f32=rng.random() < 0.4, eight=eight,
                                      clip=kind == "adamw" and rng.random() < 0.5).items() if k != "name"}


def _shapes(case):
    """A GPT's tensors: embeddings, then each layer's norms, attention and MLP."""
    d = case["width"]
    layer = [(d,), (d,), (3 * d, d), (3 * d,), (d, d), (d,), (d,), (d,), (4 * d, d), (4 * d,), (d, 4 * d), (d,)]
    return ([(case["vocab"], d), (case["context"], d)] if case["vocab"] else []) + layer * case["layers"] + [(d,), (d,)]


# ------------------------------------------------------------------------------ inputs

HYPER = {"lr": 3e-4, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "t": 100}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, sigma, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, sigma, generator=gen)

    if case["kind"] in ("forward", "backward"):
        m, k, n = case["rows"], case["in"], case["out"]
        s = {"case": case, "x": normal((m, k), 1.0), "w": normal((n, k), 0.02), "bias": None, "pre": None, "residual": None}
        if case["kind"] == "forward":
            s["bias"] = normal((n,), 0.1) if case["bias"] else None
            s["residual"] = normal((m, n), 1.0) if case["residual"] else None
            s["y"] = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
            s["pre"] = torch.empty_like(s["y"]) if case["pre"] else None
            return s
        grad = torch.float32 if case["f32"] else torch.bfloat16
        s["dy"] = normal((m, n), 1e-3)
        s["pre"] = normal((m, n), 1.0) if case["act"] != "none" else None
        s["pre_in"] = normal((m, k), 1.0) if case["act_in"] != "none" else None
        s["dx"] = torch.empty((m, k), dtype=torch.bfloat16, device="cuda")
        s["dw"] = normal((n, k), 1e-2, grad) if case["add"] else torch.empty((n, k), dtype=grad, device="cuda")
        s["dbias"] = (normal((n,), 1e-2, grad) if case["add"] else torch.empty((n,), dtype=grad, device="cuda")) if case["bias"] else None
        return s

    shapes = _shapes(case)
    sizes = [math.prod(x) for x in shapes]

    def flat(sigma, dtype):
        return normal((sum(sizes),), sigma, dtype)

    def views(x):  # one flat vector cut into the tensors, as a sharded optimizer lays them out
        return [p.view(shape) for p, shape in zip(x.split(sizes), shapes)]

    # gradients of which a tenth are exactly zero, as rows of an embedding that no token touched
    grads = flat(1e-3, torch.float32 if case["f32"] else torch.bfloat16)
    grads.mul_(torch.empty_like(grads).uniform_(0.0, 1.0, generator=gen) >= 0.1)
    s = {"case": case, "grads": views(grads)}
    if case["kind"] == "norm":
        s["max_norm"], s["out"] = 1.0, torch.empty(2, dtype=torch.float32, device="cuda")
        if own:
            import zero_partitioned_mixed_adam_gb300 as za
            s["list"] = za.grad_list(s["grads"])
            s["workspace"] = za.grad_norm_workspace()
        return s
    s["decay"] = [0.1 if len(x) == 2 else 0.0 for x in shapes]
    s["flat"] = {"master": flat(0.02, torch.float32), "m": flat(3e-4, torch.float32), "v": flat(1e-3, torch.float32).square_()}
    s["flat"]["param"] = s["flat"]["master"].bfloat16()
    s |= {name: views(x) for name, x in s["flat"].items()}
    s["scale"] = torch.full((1,), 0.37, dtype=torch.float32, device="cuda") if case["clip"] else None
    s["seed"] = seed & 0x7FFFFFFF
    s["m_scale"] = s["v_scale"] = s["m_out"] = s["v_out"] = None
    if case["eight"]:
        s["m"], s["m_scale"] = map(list, zip(*[_encode(m, torch.full_like(m, 0x8000, dtype=torch.int32), True) for m in s["m"]]))
        s["v"], s["v_scale"] = map(list, zip(*[_encode(v, torch.full_like(v, 0x8000, dtype=torch.int32), False) for v in s["v"]]))
        s["m_out"], s["v_out"] = views(s["flat"]["m"]), views(s["flat"]["v"])
    if own:
        import zero_partitioned_mixed_adam_gb300 as za
        s["list"] = za.adamw_tensors(s["grads"], s["master"], s["m"], s["v"], params=s["param"], m_scale=s["m_scale"],
                                     v_scale=s["v_scale"], weight_decay=s["decay"])
    return s


# -------------------------------------------------------------------------------- runs

def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"forward": _plain_forward, "backward": _plain_backward, "norm": _plain_norm, "adamw": _plain_adamw}[case["kind"]](case, state)


def _run_own(case, s):
    import zero_partitioned_mixed_adam_gb300 as za
    if case["kind"] == "forward":
        za.zero_linear_forward(s["x"], s["w"], s["y"], bias=s["bias"], act=ACTS[case["act"]], residual=s["residual"], pre=s["pre"])
        return [s["y"]] + ([s["pre"]] if case["pre"] else [])
    if case["kind"] == "backward":
        za.zero_linear_backward(s["dy"], s["x"], s["w"], dx=s["dx"], dw=s["dw"], dbias=s["dbias"], act=ACTS[case["act"]], pre=s["pre"],
                                act_in=ACTS[case["act_in"]], pre_in=s["pre_in"], accumulate=case["add"])
        return [s["dx"], s["dw"]] + ([s["dbias"]] if case["bias"] else [])
    if case["kind"] == "norm":
        za.zero_grad_norm(s["list"], s["out"], max_norm=s["max_norm"], workspace=s["workspace"])
        return s["out"]
    za.zero_adamw_step(s["list"], lr=HYPER["lr"], beta1=HYPER["beta1"], beta2=HYPER["beta2"], eps=HYPER["eps"], t=HYPER["t"],
                       grad_scale=s["scale"], seed=s["seed"])
    if case["eight"]:
        za.zero_adamw_state_f32(s["list"], s["m_out"], s["v_out"])  # as they go into a checkpoint
    return s["flat"]


def _act(x, name):
    if name == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    return x


def _act_grad(x, name):
    if name == "relu":
        return (x > 0).to(x.dtype)
    if name == "gelu":
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-x))
        return s * (1.0 + x * (1.0 - s))
    return torch.ones_like(x)


def _plain_forward(case, s):
    z = s["x"].float() @ s["w"].float().t()
    if case["bias"]:
        z = z + s["bias"].float()
    y = _act(z, case["act"])
    if case["residual"]:
        y = y + s["residual"].float()
    return [y.to(torch.bfloat16)] + ([z.to(torch.bfloat16)] if case["pre"] else [])


def _plain_backward(case, s):
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _act_grad(s["pre"].float(), case["act"])
    dx = dz @ s["w"].float()
    if case["act_in"] != "none":
        dx = dx * _act_grad(s["pre_in"].float(), case["act_in"])
    dw, db = dz.t() @ s["x"].float(), dz.sum(0)
    if case["add"]:
        dw = s["dw"].add_(dw)
        db = s["dbias"].add_(db) if case["bias"] else db
    return [dx.to(torch.bfloat16), dw.to(s["dw"].dtype)] + ([db.to(s["dw"].dtype)] if case["bias"] else [])


def _plain_norm(case, s):
    total = torch.stack([g.float().square().sum() for g in s["grads"]]).sum()
    norm = total.sqrt()
    coef = torch.clamp(s["max_norm"] / (norm + 1e-6), max=1.0)
    return torch.stack([norm, coef])


def _bits(x):
    return x.view(torch.int32)


def _floats(x):
    return x.to(torch.int32).view(torch.float32)


def _blocks(x):
    """A tensor's elements in rows of BLOCK, zeros after its end."""
    x = x.reshape(-1)
    rows = -(-x.numel() // BLOCK)
    full = torch.zeros(rows * BLOCK, dtype=x.dtype, device=x.device)
    full[:x.numel()] = x
    return full.view(rows, BLOCK)


def _encode(x, dither, signed):
    """8-bit codes and block scales of x: 3 bits of mantissa, 4 (signed) or 5 of exponent below the block's power of two,
    gradual underflow, and the 16-bit dither added below the last kept bit before the rest is cut off."""
    a, n = _blocks(x.abs()), x.numel()
    top = _bits(a.amax(1))
    exponent = ((top.to(torch.int64) + 0xFFFFF) >> 23).clamp(1, 253)
    fine = top < 0x7F800000
    t = a * _floats((254 - exponent) << 23)[:, None] * (2.0 ** -112 if signed else 2.0 ** -96)
    code = ((_bits(t) + (_blocks(dither).to(torch.int32) * 16 + 8)) >> 20).clamp(max=127 if signed else 255)
    code = torch.where(fine[:, None], code, torch.zeros_like(code)).reshape(-1)[:n].view(x.shape)
    if signed:
        code = code + torch.where(torch.signbit(x), 128, 0).to(torch.int32)
    scale = torch.where(fine, _floats(exponent << 23), torch.full_like(a[:, 0], float("nan")))
    return code.to(torch.uint8), scale


def _decode(code, scale, signed):
    c = code.to(torch.int32)
    a = ((c & 127) << 20).view(torch.float32) * 2.0 ** 112 if signed else (c << 20).view(torch.float32) * 2.0 ** 96
    a = (_blocks(a) * scale[:, None]).reshape(-1)[:code.numel()].view(code.shape)
    return torch.where(c >= 128, -a, a) if signed else a


def _hash(x):
    """O'Neill's 32-bit permuted congruential generator as a hash (Jarzynski and Olano, 2020), in 64-bit integers."""
    x = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    x = (((x >> ((x >> 28) + 4)) ^ x) * 277803737) & 0xFFFFFFFF
    return (x >> 22) ^ x


def _dither(seed, index, n, device):
    """32 random bits for every element of tensor `index`."""
    key = _hash(torch.tensor([seed], dtype=torch.int64, device=device))
    key = _hash((key + index) & 0xFFFFFFFF)
    return _hash((torch.arange(n, dtype=torch.int64, device=device) + key) & 0xFFFFFFFF)


def _plain_moments(case, s, i):
    """Tensor i's new moments, as the step takes them, in 32 bits."""
    g = s["grads"][i].float()
    if case["clip"]:
        g = g * s["scale"]
    m, v = s["m"][i], s["v"][i]
    if case["eight"]:
        m, v = _decode(m, s["m_scale"][i], True), _decode(v, s["v_scale"][i], False)
    m = m * HYPER["beta1"] + (1.0 - HYPER["beta1"]) * g
    v = v * HYPER["beta2"] + ((1.0 - HYPER["beta2"]) * g) * g
    return m, v


def _plain_tensor(case, s, i):
    m, v = _plain_moments(case, s, i)
    t, w = HYPER["t"], s["master"][i]
    size, root = HYPER["lr"] / (1.0 - HYPER["beta1"] ** t), math.sqrt(1.0 - HYPER["beta2"] ** t)
    w.copy_(w * (1.0 - HYPER["lr"] * s["decay"][i]) - size * m / (v.sqrt() / root + HYPER["eps"]))
    s["param"][i].copy_(w)
    if case["eight"]:
        u = _dither(s["seed"], i, m.numel(), m.device)
        m_code, m_scale = _encode(m, u >> 16, True)
        v_code, v_scale = _encode(v, u & 0xFFFF, False)
        s["m"][i].copy_(m_code), s["m_scale"][i].copy_(m_scale), s["v"][i].copy_(v_code), s["v_scale"][i].copy_(v_scale)
        return s["m_out"][i].copy_(_decode(m_code, m_scale, True)), s["v_out"][i].copy_(_decode(v_code, v_scale, False))
    return s["m"][i].copy_(m), s["v"][i].copy_(v)


def _plain_adamw(case, s):
    [_plain_tensor(case, s, i) for i in range(len(s["grads"]))]
    return s["flat"]


# --------------------------------------------------------------------- cost and values

def work(case):
    """What a pass cannot do without: each input read once, each output written once, and its products."""
    if case["kind"] in ("forward", "backward"):
        m, k, n = case["rows"], case["in"], case["out"]
        if case["kind"] == "forward":
            maps = 1 + case["residual"] + case["pre"]
            return {"bytes": 2 * (m * k + n * k + maps * m * n + case["bias"] * n), "flops": 2 * m * n * k}
        grad = (4 if case["f32"] else 2) * (2 if case["add"] else 1)
        read = m * n * (1 + (case["act"] != "none")) + m * k * (1 + (case["act_in"] != "none")) + n * k
        return {"bytes": 2 * (read + m * k) + grad * (n * k + case["bias"] * n), "flops": 4 * m * n * k}
    n = sum(math.prod(x) for x in _shapes(case))
    grad = 4 if case["f32"] else 2
    if case["kind"] == "norm":
        return {"bytes": grad * n + 8, "flops": 2 * n}
    # gradient, master in and out, parameter out; the moments in and out, and as values where they are held in 8 bits
    moments = 4 * (1 + 4 / BLOCK) + 8 if case["eight"] else 16
    return {"bytes": int((grad + 8 + 2 + moments) * n), "flops": 16 * n}


def exact(case, seed):
    """The same outputs from the definitions, in 64 bits."""
    s = prepare(case, seed)
    if case["kind"] == "forward":
        z = torch.einsum("mk,nk->mn", s["x"].double(), s["w"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        y = _exact_act(z, case["act"])[0]
        if s["residual"] is not None:
            y += s["residual"].double()
        return [y, z] if case["pre"] else [y]
    if case["kind"] == "backward":
        dz = s["dy"].double()
        if s["pre"] is not None:
            dz *= _exact_act(s["pre"].double(), case["act"])[1]
        dx = torch.einsum("mn,nk->mk", dz, s["w"].double())
        if s["pre_in"] is not None:
            dx *= _exact_act(s["pre_in"].double(), case["act_in"])[1]
        dw = torch.einsum("mn,mk->nk", dz, s["x"].double())
        db = torch.einsum("mn->n", dz)
        if case["add"]:
            dw += s["dw"].double()
            db += s["dbias"].double() if case["bias"] else 0.0
        return [dx, dw, db] if case["bias"] else [dx, dw]
    if case["kind"] == "norm":
        norm = math.sqrt(sum(float(torch.einsum("i,i->", g.double().flatten(), g.double().flatten())) for g in s["grads"]))
        return torch.tensor([norm, min(1.0, s["max_norm"] / (norm + 1e-6))], dtype=torch.float64)
    out = {name: [] for name in s["flat"]}
    for i, grad in enumerate(s["grads"]):
        g = grad.double() * (float(s["scale"]) if case["clip"] else 1.0)
        m, v, b1, b2 = s["m"][i], s["v"][i], HYPER["beta1"], HYPER["beta2"]
        if case["eight"]:
            # codes are defined on binary32 moments: every operation of them is rounded to 24 bits
            m, v = _exact_value(m, s["m_scale"][i], 4, True), _exact_value(v, s["v_scale"][i], 5, False)
            g = _r32(g)
            m = _r32(_r32(m * _c32(b1)) + _r32(_c32(1.0 - b1) * g))
            v = _r32(_r32(v * _c32(b2)) + _r32(_r32(_c32(1.0 - b2) * g) * g))
        else:
            m, v = m.double() * b1 + (1.0 - b1) * g, v.double() * b2 + (1.0 - b2) * g * g
        w = s["master"][i].double() * (1.0 - HYPER["lr"] * s["decay"][i])
        w -= HYPER["lr"] * (m / (1.0 - b1 ** HYPER["t"])) / ((v / (1.0 - b2 ** HYPER["t"])).sqrt() + HYPER["eps"])
        if case["eight"]:
            u = _exact_random(s["seed"], i, w.numel()).view(w.shape)
            m, v = _exact_round(m, torch.div(u, 65536, rounding_mode="floor"), 4), _exact_round(v, u % 65536, 5)
        for name, x in (("param", w), ("master", w), ("m", m), ("v", v)):
            out[name].append(x.flatten())
    return {name: torch.cat(x) for name, x in out.items()}


def _exact_act(x, name):
    """An activation and its derivative."""
    if name == "relu":
        return x.clamp(min=0.0), (x > 0.0).double()
    if name == "silu":
        p = torch.special.expit(x)
        return x * p, p + x * p * (1.0 - p)
    if name == "gelu":  # x times the logistic function of 2u, u = sqrt(2/pi) (x + 0.044715 x^3)
        p = torch.special.expit(math.sqrt(8.0 / math.pi) * (x + 0.044715 * x ** 3))
        return x * p, p + x * p * (1.0 - p) * math.sqrt(8.0 / math.pi) * (1.0 + 0.134145 * x ** 2)
    return x, torch.ones_like(x)


def _r32(x):
    return x.float().double()


def _c32(x):
    """A number's binary32 value."""
    return float(torch.tensor(x, dtype=torch.float32))


def _exact_value(code, scale, exponents, signed):
    """The numbers that 8-bit codes stand for: f/8 2^(e - top) or, for e = 0, f/8 2^(1 - top), times the block's scale."""
    c = code.flatten().double()
    sign = torch.ones_like(c)
    if signed:
        sign, c = torch.where(c >= 128, -1.0, 1.0), c % 128
    e, f, top = (c / 8).floor(), c % 8, 2 ** exponents - 1
    x = torch.where(e > 0, (1 + f / 8) * torch.exp2(e - top), f / 8 * 2.0 ** (1 - top)) * sign
    return (x * scale.double().repeat_interleave(BLOCK)[:x.numel()]).view(code.shape)


def _exact_round(x, dither, exponents):
    """The value that x is held as: a multiple of its step, up where the dither reaches over the rest."""
    n, top = x.numel(), 2 ** exponents - 1
    a = torch.zeros(-(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    a[:n] = x.abs().flatten()
    a = a.view(-1, BLOCK)
    most = a.amax(1, keepdim=True)
    # the least power of two 2^e for which most, rounded up to four significant bits, is below 2^(e+1)
    e = torch.floor(torch.log2(most.clamp(min=2.0 ** -126)))
    e = e + (most > 2.0 ** e * 1.875).double()
    a = (a / torch.exp2(e)).flatten()[:n].view(x.shape)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** (1 - top)))) - 3)
    whole = torch.floor(a / step)
    low = torch.round((a / step - whole) * 2 ** 20)
    a = (whole + (low + dither * 16 + 8 >= 2 ** 20).double()) * step
    return a * torch.exp2(e).repeat_interleave(BLOCK)[:n].view(x.shape) * torch.where(x < 0, -1.0, 1.0)


def _exact_random(seed, index, n):
    def mix(x):
        x = (x * 747796405 + 2891336453) % 2 ** 32
        x = ((x // 2 ** (x // 2 ** 28 + 4)) ^ x) * 277803737 % 2 ** 32
        return (x // 2 ** 22) ^ x

    key = (mix((mix(seed) + index) % 2 ** 32))
    x = (torch.arange(n, dtype=torch.int64, device="cuda") + key) % 2 ** 32
    x = (x * 747796405 + 2891336453) % 2 ** 32
    x = torch.bitwise_xor(torch.bitwise_right_shift(x, torch.bitwise_right_shift(x, 28) + 4), x) * 277803737 % 2 ** 32
    return torch.bitwise_xor(torch.bitwise_right_shift(x, 22), x)
