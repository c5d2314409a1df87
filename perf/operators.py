"""Cases of the optimizer operators over many tensors: global gradient norm and
clipping, the AdamW step with moments in 32 and in 8 bits, and the 8-bit
moments' way in and out.  Each has its plain form in torch, and the calls a
user makes of this repository's kernels.

A case's tensors lie in flat buffers, each tensor at a multiple of 256
elements (as the views of a gradient bucket do), so that the plain form works
on a whole buffer at once: a row of 256 is one block of one tensor.
"""

import math

import torch

own = False

BLOCK = 256
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "": 0}
MASK = 0xFFFFFFFF
# odd 32-bit multipliers of the rounding draws' hash
WEYL, MUL_A, MUL_B, MUL_C = 0x9E3779B9, 0x6A09E667, 0xBB67AE85, 0x3C6EF373
BETA1, BETA2 = (float(torch.tensor(b, dtype=torch.float32)) for b in (0.9, 0.999))
EPS = float(torch.tensor(1e-8, dtype=torch.float32))
LR, DECAY = (float(torch.tensor(x, dtype=torch.float32)) for x in (1e-3, 0.1))


def sizes(case):
    """Elements of each tensor, and whether weight decay applies to it."""
    d, f, layers = case["width"], case["ff"], case["layers"]
    vectors = [(d, False)] * (2 * layers + 1)
    tables = [(case["rows"] * d, True), (case["rows2"] * d, True)]
    matrices = ([(d * d, True)] * 4 + [(d * f, True)] * 3) * layers
    return {"vectors": vectors, "tables": tables, "mixed": [(4 * d * d, True)] * 3,
            "all": matrices + vectors + tables}[case["what"]]


def _case(name, op, what, width, layers=1, ff=1, rows=1, rows2=1, grad="f32", param="f32", copy="", clip=False):
    return {"name": name, "op": op, "what": what, "width": width, "layers": layers, "ff": ff, "rows": rows,
            "rows2": rows2, "grad": grad, "param": param, "copy": copy, "clip": clip}


def listed():
    llama = {"layers": 24, "ff": 5632, "rows": 32000, "rows2": 32000}
    return [
        # the norm weights of a 24-layer model: latency is all there is
        _case("norm-vectors", "norm", "vectors", 2048, layers=24),
        # every gradient of the ~1B Llama-shaped set, as bf16 training leaves them
        _case("norm-llama-bf16", "norm", "all", 2048, grad="bf16", **llama),
        # the mixed-shape sweep set, clipped in place before the Shampoo step reads it
        _case("clip-mixed", "clip", "mixed", 1024),
        # fp16 gradients under a loss scale, odd sizes throughout
        _case("clip-odd-f16", "clip", "all", 1003, layers=6, ff=2741, rows=12289, rows2=12289, grad="f16"),
        # the same norm weights stepped, clipped by the global norm
        _case("adamw32-vectors", "adamw32", "vectors", 2048, layers=24, clip=True),
        # GPT-2's embeddings beside Shampoo's matrices
        _case("adamw32-gpt2-tables", "adamw32", "tables", 768, rows=50257, rows2=1024),
        # embedding and head of the Llama-shaped set: fp32 master, bf16 gradients and model weights
        _case("adamw32-llama-ends", "adamw32", "tables", 2048, rows=32000, rows2=32000, grad="bf16", copy="bf16",
              clip=True),
        # a few odd-sized vectors in pure bf16: latency, partial blocks
        _case("adamw8-odd-vectors", "adamw8", "vectors", 1003, layers=6, grad="bf16", param="bf16"),
        # GPT-2's embeddings with 8-bit moments
        _case("adamw8-gpt2-tables", "adamw8", "tables", 768, rows=50257, rows2=1024),
        # the whole Llama-shaped set in pure bf16 with 8-bit moments
        _case("adamw8-llama-bf16", "adamw8", "all", 2048, grad="bf16", param="bf16", **llama),
        # a small model's 32-bit moments taken into 8 bits and read back
        _case("moments-odd", "moments", "all", 259, layers=2, ff=701, rows=4099, rows2=515),
        # a checkpoint of the Llama-shaped set's embedding and head
        _case("moments-llama-ends", "moments", "tables", 2048, rows=32000, rows2=32000),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["norm", "clip", "adamw32", "adamw8", "moments"])
    what = rng.choice(["vectors", "tables", "mixed", "all"])
    width = log(96, 2048) if what != "mixed" else log(96, 1500)
    grad = rng.choice(["f32", "bf16", "f16"])
    param = rng.choice(["f32", "bf16"]) if op.startswith("adamw") else "f32"
    copy = rng.choice(["", "bf16", "f16"]) if op.startswith("adamw") and param == "f32" else ""
    c = _case("", op, what, width, layers=log(1, 24) if what == "vectors" else log(1, 8), ff=log(width, 3 * width),
              rows=log(500, 32000), rows2=log(100, 32000), grad=grad, param=param, copy=copy,
              clip=op.startswith("adamw") and rng.random() < 0.5)
    del c["name"]
    return c


def _layout(case):
    """Per tensor (start, elements), in elements of a flat buffer, and the buffer's size."""
    at, spans = 0, []
    for n, _ in sizes(case):
        spans.append((at, n))
        at += -(-n // BLOCK) * BLOCK
    return spans, at


def _views(flat, spans):
    return [flat[a:a + n] for a, n in spans]


def prepare(case, seed):
    spans, total = _layout(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "spans": spans, "seed": seed % 1000003, "t": 0, "n": sum(n for _, n in spans)}
    dev = "cuda"
    # which entries belong to a tensor, as bounds of the padding behind each
    pads = [(a + n, a + -(-n // BLOCK) * BLOCK) for a, n in spans if n % BLOCK]

    def filled(std, dtype, spread=False):
        x = torch.randn(total, generator=gen, device=dev)
        if spread:  # rows of very different scales, as gradients and moments have
            x.view(-1, BLOCK).mul_(torch.randn(total // BLOCK, 1, generator=gen, device=dev).mul_(1.5).exp_())
        x = x.mul_(std).to(dtype)
        for a, b in pads:
            x[a:b] = 0
        return x

    op = case["op"]
    if op == "moments":
        s["m_in"] = filled(1e-3, torch.float32, True)
        s["v_in"] = filled(1e-3, torch.float32, True).square_()
    else:
        s["grad"] = filled(1e-2, TYPES[case["grad"]], True)
    if op in ("norm", "clip"):
        # half of four times the norm that these gradients have, about
        s["max_norm"] = 2.0 * 1e-2 * math.exp(1.5 ** 2) * math.sqrt(s["n"]) if op == "clip" else 1.0
    if op.startswith("adamw") or op == "moments":
        s["param"] = filled(0.02, TYPES[case["param"]])
        if case["copy"]:
            s["copy"] = torch.zeros(total, dtype=TYPES[case["copy"]], device=dev)
        bits = 32 if op == "adamw32" else 8
        if bits == 32:
            s["m"], s["v"] = (torch.zeros(total, device=dev) for _ in "mv")
        else:
            s["m"], s["v"] = (torch.zeros(total, dtype=torch.uint8, device=dev) for _ in "mv")
            s["m_scale"], s["v_scale"] = (torch.zeros(total // BLOCK, dtype=torch.uint8, device=dev) for _ in "mv")
            s["m_out"], s["v_out"] = (torch.empty(total, dtype=torch.bfloat16, device=dev) for _ in "mv")
    if not own:
        # per block: its tensor, its place in the tensor, its weight decay
        blocks = torch.tensor([-(-n // BLOCK) for _, n in spans], device=dev)
        first = torch.tensor([a // BLOCK for a, _ in spans], device=dev)
        tensor = torch.repeat_interleave(torch.arange(len(spans), device=dev), blocks)
        decay = torch.tensor([DECAY if w else 0.0 for _, w in sizes(case)], device=dev)
        s["tensor"], s["decay"] = tensor, decay[tensor].unsqueeze(1)
        s["at"] = ((torch.arange(total // BLOCK, device=dev) - first[tensor]) * BLOCK).unsqueeze(1)
        s["count"] = len(spans)
    else:
        from matrix_inverse_roots_stack_b200 import binding as bd
        if "grad" in s:
            grads = _views(s["grad"], spans)
            s["clipper"] = bd.GradClip(grads)
        if "param" in s:
            per_block = [(a // BLOCK, -(-n // BLOCK)) for a, n in spans]
            eight = {} if bits == 32 else {"m_scale": _views(s["m_scale"], per_block),
                                           "v_scale": _views(s["v_scale"], per_block)}
            s["opt"] = bd.AdamW(_views(s["param"], spans), grads if "grad" in s else _views(s["m_in"], spans),
                                hp=bd.make_adamw_hparams(beta1=BETA1, beta2=BETA2, adam_eps=EPS, seed=s["seed"]),
                                copies=_views(s["copy"], spans) if case["copy"] else None, state_bits=bits,
                                m=_views(s["m"], spans), v=_views(s["v"], spans),
                                weight_decay=[DECAY if w else 0.0 for _, w in sizes(case)], **eight)
    return s


# ------------------------------------------------------------------ plain form

def _norm(s, max_norm, inv_scale):
    """Norm of the unscaled gradients, and the factor that unscales and clips them: sums in 64 bits."""
    norm = s["grad"].double().square().sum().sqrt() * inv_scale
    coef = torch.where(norm > max_norm, max_norm / norm, torch.ones_like(norm)) * inv_scale
    coef = torch.where(torch.isfinite(norm), coef, torch.full_like(norm, math.nan))
    return norm.float(), coef.float()


def _key(words):
    x = 0
    for w in words:
        x ^= w
        for c in (MUL_A, MUL_B):
            x ^= x >> 16
            x = x * c & MASK
        x ^= x >> 15
        x = x + WEYL & MASK
    return x


def _draws(s):
    """32 bits for each element, from the seed, the step, the tensor and the element's place in it."""
    x = torch.full((s["count"],), _key((s["seed"], 0, s["t"])), dtype=torch.int64, device="cuda")
    at = s["at"] + torch.arange(BLOCK, device="cuda")
    for w in (torch.arange(s["count"], device="cuda"), 0):  # every place here is below 2^32
        x = x ^ w
        x = (x ^ (x >> 16)) * MUL_A & MASK
        x = (x ^ (x >> 16)) * MUL_B & MASK
        x = (x ^ (x >> 15)) + WEYL & MASK
    x = at * WEYL + x[s["tensor"]].unsqueeze(1) & MASK
    x = (x ^ (x >> 16)) * MUL_A & MASK
    x = (x ^ (x >> 15)) * MUL_B & MASK
    return x ^ (x >> 16)


def _powers():
    """2^(i - 127) for i = 0 .. 254; a scale of 0 is a block of zeros, one of 255 is not finite."""
    p = [0.0] + [math.ldexp(1.0, i - 127) for i in range(1, 255)] + [math.inf]
    return torch.tensor(p, device="cuda")


def _encode(x, mantissa, draw):
    """Codes and scales of the magnitudes in x (blocks by rows): `mantissa` bits behind four of exponent; the
    scale is the least power of two that holds the block's maximum.  draw: 16 bits for each element, or None
    to round to nearest, ties to even."""
    # the largest code stands for 1.75 * 2^8 (seven bits) or 1.9375 * 2^14 (eight bits)
    slack, top = ((1 << 21) - 1, 8) if mantissa == 3 else ((1 << 19) - 1, 14)
    most = x.amax(1, keepdim=True)
    scale = (((most.view(torch.int32) + slack) >> 23) - top).clamp(1, 254)
    unit = _powers()[254 - scale]
    # as bits of a float whose smallest normal number is the format's: its low bits are what rounding drops
    low = 23 - mantissa
    y = x * unit * math.ldexp(1.0, -120 if mantissa == 3 else -126)
    bits = y.view(torch.int32)
    if draw is None:
        bits = bits + ((1 << (low - 1)) - 1) + ((bits >> low) & 1)
    else:
        bits = bits + (draw << (low - 16))
    return bits >> low, scale


def _decode(codes, scale, mantissa):
    """The magnitudes that codes (blocks by rows) and scales stand for."""
    y = (codes << (23 - mantissa)).view(torch.float32)
    y = y * math.ldexp(1.0, 120 if mantissa == 3 else 126)
    return y * _powers()[scale]


def _read(s):
    """First moment, and root of the second, from 8 bits."""
    m = s["m"].view(-1, BLOCK).int()
    v = s["v"].view(-1, BLOCK).int()
    a = _decode(m & 127, s["m_scale"].int().unsqueeze(1), 3)
    return torch.where(m > 127, -a, a), _decode(v, s["v_scale"].int().unsqueeze(1), 4)


def _store(s, m, root, draws):
    code, scale = _encode(m.abs(), 3, None if draws is None else (draws >> 16).int())
    s["m"].view(-1, BLOCK).copy_(torch.where(m.view(torch.int32) < 0, code + 128, code))
    s["m_scale"].copy_(scale.squeeze(1))
    code, scale = _encode(root, 4, None if draws is None else (draws & 0xFFFF).int())
    s["v"].view(-1, BLOCK).copy_(torch.where(root > 0, code.clamp(min=1), code))  # never rounded away
    s["v_scale"].copy_(scale.squeeze(1))


def _values(s):
    m, root = _read(s)
    s["m_out"].copy_(m.view(-1))
    s["v_out"].copy_((root * root).view(-1))
    return [s["m_out"], s["v_out"]]


def _adamw(s, eight):
    case = s["case"]
    s["t"] += 1
    coef = _norm(s, 1.0, 1.0)[1] if case["clip"] else None
    g = s["grad"].float()
    g = (g if coef is None else g * coef).view(-1, BLOCK)
    if eight:
        m, root = _read(s)
        v = root * root
    else:
        m, v = s["m"].view(-1, BLOCK), s["v"].view(-1, BLOCK)
    m = m * BETA1 + g * (1.0 - BETA1)
    v = v * BETA2 + g * (1.0 - BETA2) * g
    root = v.sqrt()
    c1 = 1.0 / (1.0 - BETA1 ** s["t"])
    c2 = math.sqrt(1.0 / (1.0 - BETA2 ** s["t"]))
    p = s["param"].float().view(-1, BLOCK)
    p = p - LR * (m * c1 / (root * c2 + EPS) + p * s["decay"])
    draws = _draws(s) if eight or case["param"] == "bf16" else None
    if case["param"] == "bf16":
        bits = p.view(torch.int32)
        bits = bits + ((draws * MUL_C & MASK) >> 16).int() & -65536
        p = bits.view(torch.float32)
    s["param"].copy_(p.view(-1))
    if case["copy"]:
        s["copy"].copy_(p.view(-1))
    if eight:
        _store(s, m, root, draws)
    else:
        s["m"].copy_(m.view(-1))
        s["v"].copy_(v.view(-1))
    out = [s["param"]] + ([s["copy"]] if case["copy"] else [])
    return out + (_values(s) if eight else [s["m"], s["v"]])


def _clip_args(s):
    """Every other pass unscales up and clips, the passes between scale down: the gradients keep their size."""
    return (s["max_norm"], 4.0) if s["t"] % 2 == 1 else (math.inf, 0.5)


# ------------------------------------------------------------------ one pass

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        if op == "norm":
            return [s["clipper"].norm(s["max_norm"])]
        if op == "clip":
            s["t"] += 1
            max_norm, inv_scale = _clip_args(s)
            return [s["clipper"].clip(max_norm, inv_scale), s["grad"]]
        if op == "moments":
            s["opt"].load_moments(s["m_in"], s["v_in"])
            return list(s["opt"].read_moments(m=s["m_out"], v=s["v_out"]))
        coef = s["clipper"].norm(1.0)[1:] if s["case"]["clip"] else None
        s["opt"].step(LR, coef=coef)
        out = [s["param"]] + ([s["copy"]] if s["case"]["copy"] else [])
        if op == "adamw8":
            return out + list(s["opt"].read_moments(m=s["m_out"], v=s["v_out"]))
        return out + [s["m"], s["v"]]
    if op == "norm":
        return [torch.stack(_norm(s, s["max_norm"], 1.0))]
    if op == "clip":
        s["t"] += 1
        norm, coef = _norm(s, *_clip_args(s))
        s["grad"].copy_(s["grad"].float() * coef)
        return [torch.stack([norm, coef]), s["grad"]]
    if op == "moments":
        _store(s, s["m_in"].view(-1, BLOCK), s["v_in"].sqrt().view(-1, BLOCK), None)
        return _values(s)
    return _adamw(s, op == "adamw8")


def work(case):
    n = sum(n for n, _ in sizes(case))
    blocks = sum(-(-n // BLOCK) for n, _ in sizes(case))
    g, p, c = BYTES[case["grad"]], BYTES[case["param"]], BYTES[case["copy"]]
    op = case["op"]
    if op == "norm":
        return {"bytes": n * g + 8, "flops": 2 * n}
    if op == "clip":
        return {"bytes": 2 * n * g + 8, "flops": 3 * n}
    if op == "moments":  # both moments read, held in 8 bits, and their values written as bf16
        return {"bytes": n * (8 + 2 + 4) + 2 * blocks, "flops": 6 * n}
    if op == "adamw32":
        return {"bytes": n * (2 * p + g + c + 16), "flops": 18 * n}
    # codes in and out, a scale in and out for each, and the moments' values as bf16
    return {"bytes": n * (2 * p + g + c + 4 + 4) + 4 * blocks, "flops": 24 * n}


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """The first pass's outputs in 64 bits, block rows a slab at a time."""
    s = prepare(case, seed)
    s["t"] = 1
    op, total = case["op"], _layout(case)[1]
    grad = s.get("grad")
    slabs = [(a, min(a + (1 << 26), total)) for a in range(0, total, 1 << 26)]
    inv_scale, max_norm = 1.0, s.get("max_norm", 1.0)
    if op == "clip":
        max_norm, inv_scale = _clip_args(s)
    if grad is not None:
        norm = inv_scale * math.sqrt(math.fsum(float((grad[a:b].double() ** 2).sum()) for a, b in slabs))
        coef = inv_scale * min(1.0, max_norm / norm)
    if op in ("norm", "clip"):
        scalars = torch.tensor([norm, coef], dtype=torch.float64)
        return [scalars] if op == "norm" else [scalars, grad.double() * coef]

    def power(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    def grid(y, mantissa, lowest, u):
        """|y| on the numbers of `mantissa` bits, evenly spaced below 2^lowest; u in [0, 1): rounded up where
        the dropped part and u reach a whole, None: to nearest, ties to even."""
        e = torch.frexp(y.abs())[1].sub(1).clamp(min=lowest) - mantissa
        q = y.abs() * power(-e)
        return (torch.floor(q + u) if u is not None else torch.round(q)) * power(e)

    def held(y, mantissa, lowest, largest, u):
        most = y.abs().amax(1, keepdim=True)
        e = torch.frexp(most / largest)
        scale = torch.where(e[0] == 0.5, e[1] - 1, e[1])  # least power of two that is enough
        scale = torch.where(most > 0, scale, torch.zeros_like(scale)).clamp(min=-126)
        q = grid(y * power(-scale), mantissa, lowest, u)
        if mantissa == 4:
            q = torch.where(y > 0, q.clamp(min=2.0 ** (lowest - mantissa)), q)
        return q.copysign(y) * power(scale)

    if not case["clip"]:
        coef = 1.0
    starts = torch.tensor([a for a, _ in s["spans"]], device="cuda")
    decays = torch.tensor([DECAY if w else 0.0 for _, w in sizes(case)], dtype=torch.float64, device="cuda")
    keys = torch.tensor([_key((s["seed"], 0, 1, k, 0)) for k in range(len(starts))], device="cuda")
    outs = []
    for a, b in slabs:
        rows = (torch.searchsorted(starts, torch.arange(a, b, BLOCK, device="cuda"), right=True) - 1).unsqueeze(1)
        place = torch.arange(a, b, device="cuda").view(-1, BLOCK) - starts[rows]
        if op == "moments":
            m = held(s["m_in"][a:b].double().view(-1, BLOCK), 3, -6, 448.0, None)
            r = held(s["v_in"][a:b].double().sqrt().view(-1, BLOCK), 4, 0, 31744.0, None)
            outs.append([m.view(-1), (r * r).view(-1)])
            continue
        h = (place * WEYL + keys[rows]) % 2 ** 32
        h = (h ^ h // 2 ** 16) * MUL_A % 2 ** 32
        h = (h ^ h // 2 ** 15) * MUL_B % 2 ** 32
        h = h ^ h // 2 ** 16
        g = grad[a:b].double().view(-1, BLOCK) * coef
        m, v = (1 - BETA1) * g, (1 - BETA2) * g * g
        p = s["param"][a:b].double().view(-1, BLOCK)
        p = p - LR * (g / (g.abs() + EPS) + decays[rows] * p)
        if case["param"] == "bf16":
            u = (h * MUL_C % 2 ** 32 // 2 ** 16).double() / 2 ** 16
            p = grid(p, 7, -126, u).copysign(p)
        if op == "adamw8":
            m = held(m, 3, -6, 448.0, (h // 2 ** 16).double() / 2 ** 16)
            r = held(v.sqrt(), 4, 0, 31744.0, (h % 2 ** 16).double() / 2 ** 16)
            v = r * r
        outs.append([p.view(-1)] + ([p.view(-1)] if case["copy"] else []) + [m.view(-1), v.view(-1)])
    return [torch.cat([o[k] for o in outs]) for k in range(len(outs[0]))]
