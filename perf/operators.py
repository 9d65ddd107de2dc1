"""The expert-grouped and 8-bit integer products: what is measured.

Four operators:
  grouped   rows grouped by expert times their expert's matrix (also the
            input gradient: the weights in the other order, and the
            activation's derivative in the epilogue)
  wgrad     the weight and bias gradients of a grouped product
  i8        int8 matrix product with a scale per token and per channel
  quant     int8 codes and a scale for each token

With `own` false, run() computes them with elementary torch operations in 32
bits; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32,
         "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1, "i8": 1}
DEV = "cuda"


def _lib():
    import tiled_layout_algebra_amd as tla
    return tla


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a decoding step through a square projection in 8 bits
        dict(name="i8_one_token", op="i8", m=1, n=4096, k=4096, out="bf16", bias=False, act="none"),
        # a prompt of odd length, bias and activation fused
        dict(name="i8_prompt_odd", op="i8", m=3001, n=4096, k=4096, out="f16", bias=True, act="gelu"),
        # the repository's large 8-bit size
        dict(name="i8_large", op="i8", m=8192, n=8192, k=8192, out="bf16", bias=True, act="gelu"),
        # the tokens of one decoding step put in 8 bits
        dict(name="quant_step", op="quant", m=64, k=4096, x="bf16"),
        # the tokens of a long prompt, row length not a multiple of the vector width
        dict(name="quant_prompt_odd", op="quant", m=16384, k=8191, x="bf16"),
        # one token on its two experts of eight
        dict(name="grouped_one_token", op="grouped", rows=2, g=8, n=4096, k=4096, type="bf16", out="bf16",
             b="nk", skew=0.0, empty=0, bias=False, act="none", z="none", scales=False),
        # a decoding batch over many experts: the experts' weights are what is read
        dict(name="grouped_decode", op="grouped", rows=128, g=32, n=2048, k=4096, type="bf16", out="bf16",
             b="nk", skew=0.5, empty=2, bias=False, act="none", z="none", scales=False),
        # a prompt through experts in 8 bits, scales per token and channel
        dict(name="grouped_i8_prompt", op="grouped", rows=4096, g=32, n=2048, k=4096, type="i8", out="f16",
             b="nk", skew=0.5, empty=0, bias=False, act="relu", z="none", scales=True),
        # training, forward: bias and GELU fused, the pre-activation kept for the backward pass
        dict(name="grouped_train", op="grouped", rows=16384, g=8, n=4096, k=4096, type="bf16", out="bf16",
             b="nk", skew=0.3, empty=0, bias=True, act="gelu", z="store", scales=False),
        # training, input gradient: the weights in the other order, GELU's derivative fused, ragged rows
        dict(name="grouped_train_dx", op="grouped", rows=16001, g=8, n=4096, k=4096, type="bf16", out="bf16",
             b="kn", skew=0.3, empty=1, bias=False, act="gelu", z="grad", scales=False),
        # training, weight and bias gradient
        dict(name="wgrad_train", op="wgrad", rows=16384, g=8, n=4096, k=4096, type="bf16", out="bf16",
             skew=0.3, empty=0, dbias=True),
        # a small layer's gradients: a few hundred rows over experts, one of them without any, fp32 gradients
        dict(name="wgrad_small", op="wgrad", rows=777, g=16, n=1024, k=512, type="f16", out="f32",
             skew=1.0, empty=1, dbias=True),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm; half of them multiples of 64 where they are large."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    v = min(max(v, lo), hi)
    if v >= 128 and rng.random() < 0.5:
        v = v // 64 * 64
    return v


def _largest():
    return 2.0 * 8192 ** 3


def draw(rng: random.Random):
    """Another case over the listed ones' ranges: one token to long prompts, narrow to wide layers, odd sizes."""
    op = rng.choice(["i8", "i8", "quant", "grouped", "grouped", "grouped", "wgrad"])
    while True:
        if op == "quant":
            return dict(op=op, m=_log(rng, 1, 16384), k=_log(rng, 64, 8192), x=rng.choice(["bf16", "f16", "f32"]))
        n, k = _log(rng, 256, 8192), _log(rng, 256, 8192)
        if op == "i8":
            c = dict(op=op, m=_log(rng, 1, 8192), n=n, k=k, out=rng.choice(["bf16", "f16"]), bias=rng.random() < 0.5,
                     act=rng.choice(["none", "relu", "gelu"]))
            if work(c)["flops"] <= _largest():
                return c
            continue
        g = rng.choice([2, 4, 8, 16, 32])
        rows = _log(rng, 1, 16384)
        c = dict(op=op, rows=rows, g=g, n=n, k=k, skew=rng.choice([0.0, 0.3, 1.0]),
                 empty=rng.randrange(0, max(1, g // 4) + 1))
        if op == "wgrad":
            c.update(type=rng.choice(["bf16", "f16"]), out=rng.choice(["bf16", "f32"]), dbias=rng.random() < 0.5)
        else:
            t = rng.choice(["bf16", "bf16", "f16", "i8", "e4m3"])
            train = t in ("bf16", "f16") and rows >= 256
            c.update(type=t, out="f16" if t == "f16" else "bf16", b="kn" if train and rng.random() < 0.5 else "nk",
                     bias=rng.random() < 0.5, act=rng.choice(["none", "relu", "gelu"]), z="none",
                     scales=t in ("i8", "e4m3"))
            if train and c["act"] != "none":
                c["z"] = rng.choice(["store", "grad"])
                c["bias"] = c["bias"] and c["z"] == "store"
        if work(c)["flops"] <= _largest() and g * n * k <= 1 << 28:
            return c


# ------------------------------------------------------------------- the data

def _counts(case, seed):
    """Rows of each expert: shares of a softmax of normal draws (skew: their spread), `empty` experts without any."""
    rng = random.Random(1000003 * seed + 17)
    g, rows = case["g"], case["rows"]
    w = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(g)]
    for e in rng.sample(range(g), min(case["empty"], g - 1)):
        w[e] = 0.0
    picks = rng.choices(range(g), weights=w, k=rows)
    counts = [0] * g
    for e in picks:
        counts[e] += 1
    return counts


def _normal(gen, shape, std, dtype):
    """Normal values in the storage type, drawn in pieces so that fp32 copies stay small."""
    x = torch.empty(shape, dtype=dtype, device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=gen, device=DEV) * std)
    return x


def _codes(gen, shape):
    """int8 codes as a quantizer leaves normal values: most of them small, clipped at 127."""
    x = torch.empty(shape, dtype=torch.int8, device=DEV)
    flat = x.view(-1)
    for i in range(0, flat.numel(), 1 << 26):
        part = flat[i:i + (1 << 26)]
        part.copy_((torch.randn(part.numel(), generator=gen, device=DEV) * 32).round().clamp(-127, 127))
    return x


def _operand(gen, shape, std, kind):
    return _codes(gen, shape) if kind == "i8" else _normal(gen, shape, std, TORCH[kind])


def _scale(gen, shape, mid):
    return mid * torch.exp(0.5 * torch.randn(shape, generator=gen, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "quant":
        x = _normal(gen, (case["m"], case["k"]), 1.0, TORCH[case["x"]])
        x *= _scale(gen, (case["m"], 1), 1.0).to(x.dtype)  # tokens differ in size
        s["x"] = x
        return s
    n, k = case["n"], case["k"]
    if case["op"] == "i8":
        s["a"] = _codes(gen, (case["m"], k))
        s["w"] = _codes(gen, (n, k))
        s["sa"] = _scale(gen, (case["m"],), 0.03)
        s["sb"] = _scale(gen, (n,), 0.03 / math.sqrt(k))
        s["bias"] = _normal(gen, (n,), 0.1, TORCH[case["out"]]) if case["bias"] else None
        return s
    counts = _counts(case, seed)
    ends = [sum(counts[:i]) for i in range(len(counts) + 1)]
    s["offsets"] = torch.tensor(ends, dtype=torch.int32).to(DEV)
    # what a program without grouped products keeps beside it: each row's expert and its place among that expert's rows
    s["expert"] = torch.tensor([e for e, c in enumerate(counts) for _ in range(c)]).to(DEV)
    s["place"] = torch.tensor([i for c in counts for i in range(c)]).to(DEV)
    s["most"] = max(counts)
    t = case["type"]
    s["a"] = _operand(gen, (case["rows"], k), 1.0, t)
    if case["op"] == "wgrad":
        s["y"] = _operand(gen, (case["rows"], n), 0.1, t)
        return s
    shape = (case["g"], n, k) if case["b"] == "nk" else (case["g"], k, n)
    s["w"] = _operand(gen, shape, 1 / math.sqrt(k), t)
    if t == "e4m3":  # stored at a size that e4m3 holds; the scale brings it back
        s["w"] = _operand(gen, shape, 1.0, t)
    i8 = t == "i8"
    s["sa"] = _scale(gen, (case["rows"],), 0.03 if i8 else 1.0) if case["scales"] else None
    s["sb"] = _scale(gen, (case["g"], n), (0.03 if i8 else 1.0) / math.sqrt(k)) if case["scales"] else None
    s["bias"] = _normal(gen, (case["g"], n), 0.1, TORCH[case["out"]]) if case["bias"] else None
    s["z"] = _normal(gen, (case["rows"], n), 1.0, TORCH[case["out"]]) if case["z"] == "grad" else None
    return s


# ------------------------------------------------------------- the plain form

def _act(y, act):
    if act == "relu":
        return torch.clamp(y, min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    return y


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def _by_expert(s, x):
    """x's rows in fp32 as [experts, most rows of one, columns], zeros where an expert has fewer."""
    out = torch.zeros(s["case"]["g"], s["most"], x.shape[1], device=x.device)
    out[s["expert"], s["place"]] = x.float()
    return out


def _plain(s):
    case = s["case"]
    if case["op"] == "quant":
        x = s["x"].float()
        scale = x.abs().amax(dim=1) / 127
        q = torch.round(x.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None])
        return [torch.clamp(q, -127, 127).to(torch.int8), scale]
    out = TORCH[case["out"]]
    if case["op"] == "i8":
        y = (s["a"].float() @ s["w"].float().t()) * s["sa"][:, None] * s["sb"]
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return [_act(y, case["act"]).to(out)]
    if case["op"] == "wgrad":
        y = _by_expert(s, s["y"])
        dw = torch.bmm(_by_expert(s, s["a"]).transpose(1, 2).contiguous(), y).to(out)
        return [dw, y.sum(dim=1)] if case["dbias"] else [dw]
    w = s["w"].float()
    if case["b"] == "nk":
        w = w.transpose(1, 2).contiguous()
    y = torch.bmm(_by_expert(s, s["a"]), w)[s["expert"], s["place"]]
    if case["scales"]:
        y = y * s["sa"][:, None] * s["sb"][s["expert"]]
    if s["bias"] is not None:
        y = y + s["bias"].float()[s["expert"]]
    if case["z"] == "grad":
        return [(y * _act_grad(s["z"].float(), case["act"])).to(out)]
    d = _act(y, case["act"]).to(out)
    return [d, y.to(out)] if case["z"] == "store" else [d]


# -------------------------------------------------------------- the library's

def _own(s):
    tla = _lib()
    code = {"f16": tla.F16, "bf16": tla.BF16, "f32": tla.F32, "e4m3": tla.E4M3, "i8": tla.I8}
    acts = {"none": tla.ACT_NONE, "relu": tla.ACT_RELU, "gelu": tla.ACT_GELU}
    case = s["case"]
    if case["op"] == "quant":
        m, k = case["m"], case["k"]
        q = torch.empty(m, k, dtype=torch.int8, device=DEV)
        scale = torch.empty(m, dtype=torch.float32, device=DEV)
        tla.quantize_rows(m, k, s["x"], code[case["x"]], k, q, k, scale)
        return [q, scale]
    n, k, out = case["n"], case["k"], case["out"]
    if case["op"] == "i8":
        d = torch.empty(case["m"], n, dtype=TORCH[out], device=DEV)
        tla.gemm_i8(case["m"], n, k, s["a"], k, s["w"], tla.COL_MAJOR, k, d, code[out], n,
                    scale_a=s["sa"], scale_b=s["sb"], bias=s["bias"], act=acts[case["act"]])
        return [d]
    g, rows = case["g"], case["rows"]
    if case["op"] == "wgrad":
        d = torch.empty(g, k, n, dtype=TORCH[out], device=DEV)
        db = torch.empty(g, n, dtype=torch.float32, device=DEV) if case["dbias"] else None
        tla.grouped_gemm_wgrad(g, rows, n, k, s["offsets"], s["a"], k, s["y"], n, code[case["type"]],
                               d, code[out], tla.ROW_MAJOR, n, k * n, dbias=db)
        return [d, db] if case["dbias"] else [d]
    d = torch.empty(rows, n, dtype=TORCH[out], device=DEV)
    z, mode = s["z"], tla.Z_NONE
    if case["z"] == "store":
        z, mode = torch.empty_like(d), tla.Z_STORE
    elif case["z"] == "grad":
        mode = tla.Z_GRAD
    nk = case["b"] == "nk"
    tla.grouped_gemm(g, rows, n, k, s["offsets"], s["a"], code[case["type"]], k, s["w"],
                     tla.COL_MAJOR if nk else tla.ROW_MAJOR, k if nk else n, n * k, d, code[out], n,
                     scale_a=s["sa"], scale_b=s["sb"], bias=s["bias"], Z=z, ldz=n, z_mode=mode,
                     act=acts[case["act"]])
    return [d, z] if case["z"] == "store" else [d]


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------- work

def work(case):
    """Bytes: each input read once, each output written once (the matrices of experts that can have rows); flops: two a product."""
    if case["op"] == "quant":
        e = case["m"] * case["k"]
        return {"bytes": e * (SIZE[case["x"]] + 1) + 4 * case["m"], "flops": 3 * e}
    n, k = case["n"], case["k"]
    out = SIZE[case["out"]]
    if case["op"] == "i8":
        m = case["m"]
        return {"bytes": m * k + n * k + m * n * out + 4 * (m + n) + (n * out if case["bias"] else 0), "flops": 2 * m * n * k}
    rows, g, t = case["rows"], case["g"], SIZE[case["type"]]
    if case["op"] == "wgrad":
        return {"bytes": rows * (n + k) * t + g * n * k * out + (4 * g * n if case["dbias"] else 0), "flops": 2 * rows * n * k}
    # experts with at least one row, expected for rows drawn at random
    live = g - min(case["empty"], g - 1)
    live = max(1, round(live * (1 - (1 - 1 / live) ** rows)))
    extra = (rows * n * out if case["z"] != "none" else 0) + (live * n * out if case["bias"] else 0)
    if case["scales"]:
        extra += 4 * rows + 4 * live * n
    return {"bytes": rows * k * t + live * n * k * t + rows * n * out + extra, "flops": 2 * rows * n * k}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits, one expert after another."""
    s = prepare(case, seed)
    if case["op"] == "quant":
        x = s["x"].double()
        return [None, x.abs().max(dim=1).values / 127]

    def gelu(v):
        return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))

    def gelu_slope(v):
        return 0.5 * torch.special.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)

    f = {"none": lambda v: v, "relu": lambda v: v.clamp(min=0), "gelu": gelu}
    slope = {"none": lambda v: torch.ones_like(v), "relu": lambda v: (v > 0).double(), "gelu": gelu_slope}
    if case["op"] == "i8":
        z = torch.mm(s["a"].double() * s["sa"].double().unsqueeze(1), (s["w"].double() * s["sb"].double().unsqueeze(1)).t())
        if s["bias"] is not None:
            z += s["bias"].double()
        return [f[case["act"]](z)]
    off = s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(case["g"])]
    if case["op"] == "wgrad":
        dw = torch.stack([torch.mm(s["a"][lo:hi].double().t(), s["y"][lo:hi].double()) for _, lo, hi in spans])
        db = torch.stack([s["y"][lo:hi].double().sum(0) for _, lo, hi in spans])
        return [dw, db] if case["dbias"] else [dw]
    z = torch.empty(case["rows"], case["n"], dtype=torch.float64, device=DEV)
    for e, lo, hi in spans:
        if lo == hi:
            continue
        w = s["w"][e].double()
        part = torch.mm(s["a"][lo:hi].double(), w.t() if case["b"] == "nk" else w)
        if case["scales"]:
            part = part * s["sa"][lo:hi].double().unsqueeze(1) * s["sb"][e].double()
        if s["bias"] is not None:
            part = part + s["bias"][e].double()
        z[lo:hi] = part
    if case["z"] == "grad":
        return [z * slope[case["act"]](s["z"].double())]
    d = f[case["act"]](z)
    return [d, z] if case["z"] == "store" else [d]
