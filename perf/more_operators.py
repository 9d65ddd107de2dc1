"""The gated feed-forward products and the block-scaled e4m3 product: what is measured.

Four operators:
  gated     both projections of a gated feed-forward layer, the activation and
            the product, 16 bits or e4m3 with block scales
  grad      its backward pass: the gradient of the hidden layer is never stored
  blocks    e4m3 matrix product with a scale for each block of 128
  quant     e4m3 codes and a scale for each 1 x 128 or 128 x 128 block

With `own` false, run() computes them with elementary torch operations in 32
bits; with `own` true it calls the library.
"""
import math
import random

import torch

own = False

TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"f16": 2, "bf16": 2, "f32": 4, "e4m3": 1}
DEV = "cuda"


def _lib():
    import tiled_layout_algebra_amd as tla
    return tla


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a decoding step through a dense layer
        dict(name="gated_one_token", op="gated", rows=1, g=1, n=8192, k=4096, type="bf16", out="bf16", w="nk",
             act="silu", bias=False, keep=False, skew=0.0, empty=0),
        # training, forward: gate and up kept for the backward pass
        dict(name="gated_train", op="gated", rows=8192, g=1, n=8192, k=4096, type="bf16", out="bf16", w="nk",
             act="silu", bias=False, keep=True, skew=0.0, empty=0),
        # a prompt of odd length over experts whose weights are stored [K, N], with bias
        dict(name="gated_experts_odd", op="gated", rows=3001, g=8, n=1408, k=2048, type="f16", out="f16", w="kn",
             act="gelu", bias=True, keep=False, skew=0.5, empty=1),
        # a prompt through the same kind of layer served in 8 bits
        dict(name="gated_e4m3_prompt", op="gated", rows=2048, g=1, n=8192, k=4096, type="e4m3", out="bf16", w="nk",
             act="silu", bias=False, keep=False, skew=0.0, empty=0),
        # training, backward: the down projection's weights in the other order, the hidden layer computed again
        dict(name="grad_train", op="grad", rows=8192, g=1, n=8192, k=4096, type="bf16", w="kn", act="silu",
             hidden=True, skew=0.0, empty=0),
        # a small layer of experts, odd extents, one expert without rows
        dict(name="grad_small_odd", op="grad", rows=777, g=4, n=1000, k=520, type="f16", w="nk", act="gelu",
             hidden=False, skew=0.5, empty=1),
        # one token through a square projection
        dict(name="blocks_one_token", op="blocks", m=1, g=1, n=4096, k=4096, out="bf16", bias=False, act="none",
             skew=0.0, empty=0),
        # a decoding batch over many experts: the experts' weights are what is read
        dict(name="blocks_decode", op="blocks", m=128, g=32, n=2048, k=4096, out="bf16", bias=False, act="none",
             skew=0.5, empty=2),
        # a prompt of odd length, the last block of K and of N not whole
        dict(name="blocks_prompt_odd", op="blocks", m=3001, g=1, n=4000, k=4000, out="f16", bias=True, act="gelu",
             skew=0.0, empty=0),
        # the repository's large 8-bit size
        dict(name="blocks_large", op="blocks", m=8192, g=1, n=8192, k=8192, out="bf16", bias=False, act="none",
             skew=0.0, empty=0),
        # the tokens of one decoding step put in 8 bits
        dict(name="quant_step", op="quant", m=64, k=4096, x="bf16", rows=1),
        # a weight matrix in 128 x 128 blocks, row length not a multiple of the block
        dict(name="quant_weights_odd", op="quant", m=16384, k=8191, x="bf16", rows=128),
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
    """Another case over the listed ones' ranges: one token to long prompts, narrow to wide layers, odd sizes, dense or experts."""
    op = rng.choice(["gated", "gated", "gated", "grad", "blocks", "blocks", "quant"])
    while True:
        if op == "quant":
            return dict(op=op, m=_log(rng, 1, 16384), k=_log(rng, 64, 8192), x=rng.choice(["bf16", "f16", "f32"]),
                        rows=rng.choice([1, 1, 128]))
        n, k, rows = _log(rng, 256, 8192), _log(rng, 256, 8192), _log(rng, 1, 16384)
        g = rng.choice([1, 1, 4, 8, 32])
        c = dict(op=op, g=g, n=n, k=k, skew=rng.choice([0.0, 0.3, 1.0]), empty=rng.randrange(0, max(1, g // 4) + 1))
        if op == "blocks":
            c.update(m=rows, out=rng.choice(["bf16", "f16"]), bias=rng.random() < 0.3, act=rng.choice(["none", "none", "gelu", "silu"]))
        elif op == "grad":
            c.update(rows=rows, type=rng.choice(["bf16", "f16"]), w=rng.choice(["nk", "kn"]), act=rng.choice(["silu", "gelu", "relu"]),
                     hidden=rng.random() < 0.5)
        else:
            t = rng.choice(["bf16", "f16", "e4m3"])
            c.update(rows=rows, type=t, out="f16" if t == "f16" else "bf16", w="nk" if t == "e4m3" else rng.choice(["nk", "kn"]),
                     act=rng.choice(["silu", "gelu", "relu"]), bias=rng.random() < 0.3, keep=t != "e4m3" and rows >= 256 and rng.random() < 0.5)
        if work(c)["flops"] <= _largest() and g * n * k <= 1 << 27:
            return c


# ------------------------------------------------------------------- the data

def _counts(case, rows, seed):
    """Rows of each expert: shares of a softmax of normal draws (skew: their spread), `empty` experts without any."""
    rng = random.Random(1000003 * seed + 29)
    g = case["g"]
    w = [math.exp(case["skew"] * rng.gauss(0, 1)) for _ in range(g)]
    for e in rng.sample(range(g), min(case["empty"], g - 1)):
        w[e] = 0.0
    counts = [0] * g
    for e in rng.choices(range(g), weights=w, k=rows):
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


def _up(x, to):
    return -(-x // to) * to


def _coded(gen, mats, r, c, std, tokens):
    """[mats, r, c] normal values as e4m3 codes (rows 16 bytes apart or a multiple) and their scales: a scale for each
    token's 128 values, laid out [blocks of c, mats r], or for each 128 x 128 block, [mats, blocks of r, blocks of c]."""
    rb, cb = (r, 1) if tokens else (_up(r, 128) // 128, 128)
    kb = _up(c, 128) // 128
    codes = torch.zeros(mats, r, _up(c, 16), dtype=torch.float8_e4m3fn, device=DEV)
    scales = torch.empty(mats, rb, kb, device=DEV)
    for e in range(mats):
        x = _normal(gen, (r, c), std, torch.float32)
        if tokens:
            x *= torch.exp(0.5 * torch.randn(r, 1, generator=gen, device=DEV))  # tokens differ in size
        full = torch.nn.functional.pad(x, (0, kb * 128 - c, 0, rb * cb - r)).view(rb, cb, kb, 128)
        scales[e] = full.abs().amax(dim=(1, 3)) / 448
        full = (full / scales[e].clamp(min=1e-30)[:, None, :, None]).clamp(-448, 448)
        codes[e, :, :c] = full.view(rb * cb, kb * 128)[:r, :c].to(torch.float8_e4m3fn)
    if tokens:
        return codes[0], scales[0].t().contiguous()
    return codes, scales


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    s = {"case": case}
    op, k = case["op"], case["k"]
    if op == "quant":
        x = _normal(gen, (case["m"], k), 1.0, TORCH[case["x"]])
        x *= torch.exp(0.5 * torch.randn(case["m"], 1, generator=gen, device=DEV)).to(x.dtype)  # rows differ in size
        s["x"] = x
        return s
    g, n = case["g"], case["n"]
    rows = case["m"] if op == "blocks" else case["rows"]
    counts = _counts(case, rows, seed)
    ends = [sum(counts[:i]) for i in range(g + 1)]
    s["offsets"] = torch.tensor(ends, dtype=torch.int32).to(DEV) if g > 1 else None
    # what a program without grouped products keeps beside it: each row's expert and its place among that expert's rows
    s["expert"] = torch.tensor([e for e, c in enumerate(counts) for _ in range(c)]).to(DEV)
    s["place"] = torch.tensor([i for c in counts for i in range(c)]).to(DEV)
    s["most"] = max(counts)
    std = 1 / math.sqrt(k)
    if op == "blocks":
        s["a"], s["sa"] = _coded(gen, 1, rows, k, 1.0, True)
        s["b"], s["sb"] = _coded(gen, g, n, k, std, False)
        s["bias"] = _normal(gen, (g, n), 0.1, TORCH[case["out"]]) if case["bias"] else None
        return s
    t = case["type"]
    if op == "grad":
        s["dy"] = _normal(gen, (rows, k), 1.0, TORCH[t])
        s["w"] = _normal(gen, (g, n, k) if case["w"] == "nk" else (g, k, n), std, TORCH[t])
        s["z"] = _normal(gen, (rows, 2 * n), 1.0, TORCH[t])  # gate and up side by side, as the forward pass kept them
        return s
    if t == "e4m3":
        s["x"], s["sx"] = _coded(gen, 1, rows, k, 1.0, True)
        s["wg"], s["sg"] = _coded(gen, g, n, k, std, False)
        s["wu"], s["su"] = _coded(gen, g, n, k, std, False)
    else:
        s["x"] = _normal(gen, (rows, k), 1.0, TORCH[t])
        # one buffer of both matrices: [2 N, K], or [K, 2 N]
        s["w"] = _normal(gen, (g, 2 * n, k) if case["w"] == "nk" else (g, k, 2 * n), std, TORCH[t])
    s["bg"] = _normal(gen, (g, n), 0.1, TORCH[case["out"]]) if case["bias"] else None
    s["bu"] = _normal(gen, (g, n), 0.1, TORCH[case["out"]]) if case["bias"] else None
    return s


# ------------------------------------------------------------- the plain form

def _act(y, act):
    if act == "relu":
        return torch.clamp(y, min=0)
    if act == "gelu":
        return 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    if act == "silu":
        return y / (1 + torch.exp(-y))
    return y


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    p = 1 / (1 + torch.exp(-z))
    return p + z * p * (1 - p)


def _values(codes, scales, rows, cols):
    """fp32 values of [mats, rows, >= cols] codes with a scale for each 128 x 128 block."""
    x = codes[:, :, :cols].float()
    s = scales.repeat_interleave(128, dim=1)[:, :rows].repeat_interleave(128, dim=2)[:, :, :cols]
    return x * s


def _tokens(codes, scales, cols):
    return codes[:, :cols].float() * scales.t().repeat_interleave(128, dim=1)[:, :cols]


def _product(s, x, w):
    """Rows of x (fp32) times their expert's [K, N] matrix (fp32)."""
    if w.shape[0] == 1:
        return x @ w[0]
    padded = torch.zeros(w.shape[0], s["most"], x.shape[1], device=x.device)
    padded[s["expert"], s["place"]] = x
    return torch.bmm(padded, w)[s["expert"], s["place"]]


def _round_e4m3(x):
    """x (64 bits, at most 448) to the nearest e4m3 value, ties to even."""
    _, e = torch.frexp(x)
    step = ((e.clamp(min=-5) + 1019).to(torch.int64) << 52).view(torch.float64)  # 2 ** (e - 4)
    return (torch.round(x / step) * step).to(torch.float32).to(torch.float8_e4m3fn)


def _plain(s):
    case = s["case"]
    op, k = case["op"], case["k"]
    if op == "quant":
        m, r, kb = case["m"], case["rows"], _up(k, 128) // 128
        full = torch.nn.functional.pad(s["x"], (0, kb * 128 - k, 0, _up(m, r) - m)).view(_up(m, r) // r, r, kb, 128).float()
        scale = full.abs().amax(dim=(1, 3)) / 448
        q = full.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None, :, None]
        q = _round_e4m3(q.clamp(-448, 448)).view(-1, kb * 128)[:m, :k]
        return [q, scale.t().contiguous() if r == 1 else scale]
    if op == "blocks":
        y = _product(s, _tokens(s["a"], s["sa"], k), _values(s["b"], s["sb"], case["n"], k).transpose(1, 2).contiguous())
        if s["bias"] is not None:
            y = y + s["bias"].float()[s["expert"]]
        return [_act(y, case["act"]).to(TORCH[case["out"]])]
    n, t = case["n"], case["type"]
    if op == "grad":
        w = s["w"].float()
        dh = _product(s, s["dy"].float(), w.transpose(1, 2).contiguous() if case["w"] == "nk" else w)
        gate, up = s["z"][:, :n].float(), s["z"][:, n:].float()
        hidden = _act(gate, case["act"])
        dz = torch.cat([dh * up * _act_grad(gate, case["act"]), dh * hidden], dim=1).to(TORCH[t])
        return [dz, (hidden * up).to(TORCH[t])] if case["hidden"] else [dz]
    if t == "e4m3":
        x = _tokens(s["x"], s["sx"], k)
        wg, wu = (_values(s[w], s[q], n, k).transpose(1, 2).contiguous() for w, q in (("wg", "sg"), ("wu", "su")))
    else:
        x, w = s["x"].float(), s["w"].float()
        wg, wu = ((w[:, :n].transpose(1, 2).contiguous(), w[:, n:].transpose(1, 2).contiguous()) if case["w"] == "nk"
                  else (w[:, :, :n].contiguous(), w[:, :, n:].contiguous()))
    gate, up = _product(s, x, wg), _product(s, x, wu)
    if s["bg"] is not None:
        gate, up = gate + s["bg"].float()[s["expert"]], up + s["bu"].float()[s["expert"]]
    out = TORCH[case["out"]]
    h = (_act(gate, case["act"]) * up).to(out)
    return [h, torch.cat([gate, up], dim=1).to(out)] if case["keep"] else [h]


# -------------------------------------------------------------- the library's

def _own(s):
    tla = _lib()
    code = {"f16": tla.F16, "bf16": tla.BF16, "f32": tla.F32, "e4m3": tla.E4M3}
    acts = {"none": tla.ACT_NONE, "relu": tla.ACT_RELU, "gelu": tla.ACT_GELU, "silu": tla.ACT_SILU}
    case = s["case"]
    op, k = case["op"], case["k"]
    if op == "quant":
        m, r, kb = case["m"], case["rows"], _up(k, 128) // 128
        q = torch.empty(m, _up(k, 16), dtype=torch.float8_e4m3fn, device=DEV)
        if r == 1:
            scale = torch.empty(kb, m, device=DEV)
            tla.quantize_blocks(m, k, s["x"], code[case["x"]], k, 1, q, q.shape[1], scale, tla.COL_MAJOR, m)
        else:
            scale = torch.empty(_up(m, 128) // 128, kb, device=DEV)
            tla.quantize_blocks(m, k, s["x"], code[case["x"]], k, 128, q, q.shape[1], scale, tla.ROW_MAJOR, kb)
        return [q[:, :k], scale]
    g, n = case["g"], case["n"]
    if op == "blocks":
        m, kp, nb, kb = case["m"], s["a"].shape[1], _up(n, 128) // 128, _up(k, 128) // 128
        d = torch.empty(m, n, dtype=TORCH[case["out"]], device=DEV)
        tla.gemm_blocks(g, m, n, k, s["offsets"], s["a"], kp, s["sa"], tla.COL_MAJOR, m, s["b"], kp, n * kp,
                        s["sb"], tla.ROW_MAJOR, kb, nb * kb, d, code[case["out"]], n, bias=s["bias"], act=acts[case["act"]])
        return [d]
    rows, t = case["rows"], case["type"]
    if op == "grad":
        dz = torch.empty(rows, 2 * n, dtype=TORCH[t], device=DEV)
        h = torch.empty(rows, n, dtype=TORCH[t], device=DEV) if case["hidden"] else None
        nk = case["w"] == "nk"
        tla.gated_gemm_grad(g, rows, n, k, s["offsets"], s["dy"], code[t], k, s["w"], tla.COL_MAJOR if nk else tla.ROW_MAJOR,
                            k if nk else n, n * k, s["z"], s["z"][:, n:], 2 * n, dz, dz[:, n:], code[t], 2 * n, H=h, ldh=n,
                            act=acts[case["act"]])
        return [dz, h] if case["hidden"] else [dz]
    h = torch.empty(rows, n, dtype=TORCH[case["out"]], device=DEV)
    z = torch.empty(rows, 2 * n, dtype=h.dtype, device=DEV) if case["keep"] else None
    more = dict(b_gate=s["bg"], b_up=s["bu"], act=acts[case["act"]])
    if z is not None:
        more.update(Z_gate=z, Z_up=z[:, n:], ldz=2 * n)
    if t == "e4m3":
        kp, nb, kb = s["x"].shape[1], _up(n, 128) // 128, _up(k, 128) // 128
        tla.gated_gemm(g, rows, n, k, s["offsets"], s["x"], tla.E4M3, kp, s["wg"], s["wu"], tla.COL_MAJOR, kp, n * kp,
                       h, code[case["out"]], n, scale_x=s["sx"], sx_order=tla.COL_MAJOR, ldsx=rows, scale_gate=s["sg"],
                       scale_up=s["su"], sw_order=tla.ROW_MAJOR, ldsw=kb, stride_sw=nb * kb, **more)
    else:
        nk = case["w"] == "nk"
        wu = s["w"][:, n:] if nk else s["w"][:, :, n:]
        tla.gated_gemm(g, rows, n, k, s["offsets"], s["x"], code[t], k, s["w"], wu, tla.COL_MAJOR if nk else tla.ROW_MAJOR,
                       k if nk else 2 * n, 2 * n * k, h, code[case["out"]], n, **more)
    return [h, z] if case["keep"] else [h]


def run(state):
    return _own(state) if own else _plain(state)


# ----------------------------------------------------------------------- work

def work(case):
    """Bytes: each input read once, each output written once (the matrices of experts that can have rows); flops: two a product."""
    op, k = case["op"], case["k"]
    if op == "quant":
        e = case["m"] * k
        return {"bytes": e * (SIZE[case["x"]] + 1) + 4 * _up(e, 128 * case["rows"]) // (128 * case["rows"]), "flops": 3 * e}
    n, g = case["n"], case["g"]
    rows = case["m"] if op == "blocks" else case["rows"]
    # experts with at least one row, expected for rows drawn at random
    live = g - min(case["empty"], g - 1)
    live = max(1, round(live * (1 - (1 - 1 / live) ** rows)))
    t = 1 if op == "blocks" else SIZE[case["type"]]
    kb, nb = _up(k, 128) // 128, _up(n, 128) // 128
    mats = 2 if op == "gated" else 1
    size = rows * k * t + mats * live * n * k * t
    if t == 1:
        size += 4 * (rows * kb + mats * live * nb * kb)
    if op == "grad":
        size += rows * n * t * (4 + (1 if case["hidden"] else 0))
    else:
        size += rows * n * SIZE[case["out"]] * (3 if op == "gated" and case["keep"] else 1)
        size += mats * live * n * SIZE[case["out"]] if case["bias"] else 0
    return {"bytes": size, "flops": 2 * mats * rows * n * k}


# ---------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators' definitions in 64 bits, one expert (quantizer: one block of columns) after another."""
    s = prepare(case, seed)
    op, k = case["op"], case["k"]

    def f(v):
        if case["act"] == "gelu":
            return v * 0.5 * torch.special.erfc(-v / math.sqrt(2.0))
        if case["act"] == "silu":
            return v * torch.sigmoid(v)
        return v.clamp(min=0) if case["act"] == "relu" else v

    def slope(v):
        if case["act"] == "gelu":
            return 0.5 * torch.special.erfc(-v / math.sqrt(2.0)) + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        if case["act"] == "silu":
            return torch.sigmoid(v) * (1 + v * torch.sigmoid(-v))
        return (v > 0).double()

    if op == "quant":
        x, r = s["x"].double(), case["rows"]
        top, parts = [], []
        for c in range(0, k, 128):
            part = x[:, c:c + 128]
            a = part.abs().amax(dim=1)
            if r > 1:
                a = torch.nn.functional.pad(a, (0, _up(a.numel(), r) - a.numel())).view(-1, r).amax(dim=1)
            top.append(a / 448)
            by = (a / 448).repeat_interleave(r)[:x.shape[0]]
            parts.append(part / torch.where(by > 0, by, torch.ones_like(by)).unsqueeze(1))
        return [torch.cat(parts, dim=1), torch.stack(top, dim=0 if r == 1 else 1)]

    def row_values(q, sc):
        by = sc.double().t()
        return torch.cat([q[:, c:min(c + 128, k)].double() * by[:, c // 128:c // 128 + 1] for c in range(0, k, 128)], dim=1)

    def matrix(q, sc):
        by = sc.double().repeat_interleave(128, dim=0)[:q.shape[0]]
        return torch.cat([q[:, c:min(c + 128, k)].double() * by[:, c // 128:c // 128 + 1] for c in range(0, k, 128)], dim=1).t()

    rows, n, g = case["m"] if op == "blocks" else case["rows"], case["n"], case["g"]
    off = [0, rows] if s["offsets"] is None else s["offsets"].tolist()
    spans = [(e, off[e], off[e + 1]) for e in range(g) if off[e + 1] > off[e]]

    def by_expert(x, pick, bias=None):
        y = torch.empty(rows, n, dtype=torch.float64, device=DEV)
        for e, lo, hi in spans:
            y[lo:hi] = torch.mm(x[lo:hi], pick(e))
            if bias is not None:
                y[lo:hi] += bias[e].double()
        return y

    if op == "blocks":
        return [f(by_expert(row_values(s["a"], s["sa"]), lambda e: matrix(s["b"][e], s["sb"][e]), s["bias"]))]
    if op == "grad":
        dh = by_expert(s["dy"].double(), lambda e: s["w"][e].double().t() if case["w"] == "nk" else s["w"][e].double())
        gate, up = s["z"].double().split(n, dim=1)
        dz = torch.empty(rows, 2 * n, dtype=torch.float64, device=DEV)
        dz[:, :n] = dh * (up * slope(gate))
        dz[:, n:] = dh * f(gate)
        return [dz, up * f(gate)] if case["hidden"] else [dz]
    if case["type"] == "e4m3":
        x = row_values(s["x"], s["sx"])
        gate = by_expert(x, lambda e: matrix(s["wg"][e], s["sg"][e]), s["bg"])
        up = by_expert(x, lambda e: matrix(s["wu"][e], s["su"][e]), s["bu"])
    else:
        x = s["x"].double()
        half = lambda e, lo: (s["w"][e, lo:lo + n].double().t() if case["w"] == "nk" else s["w"][e, :, lo:lo + n].double())  # noqa: E731
        gate = by_expert(x, lambda e: half(e, 0), s["bg"])
        up = by_expert(x, lambda e: half(e, n), s["bu"])
    z = torch.cat([gate, up], dim=1) if case["keep"] else None
    return [f(gate) * up, z] if case["keep"] else [f(gate) * up]
