"""What a training or serving program asks of the operators for quantised layers.

Five operators: the AdamW step over many tensors, the 4-bit group quantiser, the product with 4-bit
weights, the packing of decoded trellis states, and the product with packed trellis weights.  `run`
computes each in plain torch operations, or (`own`) through the package.  A case is a dict of plain
values; `prepare` makes its inputs on the GPU from the seed alone.
"""
import math

import torch

own = False

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256  # elements of one block of 8-bit optimiser state
M32 = 0xFFFFFFFF
TINY = 2.0 ** -100  # a block whose largest value is under this holds zeros


def listed():
    return [
        # the preimage of a 2048 x 8192 projection and its 16-bit codebook, as QAT trains them
        {"name": "adamw projection f32", "op": "adamw", "sizes": "projection", "p": "f32", "g": "f32", "bits": 32, "wd": 0.0, "clip": False},
        # two decoder layers of width 2048, bf16 weights, 8-bit states
        {"name": "adamw two layers bf16 8-bit", "op": "adamw", "sizes": "layers", "count": 2, "p": "bf16", "g": "bf16", "bits": 8, "wd": 0.1, "clip": True},
        # many small tensors of odd sizes (norms, biases, codebooks of many layers)
        {"name": "adamw 96 odd tensors 8-bit", "op": "adamw", "sizes": "odd", "count": 96, "top": 20011, "p": "f32", "g": "bf16", "bits": 8, "wd": 0.01, "clip": False},
        # the projection, quantised with symmetric groups
        {"name": "quantize projection f32", "op": "quantize", "rows": 2048, "cols": 8192, "group": 128, "zero": False, "w": "f32", "scale": "f32"},
        # a small layer of odd sizes with zero points
        {"name": "quantize odd bf16 zero", "op": "quantize", "rows": 1001, "cols": 1100, "group": 32, "zero": True, "w": "bf16", "scale": "bf16"},
        # decoding one token through a square layer
        {"name": "int4 1 token bf16", "op": "int4", "tokens": 1, "rows": 8192, "cols": 8192, "group": 128, "zero": False, "x": "bf16", "scale": "bf16"},
        # reconstruction inputs in float32, an odd layer
        {"name": "int4 3 tokens f32 odd", "op": "int4", "tokens": 3, "rows": 1001, "cols": 1100, "group": 64, "zero": True, "x": "f32", "scale": "f32"},
        # a batch of sequences decoding through a wide layer
        {"name": "int4 16 tokens f16 wide", "op": "int4", "tokens": 16, "rows": 16384, "cols": 8192, "group": 32, "zero": True, "x": "f16", "scale": "f16"},
        # the hard-decoded projection, packed for serving
        {"name": "pack projection L16 k2", "op": "pack", "nseq": 65536, "len": 256, "L": 16, "k": 2},
        # a short odd layer
        {"name": "pack odd L11 k3", "op": "pack", "nseq": 999, "len": 77, "L": 11, "k": 3},
        # one token through the packed projection, the codebook as it was trained
        {"name": "trellis 1 token L16 k2", "op": "trellis", "tokens": 1, "rows": 2048, "per_row": 32, "len": 256, "L": 16, "k": 2, "x": "bf16", "c": "f32", "group": 0},
        # eight sequences decoding, a codebook kept in 16 bits, group scales
        {"name": "trellis 8 tokens L16 k4", "op": "trellis", "tokens": 8, "rows": 8192, "per_row": 8, "len": 256, "L": 16, "k": 4, "x": "bf16", "c": "bf16", "group": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "quantize", "int4", "int4", "int4", "pack", "trellis", "trellis", "trellis"])
    t = ["f32", "f16", "bf16"]
    if op == "adamw":
        count = _log(rng, 1, 120)
        p = rng.choice(t)
        return {"op": op, "sizes": "odd", "count": count, "top": _log(rng, 300, 20_000_000 // count), "p": p, "g": rng.choice([p, "f32"]),
                "bits": rng.choice([8, 32]), "wd": rng.choice([0.0, 0.01, 0.1]), "clip": rng.random() < 0.5}
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 4096), "cols": _log(rng, 32, 8192), "group": rng.choice([0, 32, 64, 128, 256]),
                "zero": rng.random() < 0.5, "w": rng.choice(t), "scale": rng.choice(["f32", "bf16"])}
    if op == "int4":
        return {"op": op, "tokens": _log(rng, 1, 33), "rows": _log(rng, 16, 8192), "cols": _log(rng, 32, 8192), "group": rng.choice([0, 32, 64, 128, 256]),
                "zero": rng.random() < 0.5, "x": rng.choice(t), "scale": rng.choice(t)}
    k = rng.randint(1, 4)
    L = rng.randint(max(4, 2 * k), 16)
    n = _log(rng, 16, 512)
    if op == "pack":
        return {"op": op, "nseq": _log(rng, 1, 16384), "len": n, "L": L, "k": k}
    per_row = max(1, _log(rng, 64, 8192) // n)
    return {"op": op, "tokens": _log(rng, 1, 12), "rows": _log(rng, 1, 4096), "per_row": per_row, "len": n, "L": L, "k": k, "x": rng.choice(t),
            "c": rng.choice(t), "group": rng.choice([0, n])}


# ---- sizes -----------------------------------------------------------------------------------------------------------

def _sizes(case):
    if case["sizes"] == "projection":
        return [2048 * 8192, 65536]
    if case["sizes"] == "layers":
        return ([2048 * 2048] * 4 + [2048 * 8192] * 3 + [2048] * 2) * case["count"]
    return [1 + (i * 7919 + 12345) * 104729 % case["top"] for i in range(case["count"])]


def _up(n, m):
    return -(-n // m) * m


def _group(case):
    return case["group"] or _up(case["cols"], 128)


def _words(case):
    return -(-(case["len"] * case["k"] + case["L"] - case["k"]) // 32)


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (2 * SIZE[case["p"]] + SIZE[case["g"]] + state), "flops": 14 * n}
    if op == "quantize":
        R, C = case["rows"], case["cols"]
        groups = R * -(-C // _group(case))
        return {"bytes": R * C * (SIZE[case["w"]] + 0.5) + groups * (SIZE[case["scale"]] + case["zero"]), "flops": 4 * R * C}
    if op == "int4":
        R, C, m = case["rows"], case["cols"], case["tokens"]
        groups = R * -(-C // _group(case))
        return {"bytes": R * C / 2 + groups * (SIZE[case["scale"]] + case["zero"]) + m * (R + C) * SIZE[case["x"]], "flops": 2 * m * R * C}
    if op == "pack":
        return {"bytes": case["nseq"] * (case["len"] + _words(case)) * 4, "flops": 4 * case["nseq"] * case["len"]}
    R, C, m = case["rows"], case["per_row"] * case["len"], case["tokens"]
    groups = R * (C // case["group"]) if case["group"] else 0
    return {"bytes": R * case["per_row"] * _words(case) * 4 + (SIZE[case["c"]] << case["L"]) + 4 * groups + m * (R + C) * SIZE[case["x"]], "flops": 2 * m * R * C}


# ---- inputs ----------------------------------------------------------------------------------------------------------

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _round_bits(t, rnd):
    """e4m3 codes (without sign) of t in [0, 448]: its bits cut after three of the mantissa, once `rnd` (20 bits) is added."""
    y = (t * 2.0 ** -120).view(torch.int32).long()
    return ((y + rnd) >> 20).clamp(max=0x7E)


def _encode(x, floor_one, rnd):
    """(codes as float8, scale of each block) of a flat x of whole blocks, signed or not."""
    top = x.abs().view(-1, BLOCK).amax(1)
    held = ~(top < TINY)
    inv = torch.where(held, 448.0 / top, torch.zeros_like(top))
    code = _round_bits((x.abs().view(-1, BLOCK) * inv[:, None]).view(-1), rnd)
    if floor_one:
        code = torch.where((code == 0) & (x > 0) & held.repeat_interleave(BLOCK), torch.ones_like(code), code)
    else:
        code = code + (x < 0) * 128
    return code.to(torch.uint8).view(torch.float8_e4m3fn), torch.where(held, top / 448.0, torch.zeros_like(top))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op == "adamw":
        sizes = _sizes(case)
        at = [0]
        for n in sizes:
            at.append(at[-1] + _up(n, BLOCK))
        used = torch.zeros(at[-1], device="cuda")
        for n, a in zip(sizes, at):
            used[a:a + n] = 1.0
        # weights of a layer, gradients over several orders of magnitude, states in the middle of training
        p = (_normal(gen, at[-1]) * 0.02 * used).to(DT[case["p"]])
        spread = torch.exp(_normal(gen, at[-1]))
        g = (_normal(gen, at[-1]) * 1e-3 * spread * used).to(DT[case["g"]])
        m = _normal(gen, at[-1]) * 3e-4 * spread * used
        r = _normal(gen, at[-1]).abs() * 1e-3 * spread * used
        s = {"p": p, "g": g, "params": [p[a:a + n] for n, a in zip(sizes, at)], "grads": [g[a:a + n] for n, a in zip(sizes, at)], "step": 100,
             "clip": torch.full((), 0.5, device="cuda") if case["clip"] else None, "scales": None}
        if case["bits"] == 32:
            s["first"], s["second"] = m, r * r
        else:
            s["first"], a = _encode(m, False, 0x80000)
            s["second"], b = _encode(r, True, 0x80000)
            s["scales"] = torch.stack([a, b])
    elif op == "quantize":
        w = _normal(gen, case["rows"], case["cols"]) * 0.02
        s = {"w": w.to(DT[case["w"]])}
    elif op == "int4":
        R, C = case["rows"], case["cols"]
        groups = -(-C // _group(case))
        # any bytes are weights; scales as the quantiser gives for weights of 0.02
        s = {"x": _normal(gen, case["tokens"], C).to(DT[case["x"]]),
             "packed": torch.randint(0, 256, (_up(R, 16) // 16, _up(C, 128) // 128, 1024), generator=gen, device="cuda", dtype=torch.uint8),
             "scales": (0.004 + 0.01 * torch.rand(groups, R, generator=gen, device="cuda")).to(DT[case["scale"]]),
             "zeros": torch.randint(0, 16, (groups, R), generator=gen, device="cuda", dtype=torch.uint8) if case["zero"] else None}
    else:
        # any bits are a path through the trellis; those behind a sequence's end are zero
        N = case["nseq"] if op == "pack" else case["rows"] * case["per_row"]
        words = _words(case)
        packed = torch.randint(-2 ** 31, 2 ** 31, (N, words), generator=gen, device="cuda", dtype=torch.int64)
        behind = words * 32 - (case["len"] * case["k"] + case["L"] - case["k"])
        packed[:, -1] = (packed[:, -1] >> behind) << behind
        packed = packed.to(torch.int32)
        if op == "pack":
            s = {"states": _windows(packed, case["len"], case["L"], case["k"]).to(torch.int32)}
        else:
            C = case["per_row"] * case["len"]
            s = {"packed": packed, "x": _normal(gen, case["tokens"], C).to(DT[case["x"]]), "codebook": _normal(gen, 1 << case["L"]).to(DT[case["c"]]),
                 "scales": 0.01 + 0.02 * torch.rand(C // case["group"], case["rows"], generator=gen, device="cuda") if case["group"] else None}
    s["case"] = case
    return s


# ---- the plain forms -------------------------------------------------------------------------------------------------

def _windows(packed, n, L, k):
    """The state of every step: bits [t k, t k + L) of each sequence's stream, the first bit the highest of its word."""
    at = torch.arange(n, device=packed.device) * k
    w = packed.long() & M32
    j = at // 32
    pair = (w[:, j] << 32) | w[:, (j + 1).clamp(max=w.shape[1] - 1)]
    return (pair >> (64 - at % 32 - L)) & ((1 << L) - 1)


def _adamw(s):
    case = s["case"]
    lr, b1, b2, eps, wd, t = 1e-3, 0.9, 0.99, 1e-8, case["wd"], s["step"]
    g = s["g"].float()
    if s["clip"] is not None:
        g = g * s["clip"]
    if case["bits"] == 32:
        m, v = s["first"], s["second"]
    else:
        a, b = s["scales"][0].repeat_interleave(BLOCK), s["scales"][1].repeat_interleave(BLOCK)
        m, r = s["first"].float() * a, s["second"].float() * b
        v = r * r
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    r = torch.sqrt(v)
    p = s["p"].float() * (1 - lr * wd) - (m / (r * (1 / math.sqrt(1 - b2 ** t)) + eps)) * (lr / (1 - b1 ** t))
    s["p"].copy_(p)
    if case["bits"] == 32:
        s["first"].copy_(m)
        s["second"].copy_(v)
    else:
        # 16 random bits for each of the two roundings: a hash of the element's place, the step and the seed
        h = (torch.arange(m.numel(), device="cuda") * 0x9E3779B1 + (t * 0x632BE5AB + 1 * 0x85157AF5)) & M32
        h = ((h ^ (h >> 15)) * 0x2C1B3C6D) & M32
        h = ((h ^ (h >> 12)) * 0x297A2D39) & M32
        h = h ^ (h >> 15)
        m8, a = _encode(m, False, ((h >> 16) << 4) | 8)
        r8, b = _encode(r, True, ((h & 0xFFFF) << 4) | 8)
        s["first"].copy_(m8)
        s["second"].copy_(r8)
        s["scales"].copy_(torch.stack([a, b]))


def _quantize(s):
    case = s["case"]
    R, C, G = case["rows"], case["cols"], _group(case)
    groups, blocks, tiles = -(-C // G), _up(C, 128) // 128, _up(R, 16) // 16
    w = torch.zeros(R, groups * G, device="cuda")
    w[:, :C] = s["w"]
    w = w.view(R, groups, G)
    if case["zero"]:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).to(DT[case["scale"]])
    else:
        scale = (w.abs().amax(2) / 7).to(DT[case["scale"]])
    held = scale > 0
    inv = torch.where(held, 1.0 / scale.float(), torch.zeros(1, device="cuda"))
    zero = torch.round(-lo * inv).clamp(0, 15) if case["zero"] else torch.full_like(inv, 8)
    q = (torch.round(w * inv[:, :, None]) + zero[:, :, None]).clamp(0, 15)
    full = torch.full((tiles * 16, blocks * 128), 8, device="cuda", dtype=torch.uint8)
    full[:R, :C] = q.view(R, -1)[:, :C].to(torch.uint8)
    # [tile, half, row, block, 32-column part, lane, pair, odd] -> [tile, block, half, row, lane, part, odd, pair]
    nib = full.view(tiles, 2, 8, blocks, 4, 4, 4, 2).permute(0, 3, 1, 2, 5, 4, 7, 6).reshape(tiles, blocks, 1024, 2)
    packed = nib[..., 0] | (nib[..., 1] << 4)
    return packed, scale.t().contiguous(), zero.t().contiguous().to(torch.uint8) if case["zero"] else None


def _int4(s):
    case = s["case"]
    R, C, G = case["rows"], case["cols"], _group(case)
    tiles, blocks, groups = _up(R, 16) // 16, _up(C, 128) // 128, -(-C // G)
    b = s["packed"]
    nib = torch.stack([b & 15, b >> 4], -1).view(tiles, blocks, 2, 8, 4, 4, 2, 4).permute(0, 2, 3, 1, 5, 4, 7, 6).reshape(tiles * 16, blocks * 128)
    part = torch.arange(C, device="cuda") // G
    zero = s["zeros"].float().t()[:, part] if s["zeros"] is not None else 8.0
    w = (nib[:R, :C].float() - zero) * s["scales"].float().t()[:, part]
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def _pack(s):
    case = s["case"]
    L, k, n = case["L"], case["k"], case["len"]
    st = s["states"].long()
    fresh = (st[:, 1:, None] >> torch.arange(k - 1, -1, -1, device="cuda")) & 1
    first = (st[:, :1] >> torch.arange(L - 1, -1, -1, device="cuda")) & 1
    words = _words(case)
    bits = torch.zeros(st.shape[0], words * 32, device="cuda", dtype=torch.int64)
    bits[:, :L] = first
    bits[:, L:L + (n - 1) * k] = fresh.reshape(st.shape[0], -1)
    return (bits.view(-1, words, 32) << torch.arange(31, -1, -1, device="cuda")).sum(2).to(torch.int32)


def _trellis(s):
    case = s["case"]
    R, C = case["rows"], case["per_row"] * case["len"]
    w = s["codebook"].float()[_windows(s["packed"], case["len"], case["L"], case["k"]).view(R, C)]
    if s["scales"] is not None:
        w = w * s["scales"].t().repeat_interleave(case["group"], 1)
    return (s["x"].float() @ w.t()).to(s["x"].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import differentiable_bcjr_b200 as B
    if op == "adamw":
        s["step"] += 1
        if own:
            B.adamw_step(s["params"], s["grads"], s["first"], s["second"], s["step"], lr=1e-3, betas=(0.9, 0.99), eps=1e-8, weight_decay=case["wd"],
                         scales=s["scales"], grad_scale=s["clip"], seed=1)
        else:
            _adamw(s)
        return {"p": s["p"], "first": s["first"], "second": s["second"], "scales": s["scales"]}
    if op == "quantize":
        return B.int4_quantize(s["w"], group_size=case["group"], zero_point=case["zero"], scale_dtype=DT[case["scale"]]) if own else _quantize(s)
    if op == "int4":
        return B.int4_matmul(s["x"], s["packed"], s["scales"], s["zeros"], group_size=case["group"]) if own else _int4(s)
    if op == "pack":
        return B.trellis_pack(s["states"], case["L"], case["k"]) if own else _pack(s)
    if own:
        return B.trellis_matmul(s["x"], s["packed"], s["codebook"], case["L"], case["k"], case["len"], scales=s["scales"], group_size=case["group"])
    return _trellis(s)


# ---- in 64 bits ------------------------------------------------------------------------------------------------------

def exact(case, seed):
    """The outputs from the definitions in 64 bits.  Codes (whole numbers, or rounded to 8 bits by chance) have no such value."""
    op = case["op"]
    if op == "pack":
        return None
    s = prepare(case, seed)
    d = torch.float64
    if op == "adamw":
        t = s["step"] + 1
        first, second = s["first"].to(torch.float32).to(d), s["second"].to(torch.float32).to(d)
        if case["bits"] == 8:
            first = (first.view(-1, BLOCK) * s["scales"][0].to(d).unsqueeze(1)).flatten()
            second = (second.view(-1, BLOCK) * s["scales"][1].to(d).unsqueeze(1)).flatten().square()
        grad = s["g"].to(d) * (0.5 if case["clip"] else 1.0)
        first += (grad - first) * 0.1
        second += (grad.square() - second) * 0.01
        step = first / (1 - 0.9 ** t) / ((second / (1 - 0.99 ** t)).sqrt() + 1e-8)
        weights = s["p"].to(d)
        weights = weights - 1e-3 * (step + case["wd"] * weights)
        scales = None
        if case["bits"] == 8:
            scales = torch.stack([x.view(-1, BLOCK).abs().max(1).values / 448 for x in (first, second.sqrt())])
        return {"p": weights, "first": first if case["bits"] == 32 else None, "second": second if case["bits"] == 32 else None, "scales": scales}
    if op == "quantize":
        R, C, G = case["rows"], case["cols"], _group(case)
        w, out = s["w"].to(d), []
        for c in range(0, C, G):
            part = w[:, c:c + G]
            if case["zero"]:
                out.append((part.max(1).values.clamp(min=0) - part.min(1).values.clamp(max=0)) / 15)
            else:
                out.append(torch.maximum(part.max(1).values, -part.min(1).values) / 7)
        return None, torch.stack(out), None
    if op == "int4":
        R, C, G = case["rows"], case["cols"], _group(case)
        y = torch.zeros(case["tokens"], R, dtype=d, device="cuda")
        r = torch.arange(R, device="cuda")
        flat = s["packed"].view(-1, 1024)
        for c0 in range(0, C, 128):
            c = torch.arange(c0, min(c0 + 128, C), device="cuda")
            i = c % 128
            # the byte and the half of it that hold row r, column c
            o = i % 8
            nibble = o // 2 + 4 * (o % 2)
            byte = (r // 8 % 2 * 512 + r % 8 * 64)[:, None] + (i % 32 // 8 * 16 + i // 32 * 4 + nibble // 2)[None]
            tile = (r // 16 * (_up(C, 128) // 128) + c0 // 128)[:, None]
            code = (flat[tile, byte].long() >> (4 * (nibble % 2))[None]) & 15
            g = c // G
            zero = s["zeros"][g].long().t() if s["zeros"] is not None else 8
            y += s["x"][:, c].to(d) @ ((code - zero).to(d) * s["scales"][g].to(d).t()).t()
        return y
    L, k, n, R, N = case["L"], case["k"], case["len"], case["rows"], case["rows"] * case["per_row"]
    word = s["packed"].long() & M32
    state = torch.zeros(N, dtype=torch.int64, device="cuda")
    values = torch.empty(N, n, dtype=d, device="cuda")
    table, bit = s["codebook"].to(d), 0
    for t in range(n):
        for _ in range(k if t else L):
            state = (state * 2 + ((word[:, bit // 32] >> (31 - bit % 32)) & 1)) % (1 << L)
            bit += 1
        values[:, t] = table[state]
    values = values.view(R, -1)
    if s["scales"] is not None:
        values = (values.view(R, -1, case["group"]) * s["scales"].to(d).t()[:, :, None]).reshape(R, -1)
    return s["x"].to(d) @ values.t()
