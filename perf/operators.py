"""Cases that measure the operators of a mixture of experts in 8- and 4-bit formats.

  quantize   bf16 -> E4M3 codes with one FP32 scale for each block of 128: a scale per 1 x 128 (activations) or per
             128 x 128 (weights)
  gemm       the product of two such matrices, bf16 out
  grouped    the experts' products: rows grouped by expert, ragged groups, one weight matrix each; optional GELU
  dispatch   expert ids -> group offsets and slots, then the tokens' rows gathered by expert and quantized
  combine    each token's weighted sum over the experts' output rows

``run`` computes them in plain torch operations, or with the framework's own calls where ``own`` is true.
"""
import math

import torch

own = False

BLOCK = 128          # K elements per scale of the block formats
E4M3_MAX = 448.0


def listed():
    return [
        # one decoding step of 16 sequences: the activation of a Linear layer, where launch latency counts
        {"name": "quantize rows 16x8192", "op": "quantize", "rows": 16, "cols": 8192, "tile": 1},
        # a large weight matrix quantized at load time, its rows not a multiple of the block
        {"name": "quantize tiles 28600x8192", "op": "quantize", "rows": 28600, "cols": 8192, "tile": 128},
        # decode: the weight stream of the skinny Linear layer of this repository's benchmark
        {"name": "gemm 16x28672x8192", "op": "gemm", "m": 16, "n": 28672, "k": 8192},
        # odd sizes: a short ragged batch, an output width that no vector divides
        {"name": "gemm 1000x2179x1152", "op": "gemm", "m": 1000, "n": 2179, "k": 1152},
        # prefill or a training batch: bound by the tensor cores
        {"name": "gemm 8192x8192x8192", "op": "gemm", "m": 8192, "n": 8192, "k": 8192},
        # decode of 64 tokens with 8 choices each among 64 experts: the weight stream of nearly all experts
        {"name": "grouped decode fp8 64x512", "op": "grouped", "fmt": "fp8_b128", "experts": 64, "rows": 512, "n": 4096,
         "k": 2048, "skew": 1.0, "gelu": False},
        # prefill: unequal groups, the first product of an experts' MLP with its activation
        {"name": "grouped prefill fp8 16x16384", "op": "grouped", "fmt": "fp8_b128", "experts": 16, "rows": 16384,
         "n": 4096, "k": 4096, "skew": 1.0, "gelu": True},
        # a mid-sized batch in the 4-bit format of this framework, some experts without a row
        {"name": "grouped batch nvfp4 32x4000", "op": "grouped", "fmt": "nvfp4", "experts": 32, "rows": 4000, "n": 4096,
         "k": 4096, "skew": 8.0, "gelu": False},
        # decode: 32 tokens, 8 of 64 experts each
        {"name": "dispatch fp8 32x8", "op": "dispatch", "fmt": "fp8_b128", "tokens": 32, "choices": 8, "experts": 64,
         "cols": 4096, "pad": 0.0},
        # prefill, the batch padded at its end (ids of -1)
        {"name": "dispatch mxfp8 16384x4", "op": "dispatch", "fmt": "mxfp8", "tokens": 16384, "choices": 4,
         "experts": 128, "cols": 4096, "pad": 0.1},
        # decode: the same tokens' outputs put together
        {"name": "combine 32x8", "op": "combine", "tokens": 32, "choices": 8, "cols": 4096, "drop": 0.0},
        # prefill, some choices dropped
        {"name": "combine 16384x8", "op": "combine", "tokens": 16384, "choices": 8, "cols": 4096, "drop": 0.05},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("quantize", "gemm", "grouped", "grouped", "dispatch", "combine"))
    k = BLOCK * _log(rng, 1, 64)
    if op == "quantize":
        return {"op": op, "rows": _log(rng, 1, 28600), "cols": k, "tile": rng.choice((1, 128))}
    if op == "gemm":
        n = _log(rng, 1, 28672)
        return {"op": op, "m": _log(rng, 1, max(1, min(8192, 8192 ** 3 // (n * k)))), "n": n, "k": k}
    if op == "grouped":
        k = BLOCK * _log(rng, 1, 32)
        experts, n = _log(rng, 1, 128), _log(rng, 1, 4096)
        return {"op": op, "fmt": rng.choice(("fp8_b128", "fp8_b128", "mxfp8", "mxfp4", "nvfp4")),
                "experts": max(1, min(experts, 2 ** 29 // (n * k))), "rows": _log(rng, 1, 16384), "n": n, "k": k,
                "skew": rng.choice((0.0, 1.0, 3.0, 8.0)), "gelu": rng.random() < 0.5}
    if op == "dispatch":
        experts = _log(rng, 1, 256)
        return {"op": op, "fmt": rng.choice(("fp8_b128", "mxfp8")), "tokens": _log(rng, 1, 16384),
                "choices": rng.randint(1, min(4, experts)), "experts": experts, "cols": BLOCK * _log(rng, 1, 32),
                "pad": rng.choice((0.0, 0.1, 0.5))}
    return {"op": op, "tokens": _log(rng, 1, 16384), "choices": rng.randint(1, 8), "cols": _log(rng, 1, 4096),
            "drop": rng.choice((0.0, 0.05, 0.5))}


# ---------------------------------------------------------------- layouts
def _pitch(rows):
    """Row pitch of the 1 x 128 scales, which are stored K block by K block."""
    return -(-rows // 4) * 4


def _bands(rows, groups):
    """128-row bands that any split of the rows into the groups fits in."""
    return min(rows, (rows + 127 * groups) // 128)


def _swizzled(s, bands):
    """Scale bytes [bands * 128, C] -> 512-byte tiles of 128 rows x 4 columns."""
    c4 = -(-s.shape[1] // 4) * 4
    s = torch.nn.functional.pad(s, (0, c4 - s.shape[1], 0, bands * 128 - s.shape[0]))
    return s.view(bands, 4, 32, c4 // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _unswizzled(t, cols):
    c4 = -(-cols // 4)
    return t.view(-1, c4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, c4 * 4)[:, :cols]


def _counts(case):
    """Rows of each expert: shares that fall off exponentially with `skew`, in a scattered order."""
    e, t = case["experts"], case["rows"]
    share = [math.exp(-case["skew"] * i / e) for i in range(e)]
    edge, total, got = 0.0, sum(share), []
    for v in share:
        got.append(int(round((edge + v) / total * t)) - int(round(edge / total * t)))
        edge += v
    step = next(s for s in range(max(1, int(e * 0.618)), 2 * e + 2) if math.gcd(s, e) == 1)
    return [got[(i * step) % e] for i in range(e)]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, rows, cols):
    """N(0, 1) with a few outlier channels, as the inputs of Linear layers have."""
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float32)
    at = torch.randint(0, cols, (max(1, cols // 512),), generator=g, device="cuda")
    x[:, at] *= 20.0
    return x.bfloat16()


def _weights(g, rows, cols):
    return (torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float32) * 0.02).bfloat16()


E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _mx_operand(x, fmt):
    """(codes, scale bytes [rows, cols / block], g) of a bf16 matrix: operands for the products."""
    rows, cols = x.shape
    x = x.float()
    block = 16 if fmt == "nvfp4" else 32
    top = E4M3_MAX if fmt == "mxfp8" else 6.0
    v = x.view(rows, cols // block, block)
    amax = v.abs().amax(2)
    g = None
    if fmt == "nvfp4":
        g = (x.abs().max() / 2688.0).clamp(min=1e-30)
        s = (amax / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn)
        sb, step = s.view(torch.uint8), s.float() * g
    else:
        e = torch.ceil(torch.log2((amax / top).clamp(min=1e-30))).clamp(-126, 126)
        sb, step = (e + 127).to(torch.uint8), torch.exp2(e)
    q = torch.where(step[..., None] > 0, v / step[..., None], torch.zeros_like(v)).clamp(-top, top).view(rows, cols)
    if fmt == "mxfp8":
        return q.to(torch.float8_e4m3fn).view(torch.uint8), sb, g
    mids = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=x.device)
    c = torch.bucketize(q.abs(), mids).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    return c[:, 0::2] | (c[:, 1::2] << 4), sb, g


def _e4m3(x, s):
    """E4M3 codes of the quotient x / s, saturating (the signed zero of x where s is 0).  In FP64: a quotient of a bf16
    value and an FP32 scale is often next to the middle of two codes, and an FP32 division would round it there."""
    q = torch.where(s > 0, x.double() / s.double(), x.double() * 0.0)
    step = torch.ldexp(torch.ones_like(q), torch.frexp(q)[1].clamp(min=-5) - 4)
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX).float().to(torch.float8_e4m3fn)


def _b128_rows(x):
    """E4M3 codes [rows, cols] and FP32 scales [cols / 128, pitch] of a bf16 matrix, one scale per 1 x 128."""
    rows, cols = x.shape
    v = x.float().view(rows, cols // BLOCK, BLOCK)
    s = v.abs().amax(2)
    s = s / torch.full_like(s, E4M3_MAX)
    scales = torch.zeros(cols // BLOCK, _pitch(rows), device=x.device)
    scales[:, :rows] = s.t()
    return _e4m3(v, s[..., None]).view(rows, cols), scales


def _b128_tiles(x):
    """The same with one scale per 128 x 128: scales [ceil(rows / 128), cols / 128]."""
    rows, cols = x.shape
    bands = -(-rows // BLOCK)
    v = torch.nn.functional.pad(x, (0, 0, 0, bands * BLOCK - rows)).view(bands, BLOCK, cols // BLOCK, BLOCK)
    s = v.abs().amax((1, 3)).float()
    s = s / torch.full_like(s, E4M3_MAX)
    return _e4m3(v, s[:, None, :, None]).view(bands * BLOCK, cols)[:rows], s


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op == "quantize":
        x = _activations if case["tile"] == 1 else _weights
        s["x"] = x(g, case["rows"], case["cols"])
    elif op == "gemm":
        a, sa = _b128_rows(_activations(g, case["m"], case["k"]))
        b, sb = _b128_tiles(_weights(g, case["n"], case["k"]))
        s.update(a=a.view(torch.uint8), sa=sa, b=b.view(torch.uint8), sb=sb)
    elif op == "grouped":
        counts = _counts(case)
        offsets = [0]
        for c in counts:
            offsets.append(offsets[-1] + c)
        rows, n, k, e = case["rows"], case["n"], case["k"], case["experts"]
        s.update(offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"), most=max(counts))
        x = _activations(g, rows, k)
        if case["fmt"] == "fp8_b128":
            a, sa = _b128_rows(x)
            s.update(a=a.view(torch.uint8), sa=sa)
            w = [_b128_tiles(_weights(g, n, k)) for _ in range(e)]
            s["b"] = torch.stack([c.view(torch.uint8) for c, _ in w])
            s["sb"] = torch.stack([torch.nn.functional.pad(v.view(-1), (0, -v.numel() % 4)) for _, v in w])
        else:
            codes, sb, ga = _mx_operand(x, case["fmt"])
            bands = _bands(rows, e)
            laid = torch.zeros(bands * 128, sb.shape[1], dtype=torch.uint8, device="cuda")
            band = 0
            for c, o in zip(counts, offsets):
                laid[band * 128:band * 128 + c] = sb[o:o + c]
                band += -(-c // 128)
            s.update(a=codes, sa=_swizzled(laid, bands))
            w = [_mx_operand(_weights(g, n, k), case["fmt"]) for _ in range(e)]
            s["b"] = torch.stack([c for c, _, _ in w])
            s["sb"] = torch.stack([_swizzled(v, -(-n // 128)) for _, v, _ in w])
            if ga is not None:
                s.update(ga=ga.view(1), gb=torch.stack([v for _, _, v in w]))
    elif op == "dispatch":
        t, c, e = case["tokens"], case["choices"], case["experts"]
        s["x"] = _activations(g, t, case["cols"])
        logits = torch.randn(t, e, generator=g, device="cuda") + torch.randn(e, generator=g, device="cuda")
        s["ids"] = torch.topk(logits, c, 1).indices.int()
        s["ids"][t - int(t * case["pad"]):] = -1
        block = BLOCK if case["fmt"] == "fp8_b128" else 32
        s["codes"] = torch.zeros(t * c, case["cols"], dtype=torch.uint8, device="cuda")
        if case["fmt"] == "fp8_b128":
            s["scales"] = torch.zeros(case["cols"] // block, _pitch(t * c), device="cuda")
        else:
            s["scales"] = torch.zeros(_bands(t * c, e) * 128 * (case["cols"] // block), dtype=torch.uint8, device="cuda")
    else:
        t, c = case["tokens"], case["choices"]
        s["y"] = _activations(g, t * c, case["cols"])
        slot = torch.randperm(t * c, generator=g, device="cuda").int().view(t, c)
        s["slot"] = torch.where(torch.rand(t, c, generator=g, device="cuda") < case["drop"], -1, slot)
        s["weights"] = torch.softmax(torch.randn(t, c, generator=g, device="cuda"), 1)
    return s


# ---------------------------------------------------------------- the framework's own calls
def _run_own(s):
    from fp8_quantization_block_b200 import mx
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        q = mx.quantize(s["x"], mx.MX_FP8_B128 if case["tile"] == 1 else mx.MX_FP8_B128X128)
        rows, cols = case["rows"], case["cols"]
        scales = q.scales.view(torch.float32)
        shape = (cols // BLOCK, _pitch(rows)) if case["tile"] == 1 else (-(-rows // BLOCK), cols // BLOCK)
        return [q.codes.view(torch.float8_e4m3fn).view(rows, cols), scales[:shape[0] * shape[1]].view(shape)]
    if op == "gemm":
        a = mx.MxTensor(mx.MX_FP8_B128, case["m"], case["k"], s["a"], s["sa"], None)
        return mx.gemm(a, mx.MxTensor(mx.MX_FP8_B128X128, case["n"], case["k"], s["b"], s["sb"], None))
    if op == "grouped":
        fa, fb = {"fp8_b128": (mx.MX_FP8_B128, mx.MX_FP8_B128X128), "mxfp8": (mx.MX_MXFP8_E4M3,) * 2,
                  "mxfp4": (mx.MX_MXFP4,) * 2, "nvfp4": (mx.MX_NVFP4,) * 2}[case["fmt"]]
        a = mx.MxTensor(fa, case["rows"], case["k"], s["a"], s["sa"], s.get("ga"))
        b = mx.MxTensor(fb, case["n"], case["k"], s["b"], s["sb"], s.get("gb"))
        return mx.gemm_grouped(a, b, s["offsets"], epilogue=mx.MX_EPI_GELU if case["gelu"] else mx.MX_EPI_NONE)
    if op == "dispatch":
        fmt = mx.MX_FP8_B128 if case["fmt"] == "fp8_b128" else mx.MX_MXFP8_E4M3
        r = mx.route(s["ids"], case["experts"])
        out = mx.MxTensor(fmt, case["tokens"] * case["choices"], case["cols"], s["codes"], s["scales"], None)
        mx.quantize_grouped(s["x"], r.offsets, fmt, row_index=r.row_token, out=out)
        return [r.offsets, r.row_token, r.slot, s["codes"].view(torch.float8_e4m3fn), s["scales"]]
    return mx.combine(s["y"], s["slot"], s["weights"])


# ---------------------------------------------------------------- plain forms
def _routed(ids, experts):
    """Offsets [experts + 1], the token of each slot (-1 behind the last), the slot of each choice (-1 where it has none)."""
    flat = ids.reshape(-1)
    hot = flat[:, None] == torch.arange(experts, device=ids.device, dtype=torch.int32)
    before = hot.cumsum(0, dtype=torch.int32)
    offsets = torch.nn.functional.pad(before[-1].cumsum(0, dtype=torch.int32), (1, 0))
    known = (flat >= 0) & (flat < experts)
    e = flat.clamp(0, experts - 1).long()
    slot = torch.where(known, offsets[e] + before.gather(1, e[:, None])[:, 0] - 1, -1)
    token = torch.full((flat.numel() + 1,), -1, dtype=torch.int32, device=ids.device)
    token[torch.where(known, slot, flat.numel()).long()] = (
        torch.arange(flat.numel(), device=ids.device, dtype=torch.int32) // ids.shape[1])
    return offsets, token[:-1], slot.view_as(ids)


def _group_of(offsets, rows):
    """Group of each row (the number of groups for rows behind the last) and the row's place in its group."""
    t = torch.arange(rows, device=offsets.device, dtype=torch.int32)
    group = (t[:, None] >= offsets[1:]).sum(1)
    return group, t - offsets[group.clamp(max=offsets.numel() - 2)]


def _band_rows(offsets, group, place):
    """Row of each grouped row in the scale buffer, whose groups each begin a 128-row band."""
    first = torch.nn.functional.pad(((offsets[1:] - offsets[:-1] + 127) // 128).cumsum(0), (1, 0))
    return first[group] * 128 + place


def _mx_values(codes, scales, fmt):
    """FP32 values of codes [..., bytes] and scale bytes [..., blocks]."""
    block = 16 if fmt == "nvfp4" else 32
    if fmt == "mxfp8":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
        q = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).flatten(-2)
    kind = torch.float8_e4m3fn if fmt == "nvfp4" else torch.float8_e8m0fnu
    return q * scales.contiguous().view(kind).float().repeat_interleave(block, -1)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return list(_b128_rows(s["x"]) if case["tile"] == 1 else _b128_tiles(s["x"]))
    if op == "gemm":
        a = s["a"].view(torch.float8_e4m3fn).float() * s["sa"][:, :case["m"]].t().repeat_interleave(BLOCK, 1)
        sb = s["sb"].repeat_interleave(BLOCK, 0)[:case["n"]].repeat_interleave(BLOCK, 1)
        return (a @ (s["b"].view(torch.float8_e4m3fn).float() * sb).t()).bfloat16()
    if op == "grouped":
        fmt, rows, n, k = case["fmt"], case["rows"], case["n"], case["k"]
        group, place = _group_of(s["offsets"], rows)
        if fmt == "fp8_b128":
            a = s["a"].view(torch.float8_e4m3fn).float() * s["sa"][:, :rows].t().repeat_interleave(BLOCK, 1)
            sb = s["sb"][:, :-(-n // BLOCK) * (k // BLOCK)].view(-1, -(-n // BLOCK), k // BLOCK)
            b = s["b"].view(torch.float8_e4m3fn).float()
            b *= sb.repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)
        else:
            c = k // (16 if fmt == "nvfp4" else 32)
            a = _mx_values(s["a"], _unswizzled(s["sa"], c)[_band_rows(s["offsets"], group, place)], fmt)
            sb = _unswizzled(s["sb"].view(-1), c).view(case["experts"], -1, c)[:, :n]
            b = _mx_values(s["b"], sb, fmt)
            if fmt == "nvfp4":
                a, b = a * s["ga"], b * s["gb"][:, None, None]
        padded = torch.zeros(case["experts"], s["most"], k, device=a.device)
        padded[group, place] = a
        out = torch.bmm(padded, b.transpose(1, 2))[group, place]
        if case["gelu"]:
            out = out * (0.5 * torch.erfc(out * -math.sqrt(0.5)))
        return out.bfloat16()
    if op == "dispatch":
        offsets, token, slot = _routed(s["ids"], case["experts"])
        rows, cols = token.numel(), case["cols"]
        x = s["x"][token.clamp(min=0).long()]
        group, place = _group_of(offsets, rows)
        live = group < case["experts"]
        if case["fmt"] == "fp8_b128":
            codes, scales = _b128_rows(x)
            scales[:, :rows] *= live
        else:
            v = x.float().view(rows, cols // 32, 32)
            m, e = torch.frexp(v.abs().amax(2))
            e = torch.where(m > 0, e - 9 + (m > 0.875).int(), -127).clamp(-127, 127)
            codes = (v * torch.exp2(-e.float())[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            bands = _bands(rows, case["experts"])
            laid = torch.zeros(bands * 128 + 1, cols // 32, dtype=torch.uint8, device=x.device)
            at = torch.where(live, _band_rows(offsets, group.clamp(max=case["experts"] - 1), place), bands * 128)
            laid[at] = (e + 127).to(torch.uint8) * live[:, None]
            codes, scales = codes.view(rows, cols), _swizzled(laid[:-1], bands)
        codes = (codes.view(torch.uint8) * live[:, None]).view(torch.float8_e4m3fn)
        return [offsets, token, slot, codes, scales]
    slot = s["slot"]
    y = s["y"][slot.clamp(min=0).long()].float()
    return (y * torch.where(slot >= 0, s["weights"], 0.0)[..., None]).sum(1).bfloat16()


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    op = case["op"]
    if op == "quantize":
        r, c, t = case["rows"], case["cols"], case["tile"]
        return {"bytes": 3 * r * c + 4 * -(-r // t) * (c // BLOCK), "flops": 2 * r * c}
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": m * k + n * k + 4 * (m + -(-n // BLOCK)) * (k // BLOCK) + 2 * m * n, "flops": 2 * m * n * k}
    if op == "grouped":
        t, n, k = case["rows"], case["n"], case["k"]
        live = sum(c > 0 for c in _counts(case))
        per = {"fp8_b128": 1.0, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32, "nvfp4": 0.5 + 1 / 16}[case["fmt"]]
        extra = 4 * (t + live * -(-n // BLOCK)) * (k // BLOCK) if case["fmt"] == "fp8_b128" else 0
        return {"bytes": per * (t + live * n) * k + extra + 2 * t * n, "flops": 2 * t * n * k}
    if op == "dispatch":
        t, c, k = case["tokens"], case["choices"], case["cols"]
        live = t - int(t * case["pad"])
        scale = 4 / BLOCK if case["fmt"] == "fp8_b128" else 1 / 32
        return {"bytes": 2 * live * k + live * c * k * (1 + scale) + 12 * t * c, "flops": 2 * live * c * k}
    t, c, n = case["tokens"], case["choices"], case["cols"]
    keep = 1.0 - case["drop"]
    return {"bytes": 2 * t * c * n * keep + 8 * t * c + 2 * t * n, "flops": 2 * t * c * n * keep}


# ---------------------------------------------------------------- the definition, in 64 bits
def _nearest_e4m3(q):
    """The E4M3 value nearest to each FP64 value, ties to the even one, saturating."""
    e = torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6)))
    step = torch.exp2(e - 3)
    return (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_block(x, amax):
    """(element values, scales in FP64) of x under the scale rule amax / 448 in FP32."""
    scale = (amax / E4M3_MAX).float().double()
    return torch.where(scale > 0, _nearest_e4m3(x / scale), x * 0.0), scale


def _exact_operand(codes, fmt):
    if fmt in ("fp8_b128", "mxfp8"):
        return codes.view(torch.float8_e4m3fn).double()
    at = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=codes.device)
    out = torch.empty(codes.shape[0], codes.shape[1] * 2, dtype=torch.float64, device=codes.device)
    out[:, 0::2], out[:, 1::2] = at[(codes & 15).long()], at[(codes >> 4).long()]
    return out


def _exact_sf(tiles, rows, cols, fmt, first_band=0):
    """Scale (r, c) of a matrix from its place in the 512-byte tiles."""
    r = torch.arange(rows, device=tiles.device)[:, None]
    c = torch.arange(cols, device=tiles.device)[None, :]
    at = ((first_band + r // 128) * -(-cols // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4
    b = tiles.view(-1)[at]
    return b.view(torch.float8_e4m3fn).double() if fmt == "nvfp4" else torch.exp2(b.double() - 127)


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "quantize":
        x, t = s["x"].double(), case["tile"]
        rows, cols = x.shape
        nb, kb = -(-rows // t), cols // BLOCK
        q, scales = torch.empty_like(x), torch.zeros(nb, kb, dtype=torch.float64, device=x.device)
        for j in range(kb):
            block = x[:, j * BLOCK:(j + 1) * BLOCK]
            amax = block.abs().amax(1)
            if t > 1:
                amax = torch.stack([v.amax() for v in amax.split(t)])
            scales[:, j] = _exact_block(amax, amax)[1]
            q[:, j * BLOCK:(j + 1) * BLOCK] = _exact_block(block, amax.repeat_interleave(t)[:rows, None])[0]
        if t > 1:
            return [q, scales]
        laid = torch.zeros(kb, _pitch(rows), dtype=torch.float64, device=x.device)
        laid[:, :rows] = scales.t()
        return [q, laid]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        out = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        for j in range(k // BLOCK):
            cut = slice(j * BLOCK, (j + 1) * BLOCK)
            a = _exact_operand(s["a"][:, cut], "fp8_b128") * s["sa"][j, :m, None].double()
            b = _exact_operand(s["b"][:, cut], "fp8_b128")
            b *= s["sb"][:, j].double().repeat_interleave(BLOCK)[:n, None]
            out.addmm_(a, b.t())
        return out
    if op == "grouped":
        fmt, n, k = case["fmt"], case["n"], case["k"]
        out = torch.zeros(case["rows"], n, dtype=torch.float64, device="cuda")
        first, band = 0, 0
        for e, c in enumerate(_counts(case)):
            if c:
                a, b = _exact_operand(s["a"][first:first + c], fmt), _exact_operand(s["b"][e], fmt)
                if fmt == "fp8_b128":
                    a *= s["sa"][:, first:first + c].t().double().repeat_interleave(BLOCK, 1)
                    sb = s["sb"][e][:-(-n // BLOCK) * (k // BLOCK)].view(-1, k // BLOCK).double()
                    b *= sb.repeat_interleave(BLOCK, 0)[:n].repeat_interleave(BLOCK, 1)
                else:
                    block = 16 if fmt == "nvfp4" else 32
                    a *= _exact_sf(s["sa"], c, k // block, fmt, band).repeat_interleave(block, 1)
                    b *= _exact_sf(s["sb"][e], n, k // block, fmt).repeat_interleave(block, 1)
                    if fmt == "nvfp4":
                        a, b = a * s["ga"].double(), b * s["gb"][e].double()
                out[first:first + c] = a @ b.t()
            first, band = first + c, band + -(-c // 128)
        if case["gelu"]:
            out = out * torch.special.ndtr(out)
        return out
    if op == "dispatch":
        ids = s["ids"].reshape(-1).tolist()
        order = sorted((i for i, e in enumerate(ids) if 0 <= e < case["experts"]), key=lambda i: (ids[i], i))
        rows, cols, live = len(ids), case["cols"], len(order)
        at = torch.tensor(order, device="cuda", dtype=torch.long) // case["choices"]
        x, q = s["x"].double()[at], torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
        if case["fmt"] != "fp8_b128":
            v = x.view(live, cols // 32, 32)
            amax = v.abs().amax(2, keepdim=True)
            e = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -140) / E4M3_MAX))
            e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, torch.where(amax <= E4M3_MAX * torch.exp2(e - 1), e - 1, e))
            q[:live] = _nearest_e4m3(v / torch.exp2(e.clamp(min=-127))).view(live, cols)
            return [None, None, None, q, None]
        scales = torch.zeros(cols // BLOCK, _pitch(rows), dtype=torch.float64, device="cuda")
        v = x.view(live, cols // BLOCK, BLOCK)
        el, sc = _exact_block(v, v.abs().amax(2, keepdim=True))
        q[:live], scales[:, :live] = el.view(live, cols), sc[..., 0].t()
        return [None, None, None, q, scales]
    out = torch.zeros(case["tokens"], case["cols"], dtype=torch.float64, device="cuda")
    for j in range(case["choices"]):
        slot = s["slot"][:, j].long()
        w = torch.where(slot >= 0, s["weights"][:, j].double(), 0.0)
        out += w[:, None] * s["y"].double()[slot.clamp(min=0)]
    return out
