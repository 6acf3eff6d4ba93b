"""Plain FP64 forms of the block-128 formats and the experts' operators (torch, elementary operations), for the tests.

They share nothing with the library but the documented layouts."""
from __future__ import annotations

import torch

from fp8_quantization_block_b200 import mx

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def e4m3_nearest(q: torch.Tensor) -> torch.Tensor:
    """Nearest E4M3 values of FP64 numbers, ties to even, saturating at 448."""
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def b128_quantize(x: torch.Tensor, tile: int):
    """(E4M3 values FP64 [rows, K], scales FP64 [ceil(rows / tile), K / 128]) of a bf16 matrix."""
    rows, K = x.shape
    xd = x.double()
    nb = -(-rows // tile)
    q = torch.zeros_like(xd)
    s = torch.zeros(nb, K // 128, dtype=torch.float64, device=x.device)
    for i in range(nb) if tile > 1 else [None]:
        r = slice(None) if i is None else slice(i * tile, (i + 1) * tile)
        v = xd[r].reshape(-1, K // 128, 128)
        amax = v.abs().amax(2) if i is None else v.abs().amax((0, 2))[None]
        sc = (amax / 448.0).float().double()
        s[r if i is None else slice(i, i + 1)] = sc
        el = torch.where(sc[..., None] > 0, e4m3_nearest(v / sc[..., None]), v * 0.0)
        q[r] = el.reshape(-1, K)
    return q, s


def b128_scales(t: mx.MxTensor) -> torch.Tensor:
    """Scales [rows or row blocks, K / 128] (float32) from an FP8_B128 / FP8_B128X128 tensor's buffer."""
    kb = t.cols // 128
    f = t.scales.view(torch.uint8).reshape(-1).view(torch.float32)
    if t.fmt == mx.MX_FP8_B128:
        pitch = -(-t.rows // 4) * 4
        return f[:kb * pitch].view(kb, pitch)[:, :t.rows].t()
    nb = -(-t.rows // 128)
    return f[:nb * kb].view(nb, kb)


def e4m3_values(codes: torch.Tensor) -> torch.Tensor:
    return codes.view(torch.float8_e4m3fn).double()


def b128_values(t: mx.MxTensor) -> torch.Tensor:
    s = b128_scales(t).double()
    if t.fmt == mx.MX_FP8_B128X128:
        s = s.repeat_interleave(128, 0)[:t.rows]
    q = e4m3_values(t.codes[:t.rows * t.cols]).view(t.rows, t.cols)
    return q * s.repeat_interleave(128, 1)


def sf_at(buf: torch.Tensor, rows: torch.Tensor, cols: int) -> torch.Tensor:
    """Scale bytes of the given rows of the 512-byte tile layout, [len(rows), cols]."""
    c = torch.arange(cols, device=buf.device)[None]
    r = rows[:, None]
    return buf.view(-1)[((r // 128) * -(-cols // 4) + c // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + c % 4]


def element_values(codes: torch.Tensor, fmt: int, rows: int, cols: int) -> torch.Tensor:
    codes = codes.view(-1)[:mx.mx_codes_bytes(fmt, rows, cols)].view(rows, -1)
    if fmt in (mx.MX_MXFP8_E4M3, mx.MX_FP8_B128, mx.MX_FP8_B128X128):
        return codes.view(torch.float8_e4m3fn).double()
    if fmt == mx.MX_MXFP8_E5M2:
        return codes.view(torch.float8_e5m2).double()
    if fmt == mx.MX_MXFP6_E3M2:
        b = codes.long().view(rows, -1, 3)
        w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
        c = torch.stack([(w >> (6 * i)) & 63 for i in range(4)], -1).view(rows, cols)
        e, m = (c >> 2) & 7, (c & 3).double()
        v = torch.where(e == 0, m * 2.0 ** -4, (1 + m / 4) * torch.exp2((e - 3).double()))
        return torch.where(c >= 32, -v, v)
    t = torch.tensor(E2M1 + [-v for v in E2M1], dtype=torch.float64, device=codes.device)
    return torch.stack((t[(codes & 15).long()], t[(codes >> 4).long()]), -1).view(rows, cols)


def scale_values(b: torch.Tensor, fmt: int) -> torch.Tensor:
    return b.contiguous().view(torch.float8_e4m3fn).double() if fmt == mx.MX_NVFP4 else torch.exp2(b.double() - 127)


def block_of(fmt: int) -> int:
    return 16 if fmt == mx.MX_NVFP4 else 32


def grouped_values(t: mx.MxTensor, offsets: list) -> torch.Tensor:
    """FP64 values of a grouped activation (rows of no group: NaN)."""
    if t.fmt == mx.MX_FP8_B128:
        v = b128_values(t)
    else:
        at = torch.zeros(t.rows, dtype=torch.long, device=t.codes.device)
        band = 0
        for a, b in zip(offsets, offsets[1:]):
            at[a:b] = torch.arange(b - a, device=at.device) + 128 * band
            band += -(-(b - a) // 128)
        blk = block_of(t.fmt)
        s = scale_values(sf_at(t.scales, at, t.cols // blk), t.fmt).repeat_interleave(blk, 1)
        v = element_values(t.codes, t.fmt, t.rows, t.cols) * s
        if t.fmt == mx.MX_NVFP4:
            v = v * t.gscale.double()
    v = v.clone()
    v[offsets[-1]:] = float("nan")
    return v


def expert_values(w: mx.MxTensor, e: int) -> torch.Tensor:
    """FP64 values of expert e's matrix in a stack."""
    cb, sb = mx.mx_codes_bytes(w.fmt, w.rows, w.cols), mx.mx_scales_bytes(w.fmt, w.rows, w.cols)
    one = mx.MxTensor(w.fmt, w.rows, w.cols, w.codes.view(-1)[e * cb:(e + 1) * cb],
                      w.scales.view(-1).view(torch.uint8)[e * sb:(e + 1) * sb], None)
    if w.fmt == mx.MX_FP8_B128X128:
        return b128_values(one)
    blk = block_of(w.fmt)
    s = scale_values(sf_at(one.scales, torch.arange(w.rows, device=w.codes.device), w.cols // blk), w.fmt)
    v = element_values(one.codes, w.fmt, w.rows, w.cols) * s.repeat_interleave(blk, 1)
    return v * w.gscale[e].double() if w.fmt == mx.MX_NVFP4 else v


def gemm_error(C: torch.Tensor, A: torch.Tensor, B: torch.Tensor, gelu: bool = False) -> float:
    """Largest |C - C_ref| / bound; at most 1 within the contract.

    The bound is the header's, 2^-8 |C_ref| + 1e-4 |A| |B|^T: one bf16 rounding, and FP32 sums, whose error is below
    (128 + K / 128 + 3) 2^-23 of the absolute sum, under 1e-4 up to K = 90,000.  With GELU the pre-activation's error
    grows by its largest slope, 1.13, and the result is rounded once more, after an evaluation within 2e-5."""
    ref, mag = A @ B.t(), A.abs() @ B.abs().t()
    if not gelu:
        bound = 2.0 ** -8 * ref.abs() + 1e-4 * mag
    else:
        pre, ref = ref, ref * torch.special.ndtr(ref)
        # the sum reaches GELU in FP32, so only its FP32 error grows by the slope
        bound = 1.13 * 1e-4 * mag + (2.0 ** -8 + 2e-5) * ref.abs() * (1 + 2.0 ** -7) + 1e-30
        del pre
    err = (C.double() - ref).abs()
    assert torch.isfinite(C.float()).all()
    return float((err / bound.clamp(min=1e-300)).max()) if err.numel() else 0.0


def offsets_of(counts, device="cuda"):
    o = [0]
    for c in counts:
        o.append(o[-1] + c)
    return o, torch.tensor(o, dtype=torch.int32, device=device)


def route_reference(ids, experts: int):
    """Offsets, the token of each slot and the slot of each choice, from lists."""
    flat = [i for row in ids for i in row]
    k = len(ids[0]) if ids else 1
    order = sorted((i for i, e in enumerate(flat) if 0 <= e < experts), key=lambda i: (flat[i], i))
    offsets = [sum(1 for i in order if flat[i] < g) for g in range(experts + 1)]
    slot = [-1] * len(flat)
    for s, i in enumerate(order):
        slot[i] = s
    return offsets, [i // k for i in order] + [-1] * (len(flat) - len(order)), slot


def activations(seed: int, rows: int, cols: int) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x[:, torch.randint(0, cols, (max(1, cols // 256),), generator=g)] *= 30.0
    return x.bfloat16().cuda()


def weights(seed: int, *shape) -> torch.Tensor:
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * 0.05).bfloat16().cuda()
