"""Quantize and dequantize of the block-128 FP8 formats: codes and scales equal the FP64 form's, bit for bit."""
import pytest
import torch

from experts_helpers import activations, b128_quantize, b128_scales, b128_values, e4m3_values
from fp8_quantization_block_b200 import mx

pytestmark = pytest.mark.gpu
FMTS = [(mx.MX_FP8_B128, 1), (mx.MX_FP8_B128X128, 128)]


def check(x, fmt, tile):
    rows, K = x.shape
    t = mx.quantize(x, fmt)
    torch.cuda.synchronize()
    q, s = b128_quantize(x, tile)
    assert torch.equal(b128_scales(t).double(), s)
    got = e4m3_values(t.codes).view(rows, K)
    assert torch.equal(got, q), (got != q).sum()
    assert torch.equal(torch.signbit(got), torch.signbit(x.double()))
    return t, q, s


@pytest.mark.parametrize("fmt,tile", FMTS)
@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (16, 8192), (127, 384), (128, 128), (129, 512), (1000, 1152)])
def test_codes_and_scales(fmt, tile, rows, K):
    check(activations(rows * 7 + K, rows, K), fmt, tile)


@pytest.mark.parametrize("fmt,tile", FMTS)
def test_edges(fmt, tile):
    """Zeros, signed zeros, subnormals, the largest bf16, one value beside zeros, and quotients on or next to the
    middle of two codes."""
    K = 128
    rows = [torch.zeros(K), -torch.zeros(K), torch.full((K,), 2.0 ** -133), torch.full((K,), 3.3e38)]
    one = torch.zeros(K)
    one[77] = -5.0
    rows.append(one)
    for top in (448.0, 1.0, 3.0, 2.0 ** -130, 2.0 ** -70, 1e38, 0.7):
        mids = torch.tensor([(2 * i + 1) / 32 for i in range(16, 32)]) * 2.0
        for e in (0, -3, -7, -9):
            r = torch.zeros(K)
            r[0] = top
            r[1:17] = mids * 2.0 ** e * (top / 4.0)
            r[17:33] = -r[1:17]
            rows.append(r)
    for r in rows:
        check(r[None].bfloat16().cuda(), fmt, tile)
    check(torch.stack(rows).bfloat16().cuda(), fmt, tile)


@pytest.mark.parametrize("fmt,tile", FMTS)
def test_row_pitch_and_dequantize(fmt, tile):
    wide = activations(5, 200, 1024)
    x = wide[:, 256:640]
    t, q, s = check(x, fmt, tile)
    d = mx.dequantize(t)
    assert torch.equal(d, b128_values(t).bfloat16())     # one rounding of the exact product: FP64 holds it
    out = torch.full((200, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    mx.dequantize(t, out=out[:, :384])
    assert torch.equal(out[:, :384], d) and (out[:, 384:] == 7).all()


def test_scale_padding_is_zero():
    x = activations(6, 5, 256)
    t = mx.empty(mx.MX_FP8_B128, 5, 256)
    t.scales.fill_(255)
    mx.quantize(x, mx.MX_FP8_B128, out=t)
    f = t.scales.view(torch.float32).view(2, 8)
    assert (f[:, 5:] == 0).all() and (f[:, :5] > 0).all()


def test_round_trip_of_representable_blocks():
    """Codes 448 2^e and below with a scale of exactly 2^e come back as they went in."""
    vals = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    x = torch.zeros(4, 128)
    x[:, :126] = vals
    x[:, 126] = 448.0
    x[1] *= 2.0 ** 9
    x[2] *= -(2.0 ** -20)
    x = x.bfloat16().cuda()
    assert torch.equal(mx.dequantize(mx.quantize(x, mx.MX_FP8_B128)), x)


def test_every_pair_of_mantissas():
    """All 128 x 128 pairs of a block's largest and another element's mantissa, at every distance of exponents that
    reaches a nonzero code: among them every tie and everything next to one."""
    rows = []
    for top in range(128, 256):
        others = torch.tensor([[m * 2.0 ** -k for k in range(0, 21)] for m in range(128, 256)]).reshape(-1)
        others = others[others <= top]
        others = torch.where(torch.arange(others.numel()) % 2 == 0, others, -others)
        pad = torch.zeros(-others.numel() % 127)
        block = torch.cat((others, pad)).view(-1, 127)
        rows.append(torch.cat((torch.full((block.shape[0], 1), float(top)), block), 1))
    x = torch.cat(rows)
    for scale in (1.0, 2.0 ** -60, 2.0 ** -75, 2.0 ** 100):
        check((x * scale).bfloat16().cuda(), mx.MX_FP8_B128, 1)
