"""GEMM of block-128 FP8 matrices against the FP64 product of the dequantized operands, within the header's contract."""
import pytest
import torch

from experts_helpers import activations, b128_values, gemm_error, weights
from fp8_quantization_block_b200 import mx

pytestmark = pytest.mark.gpu


def operands(M, N, K, seed=0):
    return (mx.quantize(activations(seed + 1, M, K), mx.MX_FP8_B128),
            mx.quantize(weights(seed + 2, N, K), mx.MX_FP8_B128X128))


def run(M, N, K, seed=0, out=None):
    a, b = operands(M, N, K, seed)
    c = mx.gemm(a, b, out=out)
    torch.cuda.synchronize()
    mx.check_device_error()
    err = gemm_error(c, b128_values(a), b128_values(b))
    assert err <= 1.0, err
    return a, b, c


@pytest.mark.parametrize("M", [1, 16, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("N,K", [(256, 128), (1000, 640), (4096, 1024)])
def test_few_rows(M, N, K):
    run(M, N, K)


@pytest.mark.parametrize("M,N,K", [(129, 129, 128), (256, 256, 512), (300, 520, 384), (1000, 2179, 1152),
                                   (513, 96, 256), (2048, 8, 128), (777, 1, 256), (4096, 4096, 2048)])
def test_many_rows(M, N, K):
    run(M, N, K)


@pytest.mark.parametrize("M,N,K", [(300, 700, 256), (40, 700, 256)])
def test_several_tiles_per_cta(M, N, K):
    """The grid cap makes every CTA walk several tiles; the grid does not change how a tile is summed."""
    try:
        mx.check(mx.mx_debug_set(mx.MX_DEBUG_MAX_GEMM_CTAS, 2))
        _, _, c2 = run(M, N, K)
    finally:
        mx.mx_debug_set(mx.MX_DEBUG_MAX_GEMM_CTAS, 0)
    _, _, c = run(M, N, K)
    assert torch.equal(c, c2)


def test_row_pitch_leaves_the_rest():
    out = torch.full((70, 400), 3.0, dtype=torch.bfloat16, device="cuda")
    run(70, 320, 256, out=out[:, :320])
    assert (out[:, 320:] == 3).all()
    out = torch.full((70, 333), 3.0, dtype=torch.bfloat16, device="cuda")
    run(70, 320, 256, out=out[:, :320])
    assert (out[:, 320:] == 3).all()


def test_scales_reach_their_block():
    """One nonzero block at a time: C is the product of exactly those scales."""
    M, N, K = 200, 300, 512
    a, b = mx.empty(mx.MX_FP8_B128, M, K), mx.empty(mx.MX_FP8_B128X128, N, K)
    a.codes.fill_(0x38)     # 1.0
    b.codes.fill_(0x38)
    sa = a.scales.view(torch.float32).view(K // 128, 200)
    sb = b.scales.view(torch.float32)[:3 * 4].view(3, 4)
    sa.copy_(torch.arange(1, 801, device="cuda").view(4, 200).float() / 1024)
    sb.copy_(torch.arange(1, 13, device="cuda").view(3, 4).float())
    c = mx.gemm(a, b)
    ref = 128 * (sa.double().t() @ sb.double().t()).repeat_interleave(128, 1)[:, :N]
    assert torch.equal(c, ref.bfloat16()) or ((c.double() - ref).abs() <= 2.0 ** -8 * ref).all()


def test_zero_blocks_and_extreme_scales():
    M, N, K = 64, 256, 384
    x = activations(3, M, K)
    x[5] = 0
    x[:, 128:256] *= 1e-30
    x[7] *= 1e20
    a, b = mx.quantize(x, mx.MX_FP8_B128), mx.quantize(weights(4, N, K), mx.MX_FP8_B128X128)
    c = mx.gemm(a, b)
    assert (c[5] == 0).all()
    assert gemm_error(c, b128_values(a), b128_values(b)) <= 1.0


@pytest.mark.parametrize("gelu", [False, True])
def test_fused_call_is_quantize_then_gemm(gelu):
    M, N, K = 150, 400, 640
    x = activations(8, M, K)
    w = mx.quantize(weights(9, N, K), mx.MX_FP8_B128X128)
    c = mx.gemm_fused_act(x, w, x_fmt=mx.MX_FP8_B128, epilogue=mx.MX_EPI_GELU if gelu else mx.MX_EPI_NONE)
    a = mx.quantize(x, mx.MX_FP8_B128)
    if not gelu:
        assert torch.equal(c, mx.gemm(a, w))
    assert gemm_error(c, b128_values(a), b128_values(w), gelu) <= 1.0


def test_same_bits_from_call_to_call_and_in_a_graph():
    a, b, c = run(333, 1024, 512)
    out = torch.zeros_like(c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.gemm(a, b, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, c)
    g = torch.cuda.CUDAGraph()
    out.zero_()
    with torch.cuda.graph(g):
        mx.gemm(a, b, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, c)


def test_two_streams_at_once():
    """Calls of two streams that overlap on the GPU do not touch one another."""
    a, b, c = run(200, 2048, 1024)
    a2, b2, c2 = run(16, 4096, 2048)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    o1, o2 = [torch.empty_like(c) for _ in range(8)], [torch.empty_like(c2) for _ in range(8)]
    for i in range(8):
        mx.gemm(a, b, out=o1[i], stream=s1)
        mx.gemm(a2, b2, out=o2[i], stream=s2)
    torch.cuda.synchronize()
    assert all(torch.equal(o, c) for o in o1) and all(torch.equal(o, c2) for o in o2)
    mx.check_device_error()


def test_fused_call_without_allocation_in_a_graph():
    """The fused call's quantized operand lives in the caller's workspace, through a capture and its replays."""
    M, N, K = 150, 400, 640
    x = activations(8, M, K)
    w = mx.quantize(weights(9, N, K), mx.MX_FP8_B128X128)
    ws = mx.fused_workspace(mx.MX_FP8_B128, M, K)
    want = mx.gemm(mx.quantize(x, mx.MX_FP8_B128), w)
    out = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mx.gemm_fused_act(x, w, out=out, workspace=ws)      # x_fmt: the one that goes with w
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx.gemm_fused_act(x, w, x_fmt=mx.MX_FP8_B128, out=out, workspace=ws)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("kb", [1, 2, 3, 4, 5, 6, 7, 9])
@pytest.mark.parametrize("M,N", [(5, 700), (32, 64), (33, 1000), (128, 4096), (300, 5000), (40, 333)])
def test_any_number_of_blocks(M, N, kb):
    """Stages of one, two and four K blocks with every remainder; several tiles per CTA, whose rings run on."""
    try:
        mx.check(mx.mx_debug_set(mx.MX_DEBUG_MAX_GEMM_CTAS, 3))
        _, _, c = run(M, N, 128 * kb)
    finally:
        mx.mx_debug_set(mx.MX_DEBUG_MAX_GEMM_CTAS, 0)
    a, b = mx.quantize(activations(M, M, 128 * kb), 6), mx.quantize(weights(N, N, 128 * kb), 8)
    g = mx.gemm_fused_act(activations(M, M, 128 * kb), b, epilogue=mx.MX_EPI_GELU)
    assert gemm_error(g, b128_values(a), b128_values(b), True) <= 1.0
