"""Sizes and refusals of the block-128 formats and the experts' operators (host only, no GPU)."""
import ctypes

import pytest
import torch

from fp8_quantization_block_b200 import build as mxbuild
from fp8_quantization_block_b200 import mx

BAD, SHAPE, ALIGN, OK = mx.MX_ERR_INVALID_ARG, mx.MX_ERR_UNSUPPORTED_SHAPE, mx.MX_ERR_MISALIGNED, mx.MX_OK


@pytest.fixture(scope="module", autouse=True)
def built():
    mxbuild.build()


def T(fmt, rows, cols, codes=0x1000, scales=0x2000, g=0x3000):
    return mx.MxTensorC(fmt, 0, rows, cols, codes, scales, g)


def G(count=4, offsets=0x8000):
    return mx.MxGroupsC(count, 0, offsets)


def test_sizes():
    assert mx.mx_codes_bytes(6, 5, 256) == 1280 and mx.mx_block_size(6) == 128
    assert mx.mx_scales_bytes(6, 5, 256) == 4 * 8 * 2
    assert mx.mx_scales_bytes(8, 129, 384) == 32 and mx.mx_block_size(8) == 128    # 2 x 3 floats, to 16 bytes
    assert mx.mx_codes_bytes(7, 4, 128) == 0 and mx.mx_scales_bytes(7, 4, 128) == 0 and mx.mx_block_size(7) == 0
    assert mx.mx_grouped_scales_bytes(6, 5, 9, 256) == mx.mx_scales_bytes(6, 5, 256)
    assert mx.mx_grouped_scales_bytes(0, 300, 4, 256) == (300 + 127 * 4) // 128 * 128 * 8
    assert mx.mx_grouped_scales_bytes(0, 3, 100, 256) == 3 * 128 * 8               # at most a band per row
    assert mx.mx_grouped_scales_bytes(8, 3, 1, 256) == 0 and mx.mx_grouped_scales_bytes(5, 3, 1, 256) == 0
    assert mx.mx_route_workspace_bytes(256, 8, 64) == 0
    assert mx.mx_route_workspace_bytes(257, 8, 64) == 3 * 64 * 4                    # counts of three chunks of 1024
    assert mx.mx_route_workspace_bytes(2 ** 31, 2, 4) == 0
    assert ctypes.sizeof(mx.MxGroupsC) == 16
    assert mx.MX_MAX_GROUPS == 1024


@pytest.mark.parametrize("rows,counts", [(300, [1] * 300), (300, [300]), (300, [129, 1, 127, 43]), (7, [0, 7, 0]),
                                         (1000, [128, 129, 743])])
def test_grouped_bands_fit_any_split(rows, counts):
    assert sum(-(-c // 128) for c in counts) * 128 * 8 <= mx.mx_grouped_scales_bytes(0, rows, len(counts), 256)


def test_block128_calls_refuse():
    assert mx.mx_quantize(6, 0x1000, 4, 64, 64, T(6, 4, 64), None, None) == SHAPE
    assert mx.mx_quantize(8, 0x1000, 4, 192, 192, T(8, 4, 192), None, None) == SHAPE
    assert mx.mx_quantize(7, 0x1000, 4, 128, 128, T(7, 4, 128), None, None) == BAD
    assert mx.mx_quantize(6, 0x1000, 4, 128, 128, T(8, 4, 128), None, None) == BAD
    assert mx.mx_quantize(6, 0x1000, 4, 128, 120, T(6, 4, 128), None, None) == ALIGN
    assert mx.mx_quantize(6, 0x1000, 4, 128, 128, T(6, 4, 128, scales=0x2004), None, None) == ALIGN
    assert mx.mx_quantize(6, None, 0, 128, 128, T(6, 0, 128), None, None) == OK
    A, W = T(6, 8, 256), T(8, 8, 256)
    for a, b in ((W, A), (A, A), (W, W), (A, T(0, 8, 256)), (T(0, 8, 256), W), (A, T(5, 8, 256))):
        assert mx.mx_gemm(a, b, 0x4000, 8, None) == BAD
    assert mx.mx_gemm(A, T(8, 8, 128), 0x4000, 8, None) == BAD
    assert mx.mx_gemm(A, W, 0x4000, 7, None) == BAD
    assert mx.mx_gemm(A, W, 0x4008, 8, None) == ALIGN
    assert mx.mx_gemm(T(6, 8, 64), T(8, 8, 64), 0x4000, 8, None) == SHAPE
    assert mx.mx_quantize_rht(6, 0x1000, 4, 256, 256, T(6, 4, 256), None, None) == BAD
    assert mx.mx_qsnr(T(6, 4, 256), 0x1000, 256, 0x5000, None) == BAD
    ws = mx.mx_fused_workspace_bytes(6, 4, 256)
    assert ws > 0 and mx.mx_fused_workspace_bytes(8, 4, 256) == 0
    f = lambda w, need=ws, amax=None: mx.mx_gemm_fused_act(6, 0x1000, 4, 256, 256, w, 0x4000, 8, 0, amax, None, None,  # noqa: E731
                                                           0x10000, need, None)
    assert f(T(0, 8, 256)) == BAD and f(T(6, 8, 256)) == BAD and f(W, ws - 1) == BAD


def test_quantize_grouped_refuses():
    def q(fmt=6, src=0x1000, src_rows=9, K=256, ld=256, idx=0x7000, groups=None, dst=None, g=0x9000):
        return mx.mx_quantize_grouped(fmt, src, src_rows, K, ld, idx, groups or G(), dst or T(fmt, 9, K), g, None, 0, None)
    assert q(fmt=5) == BAD and q(fmt=8) == BAD and q(fmt=7) == BAD
    assert q(groups=G(0)) == BAD and q(groups=G(4, None)) == BAD and q(groups=G(1025)) == SHAPE
    assert q(groups=G(4, 0x8002)) == ALIGN and q(idx=0x7001) == ALIGN
    assert q(dst=T(0, 9, 256)) == BAD and q(dst=T(6, 9, 128)) == BAD and q(dst=T(6, 9, 256, codes=None)) == BAD
    assert q(idx=None, src_rows=8) == BAD              # fewer source rows than rows without an index
    assert q(K=192, ld=192) == SHAPE and q(fmt=0, K=48, ld=48) == SHAPE
    assert q(ld=255) == ALIGN and q(src=0x1008) == ALIGN and q(src=None) == BAD
    assert q(fmt=3, g=None) == BAD
    assert q(dst=T(6, 0, 256)) == OK                   # no rows: nothing to do
    # the workspace of rows that go to several places
    need = mx.mx_quantize_grouped_workspace_bytes(4096, 1024, 1024)
    assert need >= 4 * 1025 + 64 * 1024 + 16 * 4096
    for rows, src in ((1024, 1024), (32 * 8, 32), (20 * 1024, 1024), (-1, 4), (4, -1)):
        assert mx.mx_quantize_grouped_workspace_bytes(rows, src, 1024) == 0
    assert mx.mx_quantize_grouped_workspace_bytes(4096, 1024, 384) == 0
    assert mx.mx_quantize_grouped_workspace_bytes(4096, 1024, 0) == 0
    def w(ws, n):  # noqa: E306
        return mx.mx_quantize_grouped(6, 0x1000, 1024, 1024, 1024, 0x7000, G(), T(6, 4096, 1024), None, ws, n, None)
    assert w(0x20000, need - 1) == BAD and w(0x20008, need) == ALIGN


def test_gemm_grouped_refuses():
    def m(a=None, b=None, groups=None, C=0x4000, ldc=16, epi=0):
        return mx.mx_gemm_grouped(a or T(6, 9, 256), b or T(8, 16, 256), groups or G(), C, ldc, epi, None)
    assert m(a=T(5, 9, 256), b=T(5, 16, 256)) == BAD
    assert m(a=T(6, 9, 256), b=T(6, 16, 256)) == BAD and m(a=T(0, 9, 256)) == BAD and m(a=T(3, 9, 256), b=T(0, 16, 256)) == BAD
    assert m(b=T(8, 16, 128)) == BAD and m(epi=2) == BAD and m(ldc=15) == BAD and m(C=None) == BAD and m(C=0x4008) == ALIGN
    assert m(a=T(0, 9, 64), b=T(0, 16, 64)) == SHAPE
    assert m(a=T(6, 9, 0), b=T(8, 16, 0)) == SHAPE
    assert m(groups=G(0)) == BAD and m(groups=G(2000)) == SHAPE
    assert m(a=T(4, 9, 256, codes=0x1010), b=T(4, 16, 256)) == ALIGN
    assert m(b=T(8, 2 ** 30, 256), ldc=2 ** 30) == SHAPE   # groups x N past 32 bits
    assert m(a=T(6, 0, 256)) == OK and m(b=T(8, 0, 256)) == OK


def test_route_and_combine_refuse():
    def r(ids=0x1000, bits=32, tokens=4, choices=2, groups=8, off=0x2000, row=0x3000, slot=0x4000, ws=None, wsb=0):
        return mx.mx_route(ids, bits, tokens, choices, groups, off, row, slot, ws, wsb, None)
    assert r(bits=16) == BAD and r(choices=0) == BAD and r(groups=0) == BAD and r(groups=1025) == SHAPE
    assert r(ids=None) == BAD and r(off=None) == BAD and r(row=None) == BAD and r(slot=None) == BAD
    assert r(ids=0x1004, bits=64) == ALIGN and r(row=0x3002) == ALIGN
    assert r(tokens=2 ** 31, choices=2) == SHAPE
    assert r(tokens=5000, ws=None) == BAD and r(tokens=5000, ws=0x9000, wsb=8) == BAD

    def c(y=0x1000, rows=8, cols=16, ldy=16, slot=0x2000, w=0x3000, tokens=4, choices=2, out=0x4000, ldo=16):
        return mx.mx_combine(y, rows, cols, ldy, slot, w, tokens, choices, out, ldo, None)
    assert c(y=None) == BAD and c(slot=None) == BAD and c(w=None) == BAD and c(out=None) == BAD
    assert c(ldy=15) == BAD and c(ldo=15) == BAD and c(choices=0) == BAD and c(rows=-1) == BAD
    assert c(y=0x1001) == ALIGN and c(w=0x3002) == ALIGN
    assert c(tokens=0) == OK and c(cols=0) == OK


def test_binding_refuses_before_it_calls():
    """Shapes, types and devices that the binding turns away (CPU tensors among them)."""
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    off = torch.tensor([0, 4], dtype=torch.int32)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call in (lambda: mx.route(ids, 3), lambda: mx.route(ids.float(), 3), lambda: mx.route(ids[:, :1], 3),
                 lambda: mx.quantize_grouped(x.float(), off, 6), lambda: mx.quantize_grouped(x, off.long(), 6),
                 lambda: mx.quantize_grouped(x, off[:1], 6), lambda: mx.quantize_grouped(x.t(), off, 6),
                 lambda: mx.quantize_grouped(x, off, 6, row_index=torch.zeros(4)),
                 lambda: mx.combine(x, ids, torch.zeros(4, 2, dtype=torch.float64)),
                 lambda: mx.combine(x, ids, torch.zeros(4, 3)), lambda: mx.combine(x, ids.long(), torch.zeros(4, 2)),
                 lambda: mx.combine(x, ids, torch.zeros(4, 2)), lambda: mx.quantize_experts(x, 8)):
        with pytest.raises(ValueError):
            call()
    a = mx.MxTensor(6, 4, 256, torch.zeros(1024, dtype=torch.uint8), torch.zeros(32, dtype=torch.uint8), None)
    w = mx.MxTensor(8, 16, 256, torch.zeros(16 * 256, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), None)
    with pytest.raises(ValueError):       # two groups, one matrix
        mx.gemm_grouped(a, w, torch.tensor([0, 2, 4], dtype=torch.int32))
    with pytest.raises(ValueError):       # a scale buffer that is too small
        mx.gemm_grouped(mx.MxTensor(6, 4, 256, a.codes, a.scales[:16], None), w, off)
    with pytest.raises(ValueError):
        mx.quantize_grouped(x, off, 6, out=mx.MxTensor(6, 4, 256, a.codes[:100], a.scales, None))
