"""Quantize and GEMM of rows grouped by expert against FP64 forms."""
import pytest
import torch

from experts_helpers import (activations, element_values, expert_values, gemm_error, grouped_values, offsets_of,
                             scale_values, sf_at, weights, block_of, b128_scales)
from fp8_quantization_block_b200 import mx

pytestmark = pytest.mark.gpu
B = (mx.MX_FP8_B128, mx.MX_FP8_B128X128)
PAIRS = [B, (0, 0), (2, 2), (3, 3), (1, 1), (4, 4), (0, 2), (0, 4), (2, 0), (1, 0)]
GROUPS = {
    "one": [1],
    "empty ends": [0, 0, 5, 0, 130, 1, 0, 33, 0],
    "all empty": [0, 0, 0],
    "exact blocks": [128, 256, 32, 64],
    "many": [(i * 37) % 19 for i in range(70)],
    "skewed": [700, 3, 0, 1, 259, 64],
}
NV_G = 0.004


def gs(fmt):
    return torch.tensor([NV_G], device="cuda") if fmt == mx.MX_NVFP4 else None


def quantized(counts, fmt, K, behind=0, seed=1):
    o, od = offsets_of(counts)
    x = activations(seed, max(o[-1] + behind, 1), K)
    return x, o, od, mx.quantize_grouped(x, od, fmt, gscale=gs(fmt))


@pytest.mark.parametrize("counts", GROUPS.values(), ids=GROUPS.keys())
@pytest.mark.parametrize("fmt", [6, 0, 1, 2, 3, 4])
def test_quantize_grouped_is_quantize_of_the_rows(fmt, counts):
    K = 384
    o, od = offsets_of(counts)
    T = max(o[-1], 1) + 3
    x = activations(11, T + 5, K)
    idx = torch.randperm(T + 5, generator=torch.Generator().manual_seed(3))[:T].int().cuda()
    out = mx.empty_grouped(fmt, T, len(counts), K)
    out.codes.fill_(0xAA)
    out.scales.fill_(0xAA)
    mx.quantize_grouped(x, od, fmt, row_index=idx, gscale=gs(fmt), out=out)
    torch.cuda.synchronize()
    ref = mx.quantize(x[idx.long()].contiguous(), fmt, gscale=gs(fmt))
    live, per = o[-1], mx.mx_codes_bytes(fmt, 1, K)
    codes, want = out.codes.view(T, per), ref.codes.view(T, per)
    assert torch.equal(codes[:live], want[:live])
    assert (codes[live:] == 0xAA).all()              # rows of no group are left as they are
    if fmt == 6:
        assert torch.equal(b128_scales(out)[:live], b128_scales(ref)[:live])
        assert (b128_scales(out)[live:].contiguous().view(torch.uint8) == 0xAA).all()
        return
    cols = K // block_of(fmt)
    band = 0
    seen = torch.zeros(mx.mx_grouped_scales_bytes(fmt, T, len(counts), K), dtype=torch.bool, device="cuda")
    for a, b in zip(o, o[1:]):
        at = torch.arange(b - a, device="cuda") + 128 * band
        mine = torch.arange(a, b, device="cuda")
        assert torch.equal(sf_at(out.scales, at, cols), sf_at(ref.scales, mine, cols))
        seen[sf_at(torch.arange(seen.numel(), device="cuda"), at, cols).reshape(-1)] = True
        band += -(-(b - a) // 128)
    assert (out.scales[~seen] == 0).all()


def test_indexes_outside_the_source_are_zero_rows():
    x = activations(2, 10, 128)
    idx = torch.tensor([3, -1, 10, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32, device="cuda")
    _, od = offsets_of([2, 4])
    for fmt in (6, 0, 3):
        t = mx.quantize_grouped(x, od, fmt, row_index=idx, gscale=gs(fmt))
        v = grouped_values(t, [0, 2, 6])
        assert (v[1:5] == 0).all() and (v[0] != 0).any() and (v[5] != 0).any()


@pytest.mark.parametrize("counts", GROUPS.values(), ids=GROUPS.keys())
@pytest.mark.parametrize("fa,fb", PAIRS)
def test_gemm_grouped(fa, fb, counts):
    N, K = 392, 640
    x, o, od, a = quantized(counts, fa, K, behind=7)
    w = mx.quantize_experts(weights(21, len(counts), N, K), fb)
    c = torch.full((a.rows, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.gemm_grouped(a, w, od, out=c)
    torch.cuda.synchronize()
    mx.check_device_error()
    v = grouped_values(a, o)
    for g, (i, j) in enumerate(zip(o, o[1:])):
        if j > i:
            err = gemm_error(c[i:j], v[i:j], expert_values(w, g))
            assert err <= 1.0, (g, i, j, err)
    assert (c[o[-1]:] == 9).all()


@pytest.mark.parametrize("fa,fb", [B, (0, 0), (3, 3), (0, 2)])
@pytest.mark.parametrize("N", [1, 31, 128, 257, 1003])
def test_gelu_and_odd_widths(fa, fb, N):
    counts, K = [40, 0, 200, 1], 256
    x, o, od, a = quantized(counts, fa, K)
    w = mx.quantize_experts(weights(22, 4, N, K), fb)
    c = mx.gemm_grouped(a, w, od, epilogue=mx.MX_EPI_GELU)
    v = grouped_values(a, o)
    for g, (i, j) in enumerate(zip(o, o[1:])):
        if j > i:
            err = gemm_error(c[i:j], v[i:j], expert_values(w, g), gelu=True)
            assert err <= 1.0, (g, err)


@pytest.mark.parametrize("fa,fb", [B, (0, 0), (2, 2), (3, 3)])
@pytest.mark.parametrize("gelu", [False, True])
def test_several_tiles_per_cta(fa, fb, gelu):
    counts, N, K = [300, 0, 17, 129, 64], 1000, 512
    x, o, od, a = quantized(counts, fa, K)
    w = mx.quantize_experts(weights(23, 5, N, K), fb)
    epi = mx.MX_EPI_GELU if gelu else mx.MX_EPI_NONE
    c = mx.gemm_grouped(a, w, od, epilogue=epi)
    try:
        mx.check(mx.mx_debug_set(mx.MX_DEBUG_MAX_GEMM_CTAS, 2))
        c2 = mx.gemm_grouped(a, w, od, epilogue=epi)
        torch.cuda.synchronize()
    finally:
        mx.mx_debug_set(mx.MX_DEBUG_MAX_GEMM_CTAS, 0)
    mx.check_device_error()
    assert torch.equal(c, c2)
    v = grouped_values(a, o)
    for g, (i, j) in enumerate(zip(o, o[1:])):
        if j > i:
            assert gemm_error(c[i:j], v[i:j], expert_values(w, g), gelu) <= 1.0


def test_groups_of_several_blocks():
    counts, N, K = [600, 1, 333, 256], 520, 384
    x, o, od, a = quantized(counts, 6, K)
    w = mx.quantize_experts(weights(24, 4, N, K), 8)
    c = mx.gemm_grouped(a, w, od)
    v = grouped_values(a, o)
    for g, (i, j) in enumerate(zip(o, o[1:])):
        assert gemm_error(c[i:j], v[i:j], expert_values(w, g)) <= 1.0


def test_offsets_outside_the_rows_are_clipped():
    """No offsets make a call leave its matrices; rows inside keep their products."""
    N, K = 256, 256
    x = activations(5, 100, K)
    w8, w0 = (mx.quantize_experts(weights(25, 3, N, K), f) for f in (8, 0))
    od = torch.tensor([-5, 40, 30, 1000], dtype=torch.int32, device="cuda")   # groups [0, 40), none, [30, 100)
    for fa, w in ((6, w8), (0, w0)):
        a = mx.quantize_grouped(x, od, fa)
        big = torch.full((300, N), 4.0, dtype=torch.bfloat16, device="cuda")
        mx.gemm_grouped(a, w, od, out=big[100:200])
        torch.cuda.synchronize()
        mx.check_device_error()
        assert (big[:100] == 4).all() and (big[200:] == 4).all()


def test_graph_follows_its_offsets():
    """A captured call reads the offsets of the replay, not of the capture."""
    N, K = 264, 256
    x = activations(6, 300, K)
    _, od = offsets_of([100, 100, 100])
    for fa, fb in (B, (0, 0), (3, 3)):
        w = mx.quantize_experts(weights(26, 3, N, K), fb)
        od.copy_(torch.tensor([0, 100, 200, 300], dtype=torch.int32))
        a = mx.quantize_grouped(x, od, fa, gscale=gs(fa))
        c = torch.empty(300, N, dtype=torch.bfloat16, device="cuda")
        mx.gemm_grouped(a, w, od, out=c)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx.quantize_grouped(x, od, fa, gscale=gs(fa) if fa != 3 else a.gscale, out=a)
            mx.gemm_grouped(a, w, od, out=c)
        for o in ([0, 1, 299, 300], [0, 0, 130, 290]):
            od.copy_(torch.tensor(o, dtype=torch.int32))
            g.replay()
            torch.cuda.synchronize()
            v = grouped_values(a, o)
            for e, (i, j) in enumerate(zip(o, o[1:])):
                if j > i:
                    assert gemm_error(c[i:j], v[i:j], expert_values(w, e)) <= 1.0


def test_helpers_read_the_layouts():
    """The FP64 readers of the tests agree with the library's dequantize on ungrouped matrices."""
    for fmt in (0, 1, 2, 4):
        x = activations(9, 70, 256)
        t = mx.quantize(x, fmt)
        s = scale_values(sf_at(t.scales, torch.arange(70, device="cuda"), 8), fmt).repeat_interleave(32, 1)
        assert torch.equal((element_values(t.codes, fmt, 70, 256) * s).bfloat16(), mx.dequantize(t))


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    """Groups, widths and depths at random, empty groups and groups of one row among them."""
    g = torch.Generator().manual_seed(seed)

    def r(lo, hi):
        return int(torch.randint(lo, hi + 1, (1,), generator=g))
    fa, fb = PAIRS[seed % len(PAIRS)]
    E, N, K = r(1, 40) if seed % 6 else 300, r(1, 700), 128 * r(1, 9)
    counts = [r(0, 90) * (r(0, 3) > 0) * (1 if r(0, 9) else 6) for _ in range(E)]
    x, o, od, a = quantized(counts, fa, K, behind=r(0, 5), seed=seed)
    w = mx.quantize_experts(weights(seed, E, N, K), fb)
    gelu = seed % 3 == 0
    c = torch.full((a.rows, N), 9.0, dtype=torch.bfloat16, device="cuda")
    mx.gemm_grouped(a, w, od, out=c, epilogue=mx.MX_EPI_GELU if gelu else mx.MX_EPI_NONE)
    torch.cuda.synchronize()
    mx.check_device_error()
    v = grouped_values(a, o)
    for e, (i, j) in enumerate(zip(o, o[1:])):
        if j > i:
            assert gemm_error(c[i:j], v[i:j], expert_values(w, e), gelu) <= 1.0, (E, N, K, e)
    assert (c[o[-1]:] == 9).all()


@pytest.mark.parametrize("fa,fb", [B, (0, 0)])
def test_a_nan_stays_in_its_row_and_column(fa, fb):
    """NaN codes in the rows behind the last group, in another group and in one weight row touch nothing else."""
    counts, N, K = [20, 30], 300, 256
    x, o, od, a = quantized(counts, fa, K, behind=14)
    w = mx.quantize_experts(weights(41, 2, N, K), fb)
    want = mx.gemm_grouped(a, w, od)[:50].clone()
    codes = a.codes.view(-1, K)
    codes[50:] = 0x7F
    codes[25] = 0x7F
    w.codes.view(2, N, K)[1, 7] = 0x7F
    c = mx.gemm_grouped(a, w, od)[:50]
    assert c[25].isnan().all() and c[20:, 7].isnan().all()
    keep = torch.ones(50, N, dtype=torch.bool, device="cuda")
    keep[25] = False
    keep[20:, 7] = False
    assert torch.equal(c[keep], want[keep])


@pytest.mark.parametrize("fa,fb", [(6, 8), (0, 0), (3, 3), (1, 2)])
def test_a_stalled_producer_is_reported(fa, fb):
    """The producer issues nothing: the bounded waits run out, the call ends and is reported, and the next is right."""
    counts, N, K = [40, 0, 9], 300, 2560
    x, o, od, a = quantized(counts, fa, K)
    w = mx.quantize_experts(weights(51, 3, N, K), fb)
    c = mx.gemm_grouped(a, w, od)
    torch.cuda.synchronize()
    assert mx.mx_check_device_error()[0] == mx.MX_OK
    try:
        mx.check(mx.mx_debug_set(mx.MX_DEBUG_WAIT_LIMIT_NS, 50_000_000))
        mx.check(mx.mx_debug_set(mx.MX_DEBUG_SKIP_PRODUCER, 1))
        mx.gemm_grouped(a, w, od)
        status, info = mx.mx_check_device_error()
    finally:
        mx.mx_debug_set(mx.MX_DEBUG_SKIP_PRODUCER, 0)
        mx.mx_debug_set(mx.MX_DEBUG_WAIT_LIMIT_NS, 1_000_000_000)
    assert status == mx.MX_ERR_TIMEOUT and info[0] & 1 and info[3] >= 1
    assert mx.mx_check_device_error()[0] == mx.MX_OK
    assert torch.equal(mx.gemm_grouped(a, w, od), c)
    assert mx.mx_check_device_error()[0] == mx.MX_OK


def scattered(seed, tokens, T, how):
    g = torch.Generator().manual_seed(seed)
    if how == "one":
        idx = torch.full((T,), 3)
    elif how == "outside":
        idx = torch.randint(-tokens, 2 * tokens, (T,), generator=g)
        idx[0], idx[1] = -2 ** 31, 2 ** 31 - 1
    else:
        idx = torch.randint(0, tokens, (T,), generator=g)
    return idx.int().cuda()


@pytest.mark.parametrize("fmt", [6, 0, 1, 2, 3, 4])
@pytest.mark.parametrize("tokens,T,K,how", [(700, 2100, 2048, "random"), (600, 4800, 640, "random"), (300, 1500, 4096, "one"),
                                            (400, 2000, 1536, "outside"), (300, 2400, 1152, "random")])
def test_rows_to_several_places(fmt, tokens, T, K, how):
    """Read once and stored at every place (a workspace given), or gathered place by place: the same bytes."""
    counts = [T // 3, 0, 1, T // 2, 100]
    o, od = offsets_of(counts)
    x = torch.full((tokens, K + 8), 5.0, dtype=torch.bfloat16, device="cuda")[:, :K]
    x.copy_(activations(K, tokens, K))
    idx = scattered(T, tokens, T, how)
    need = mx.mx_quantize_grouped_workspace_bytes(T, tokens, K)
    assert need > 0
    got, want = (mx.empty_grouped(fmt, T, len(counts), K) for _ in range(2))
    for t in (got, want):
        t.codes.fill_(0xA5)
        t.scales.fill_(0x5A)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    for _ in range(2):                                  # a used workspace is as good as a new one
        mx.quantize_grouped(x, od, fmt, row_index=idx, gscale=gs(fmt), out=got, workspace=ws)
    groups = mx.MxGroupsC(len(counts), 0, od.data_ptr())
    g = gs(fmt)
    mx.check(mx.mx_quantize_grouped(fmt, x.data_ptr(), tokens, K, K + 8, idx.data_ptr(), groups, want.c(),
                                    None if g is None else g.data_ptr(), None, 0, mx._stream()))
    assert torch.equal(got.codes, want.codes) and torch.equal(got.scales, want.scales)
    if g is not None:
        assert torch.equal(got.gscale, g)
    # and the codes are those of the rows themselves
    live = idx[:o[-1]].long()
    rows = torch.where(((live >= 0) & (live < tokens))[:, None], x[live.clamp(0, tokens - 1)], 0)
    q = mx.quantize(rows.contiguous(), fmt, gscale=g)
    n = mx.mx_codes_bytes(fmt, o[-1], K)
    assert torch.equal(got.codes[:n], q.codes[:n]) and (got.codes[n:] == 0xA5).all()


def test_rows_to_several_places_in_two_graphs_at_once():
    """Two captured calls have workspaces of their own and run together."""
    T, tokens, K, E = 4096, 1024, 2048, 16
    cases = []
    for seed in (1, 2):
        x = activations(seed, tokens, K)
        ids = torch.randint(0, E, (tokens, 4), generator=torch.Generator().manual_seed(seed)).int().cuda()
        r = mx.route(ids, E)
        want = mx.quantize_grouped(x, r.offsets, 6, row_index=r.row_token)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            got = [mx.quantize_grouped(x, r.offsets, 6, row_index=r.row_token) for _ in range(4)]
        cases.append((s, g, got, want, x, r))
    torch.cuda.synchronize()
    for _ in range(3):
        for s, g, *_ in cases:
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for _, _, got, want, *_ in cases:
        for t in got:
            assert torch.equal(t.codes, want.codes) and torch.equal(t.scales, want.scales)


@pytest.mark.parametrize("fmt", [6, 0, 3])
def test_rows_to_several_places_with_overlapping_offsets(fmt):
    """Offsets that descend enter rows twice: nothing is written outside the buffers, and both ways agree."""
    tokens, T, K = 400, 2000, 1536
    od = torch.tensor([-5, 1600, 800, 10 ** 6], dtype=torch.int32, device="cuda")   # [0, 1600), none, [800, 2000)
    x, idx, g = activations(1, tokens, K), scattered(2, tokens, T, "random"), gs(fmt)
    assert mx.mx_quantize_grouped_workspace_bytes(T, tokens, K) > 0
    codes, scales = mx.mx_codes_bytes(fmt, T, K), mx.mx_grouped_scales_bytes(fmt, T, 3, K)
    got = []
    for ws in (True, False):
        c, s = (torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda") for n in (codes, scales))
        out = mx.MxTensor(fmt, T, K, c, s, None if g is None else torch.empty(1, device="cuda"))
        if ws:
            mx.quantize_grouped(x, od, fmt, row_index=idx, gscale=g, out=out)
        else:
            mx.check(mx.mx_quantize_grouped(fmt, x.data_ptr(), tokens, K, K, idx.data_ptr(), mx.MxGroupsC(3, 0, od.data_ptr()),
                                            out.c(), None if g is None else g.data_ptr(), None, 0, mx._stream()))
        torch.cuda.synchronize()
        assert (c[codes:] == 0x5A).all() and (s[scales:] == 0x5A).all()
        got.append((c, s))
    assert torch.equal(got[0][0], got[1][0])
