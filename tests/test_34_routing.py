"""Route and combine against plain forms, and the experts' operators run together."""
import pytest
import torch

from experts_helpers import activations, expert_values, grouped_values, route_reference, weights
from fp8_quantization_block_b200 import mx

pytestmark = pytest.mark.gpu


def ids_of(seed, tokens, choices, experts, bad=0.0, dtype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, experts, (tokens, choices), generator=g)
    drop = torch.rand(tokens, choices, generator=g) < bad
    return torch.where(drop, torch.where(ids % 2 == 0, -1, experts + ids), ids).to(dtype)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("tokens,choices,experts,bad", [
    (1, 1, 1, 0.0), (1, 8, 64, 0.0), (33, 2, 5, 0.3), (100, 3, 1000, 0.1), (1024, 8, 128, 0.0), (1025, 8, 128, 0.2),
    (5000, 4, 1024, 0.05), (20000, 2, 3, 0.5), (40, 1, 7, 1.0), (3000, 6, 1, 0.0)])
def test_route(tokens, choices, experts, bad, dtype):
    ids = ids_of(tokens + experts, tokens, choices, experts, bad, dtype)
    r = mx.route(ids.cuda(), experts)
    o, t, s = route_reference(ids.tolist(), experts)
    assert r.offsets.tolist() == o
    assert r.row_token.tolist() == t
    assert r.slot.view(-1).tolist() == s


def test_route_of_nothing_and_far_ids():
    r = mx.route(torch.zeros(0, 4, dtype=torch.int32, device="cuda"), 5)
    assert r.offsets.tolist() == [0] * 6 and r.slot.shape == (0, 4)
    r = mx.route(torch.tensor([[2 ** 40, 1], [-2 ** 40, 2 ** 32 + 1]], device="cuda"), 3)
    assert r.offsets.tolist() == [0, 0, 1, 1] and r.slot.tolist() == [[-1, 0], [-1, -1]]


def test_one_expert_twice_in_a_token():
    r = mx.route(torch.tensor([[1, 1], [0, 1]], dtype=torch.int32, device="cuda"), 2)
    assert r.offsets.tolist() == [0, 1, 4] and r.slot.tolist() == [[1, 2], [0, 3]]
    assert r.row_token.tolist() == [1, 0, 0, 1]


def combine_reference(y, slot, w):
    out = torch.zeros(slot.shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    mag = out.clone()
    for j in range(slot.shape[1]):
        s = slot[:, j].long()
        ok = (s >= 0) & (s < y.shape[0])
        v = torch.where(ok[:, None], y.double()[s.clamp(0, y.shape[0] - 1)] * w[:, j, None].double(), 0.0)
        out += v
        mag += v.abs()
    return out, mag


@pytest.mark.parametrize("tokens,choices,cols", [(1, 1, 8), (32, 8, 4096), (7, 3, 1), (50, 9, 100), (64, 2, 2050),
                                                 (200, 17, 264)])
def test_combine(tokens, choices, cols):
    g = torch.Generator().manual_seed(tokens)
    y = activations(tokens, tokens * choices, cols)
    slot = torch.randperm(tokens * choices, generator=g).int().view(tokens, choices).cuda()
    slot[0, 0] = -1
    slot[-1, -1] = tokens * choices            # outside y: dropped too
    w = torch.rand(tokens, choices, generator=g).cuda()
    w[0, 0] = float("nan")                     # a dropped choice's weight is not looked at
    out = mx.combine(y, slot, w)
    ref, mag = combine_reference(y, slot, torch.nan_to_num(w))
    # one bf16 rounding, and `choices` FP32 fmas of half a step each
    bound = 2.0 ** -8 * ref.abs() + (choices + 1) * 2.0 ** -24 * mag + 1e-38
    assert ((out.double() - ref).abs() <= bound).all()


def test_combine_pitches_and_repeated_slots():
    y = activations(1, 20, 48)
    wide = torch.zeros(20, 64, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:51] = y
    slot = torch.tensor([[4, 4], [19, 0]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[0.5, 0.25], [1.0, -1.0]], device="cuda")
    out = torch.full((2, 50), 5.0, dtype=torch.bfloat16, device="cuda")
    mx.combine(wide[:, 3:51], slot, w, out=out[:, 1:49])
    assert torch.equal(out[:, 1:49], mx.combine(y, slot, w))
    assert (out[:, 0] == 5).all() and (out[:, 49] == 5).all()


def test_combine_of_no_rows_is_zero():
    y = torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    slot = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    assert (mx.combine(y, slot, torch.ones(3, 2, device="cuda")) == 0).all()


def experts_case(fa, fb, tokens=70, choices=3, experts=6, K=256, N=512):
    x = activations(1, tokens, K)
    ids = ids_of(2, tokens, choices, experts, 0.1).cuda()
    ids[-5:] = -1                              # a batch padded at its end
    p = torch.softmax(torch.randn(tokens, choices, generator=torch.Generator().manual_seed(4)), 1).cuda()
    W1 = mx.quantize_experts(weights(5, experts, N, K), fb)
    W2 = mx.quantize_experts(weights(6, experts, K, N), fb)
    return x, ids, p, W1, W2


@pytest.mark.parametrize("fa,fb", [(6, 8), (0, 0), (0, 2), (3, 3), (2, 2)])
def test_experts_mlp_is_its_steps(fa, fb):
    """The path as a user runs it, each step checked against FP64 on the step's own inputs, and every token's result
    against the experts' products of that token alone."""
    x, ids, p, W1, W2 = experts_case(fa, fb)
    g1 = torch.tensor([0.02], device="cuda") if fa == 3 else None
    g2 = torch.tensor([0.01], device="cuda") if fa == 3 else None
    out = mx.experts_mlp(x, ids, p, W1, W2, x_gscale=g1, h_gscale=g2, act_fmt=fa)
    torch.cuda.synchronize()
    mx.check_device_error()
    r = mx.route(ids, 6)
    o = r.offsets.tolist()
    a = mx.quantize_grouped(x, r.offsets, fa, row_index=r.row_token, gscale=g1)
    h = mx.gemm_grouped(a, W1, r.offsets, epilogue=mx.MX_EPI_GELU)
    b = mx.quantize_grouped(h, r.offsets, fa, gscale=g2)
    y = mx.gemm_grouped(b, W2, r.offsets)
    av, bv = grouped_values(a, o), grouped_values(b, o)
    href, yref = torch.zeros(a.rows, W1.rows, dtype=torch.float64, device="cuda"), None
    yref = torch.zeros(a.rows, W2.rows, dtype=torch.float64, device="cuda")
    ymag = yref.clone()
    for e, (i, j) in enumerate(zip(o, o[1:])):
        pre = av[i:j] @ expert_values(W1, e).t()
        href[i:j] = pre * torch.special.ndtr(pre)
        w2 = expert_values(W2, e)
        yref[i:j], ymag[i:j] = bv[i:j] @ w2.t(), bv[i:j].abs() @ w2.abs().t()
    live = o[-1]
    assert ((h[:live].double() - href[:live]).abs() <= 2.0 ** -7 * href[:live].abs() + 2e-3).all()
    assert ((y[:live].double() - yref[:live]).abs() <= 2.0 ** -8 * yref[:live].abs() + 1e-4 * ymag[:live]).all()
    ref, mag = combine_reference(y, r.slot, p)
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 4 * 2.0 ** -24 * mag + 1e-38).all()
    assert (out[-5:] == 0).all()


def test_experts_mlp_in_a_graph_and_on_a_stream():
    x, ids, p, W1, W2 = experts_case(6, 8)
    want = mx.experts_mlp(x, ids, p, W1, W2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = mx.experts_mlp(x, ids, p, W1, W2)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = mx.experts_mlp(x, ids, p, W1, W2)
    x2, ids2 = activations(77, *x.shape), ids.roll(3, 0)
    want2 = mx.experts_mlp(x2, ids2, p, W1, W2)
    x.copy_(x2)
    ids.copy_(ids2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want2)


def test_a_named_stream_owns_what_the_call_allocates():
    """The call's own tensors belong to the named stream: what is allocated and written right after it on the current
    stream does not touch them."""
    x, ids, p, W1, W2 = experts_case(6, 8, tokens=2000, choices=4, N=1024)
    want = mx.experts_mlp(x, ids, p, W1, W2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        got = mx.experts_mlp(x, ids, p, W1, W2, stream=s)
        junk = [torch.full((1 << 20,), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(40)]
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del junk
    ids2 = torch.randint(0, 9, (3000, 8), device="cuda")
    a, b = mx.route(ids2, 9), mx.route(ids2, 9, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.slot, b.slot) and torch.equal(a.row_token, b.row_token)


@pytest.mark.parametrize("n,experts", [(600_000, 40), (300_000, 1024), (262_145, 2)])
def test_route_of_many_choices(n, experts):
    """Over 128 chunks' worth: larger chunks."""
    ids = torch.randint(-1, experts + 1, (n, 1), generator=torch.Generator().manual_seed(n)).int()
    r = mx.route(ids.cuda(), experts)
    flat = ids.view(-1)
    ok = (flat >= 0) & (flat < experts)
    order = torch.argsort(torch.where(ok, flat, experts), stable=True)[:int(ok.sum())]
    slot = torch.full((n,), -1, dtype=torch.int32)
    slot[order] = torch.arange(order.numel(), dtype=torch.int32)
    assert torch.equal(r.slot.view(-1).cpu(), slot)
    assert torch.equal(r.row_token[:order.numel()].cpu(), order.int()) and (r.row_token[order.numel():] == -1).all()
    assert torch.equal(r.offsets.cpu(), torch.nn.functional.pad(
        torch.bincount(flat[ok], minlength=experts).cumsum(0), (1, 0)).int())


def test_offsets_past_32_bits():
    """Rows whose element offset needs 64 bits: the gather's source, combine's rows, the product's output."""
    rows, cols = 540_000, 4096                       # 2.2 G elements
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    tail = activations(3, 40, cols)
    y[-40:] = tail
    slot = torch.arange(rows - 40, rows, dtype=torch.int32, device="cuda").view(20, 2)
    w = torch.rand(20, 2, generator=torch.Generator().manual_seed(1)).cuda()
    near = torch.arange(40, dtype=torch.int32, device="cuda").view(20, 2)
    assert torch.equal(mx.combine(y, slot, w), mx.combine(tail, near, w))
    off = torch.tensor([0, 25, 40], dtype=torch.int32, device="cuda")
    for fmt in (6, 0):
        a = mx.quantize_grouped(y, off, fmt, row_index=slot.view(-1))
        b = mx.quantize_grouped(tail, off, fmt, row_index=near.view(-1))
        assert torch.equal(a.codes, b.codes)
    del y
    M, N = 34_000, 65_536                            # 2.2 G elements of output
    a = mx.quantize(activations(4, M, 128), 6)
    b = mx.quantize(weights(5, N, 128), 8)
    c = mx.gemm(a, b)
    last = mx.MxTensor(6, 100, 128, a.codes[(M - 100) * 128:], a.scales.view(torch.float32)[M - 100:M].contiguous(), None)
    assert torch.equal(c[-100:], mx.gemm(last, b))
