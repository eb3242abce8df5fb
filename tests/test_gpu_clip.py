"""lora_clip_gradients against its definition in 64 bits (GPU)."""
import math

import pytest
import torch

import expand_gemm_gb300 as eg

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def expected(grads, groups, max_norm, eps):
    total = sum(g.double().reshape(groups, -1).square().sum(1) for g in grads)
    norms = total.sqrt()
    f = (max_norm / (norms + eps)).clamp(max=1.0)
    return norms, [(g.double().reshape(groups, -1) * f[:, None]).reshape(g.shape) for g in grads]


def check(grads, groups, max_norm, eps=1e-6, out=False, norms=None):
    want_norms, want = expected(grads, groups, max_norm, eps)
    got = [torch.full_like(g, 5.0) for g in grads] if out else [g.clone() for g in grads]
    norms = torch.empty(groups, device="cuda") if norms is None else norms
    if out:
        keep = [g.clone() for g in grads]
        eg.lora_clip_gradients(eg.LoRAGradients.make(grads, groups, out=got), max_norm, norms, eps=eps)
        assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    else:
        eg.lora_clip_gradients(got, max_norm, norms, eps=eps)
    # a unit's partial sum of at most 33 squares is fp32, the rest fp64; the root halves the
    # error, the norm is rounded once more
    # (beyond 3.4e38, the largest fp32, to infinity)
    assert bool((((norms.double() - want_norms).abs() <= 20 * 2.0 ** -24 * want_norms)
                 | (torch.isinf(norms) & torch.isinf(want_norms.float()))).all())
    for g, w in zip(got, want):
        step = 2.0 ** -8 if g.dtype is BF16 else 2.0 ** -24
        # the factor is that of the norm above, and rounded once
        limit = w.abs() * (step + 22 * 2.0 ** -24) + (2.0 ** -134 if g.dtype is BF16 else 2.0 ** -150)
        assert bool(((g.double() - w).abs() <= limit).all())
    return norms, got


def tensors(shapes, dtypes, seed=0, std=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(s, generator=g) * std).to("cuda", d) for s, d in zip(shapes, dtypes)]


@pytest.mark.parametrize("out", [False, True])
@pytest.mark.parametrize("groups, shapes, dtypes", [
    (1, [(1,)], [F32]), (1, [(1,)], [BF16]), (1, [(5, 7)], [BF16]), (1, [()], [F32]),
    (1, [(16385,), (3,), (16384,)], [BF16, F32, BF16]), (3, [(3, 5, 7), (3, 1), (3, 40, 8)], [BF16, F32, BF16]),
    (8, [(8, 16, 512), (8, 512, 16)] * 3, [BF16] * 6), (2, [(2, 100003), (2, 9)], [F32, BF16]),
    (64, [(64, 8, 33), (64, 33, 8)], [BF16, F32]), (1, [(4, 300, 301)] * 2, [F32, BF16]),
    (700, [(700, 3)], [F32]), (1024, [(1024, 24), (1024, 1)], [BF16, BF16])], ids=str)
def test_norms_and_gradients(groups, shapes, dtypes, out):
    grads = tensors(shapes, dtypes)
    usual = 1e-2 * math.sqrt(sum(g.numel() for g in grads) / groups)
    for max_norm in (0.3 * usual, usual, 30 * usual):
        check(grads, groups, max_norm, out=out)


@pytest.mark.parametrize("count", [2, 64, 65, 1024, 1025, 2300])
def test_many_tensors(count):
    shapes = [(2, 3 + i % 5, 8 if i % 3 else 7) for i in range(count)]
    grads = tensors(shapes, [BF16 if i % 2 else F32 for i in range(count)], std=1.0)
    check(grads, 2, 1.5)
    check(grads, 1, 1.5)


@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_tensors_off_a_16_byte_boundary(offset, dtype):
    """Slices in the middle of a larger buffer, in place and to another alignment."""
    store = torch.randn(120000, device="cuda").to(dtype)
    before = store.clone()

    def parts(t):
        return [t[offset:offset + 2 * 17001].view(2, 17001), t[50001:50001 + 2 * 11].view(2, 11)]
    want_norms, want = expected(parts(before), 2, 2.0, 1e-6)
    step = (2.0 ** -8 if dtype is BF16 else 2.0 ** -24) + 22 * 2.0 ** -24
    norms = torch.empty(2, device="cuda")
    eg.lora_clip_gradients(parts(store), 2.0, norms)
    assert bool(((norms.double() - want_norms).abs() <= 20 * 2.0 ** -24 * want_norms).all())
    for g, w in zip(parts(store), want):
        assert bool(((g.double() - w).abs() <= step * w.abs()).all())
    touched = torch.zeros_like(store, dtype=torch.bool)
    for t in parts(touched):
        t.fill_(True)
    assert torch.equal(store[~touched], before[~touched])
    out = torch.zeros(40000, dtype=dtype, device="cuda")
    o = [out[:2 * 17001].view(2, 17001), out[34003:34003 + 22].view(2, 11)]
    eg.lora_clip_gradients(eg.LoRAGradients.make(parts(before), 2, out=o), 2.0, norms)
    for g, w in zip(o, want):
        assert bool(((g.double() - w).abs() <= step * w.abs()).all())
    assert not bool(out[34002]) and not bool(out[34025:].any())


def test_gradients_below_the_limit_are_left_as_they_are():
    grads = tensors([(2, 1000), (2, 31)], [BF16, F32])
    keep = [g.clone() for g in grads]
    norms = torch.empty(2, device="cuda")
    eg.lora_clip_gradients(grads, 1e6, norms)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    eg.lora_clip_gradients(grads, None, norms)
    assert all(torch.equal(a, b) for a, b in zip(grads, keep))
    assert bool((norms > 0).all())


def test_zero_gradients():
    grads = [torch.zeros(3, 50, device="cuda"), torch.zeros(3, 8, device="cuda").bfloat16()]
    norms = torch.ones(3, device="cuda")
    for max_norm, eps in ((1.0, 1e-6), (0.0, 1e-6), (0.0, 0.0), (1.0, 0.0)):
        eg.lora_clip_gradients(grads, max_norm, norms, eps=eps)
        assert not bool(norms.any()) and not any(bool(g.any()) for g in grads)


def test_empty_tensors():
    grads = [torch.zeros(3, 0, device="cuda"), torch.ones(3, 4, device="cuda"), torch.zeros(3, 0, 5, device="cuda").bfloat16()]
    norms = torch.zeros(3, device="cuda")
    eg.lora_clip_gradients(grads, 1.0, norms, eps=0.0)
    assert torch.equal(norms, torch.full((3,), 2.0, device="cuda"))
    assert torch.equal(grads[1], torch.full((3, 4), 0.5, device="cuda"))
    eg.lora_clip_gradients([grads[0]], 1.0, norms)
    assert not bool(norms.any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e-40, 1e-38, 1e-30, 1e-24, 1e-15, 1e15, 1e19, 1e25, 1e37])
def test_sizes_whose_squares_leave_32_bits(size, dtype):
    g = torch.Generator().manual_seed(1)
    v = torch.rand(2, 20001, generator=g) + 0.5
    v[1] *= 0.125
    grads = [(v * size).to("cuda", dtype)]
    norms, _ = check(grads, 2, float(torch.tensor(size).float()), eps=0.0)
    # 1e-40 in bf16: the second row (at most 1.9e-41) rounds to zeros, the smallest number being 9.2e-41
    assert torch.equal(norms > 0, grads[0].any(1))


def test_large_and_small_values_together():
    v = torch.full((1, 5000), 1e-30, device="cuda")
    v[0, 17], v[0, 4000] = 3e30, 1.0
    norms, got = check([v], 1, 1.0)
    assert float(norms[0]) == float(torch.tensor(3e30).float())


def test_a_norm_beyond_32_bits_still_scales():
    grads = [torch.full((1, 4096), 3e38, device="cuda")]
    norms = torch.empty(1, device="cuda")
    eg.lora_clip_gradients(grads, 64.0, norms, eps=0.0)
    assert math.isinf(float(norms[0]))                      # 64 x 3e38
    assert bool(((grads[0] - 1.0).abs() <= 8 * 2.0 ** -24).all())   # the factor is subnormal


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_and_infinity_stay_in_their_adapter(dtype):
    grads = [t.to(dtype) for t in tensors([(4, 3000), (4, 5, 7)], [F32, F32], std=1.0)]
    clean = [g.clone() for g in grads]
    norms = torch.empty(4, device="cuda")
    eg.lora_clip_gradients(clean, 1.0, norms)
    before = norms.clone()
    grads[1][1, 2, 3] = float("nan")
    grads[0][3, 2999] = float("-inf")
    eg.lora_clip_gradients(grads, 1.0, norms)
    assert math.isnan(float(norms[1])) and math.isinf(float(norms[3]))
    assert torch.equal(norms[0::2], before[0::2])
    for g, c in zip(grads, clean):
        assert torch.equal(g[0], c[0]) and torch.equal(g[2], c[2])
        assert bool(torch.isnan(g[1]).all())
    assert not bool(grads[1][3].any()) and int(torch.isnan(grads[0][3]).sum()) == 1


def test_nan_among_zeros_shows():
    g = torch.zeros(1, 64, device="cuda")
    g[0, 9] = float("nan")
    norms = torch.empty(1, device="cuda")
    eg.lora_clip_gradients([g], 1.0, norms)
    assert math.isnan(float(norms[0])) and bool(torch.isnan(g).all())


def test_offsets_beyond_32_bits():
    """A stack of more than 2^31 elements; its last slice and element are reached."""
    g = torch.zeros(3, (1 << 30) + 5, dtype=BF16, device="cuda")
    g[2, -1] = 4.0
    g[1, 0] = 3.0
    norms = torch.empty(3, device="cuda")
    eg.lora_clip_gradients([g], 1.0, norms, eps=0.0)
    assert norms.tolist() == [0.0, 3.0, 4.0]
    assert float(g[2, -1]) == 1.0 and float(g[1, 0]) == 1.0
    assert int(torch.count_nonzero(g)) == 2


def test_equal_calls_give_equal_bits_and_a_graph_replays():
    grads = tensors([(5, 4097, 3), (5, 33)], [BF16, F32], std=1.0)
    out = [torch.empty_like(g) for g in grads]
    norms = torch.empty(5, device="cuda")
    handle = eg.LoRAGradients.make(grads, 5, out=out)
    eg.lora_clip_gradients(handle, 2.0, norms)
    first = [norms.clone()] + [o.clone() for o in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.lora_clip_gradients(handle, 2.0, norms)
    for _ in range(2):
        for t in [norms] + out:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip([norms] + out, first))
    for g in grads:
        g.mul_(0.5)
    graph.replay()
    want = expected(grads, 5, 2.0, 1e-6)[0]
    assert bool(((norms.double() - want).abs() <= 20 * 2.0 ** -24 * want).all())


def test_missing_gradients_are_skipped():
    grads = tensors([(2, 10), (2, 20)], [BF16, BF16], std=1.0)
    norms = torch.empty(2, device="cuda")
    want = expected(grads, 2, 1.0, 1e-6)[0]
    eg.lora_clip_gradients([None, grads[0], None, grads[1]], 1.0, norms)
    assert bool(((norms.double() - want).abs() <= 20 * 2.0 ** -24 * want).all())


def test_refusals():
    a = torch.zeros(2, 8, device="cuda")
    norms = torch.zeros(2, device="cuda")
    for bad, error in (([a.half()], TypeError), ([a.cpu()], ValueError), ([a.t()], ValueError), ([torch.zeros(3, 8, device="cuda")], ValueError),
                       ([], ValueError), ([None], ValueError), ([3.0], TypeError)):
        with pytest.raises(error):
            eg.lora_clip_gradients(bad, 1.0, norms)
    for kw in (dict(out=[a.bfloat16()]), dict(out=[]), dict(out=[None]), dict(out=[a[:, :4]])):
        with pytest.raises((TypeError, ValueError)):
            eg.LoRAGradients.make([a], 2, **kw)
    with pytest.raises(ValueError):
        eg.lora_clip_gradients([a], -1.0, norms)
    with pytest.raises(ValueError):
        eg.lora_clip_gradients([a], float("nan"), norms)
    with pytest.raises((TypeError, ValueError)):
        eg.lora_clip_gradients([a], 1.0, norms.double())
    with pytest.raises(ValueError):
        eg.lora_clip_gradients(eg.LoRAGradients.make([a], 2), 1.0, torch.zeros(3, device="cuda"))


def test_overlapping_tensors_are_refused():
    flat, other = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    norms = torch.zeros(1, device="cuda")
    for bad in ([flat[:20], flat[19:40]], [flat, flat], [flat[:32], flat[8:16]]):
        with pytest.raises(ValueError, match="overlaps"):
            eg.lora_clip_gradients(bad, 1.0, norms)
    for grads, out in (([flat[:16]], [flat[8:24]]), ([flat[:16], flat[16:32]], [other[:16], other[8:24]]),
                       ([flat[:16], flat[16:32]], [flat[16:32], other[:16]])):
        with pytest.raises(ValueError, match="overlaps"):
            eg.LoRAGradients.make(grads, 1, out=out)
    # read by two, written by none, and one's own place
    eg.LoRAGradients.make([flat[:16], flat[8:24]], 1, out=[other[:16], other[16:32]])
    eg.LoRAGradients.make([flat[:16], flat[16:32]], 1, out=[flat[:16], other[:16]])
