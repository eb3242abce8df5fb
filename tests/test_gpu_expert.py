"""lora_expert_linear and lora_expert_linear_backward against their
definitions in 64 bits (GPU)."""
import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref

pytestmark = pytest.mark.gpu

# tokens, fan out, experts, hidden, width, share of rows without an expert
SIZES = [
    (1, 1, 1, 8, 1, 0.0), (1, 2, 8, 64, 64, 0.0), (1, 4, 4, 4096, 129, 0.0), (2, 1, 2, 72, 33, 0.0),
    (7, 3, 5, 1000, 523, 0.3), (16, 2, 4, 256, 256, 0.0), (33, 1, 3, 40, 130, 0.5), (64, 2, 8, 512, 200, 0.1),
    (65, 1, 1, 96, 257, 0.0), (129, 2, 16, 128, 64, 0.2), (256, 1, 1, 320, 384, 0.0), (257, 4, 7, 200, 75, 0.1),
    (700, 1, 2, 136, 520, 0.0), (1500, 2, 3, 64, 40, 0.4), (40, 8, 64, 32, 96, 0.0), (3, 2, 1000, 64, 24, 0.0),
]
FOUR = [s for s in SIZES if s[3] % 32 == 0] + [(5, 1, 2, 4096, 65, 0.0), (300, 2, 5, 96, 203, 0.2)]


def inputs(tokens, fan, experts, hidden, width, none, four=False, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(seed + tokens * 31 + width)
    rows = tokens * fan
    ids = torch.randint(0, experts, (rows,), generator=g, dtype=torch.int32)
    ids[torch.rand(rows, generator=g) < none] = -1
    x = torch.randn(tokens, hidden, generator=g).bfloat16()
    w = (torch.randn(experts, width, hidden, generator=g) * hidden ** -0.5).bfloat16()
    dy = torch.randn(rows, width, generator=g).bfloat16()
    ids, x, w, dy = (t.to(device) for t in (ids, x, w, dy))
    if not four:
        return ids, x, (w, None), w, dy
    codes, scales = ref.encode(w)
    return ids, x, (codes, scales), ref.decode(codes, scales), dy


def meta_of(ids, experts):
    meta = eg.LoRAKernelMeta.make(experts, max(1, len(ids)), ids.device)
    meta.prepare_tensors(ids)
    return meta


def check_forward(size, four, add=False, seed=0):
    ids, x, (w, scale), values, _ = inputs(*size, four=four, seed=seed)
    meta = meta_of(ids, size[2])
    y = torch.randn(len(ids), size[4], device="cuda").bfloat16()
    was = y.clone()
    eg.lora_expert_linear(x, w, y, meta, weight_scale=scale, add_inputs=add)
    want, sums = ref.forward(x, values, ids, size[1])
    has = (ids >= 0)[:, None]
    assert torch.equal(torch.where(has, torch.zeros_like(y), y), torch.where(has, torch.zeros_like(y), was))
    if add:
        want, sums = want + was.double(), sums + was.double().abs()
    want = torch.where(has, want, was.double())
    ref.within(y, want, torch.where(has, ref.bound(want, sums, size[3] + 1), torch.zeros_like(want)), "y")
    assert int(meta.error_word) == 0


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("add", [False, True])
def test_forward(size, add):
    check_forward(size, False, add)


@pytest.mark.parametrize("size", FOUR, ids=str)
@pytest.mark.parametrize("add", [False, True])
def test_forward_of_weights_in_4_bits(size, add):
    check_forward(size, True, add)


def check_backward(size, four, add=False, want_dx=True, want_dw=True):
    tokens, fan, experts, hidden, width, _ = size
    ids, x, (w, scale), values, dy = inputs(*size, four=four)
    meta = meta_of(ids, experts)
    dx = torch.randn(tokens, hidden, device="cuda").bfloat16()
    was = dx.clone()
    dw = torch.full((experts, width, hidden), 7.0, device="cuda").bfloat16()
    eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=dx if want_dx else None, add_inputs=add,
                                   d_weight=dw if want_dw else None)
    rx, rw, sx, sw = ref.backward(dy, x, values, ids, fan)
    if want_dx:
        if add:
            rx, sx = rx + was.double(), sx + was.double().abs()
        none = (ids.view(tokens, fan) < 0).all(1)
        if add:
            assert torch.equal(dx[none], was[none])
        else:
            assert not bool(dx[none].any())
        ref.within(dx, rx, ref.bound(rx, sx, width + fan + 1), "dx")
    if want_dw:
        count = torch.stack([(ids == e).sum() for e in range(experts)])
        ref.within(dw, rw, ref.bound(rw, sw, count.double()[:, None, None] + 1), "dw")
        assert not bool(dw[count == 0].any())
    assert int(meta.error_word) == 0


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("add", [False, True])
def test_backward(size, add):
    check_backward(size, False, add)


@pytest.mark.parametrize("size", FOUR[::2], ids=str)
def test_backward_of_weights_in_4_bits(size):
    check_backward(size, True)


@pytest.mark.parametrize("size", [SIZES[4], SIZES[11]], ids=str)
@pytest.mark.parametrize("dx, dw", [(True, False), (False, True), (False, False)])
def test_backward_of_one_output(size, dx, dw):
    check_backward(size, False, want_dx=dx, want_dw=dw)


@pytest.mark.parametrize("four", [False, True])
def test_no_row_has_an_expert(four):
    ids, x, (w, scale), _, dy = inputs(6, 2, 3, 64, 48, 0.0, four=four)
    ids.fill_(-1)
    meta = meta_of(ids, 3)
    y = torch.randn(12, 48, device="cuda").bfloat16()
    was = y.clone()
    eg.lora_expert_linear(x, w, y, meta, weight_scale=scale)
    assert torch.equal(y, was)
    dx, dw = torch.ones_like(x), torch.ones((3, 48, 64), device="cuda").bfloat16()
    eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=dx, d_weight=dw)
    assert not bool(dx.any()) and not bool(dw.any())
    one = torch.ones_like(x)
    eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=one, add_inputs=True)
    assert torch.equal(one, torch.ones_like(x))
    # one row a token: cleared by another kernel
    x1 = torch.randn(12, 64, device="cuda").bfloat16()
    dx1 = torch.ones_like(x1)
    eg.lora_expert_linear_backward(dy, x1, w, meta, weight_scale=scale, dx=dx1)
    assert not bool(dx1.any())


def test_no_rows_at_all():
    meta = eg.LoRAKernelMeta.make(3, 4, "cuda")
    meta.prepare_tensors(torch.empty(0, dtype=torch.int32, device="cuda"))
    x, y = torch.empty(0, 64, device="cuda").bfloat16(), torch.empty(0, 48, device="cuda").bfloat16()
    w = torch.randn(3, 48, 64, device="cuda").bfloat16()
    eg.lora_expert_linear(x, w, y, meta)
    dw = torch.ones_like(w)
    eg.lora_expert_linear_backward(y, x, w, meta, dx=torch.empty_like(x), d_weight=dw)
    assert not bool(dw.any())


def test_ids_out_of_range_are_rows_without_an_expert():
    ids, x, (w, _), _, dy = inputs(30, 2, 4, 64, 40, 0.0)
    bad = ids.clone()
    bad[::7] = 4
    bad[3::11] = -5
    meta = meta_of(bad, 4)
    count = int(((bad < -1) | (bad > 3)).sum())
    assert int(meta.error_word) == count
    none = torch.where((bad < 0) | (bad > 3), torch.full_like(bad, -1), bad)
    y = torch.zeros(60, 40, device="cuda").bfloat16()
    eg.lora_expert_linear(x, w, y, meta)
    want, sums = ref.forward(x, w, none, 2)
    ref.within(y, want, ref.bound(want, sums, 64), "y")
    dx = torch.ones_like(x)
    eg.lora_expert_linear_backward(dy, x, w, meta, dx=dx)
    rx, _, sx, _ = ref.backward(dy, x, w, none, 2)
    ref.within(dx, rx, ref.bound(rx, sx, 42), "dx")


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("tokens", [5, 300])
def test_values_of_others_stay_out(bad, tokens):
    """NaN and infinities in the weights of experts without rows, in rows without an
    expert and in the neighbours of the last rows and columns."""
    fan, experts, hidden, width = 2, 5, 72, 43
    ids, x, _, w, dy = inputs(tokens, fan, experts, hidden, width, 0.3)
    ids[ids == 2] = 1
    ids[:2] = -1                                            # token 0 has no expert
    w, x, dy = w.clone(), x.clone(), dy.clone()
    w[2] = bad
    x[0] = bad
    dy[ids < 0] = bad
    wide = torch.full((tokens, hidden + 8), bad, device="cuda").bfloat16()
    wide[:, :hidden] = x
    dwide = torch.full((tokens * fan, width + 5), bad, device="cuda").bfloat16()
    dwide[:, :width] = dy
    meta = meta_of(ids, experts)
    y = torch.zeros(tokens * fan, width, device="cuda").bfloat16()
    eg.lora_expert_linear(wide[:, :hidden], w, y, meta)
    clean = [torch.nan_to_num(t.float(), 0.0, 0.0, 0.0).bfloat16() for t in (x, w, dy)]
    want, sums = ref.forward(clean[0], clean[1], ids, fan)
    ref.within(y, want, ref.bound(want, sums, hidden), "y")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    eg.lora_expert_linear_backward(dwide[:, :width], wide[:, :hidden], w, meta, dx=dx, d_weight=dw)
    rx, rw, sx, sw = ref.backward(clean[2], clean[0], clean[1], ids, fan)
    ref.within(dx, rx, ref.bound(rx, sx, width + fan), "dx")
    ref.within(dw, rw, ref.bound(rw, sw, tokens * fan), "dw")


def test_nan_and_infinity_of_ones_own_show():
    ids, x, _, w, dy = inputs(20, 1, 2, 64, 40, 0.0)
    ids[:] = torch.arange(20, device="cuda") % 2
    meta = meta_of(ids, 2)
    x = x.clone()
    x[3, 5] = float("nan")
    w = w.clone()
    w[0, 7, 0] = float("inf")
    y = torch.zeros(20, 40, device="cuda").bfloat16()
    eg.lora_expert_linear(x, w, y, meta)
    want = ref.forward(x, w, ids, 1)[0]
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.isinf(y), torch.isinf(want))
    assert bool(torch.isnan(y[3]).all()) and bool(torch.isinf(y[0::2, 7]).all())


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("offset, pad", [(0, 8), (1, 3), (4, 4), (8, 1)])
def test_strides_and_alignments(offset, pad, four):
    tokens, fan, experts, hidden, width = 70, 2, 3, 96, 88
    ids, x, (w, scale), values, dy = inputs(tokens, fan, experts, hidden, width, 0.1, four=four)
    meta = meta_of(ids, experts)

    def spread(t, fill=9.0):
        flat = torch.full((t.shape[0] * (t.shape[1] + pad) + offset,), fill, device="cuda").bfloat16()
        v = flat[offset:].view(t.shape[0], -1)[:, :t.shape[1]]
        v.copy_(t)
        return flat, v
    y0 = torch.randn(tokens * fan, width, device="cuda").bfloat16()
    flat, y = spread(y0)
    whole = flat.clone()
    xs, dys = spread(x)[1], spread(dy)[1]
    for add in (False, True):
        y.copy_(y0)
        eg.lora_expert_linear(xs, w, y, meta, weight_scale=scale, add_inputs=add)
        want, sums = ref.forward(x, values, ids, fan)
        has = (ids >= 0)[:, None]
        base = y0.double() * (1.0 if add else 0.0)
        want = torch.where(has, want + base, y0.double())
        ref.within(y, want, torch.where(has, ref.bound(want, sums + base.abs(), hidden + 1), torch.zeros_like(want)), "y")
    y.copy_(y0)
    assert torch.equal(flat, whole)                         # nothing between the rows
    flat, dx = spread(torch.zeros_like(x))
    between = flat.clone()
    dw = torch.empty((experts, width, hidden), device="cuda").bfloat16()
    eg.lora_expert_linear_backward(dys, xs, w, meta, weight_scale=scale, dx=dx, d_weight=dw)
    rx, rw, sx, sw = ref.backward(dy, x, values, ids, fan)
    ref.within(dx, rx, ref.bound(rx, sx, width + fan), "dx")
    ref.within(dw, rw, ref.bound(rw, sw, tokens * fan), "dw")
    dx.zero_()
    assert torch.equal(flat, between)


def test_gradients_by_differences():
    """The gradient of a weighted sum of y, against differences of that sum in 64 bits."""
    tokens, fan, experts, hidden, width = 9, 2, 3, 16, 24
    ids, x, _, w, dy = inputs(tokens, fan, experts, hidden, width, 0.2)
    meta = meta_of(ids, experts)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    eg.lora_expert_linear_backward(dy, x, w, meta, dx=dx, d_weight=dw)

    def total(x, w):
        return float((ref.forward(x, w, ids, fan)[0] * dy.double()).sum())
    for (t, c) in ((0, 0), (3, 7), (8, 15)):
        up, down = x.double(), x.double()
        up[t, c] += 0.5
        down[t, c] -= 0.5
        got = total(up, w.double()) - total(down, w.double())   # linear: exact but for roundings
        assert abs(got - float(dx[t, c])) <= 2.0 ** -8 * abs(got) + 1e-4
    for (e, n, c) in ((0, 0, 0), (1, 23, 5), (2, 11, 15)):
        up, down = w.double(), w.double()
        up[e, n, c] += 0.5
        down[e, n, c] -= 0.5
        got = total(x.double(), up) - total(x.double(), down)
        assert abs(got - float(dw[e, n, c])) <= 2.0 ** -8 * abs(got) + 1e-4


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens", [4, 500])
def test_equal_calls_give_equal_bits(tokens, four):
    ids, x, (w, scale), _, dy = inputs(tokens, 2, 6, 128, 200, 0.1, four=four)
    meta = meta_of(ids, 6)
    outs = []
    for _ in range(3):
        y = torch.zeros(tokens * 2, 200, device="cuda").bfloat16()
        dx, dw = torch.empty_like(x), torch.empty((6, 200, 128), device="cuda").bfloat16()
        eg.lora_expert_linear(x, w, y, meta, weight_scale=scale)
        eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=dx, d_weight=dw)
        outs.append((y, dx, dw))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("tokens", [4, 300])
def test_captured_and_replayed_with_other_inputs(tokens, four):
    size = (tokens, 2, 5, 96, 72, 0.2)
    ids, x, (w, scale), values, dy = inputs(*size, four=four)
    meta = eg.LoRAKernelMeta.make(5, tokens * 2, "cuda")
    y = torch.zeros(tokens * 2, 72, device="cuda").bfloat16()
    dx, dw = torch.empty_like(x), torch.empty((5, 72, 96), device="cuda").bfloat16()
    ws = [torch.empty(eg.lora_expert_linear_workspace(tokens * 2, 96, 72, 5, quantized=four), dtype=torch.uint8,
                      device="cuda"),
          torch.empty(eg.lora_expert_linear_backward_workspace(tokens * 2, 96, 72, 5, fan_out=2, weight_grad=True,
                                                               quantized=four), dtype=torch.uint8, device="cuda")]

    def step():
        meta.prepare_tensors(ids)
        eg.lora_expert_linear(x, w, y, meta, weight_scale=scale, workspace=ws[0])
        eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=dx, d_weight=dw, workspace=ws[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        other = inputs(*size, seed=seed)
        ids.copy_(other[0])
        if seed == 2:
            ids.fill_(-1)
        x.copy_(other[1])
        dy.copy_(other[4])
        y.zero_()
        graph.replay()
        want, sums = ref.forward(x, values, ids, 2)
        ref.within(y, want, ref.bound(want, sums, 96), "y")
        rx, rw, sx, sw = ref.backward(dy, x, values, ids, 2)
        ref.within(dx, rx, ref.bound(rx, sx, 74), "dx")
        ref.within(dw, rw, ref.bound(rw, sw, tokens * 2), "dw")


def test_on_a_stream_of_ones_own():
    ids, x, _, w, _ = inputs(200, 1, 4, 128, 96, 0.0)
    y = torch.zeros(200, 96, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        meta = meta_of(ids, 4)
        eg.lora_expert_linear(x, w, y, meta)
    side.synchronize()
    want, sums = ref.forward(x, w, ids, 1)
    ref.within(y, want, ref.bound(want, sums, 128), "y")


def test_workspaces_end_where_they_say():
    for four in (False, True):
        for tokens in (3, 300):
            ids, x, (w, scale), _, dy = inputs(tokens, 2, 5, 96, 75, 0.1, four=four)
            meta = meta_of(ids, 5)
            y = torch.zeros(tokens * 2, 75, device="cuda").bfloat16()
            dx, dw = torch.empty_like(x), torch.empty((5, 75, 96), device="cuda").bfloat16()
            for need, call in (
                    (eg.lora_expert_linear_workspace(tokens * 2, 96, 75, 5, quantized=four),
                     lambda ws: eg.lora_expert_linear(x, w, y, meta, weight_scale=scale, workspace=ws)),
                    (eg.lora_expert_linear_backward_workspace(tokens * 2, 96, 75, 5, fan_out=2, weight_grad=True,
                                                              quantized=four),
                     lambda ws: eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=dx, d_weight=dw,
                                                               workspace=ws))):
                # full of NaN, as a workspace may be left
                ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
                call(ws[:need])
                assert bool((ws[need:] == 255).all())
                with pytest.raises(ValueError, match="workspace must have at least %d bytes" % need):
                    call(ws[:need - 1])
            assert not bool(torch.isnan(y).any() | torch.isnan(dx).any() | torch.isnan(dw).any())


def test_weights_of_more_experts_than_the_metadata_names():
    ids, x, _, w, dy = inputs(40, 1, 6, 64, 48, 0.0)
    ids.clamp_(max=3)
    meta = meta_of(ids, 4)
    y = torch.zeros(40, 48, device="cuda").bfloat16()
    eg.lora_expert_linear(x, w, y, meta)
    want, sums = ref.forward(x, w, ids, 1)
    ref.within(y, want, ref.bound(want, sums, 64), "y")
    dw = torch.ones_like(w)
    eg.lora_expert_linear_backward(dy, x, w, meta, d_weight=dw)
    _, rw, _, sw = ref.backward(dy, x, w, ids, 1)
    ref.within(dw, rw, ref.bound(rw, sw, 40), "dw")


def test_adapters_over_experts():
    """The expert product, then adapters of their own ids added to it; gradients of both into one dx."""
    tokens, hidden, width, rank = 90, 128, 96, 16
    ids, x, _, w, dy = inputs(tokens, 1, 4, hidden, width, 0.0)
    g = torch.Generator().manual_seed(5)
    lora = torch.randint(-1, 3, (tokens,), generator=g, dtype=torch.int32).cuda()
    A = (torch.randn(3, rank, hidden, generator=g) * 0.1).bfloat16().cuda()
    B = (torch.randn(3, width, rank, generator=g) * 0.1).bfloat16().cuda()
    experts, adapters = meta_of(ids, 4), meta_of(lora, 3)
    y = torch.zeros(tokens, width, device="cuda").bfloat16()
    buffer = torch.zeros(1, tokens, rank, device="cuda")
    eg.lora_expert_linear(x, w, y, experts)
    eg.add_lora_linear(y, x, [A], [B], None, 0.5, [width], adapters, buffer=buffer)
    want, sums = ref.forward(x, w, ids, 1)
    add, off = torch.zeros_like(want), torch.zeros_like(want)
    for a in range(3):
        at = (lora == a).nonzero()[:, 0]
        u = 0.5 * x[at].double() @ A[a].double().T
        add[at] = u @ B[a].double().T
        # the buffer is rounded to bf16 before the second product
        off[at] = 1.1 * 2.0 ** -8 * (u.abs() @ B[a].double().abs().T)
    ref.within(y, want + add, ref.bound(want, sums, hidden) + ref.bound(want + add, sums, hidden) + off, "y")
    dx, dA, dB = torch.empty_like(x), torch.empty_like(A), torch.empty_like(B)
    eg.lora_expert_linear_backward(dy, x, w, experts, dx=dx)
    base = dx.clone()
    eg.lora_linear_backward(dy, x, buffer, [A], [B], 0.5, adapters, dx=dx, d_lora_a=[dA], d_lora_b=[dB])
    none = lora < 0
    assert torch.equal(dx[none], base[none]) and not torch.equal(dx, base)


# ------------------------------------------------------------ borders between kernels, large sizes, odd calls

@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("rows", [11, 12, 13, 31, 32, 33, 64])
@pytest.mark.parametrize("experts", [1, 3, 256, 257])
def test_forward_where_the_kernels_change(rows, experts, four):
    """Batches of up to 12 and 32 rows, and up to 256 experts, take no copy of x."""
    check_forward((rows, 1, experts, 544, 150, 0.1), four, seed=rows)


@pytest.mark.parametrize("mean", [12, 13, 32, 33, 96, 97, 128, 129])
@pytest.mark.parametrize("four", [False, True])
def test_forward_by_rows_an_expert(mean, four):
    check_forward((3 * mean, 1, 3, 96, 140, 0.0), four)


@pytest.mark.parametrize("tokens", [1024, 1025])
def test_forward_of_4_bits_where_weights_are_decoded_first(tokens):
    check_forward((tokens, 1, 1, 64, 300, 0.1), True)


@pytest.mark.parametrize("width", [127, 128, 129, 4 * 128, 19 * 128, 38 * 128 + 1, 76 * 128 + 1])
@pytest.mark.parametrize("four", [False, True])
def test_clusters_that_share_a_tile(width, four):
    """Few tiles: a cluster of four, two or one CTA each; sums of K in several parts, some of them empty."""
    for hidden in (32, 64, 96, 288, 1056):
        check_forward((2, 1, 1, hidden, width, 0.0), four)


@pytest.mark.parametrize("size", [(12, 1, 3, 32 * 9, 131, 0.0), (30, 2, 5, 32 * 21, 67, 0.1), (7, 1, 2, 32 * 34, 33, 0.0),
                                  (90, 1, 2, 32 * 43, 257, 0.0), (3, 2, 4, 32 * 115, 301, 0.0), (200, 1, 1, 32 * 47, 129, 0.0),
                                  (5, 1, 3, 32 * 8, 65, 0.0), (5, 1, 3, 32 * 7, 65, 0.0), (20, 1, 3, 32 * 17, 3, 0.0)], ids=str)
def test_scales_at_any_alignment(size):
    """Rows of scales whose bytes are no whole words, in number or in place."""
    check_forward(size, True)


@pytest.mark.parametrize("blocks", [3, 9, 10, 11, 13])
def test_scales_end_with_their_array(blocks):
    """The last row's scales, with NaN behind them: they are not this weight's."""
    T, N, K = 20, 67, 32 * blocks
    ids, x, (codes, scales), values, _ = inputs(T, 1, 2, K, N, 0.0, four=True)
    room = torch.full((scales.numel() + 64,), 255, dtype=torch.uint8, device="cuda")
    room[:scales.numel()] = scales.view(-1)
    y = torch.zeros(T, N, device="cuda").bfloat16()
    eg.lora_expert_linear(x, codes, y, meta_of(ids, 2), weight_scale=room[:scales.numel()].view(scales.shape))
    want, sums = ref.forward(x, values, ids, 1)
    ref.within(y, want, ref.bound(want, sums, K), "y")


@pytest.mark.parametrize("size", [(1, 1, 1, 2560, 129, 0.0), (9, 1, 1, 1536, 200, 0.0), (20, 2, 3, 512, 140, 0.1),
                                  (40, 1, 2, 6656, 257, 0.0), (300, 1, 2, 1536, 100, 0.1), (1, 2, 4, 2560, 64, 0.0),
                                  (6, 2, 5, 7680, 300, 0.0)], ids=str)
def test_scales_in_boxes_of_two_blocks(size):
    """Hidden sizes whose blocks of 256 are even and odd in number, also in the parts of a cluster."""
    check_forward(size, True)


def test_rows_of_x_off_a_16_byte_boundary_in_a_small_batch():
    ids, x, _, w, _ = inputs(5, 2, 3, 64, 40, 0.0)
    wide = torch.zeros(5, 67, device="cuda").bfloat16()
    wide[:, 1:65] = x
    y = torch.zeros(10, 40, device="cuda").bfloat16()
    eg.lora_expert_linear(wide[:, 1:65], w, y, meta_of(ids, 3))
    want, sums = ref.forward(x, w, ids, 2)
    ref.within(y, want, ref.bound(want, sums, 64), "y")


def test_products_with_the_smallest_scales():
    """Scales down to 2^-127, whose elements are subnormal in bf16, times large rows."""
    codes = torch.randint(0, 256, (1, 40, 16), dtype=torch.uint8, device="cuda")
    scales = (torch.arange(40, dtype=torch.int32) // 2).to(torch.uint8).view(1, 40, 1).cuda()
    for rows in (3, 40):
        ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
        x = (torch.randint(-3, 4, (rows, 32), device="cuda").float() * 2.0 ** 110).bfloat16()
        y = torch.zeros(rows, 40, device="cuda").bfloat16()
        eg.lora_expert_linear(x, codes, y, meta_of(ids, 1), weight_scale=scales)
        want, sums = ref.forward(x, ref.decode(codes, scales), ids, 1)
        ref.within(y, want, ref.bound(want, sums, 32), "y")


@pytest.mark.parametrize("four", [False, True])
def test_weights_beyond_32_bit_offsets(four):
    """The last expert of a stack of more than 2^31 weights, and with few rows and many."""
    experts, width, hidden = 3, 90000, 8192
    w = torch.zeros(experts, width, hidden // 2 if four else hidden, dtype=torch.uint8 if four else torch.bfloat16,
                    device="cuda")
    last = torch.randn(257, hidden, device="cuda").bfloat16() * 0.01
    scale = None
    if four:
        codes, scales = ref.encode(last)
        scale = torch.full((experts, width, hidden // 32), 127, dtype=torch.uint8, device="cuda")
        w[2, -257:], scale[2, -257:] = codes, scales
        last = ref.decode(codes, scales)
    else:
        w[2, -257:] = last
    for rows in (3, 500):
        ids = torch.full((rows,), 2, dtype=torch.int32, device="cuda")
        ids[0] = 0
        x = torch.randn(rows, hidden, device="cuda").bfloat16()
        y = torch.ones(rows, width, device="cuda").bfloat16()
        eg.lora_expert_linear(x, w, y, meta_of(ids, experts), weight_scale=scale)
        assert not bool(y[0].any()) and not bool(y[:, :-257].any())
        want, sums = ref.forward(x[1:], last[None], torch.zeros_like(ids[1:]), 1)
        ref.within(y[1:, -257:], want, ref.bound(want, sums, hidden), "y")
        del x, y


def test_rows_beyond_32_bit_offsets():
    rows, width, hidden = 40000, 60000, 8                   # y has 2.4e9 values
    ids = torch.zeros(rows, dtype=torch.int32, device="cuda")
    x = torch.randn(rows, hidden, device="cuda").bfloat16()
    w = torch.randn(1, width, hidden, device="cuda").bfloat16()
    y = torch.zeros(rows, width, device="cuda").bfloat16()
    meta = meta_of(ids, 1)
    eg.lora_expert_linear(x, w, y, meta)
    for at in (slice(0, 3), slice(-300, None)):
        want, sums = ref.forward(x[at], w, ids[at], 1)
        ref.within(y[at], want, ref.bound(want, sums, hidden), "y")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    eg.lora_expert_linear_backward(y, x, w, meta, dx=dx, d_weight=dw)
    want = y[-5:].double() @ w[0].double()
    size = y[-5:].double().abs() @ w[0].double().abs()
    ref.within(dx[-5:], want, ref.bound(want, size, width), "dx")
    want, size = y[:, -40:].double().T @ x.double(), y[:, -40:].double().abs().T @ x.double().abs()
    ref.within(dw[0, -40:], want, ref.bound(want, size, rows), "dw")


def test_two_calls_at_once():
    """On two streams, with workspaces of their own and metadata in common."""
    sets = []
    ids, *_ = inputs(300, 2, 6, 128, 200, 0.1)
    meta = meta_of(ids, 6)
    for seed in (1, 2):
        _, x, _, w, dy = inputs(300, 2, 6, 128, 200, 0.1, seed=seed)
        sets.append(dict(x=x, w=w, dy=dy, y=torch.zeros_like(dy), dx=torch.empty_like(x), dw=torch.empty_like(w),
                         stream=torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s in sets:
            with torch.cuda.stream(s["stream"]):
                eg.lora_expert_linear(s["x"], s["w"], s["y"], meta)
                eg.lora_expert_linear_backward(s["dy"], s["x"], s["w"], meta, dx=s["dx"], d_weight=s["dw"])
    torch.cuda.synchronize()
    for s in sets:
        want, sums = ref.forward(s["x"], s["w"], ids, 2)
        ref.within(s["y"], want, ref.bound(want, sums, 128), "y")
        rx, rw, sx, sw = ref.backward(s["dy"], s["x"], s["w"], ids, 2)
        ref.within(s["dx"], rx, ref.bound(rx, sx, 202), "dx")
        ref.within(s["dw"], rw, ref.bound(rw, sw, 600), "dw")


@pytest.mark.parametrize("rows", [6, 200])
def test_metadata_of_a_larger_batch_write_nothing_beyond_the_call_s_rows(rows):
    """Not a documented call; rows that the call does not have are left out."""
    ids, x, _, w, dy = inputs(3 * rows, 1, 4, 64, 48, 0.0)
    meta = meta_of(ids, 4)
    flat = torch.zeros(3 * rows, 48, device="cuda").bfloat16()
    eg.lora_expert_linear(x[:rows], w, flat[:rows], meta)
    assert not bool(flat[rows:].any())
    full, dw = torch.zeros(3 * rows, 64, device="cuda").bfloat16(), torch.empty_like(w)
    need = eg.lora_expert_linear_backward_workspace(rows, 64, 48, 4, weight_grad=True)
    ws = torch.full((need + 65536,), 7, dtype=torch.uint8, device="cuda")
    eg.lora_expert_linear_backward(dy[:rows], x[:rows], w, meta, dx=full[:rows], d_weight=dw, workspace=ws[:need])
    assert not bool(full[rows:].any()) and bool((ws[need:] == 7).all())


@pytest.mark.parametrize("four", [False, True])
def test_calls_one_after_another_share_a_workspace(four):
    """No call begins to write what the one before still reads: batches that gather, copy and run on pairs."""
    cases = []
    for k, tokens in enumerate((1, 30, 700, 3, 64, 200, 40, 9, 2000, 26)):
        ids, x, (w, scale), _, _ = inputs(tokens, 2, 3, 512, 384, 0.1, four=four, seed=k)
        cases.append((ids, x, w, scale, meta_of(ids, 3)))
    y = [torch.zeros(len(c[0]), 384, device="cuda").bfloat16() for c in cases]
    alone = []
    for (ids, x, w, scale, meta), out in zip(cases, y):
        eg.lora_expert_linear(x, w, out, meta, weight_scale=scale)
        torch.cuda.synchronize()
        alone.append(out.clone())
    workspace = torch.empty(eg.lora_expert_linear_workspace(4000, 512, 384, 3, quantized=four), dtype=torch.uint8,
                            device="cuda")
    for _ in range(20):
        for out in y:
            out.zero_()
        for n, (ids, x, w, scale, meta) in enumerate(cases * 3):
            if n % 4 == 0:
                meta.prepare_tensors(ids)
            eg.lora_expert_linear(x, w, y[n % len(y)], meta, weight_scale=scale, workspace=workspace)
        for out, want in zip(y, alone):
            assert torch.equal(out, want)


def test_refusals():
    ids, x, _, w, dy = inputs(8, 2, 3, 64, 48, 0.0)
    meta = meta_of(ids, 3)
    y = torch.zeros(16, 48, device="cuda").bfloat16()
    codes, scales = ref.encode(w)
    ok = dict(x=x, weight=w, y=y, meta=meta)
    four = dict(ok, weight=codes, weight_scale=scales)
    for bad, error in (
            (dict(ok, x=x.float()), TypeError), (dict(ok, x=None), TypeError), (dict(ok, x=x.cpu()), (TypeError, ValueError)),
            (dict(ok, y=y.cpu()), (TypeError, ValueError)), (dict(ok, weight=w.half()), TypeError),
            (dict(ok, weight=None), TypeError), (dict(ok, weight=w[:2]), ValueError), (dict(ok, weight=w[0]), ValueError),
            (dict(ok, weight=w.transpose(1, 2)), ValueError), (dict(ok, y=y[:15]), ValueError),
            (dict(ok, y=y[:, :40]), ValueError), (dict(ok, y=y[:0]), ValueError), (dict(ok, x=x[:0]), ValueError),
            (dict(ok, x=x.t()), ValueError), (dict(ok, weight=codes), TypeError), (dict(four, weight=w), TypeError),
            (dict(four, weight_scale=scales[:, :, :1]), ValueError), (dict(four, weight=codes[:, :, :16]), ValueError),
            (dict(ok, workspace=torch.zeros(1 << 20, device="cuda")), TypeError),
            (dict(ok, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda")), ValueError),
            (dict(ok, x=x, y=x, weight=torch.zeros(3, 64, 64, device="cuda").bfloat16()), ValueError)):
        with pytest.raises(error):
            eg.lora_expert_linear(**bad)
    with pytest.raises(eg.LoraError):
        eg.lora_expert_linear(x[:, :60], w[:, :, :60].contiguous(), y, meta)
    assert not bool(y.any())
    ok = dict(dy=dy, x=x, weight=w, meta=meta)
    for bad, error in (
            (dict(ok, dy=dy[:, :40]), ValueError), (dict(ok, dy=None), TypeError), (dict(ok, dx=x), ValueError),
            (dict(ok, dx=torch.zeros(8, 72, device="cuda").bfloat16()), ValueError),
            (dict(ok, dx=torch.zeros(8, 64, device="cuda")), TypeError),
            (dict(ok, d_weight=torch.zeros(3, 48, 72, device="cuda").bfloat16()), ValueError),
            (dict(ok, d_weight=w.transpose(1, 2)), ValueError), (dict(ok, d_weight=w.float()), TypeError)):
        with pytest.raises(error):
            eg.lora_expert_linear_backward(**bad)


@pytest.mark.parametrize("rows, experts, width, hidden", [(20, 3, 20000, 8192), (200, 3, 20000, 8192), (500, 3, 20000, 8192),
                                                          (900, 1, 20000, 2048), (10, 3, 20000, 8192)], ids=str)
@pytest.mark.parametrize("four", [False, True])
def test_long_runs_of_stages_repeat(rows, experts, width, hidden, four):
    """Hundreds of thousands of stages through the rings: every call gives the same bits, and the right ones."""
    g = torch.Generator(device="cuda").manual_seed(3)
    ids = torch.randint(0, experts, (rows,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn(rows, hidden, generator=g, device="cuda").bfloat16()
    scale = None
    if four:
        w = torch.randint(0, 256, (experts, width, hidden // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = torch.randint(115, 125, (experts, width, hidden // 32), generator=g, device="cuda", dtype=torch.uint8)
    else:
        w = (torch.randn(experts, width, hidden, generator=g, device="cuda") * 0.02).bfloat16()
    meta = meta_of(ids, experts)
    first = None
    for _ in range(20):
        y = torch.zeros(rows, width, device="cuda").bfloat16()
        eg.lora_expert_linear(x, w, y, meta, weight_scale=scale)
        if first is None:
            first = y
            for e in range(experts):
                at = (ids == e).nonzero()[:, 0]
                we = (ref.decode(w[e], scale[e]) if four else w[e].double())
                want, size = x[at].double() @ we.T, x[at].double().abs() @ we.abs().T
                ref.within(y[at], want, ref.bound(want, size, hidden), "y")
        else:
            assert torch.equal(y, first)
    assert int(meta.error_word) == 0
