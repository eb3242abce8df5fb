"""lora_expert_linear where the kernel asks for weights before x has been copied,
right behind what writes its inputs: in a stream and in graphs (GPU)."""
import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref
from test_gpu_expert import inputs, meta_of

pytestmark = pytest.mark.gpu

# tokens, fan out, experts, hidden, width: gathered; copied beside the weights, tiles of 16 and of 64 rows; by a table; on pairs
SIZES = [(5, 2, 3, 544, 520), (18, 2, 3, 544, 520), (40, 2, 3, 1024, 1500), (150, 2, 300, 256, 200), (600, 2, 3, 544, 520)]


def sets(size, four, count=3):
    made = []
    for seed in range(count):
        ids, x, (w, scale), values, _ = inputs(*size, 0.1, four=four, seed=seed)
        y = torch.zeros(len(ids), size[4], device="cuda").bfloat16()
        eg.lora_expert_linear(x, w, y, meta_of(ids, size[2]), weight_scale=scale)
        want, sums = ref.forward(x, values, ids, size[1])
        ref.within(y, want, ref.bound(want, sums, size[3]), "y")
        made.append((ids, x, w, scale, y))
    torch.cuda.synchronize()
    return made


def buffers(one):
    ids, x, w, scale, y = one
    return [t if t is None else torch.empty_like(t) for t in (ids, x, w, scale, y)]


def fill(held, one):
    for to, t in zip(held[:4], one):
        if t is not None:
            to.copy_(t)


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("four", [False, True])
def test_inputs_written_right_before_the_call(size, four):
    made = sets(size, four)
    held, meta = buffers(made[0]), eg.LoRAKernelMeta.make(size[2], size[0] * size[1], "cuda")
    ids, x, w, scale, _ = held
    outs = []
    for n in range(30):
        fill(held, made[n % 3])
        y = torch.zeros_like(held[4])
        meta.prepare_tensors(ids)
        eg.lora_expert_linear(x, w, y, meta, weight_scale=scale)
        outs.append(y)
    for n, y in enumerate(outs):
        assert torch.equal(y, made[n % 3][4]), n


@pytest.mark.parametrize("size", SIZES, ids=str)
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("prepare", [False, True])
def test_inputs_written_right_before_a_replay(size, four, prepare):
    made = sets(size, four)
    held, meta = buffers(made[0]), eg.LoRAKernelMeta.make(size[2], size[0] * size[1], "cuda")
    ids, x, w, scale, y = held
    fill(held, made[0])
    meta.prepare_tensors(ids)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        if prepare:
            meta.prepare_tensors(ids)
        eg.lora_expert_linear(x, w, y, meta, weight_scale=scale)
    outs = []
    for n in range(30):
        fill(held, made[n % 3])
        y.zero_()
        if not prepare:
            meta.prepare_tensors(ids)
        graph.replay()
        outs.append(y.clone())
    for n, got in enumerate(outs):
        assert torch.equal(got, made[n % 3][4]), n


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_weights_quantised_right_before_the_call(size):
    made = [inputs(*size, 0.1, seed=s) for s in range(3)]
    E, H, N = size[2:]
    held = torch.empty(E, N, H, dtype=torch.bfloat16, device="cuda")
    codes = torch.empty(E, N, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, H // 32, dtype=torch.uint8, device="cuda")
    metas = [meta_of(m[0], E) for m in made]
    outs = []
    for n in range(12):
        ids, x, (w, _), _, _ = made[n % 3]
        held.copy_(w)
        y = torch.zeros(len(ids), N, device="cuda").bfloat16()
        eg.lora_quantize_mxfp4(held, codes, scales)
        eg.lora_expert_linear(x, codes, y, metas[n % 3], weight_scale=scales)
        outs.append(y)
    for n, y in enumerate(outs):
        ids, x, (w, _), _, _ = made[n % 3]
        assert torch.equal(y, outs[n % 3])
        if n < 3:
            want, sums = ref.forward(x, ref.decode(*ref.encode(w)), ids, size[1])
            ref.within(y, want, ref.bound(want, sums, H), "y")
