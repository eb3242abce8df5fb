"""The layers under the adapters, the adapters, and what follows their
gradients, as a training step runs them: experts in 4 bits, adapters over
them, the loss, the gradients through both, clipping for each adapter and the
orthogonalised update; and the example with these layers."""
import importlib.util
import math
import os

import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_a_step_over_experts_in_4_bits():
    T, E, L, H, N, V, r, scale = 200, 4, 3, 96, 160, 300, 16, 0.5
    g = torch.Generator().manual_seed(11)
    experts = torch.randint(0, E, (T,), generator=g, dtype=torch.int32).cuda()
    adapters = torch.randint(-1, L, (T,), generator=g, dtype=torch.int32).cuda()
    x = torch.randn(T, H, generator=g).bfloat16().cuda()
    W = (torch.randn(E, N, H, generator=g) * H ** -0.5).bfloat16().cuda()
    A = (torch.randn(L, r, H, generator=g) * H ** -0.5).bfloat16().cuda()
    B = (torch.randn(L, N, r, generator=g) * 0.1).bfloat16().cuda()
    head = (torch.randn(V, N, generator=g) * N ** -0.5).bfloat16().cuda()
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32).cuda()
    codes = torch.empty(E, N, H // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E, N, H // 32, dtype=torch.uint8, device="cuda")
    eg.lora_quantize_mxfp4(W, codes, scales)
    by_expert, by_adapter = eg.LoRAKernelMeta.make(E, T, "cuda"), eg.LoRAKernelMeta.make(L, T, "cuda")
    by_expert.prepare_tensors(experts)
    by_adapter.prepare_tensors(adapters)
    y = torch.empty(T, N, device="cuda", dtype=torch.bfloat16)
    buffer = torch.zeros(1, T, r, device="cuda")
    eg.lora_expert_linear(x, codes, y, by_expert, weight_scale=scales)
    eg.add_lora_linear(y, x, [A], [B], None, scale, [N], by_adapter, buffer=buffer)
    loss, dy = torch.empty(T, device="cuda"), torch.empty_like(y)
    eg.lora_cross_entropy(y, head, targets, loss, hidden_grad=dy)
    dx, dA, dB = torch.empty_like(x), torch.empty_like(A), torch.empty_like(B)
    eg.lora_expert_linear_backward(dy, x, codes, by_expert, weight_scale=scales, dx=dx)
    eg.lora_linear_backward(dy, x, buffer, [A], [B], scale, by_adapter, dx=dx, d_lora_a=[dA], d_lora_b=[dB])
    norms = torch.empty(L, device="cuda")
    raw = [dA.clone(), dB.clone()]
    eg.lora_clip_gradients([dA, dB], 0.5, norms)
    update = torch.empty_like(dA)
    eg.lora_orthogonalize(dA, update)

    # in 64 bits, each part from what the part before it gave, so that its bound is its own
    w = ref.decode(codes, scales)
    want, size = ref.forward(x, w, experts, 1)
    off = torch.zeros_like(want)
    for a in range(L):
        at = (adapters == a).nonzero()[:, 0]
        u = scale * x[at].double() @ A[a].double().T
        want[at] += u @ B[a].double().T
        off[at] = 1.1 * 2.0 ** -8 * (u.abs() @ B[a].double().abs().T)
    base = ref.forward(x, w, experts, 1)[0]
    ref.within(y, want, ref.bound(base, size, H) + ref.bound(want, size, H) + off, "y")
    logits = y.double() @ head.double().T
    right = torch.logsumexp(logits, 1) - logits[torch.arange(T), targets.long()]
    assert bool(((loss.double() - right).abs() <= 1e-4 * (1 + right)).all())
    dbase, _, sx, _ = ref.backward(dy, x, w, experts, 1)
    more, off = torch.zeros_like(dbase), torch.zeros_like(dbase)
    for a in range(L):
        at = (adapters == a).nonzero()[:, 0]
        gr = dy[at].double() @ B[a].double()
        more[at] = scale * gr @ A[a].double()
        off[at] = 1.1 * 2.0 ** -8 * scale * (gr.abs() @ A[a].double().abs())
    ref.within(dx, dbase + more, ref.bound(dbase, sx, N) + ref.bound(dbase + more, sx, N) + off, "dx")
    right = sum(v.double().square().sum((1, 2)) for v in raw).sqrt()
    assert bool(((norms.double() - right).abs() <= 20 * 2.0 ** -24 * right).all())
    f = (0.5 / (right + 1e-6)).clamp(max=1.0)[:, None, None]
    for got, v in zip((dA, dB), raw):
        ref.within(got, v.double() * f, v.double().abs() * f * (2.0 ** -8 + 22 * 2.0 ** -24), "clipped")
    clipped = sum(v.double().square().sum((1, 2)) for v in (dA, dB)).sqrt()
    assert bool((clipped <= 0.5 * (1 + 2.0 ** -8)).all()) and bool(torch.isfinite(update).all())


def _example():
    spec = importlib.util.spec_from_file_location("train_adapters", os.path.join(ROOT, "examples", "train_adapters.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("clip", [None, 1e-3])
def test_the_example_runs_on_layers_in_4_bits_and_clipped(clip):
    history = _example().train(steps=4, tokens=200, hidden=128, vocab=300, rank=16, loras=3, four=True, clip=clip)
    assert len(history) == 4 and all(math.isfinite(v) for v in history)


def test_a_layer_of_the_example_in_4_bits_has_the_gradient_of_its_weights_values():
    mod = _example()
    gen = torch.Generator().manual_seed(2)
    layer = mod.Layer(128, 16, 2, 0.5, 60, "cuda", gen, four=True)
    layer.weights[1].copy_(torch.randn(2, 128, 16, generator=gen) * 0.1)
    meta = eg.LoRAKernelMeta.make(2, 60, "cuda")
    meta.prepare_tensors(torch.full((60,), -1, dtype=torch.int32, device="cuda"))
    x, dy = (torch.randn(60, 128, generator=gen).bfloat16().cuda() for _ in range(2))
    y = layer.forward(x, meta)
    w = ref.decode(layer.codes, layer.scales)[0]
    want, size = x.double() + x.double() @ w.T, x.double().abs() + x.double().abs() @ w.abs().T
    ref.within(y, want, ref.bound(want, size, 129), "y")
    dx = layer.backward(dy, meta, None)
    want, size = dy.double() + dy.double() @ w, dy.double().abs() + dy.double().abs() @ w.abs()
    ref.within(dx, want, ref.bound(want, size, 129), "dx")
