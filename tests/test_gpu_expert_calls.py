"""Calls of lora_expert_linear and its gradients with metadata that name more
rows than the call has (GPU): what the call has of them is right, the rest
stays as it was, and no wait runs out."""
import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref
from test_gpu_expert import inputs, meta_of

pytestmark = pytest.mark.gpu


def seen(ids, rows):
    """Of the first `rows` rows, those among the first `rows` of the stable order by id."""
    order = torch.sort(ids, stable=True).indices[:rows]
    mine = torch.zeros(rows, dtype=torch.bool, device=ids.device)
    mine[order[order < rows]] = True
    return mine


# rows of the call, experts: gathered and shared by clusters, copied beside the weights, by a table, on pairs
@pytest.mark.parametrize("rows, experts", [(1, 4), (6, 4), (12, 2), (24, 3), (40, 4), (40, 300), (200, 4), (500, 1)])
@pytest.mark.parametrize("factor", [2, 40])
@pytest.mark.parametrize("width", [48, 1500, 4000])
@pytest.mark.parametrize("four", [False, True])
def test_forward_by_metadata_of_a_larger_batch(rows, experts, factor, width, four):
    hidden = 320 if experts < 100 else 96
    ids, x, (w, scale), values, _ = inputs(factor * rows, 1, experts, hidden, width, 0.1, four=four)
    meta = meta_of(ids, experts)
    was = torch.randn(factor * rows, width, device="cuda").bfloat16()
    flat = was.clone()
    eg.lora_expert_linear(x[:rows], w, flat[:rows], meta, weight_scale=scale)
    assert torch.equal(flat[rows:], was[rows:])
    mine = seen(ids, rows) & (ids[:rows] >= 0)
    assert torch.equal(flat[:rows][~mine], was[:rows][~mine])
    some = torch.where(mine, ids[:rows], torch.full_like(ids[:rows], -1))
    want, sums = ref.forward(x[:rows], values, some, 1)
    ref.within(flat[:rows][mine], want[mine], ref.bound(want, sums, hidden)[mine], "y")
    assert int(meta.error_word) == 0


@pytest.mark.parametrize("rows, experts", [(6, 4), (200, 4), (500, 1), (40, 300)])
@pytest.mark.parametrize("factor", [2, 40])
@pytest.mark.parametrize("four", [False, True])
def test_gradients_by_metadata_of_a_larger_batch(rows, experts, factor, four):
    hidden, width = 320 if experts < 100 else 96, 130
    ids, x, (w, scale), values, dy = inputs(factor * rows, 1, experts, hidden, width, 0.1, four=four)
    meta = meta_of(ids, experts)
    was = torch.randn(factor * rows, hidden, device="cuda").bfloat16()
    flat, dw = was.clone(), torch.empty(experts, width, hidden, device="cuda").bfloat16()
    need = eg.lora_expert_linear_backward_workspace(rows, hidden, width, experts, weight_grad=True, quantized=four)
    ws = torch.full((need + 65536,), 7, dtype=torch.uint8, device="cuda")
    eg.lora_expert_linear_backward(dy[:rows], x[:rows], w, meta, weight_scale=scale, dx=flat[:rows], d_weight=dw,
                                   workspace=ws[:need])
    assert torch.equal(flat[rows:], was[rows:]) and bool((ws[need:] == 7).all())
    mine = seen(ids, rows)
    assert torch.equal(flat[:rows][~mine], was[:rows][~mine])
    some = torch.where(mine, ids[:rows], torch.full_like(ids[:rows], -1))
    rx, rw, sx, sw = ref.backward(dy[:rows], x[:rows], values, some, 1)
    ref.within(flat[:rows][mine], rx[mine], ref.bound(rx, sx, width + 1)[mine], "dx")
    ref.within(dw, rw, ref.bound(rw, sw, rows), "dw")
    assert int(meta.error_word) == 0
