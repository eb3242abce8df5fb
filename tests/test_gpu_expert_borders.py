"""lora_expert_linear on both sides of the borders between its kernels, each
call in a workspace of exactly the size that it asks for (GPU)."""
import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref
from test_gpu_expert import inputs, meta_of

pytestmark = pytest.mark.gpu


def check(rows, experts, hidden, width, four, fan=1):
    ids, x, (w, scale), values, _ = inputs(rows // fan, fan, experts, hidden, width, 0.1, four=four, seed=rows)
    meta = meta_of(ids, experts)
    need = eg.lora_expert_linear_workspace(rows, hidden, width, experts, quantized=four)
    ws = torch.full((need + 4096,), 255, dtype=torch.uint8, device="cuda")
    was = torch.randn(rows, width, device="cuda").bfloat16()
    y = was.clone()
    eg.lora_expert_linear(x, w, y, meta, weight_scale=scale, workspace=ws[:need])
    want, sums = ref.forward(x, values, ids, fan)
    has = (ids >= 0)[:, None]
    assert torch.equal(y[ids < 0], was[ids < 0])
    ref.within(torch.where(has, y, torch.zeros_like(y)), want, ref.bound(want, sums, hidden), "y")
    assert bool((ws[need:] == 255).all()) and int(meta.error_word) == 0


@pytest.mark.parametrize("rows", [23, 24, 25, 26])
@pytest.mark.parametrize("experts, fan", [(1, 1), (5, 1), (256, 1), (257, 1), (6, 2)])
def test_up_to_24_rows_of_bf16_take_no_copy_of_x(rows, experts, fan):
    check(rows // fan * fan, experts, 544, 150, False, fan)


@pytest.mark.parametrize("experts", [1, 3, 8])
@pytest.mark.parametrize("more", [-1, 0, 1])
def test_4_bits_are_decoded_first_above_384_rows_an_expert(experts, more):
    """The average is rounded down: it reaches 385 with 385 rows of each expert."""
    check(385 * experts + more, experts, 96, 300, True)


@pytest.mark.parametrize("experts", [1, 3])
@pytest.mark.parametrize("mean, four", [(33, False), (13, True)])
@pytest.mark.parametrize("more", [-1, 0])
def test_taller_tiles_above_an_average_of_rows(mean, four, experts, more):
    check(mean * experts + more, experts, 96, 300, four)


@pytest.mark.parametrize("rows", [63, 64, 65, 223, 224, 225, 256, 257, 2431, 2432, 2433])
def test_one_layer_s_tiles_of_different_heights(rows):
    """Pairs take tiles of 64 to 256 rows, by whole rounds."""
    check(rows, 1, 72, 520, False)
