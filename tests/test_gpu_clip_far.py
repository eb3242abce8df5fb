"""lora_clip_gradients where the norm lies 2^126 largest norms and more away, so
that the factor is no normal number of 32 bits (GPU)."""
import pytest
import torch

import expand_gemm_gb300 as eg
from test_gpu_clip import BF16, F32, check

pytestmark = pytest.mark.gpu


def in_32_bits(value):
    return float(torch.tensor(value, dtype=F32))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("max_norm", [100.0, 1.0, 1e-3, 1e-7, 1e-30, 1e-45])
@pytest.mark.parametrize("out", [False, True])
def test_factors_that_are_subnormal_or_zero_in_32_bits(dtype, max_norm, out):
    v = torch.full((2, 1 << 20), 3e38)
    v[0, ::3] = -1.5e38
    v[1] *= 1e-30                                           # this one's factor is a normal number, or 1
    _, got = check([v.to("cuda", dtype)], 2, in_32_bits(max_norm), eps=0.0, out=out)
    assert max_norm < 1e-40 or bool((got[0] != 0).all())


def test_the_largest_gradients_of_all():
    _, got = check([torch.full((1 << 24,), 3e38, device="cuda")], 1, in_32_bits(1e-3), eps=0.0)
    assert bool((got[0] > 2.4e-7).all())                    # 1e-3 / 2^12


@pytest.mark.parametrize("count", [1, 64, 65, 1024, 1025])
@pytest.mark.parametrize("out", [False, True])
def test_by_many_tensors_at_any_alignment(count, out):
    """One launch, which joins the sums itself, and several."""
    store = torch.full((count * 37 + 8,), 2e38, device="cuda")
    store[::5] = -3e37
    grads = [store[1 + 37 * i:37 * (i + 1)].view(3, 12) for i in range(count)]
    check(grads, 3, 1.0, eps=0.0, out=out)
    check(grads, 1, 1e-2, eps=0.0, out=out)


def test_small_values_beside_large_ones():
    v = torch.zeros(1, 5000)
    v[0, 0], v[0, 1], v[0, 4999], v[0, 2500] = 3e38, 1e30, 1e38, 1e-10
    check([v.cuda()], 1, 1.0, eps=0.0)
    check([v.cuda().bfloat16()], 1, 1.0, eps=0.0)


def test_limits_that_32_bits_do_not_hold_are_refused():
    """Infinite in 32 bits they would leave the gradients as they are, or make them zero."""
    g, norms = torch.full((4,), 3e38, device="cuda"), torch.zeros(1, device="cuda")
    for kw in (dict(max_norm=4e38), dict(max_norm=1e300), dict(max_norm=1.0, eps=1e39), dict(max_norm=1.0, eps=float("inf"))):
        with pytest.raises(ValueError, match="max_norm"):
            eg.lora_clip_gradients([g], norms=norms, **kw)
    assert bool((g == torch.full_like(g, 3e38)).all()) and not bool(norms.any())
    eg.lora_clip_gradients([g], float(torch.finfo(F32).max), norms, eps=0.0)
    want = 3.4028234663852886e38 / (2 * float(torch.tensor(3e38))) * 3e38
    assert bool(((g.double() - want).abs() <= 22 * 2.0 ** -24 * want).all())
    eg.lora_clip_gradients([g], float("inf"), norms)
