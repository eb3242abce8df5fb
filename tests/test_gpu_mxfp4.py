"""lora_quantize_mxfp4 and lora_dequantize_mxfp4 against the format's
definition (GPU): codes, scales and values are equal."""
import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref

pytestmark = pytest.mark.gpu


def quantized(w):
    codes = torch.empty((*w.shape[:-1], w.shape[-1] // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*w.shape[:-1], w.shape[-1] // 32), dtype=torch.uint8, device="cuda")
    eg.lora_quantize_mxfp4(w, codes, scales)
    return codes, scales


@pytest.mark.parametrize("shape", [(32,), (1, 32), (3, 64), (5, 7, 96), (1003, 1024), (2, 129, 4096), (0, 32)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_codes_scales_and_values(shape, dtype):
    g = torch.Generator().manual_seed(len(shape) + shape[-1])
    w = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn((*shape[:-1], 1), generator=g))
    w = w.to("cuda", dtype)
    codes, scales = quantized(w)
    want = ref.encode(w)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    for out_type in (torch.bfloat16, torch.float32):
        out = torch.empty(shape, dtype=out_type, device="cuda")
        eg.lora_dequantize_mxfp4(codes, scales, out)
        assert torch.equal(out.double(), ref.decode(*want))


def test_borders_between_codes():
    """Every midpoint, and its neighbours on both sides, at several scales."""
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    values = [4.5, 6.0]                                     # the first fixes the scale at 1
    for m in mid + [6.5, 7.5, 7.999]:
        t = torch.tensor(m)
        values += [m, float(torch.nextafter(t, torch.tensor(0.0))), float(torch.nextafter(t, torch.tensor(9.0)))]
    block = torch.tensor(values + [-v for v in values]).view(2, 32)
    for e in (-127, -126, -125, -20, 0, 20, 100, 125):
        w = (block.double() * 2.0 ** e).float().cuda()
        codes, scales = quantized(w)
        want = ref.encode(w)
        assert torch.equal(scales, want[1]) and torch.equal(codes, want[0]), e


def test_smallest_and_largest_values():
    w = torch.zeros(6, 32)
    w[1, 3] = 1e-45                                         # the smallest number
    w[2] = torch.linspace(0, 1.1e-38, 32)
    w[3] = torch.linspace(0, 2e-38, 32)
    w[4] = torch.linspace(-3.4e38, 3.4e38, 32, dtype=torch.float64).float()     # 32 bits overflow on the way
    w[5, ::2] = -0.0
    w = w.cuda()
    codes, scales = quantized(w)
    want = ref.encode(w)
    assert torch.equal(scales, want[1]) and torch.equal(codes, want[0])
    out = torch.empty_like(w)
    eg.lora_dequantize_mxfp4(codes, scales, out)
    assert torch.equal(out.double(), ref.decode(*want))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_block_with_nan_or_infinity_is_nan(bad, dtype):
    w = torch.randn(4, 96, device="cuda").to(dtype)
    clean = quantized(w)
    w[1, 40] = bad
    codes, scales = quantized(w)
    assert int(scales[1, 1]) == 255
    out = torch.empty_like(w)
    eg.lora_dequantize_mxfp4(codes, scales, out)
    assert bool(torch.isnan(out[1, 32:64]).all()) and int(torch.isnan(out).sum()) == 32
    scales[1, 1], codes[1, 16:32] = clean[1][1, 1], clean[0][1, 16:32]
    assert torch.equal(codes, clean[0]) and torch.equal(scales, clean[1])


def test_every_code_with_every_scale():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 16, 16).expand(256, 16, 16).contiguous().cuda()
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1, 1).expand(256, 16, 1).contiguous().cuda()
    want = ref.decode(codes, scales)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty(256, 16, 32, dtype=dtype, device="cuda")
        eg.lora_dequantize_mxfp4(codes, scales, out)
        # beyond the type's largest value (4 and 6 times 2^127 in scale 254): infinity
        assert torch.equal(torch.isnan(out), torch.isnan(want))
        exact = want.to(dtype).double()
        assert torch.equal(torch.nan_to_num(out.double(), 0.5), torch.nan_to_num(exact, 0.5))
        finite = torch.isfinite(out)
        assert torch.equal(out.double()[finite], want[finite])


def test_products_with_every_scale():
    """A product's weights are the decoded ones, at every scale that leaves it finite."""
    codes = torch.randint(0, 256, (1, 230, 16), dtype=torch.uint8, device="cuda")
    scales = torch.arange(23, 253, dtype=torch.int32).to(torch.uint8).view(1, 230, 1).cuda()
    meta = eg.LoRAKernelMeta.make(1, 3, "cuda")
    meta.prepare_tensors(torch.zeros(3, dtype=torch.int32, device="cuda"))
    x = (torch.randint(-2, 3, (3, 32), device="cuda").float() * 2.0 ** -4).bfloat16()
    y = torch.zeros(3, 230, device="cuda").bfloat16()
    eg.lora_expert_linear(x, codes, y, meta, weight_scale=scales)
    want, sums = ref.forward(x, ref.decode(codes, scales), torch.zeros(3, dtype=torch.int32, device="cuda"), 1)
    ok = sums < 2.0 ** 127
    limit = torch.where(ok, ref.bound(want, sums, 32), torch.full_like(want, float("inf")))
    ref.within(torch.nan_to_num(y.double(), 0.0, 0.0, 0.0) * ok, want * ok, limit, "y")
