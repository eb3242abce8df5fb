"""lora_quantize_mxfp4 and lora_dequantize_mxfp4 beyond 32-bit offsets (GPU)."""
import pytest
import torch

import expand_gemm_gb300 as eg
import expert_reference as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype, rows", [(torch.bfloat16, (1 << 22) + 3), (torch.float32, (1 << 21) + 3)])
def test_last_rows_of_a_large_matrix(dtype, rows):
    """More than 2^32 (bf16) and 2^31 (fp32) elements."""
    n = 1024
    w = torch.zeros(rows, n, dtype=dtype, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(1)
    for at in (slice(0, 2), slice(rows // 2, rows // 2 + 2), slice(rows - 2, rows)):
        w[at] = torch.randn(2, n, generator=g, device="cuda").to(dtype)
    codes = torch.full((rows, n // 2), 7, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, n // 32), 7, dtype=torch.uint8, device="cuda")
    eg.lora_quantize_mxfp4(w, codes, scales)
    out = torch.full_like(w, 5.0)
    eg.lora_dequantize_mxfp4(codes, scales, out)
    for at in (slice(0, 4), slice(rows // 2 - 1, rows // 2 + 3), slice(rows - 4, rows)):
        want = ref.encode(w[at])
        assert torch.equal(codes[at], want[0]) and torch.equal(scales[at], want[1])
        assert torch.equal(out[at].double(), ref.decode(*want))
    assert int(torch.count_nonzero(scales)) == 6 * n // 32      # of zeros: 2^-127, stored as 0
    assert int(torch.count_nonzero(out.view(-1)[:: 1021])) <= 6 * n // 1021 + 6
