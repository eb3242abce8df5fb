"""lora_orthogonalize by norms, on spectra where the update lacks directions.

Tolerance of the norm of out - ref, from the formats before any run, with n
steps of leading coefficient a on matrices of short side r, |X0| = 1:
  2^-8 |ref|             out rounded to bf16 (2^-9), twice that allowed;
  a^n 2^-17              P, whose entries reach a^n, as two bf16 terms;
  a^n E                  the error of U U^T beside its largest eigenvalue: an
                         error between a large direction and one that U lacks
                         enters with P(0) - P(l), about a^n; E = 2^-18, and
                         2^-17 for fp32 entries (two bf16 terms, the product
                         of the low ones left out);
  2 n |b| a^n 2^-24 sqrt(r)   the same for the roundings of each step, one
                         entry in each of up to r missing directions.
The iteration on X itself (a^n above 512) rounds in fp32 throughout: beside
2^-8 |ref|, a^n 2^-20 for the 2^-24 of X0's entries and of the sums of its
first steps, sixteen in all, in directions that U lacks.
"""
import math

import pytest
import torch

import expand_gemm_gb300 as eg
from test_gpu_orthogonalize import ABC, iterate, matrix

pytestmark = pytest.mark.gpu


def spectrum(rows, cols, kind, g):
    if kind == "rank eight":        # small whole numbers: exactly of that rank in both types
        u = (torch.randint(-1, 2, (rows, 8), generator=g, dtype=torch.float64) @
             torch.randint(-1, 2, (8, cols), generator=g, dtype=torch.float64))
        return u / 1024
    if kind == "steep":             # singular values over five decades
        u = torch.randn((rows, cols), generator=g, dtype=torch.float64)
        w, _, v = torch.linalg.svd(u, full_matrices=False)
        return 1e-3 * w @ torch.diag(10.0 ** torch.linspace(0, -5, min(rows, cols), dtype=torch.float64)) @ v
    return matrix(rows, cols, kind, g)


def tolerance(ref, r, f32, steps, abc, scale=1.0):
    grown = abs(abc[0]) ** steps
    step = 2 * steps * abs(abc[1]) * 2.0 ** -24 * math.sqrt(r)
    first = 2.0 ** -20 if grown > 512 else 2.0 ** -17 + (2.0 ** -17 if f32 else 2.0 ** -18) + step
    return 2.0 ** -8 * float(torch.linalg.norm(ref)) + scale * grown * first


def run(u, f32, steps, abc=ABC, **kw):
    u = (u.float() if f32 else u.bfloat16()).cuda()
    out = torch.full(u.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    eg.lora_orthogonalize(u, out, steps=steps, coefficients=abc, **kw)
    return u.double().cpu(), out.double().cpu()


KINDS = ["noise", "decay", "steep", "dominant", "rank one", "rank eight"]


def test_many_small_matrices():
    """More than 65535 of them."""
    g = torch.Generator().manual_seed(19)
    u = (1e-3 * torch.randn((70001, 8, 8), generator=g)).bfloat16()
    v = u.cuda()
    out = torch.full(v.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    eg.lora_orthogonalize(v, out)
    assert torch.isfinite(out.float()).all()
    a, b, c = ABC
    x = u.double()
    x = x / (torch.linalg.norm(x, dim=(1, 2), keepdim=True) + 1e-7)
    for _ in range(5):
        s = x @ x.transpose(1, 2)
        x = a * x + (b * s + c * (s @ s)) @ x
    off = torch.linalg.norm(out.double().cpu() - x, dim=(1, 2))
    size = torch.linalg.norm(x, dim=(1, 2))
    grown = a ** 5 * (2.0 ** -17 + 2.0 ** -18 + 2 * 5 * abs(b) * 2.0 ** -24 * math.sqrt(8))
    assert (off <= 2.0 ** -8 * size + grown).all(), float((off - 2.0 ** -8 * size).max())
