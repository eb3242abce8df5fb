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


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(16, 512), (32, 1024), (64, 1024), (128, 1024), (1003, 24), (1024, 64), (1500, 96)])
def test_five_steps(rows, cols, kind, f32):
    g = torch.Generator().manual_seed(rows + cols)
    u, out = run(torch.stack([spectrum(rows, cols, kind, g) for _ in range(2)]), f32, 5)
    for m, o in zip(u, out):
        ref = iterate(m)
        tol, size = tolerance(ref, min(rows, cols), f32, 5, ABC), float(torch.linalg.norm(ref))
        # the tolerance tells: nothing at all, a step less and one term of P would not pass
        assert tol < 0.06 * size
        assert float(torch.linalg.norm(iterate(m, steps=4) - ref)) > 2 * tol
        assert float(torch.linalg.norm(o - ref)) <= tol, (float(torch.linalg.norm(o - ref)), tol, size)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,steps", [
    (16, 512, 6), (16, 512, 9), (32, 1024, 8), (64, 520, 7), (128, 1024, 7), (128, 1024, 9), (1003, 24, 8),
    (2050, 8, 9), (1024, 64, 6), (1500, 104, 9)])
def test_long_runs(rows, cols, steps, kind, f32):
    """Above five of the default steps, and with updates that lack directions."""
    g = torch.Generator().manual_seed(rows + cols + steps)
    u, out = run(torch.stack([spectrum(rows, cols, kind, g) for _ in range(3)]), f32, steps, scale=0.2)
    for m, o in zip(u, out):
        ref = iterate(m, steps=steps, scale=0.2)
        tol = tolerance(ref, min(rows, cols), f32, steps, ABC, 0.2)
        assert float(torch.linalg.norm(o - ref)) <= tol, (float(torch.linalg.norm(o - ref)), tol,
                                                          float(torch.linalg.norm(ref)))


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("rows,cols", [(32, 256), (128, 520), (300, 40)])
def test_twenty_steps_stay_finite(rows, cols, f32):
    g = torch.Generator().manual_seed(5)
    for kind in KINDS:
        _, out = run(spectrum(rows, cols, kind, g)[None], f32, 20)
        assert torch.isfinite(out).all()
        # singular values end between 0.6 and 1.3
        assert float(torch.linalg.svdvals(out[0])[0]) < 1.3, kind


def test_long_runs_in_place_in_groups_and_alone():
    """More matrices than the workspace holds at a time, over the input; a zero
    and a broken matrix among them."""
    g = torch.Generator().manual_seed(11)
    u = torch.stack([matrix(24, 520, "noise", g) for _ in range(300)]).bfloat16()
    u[7] = 0.0
    u[250, 3, 5] = math.nan
    v = u.cuda()
    ws = torch.full((eg.lora_orthogonalize_workspace(300, 24, 520) + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    eg.lora_orthogonalize(v, v, steps=8, workspace=ws[:-4096])
    assert (ws[-4096:] == 0xA5).all()
    v = v.cpu()
    assert (v[7] == 0).all() and torch.isnan(v[250].float()).all()
    for i in (0, 6, 8, 100, 249, 251, 299):
        ref = iterate(u[i].double(), steps=8)
        assert float(torch.linalg.norm(v[i].double() - ref)) <= tolerance(ref, 24, False, 8, ABC)


def test_one_long_matrix():
    g = torch.Generator().manual_seed(13)
    u = torch.randn((1, 8, 200008), generator=g).bfloat16()
    m, out = run(u, False, 7)
    ref = iterate(m[0], steps=7)
    assert float(torch.linalg.norm(out[0] - ref)) <= tolerance(ref, 8, False, 7, ABC)


@pytest.mark.parametrize("abc,steps", [((2.0, -1.5, 0.5), 9), ((1.5, -0.5, 0.0), 15), ((3.0, -3.2, 1.2), 5)])
def test_other_coefficients_up_to_the_limit(abc, steps):
    g = torch.Generator().manual_seed(17)
    for rows, cols in ((32, 512), (512, 96)):
        for kind in ("noise", "rank eight", "dominant"):
            u, out = run(spectrum(rows, cols, kind, g)[None], False, steps, abc)
            ref = iterate(u[0], steps=steps, abc=abc)
            tol = tolerance(ref, min(rows, cols), False, steps, abc)
            assert float(torch.linalg.norm(out[0] - ref)) <= tol, (kind, tol)


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
