"""lora_orthogonalize against the iteration in 64 bits.

Tolerance, from the formats before any run: out is rounded to bf16 once
(2^-9); U U^T in fp32 is off by E with |E| about 2^-18 of its largest
eigenvalue (2^-16 where fp32 entries enter as two bf16 terms).  out = P(G) X,
and a change E of G moves it, in the basis of the singular vectors, by
(P(l_i) - P(l_j)) / (l_i - l_j) E_ij s_j, which the test evaluates in 64
bits; P as two bf16 terms adds 2^-16 |P| s_j in the same basis.
"""
import math

import pytest
import torch

import expand_gemm_gb300 as eg

pytestmark = pytest.mark.gpu
ABC = (3.4445, -4.7750, 2.0315)


def iterate(u, steps=5, abc=ABC, eps=1e-7, scale=1.0):
    """The definition, in u's own precision."""
    a, b, c = abc
    x = u if u.shape[0] <= u.shape[1] else u.T
    x = x / (torch.linalg.norm(x) + eps)
    for _ in range(steps):
        g = x @ x.T
        x = a * x + (b * g + c * (g @ g)) @ x
    x = x if u.shape[0] <= u.shape[1] else x.T
    return scale * x


def tolerance(u, f32, steps=5, abc=ABC, eps=1e-7, scale=1.0):
    """The elementwise allowance beside 2^-8 |ref|."""
    a, b, c = abc
    s = torch.linalg.svdvals(u)
    s = s / (torch.linalg.norm(u) + eps)
    lam = s * s

    def poly(v):
        p, r = torch.ones_like(v), v.clone()
        for _ in range(steps):
            q = a + b * r + c * r * r
            p, r = p * q, r * q * q
        return p
    p = poly(lam)
    d = lam[:, None] - lam[None, :]
    h = 1e-7 * lam.max() + 1e-30
    near = d.abs() < h
    slope = (poly(lam + h) - poly((lam - h).clamp(min=0))) / (2 * h)
    dd = torch.where(near, slope[:, None].expand_as(d), (p[:, None] - p[None, :]) / torch.where(near, torch.ones_like(d), d))
    e = (2.0 ** -16 if f32 else 2.0 ** -18) * lam.max()
    moved = (dd.abs() * e * s[None, :]).max()
    terms = 2.0 ** -16 * p.abs().max() * s.max()
    return float(scale * (moved + terms)) + 1e-12


def matrix(rows, cols, kind, g):
    u = torch.randn((rows, cols), generator=g, dtype=torch.float64)
    k = min(rows, cols)
    if kind == "decay":
        w, _, v = torch.linalg.svd(u, full_matrices=False)
        u = w @ torch.diag(10.0 ** torch.linspace(0, -2.5, k, dtype=torch.float64)) @ v
    elif kind == "dominant":
        u = u + 30.0 * torch.randn((rows, 1), generator=g, dtype=torch.float64) @ torch.randn((1, cols), generator=g, dtype=torch.float64)
    elif kind == "rank one":
        u = torch.randn((rows, 1), generator=g, dtype=torch.float64) @ torch.randn((1, cols), generator=g, dtype=torch.float64)
    return 1e-3 * u


def check(u, out, f32, **kw):
    """u, out: [count, rows, cols] on the GPU."""
    for m, o in zip(u.double().cpu(), out.double().cpu()):
        ref = iterate(m, **kw)
        assert torch.isfinite(o).all()
        off = (o - ref).abs() - 2.0 ** -8 * ref.abs()
        tol = tolerance(m, f32, **kw)
        assert float(off.max()) <= tol, (float(off.max()), tol, m.shape)


SHAPES = [(1, 1, 8), (2, 8, 8), (3, 8, 64), (2, 16, 1000), (5, 24, 520), (2, 40, 2048), (2, 64, 72),
          (3, 96, 1032), (2, 128, 128), (2, 128, 3080), (2, 65, 200),
          (1, 9, 8), (2, 130, 8), (3, 1003, 16), (2, 300, 40), (2, 2050, 64), (2, 513, 104), (2, 1500, 128)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("count,rows,cols", SHAPES)
def test_shapes(count, rows, cols, f32):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    u = torch.stack([matrix(rows, cols, "decay" if i % 2 else "noise", g) for i in range(count)])
    u = (u.float() if f32 else u.bfloat16()).cuda()
    out = torch.full(u.shape, math.nan, dtype=torch.bfloat16, device="cuda")
    eg.lora_orthogonalize(u, out)
    check(u, out, f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("kind", ["dominant", "rank one", "decay"])
def test_spectra(kind, f32):
    g = torch.Generator().manual_seed(3)
    for rows, cols in ((128, 1024), (1024, 64)):
        u = matrix(rows, cols, kind, g)[None]
        u = (u.float() if f32 else u.bfloat16()).cuda()
        out = torch.empty(u.shape, dtype=torch.bfloat16, device="cuda")
        eg.lora_orthogonalize(u, out)
        check(u, out, f32)


@pytest.mark.parametrize("steps", [1, 2, 7])
def test_other_steps_coefficients_and_scale(steps):
    g = torch.Generator().manual_seed(5)
    u = matrix(32, 256, "noise", g)[None].bfloat16().cuda()
    out = torch.empty_like(u)
    kw = dict(steps=steps, abc=(2.0, -1.5, 0.5), eps=1e-3, scale=0.2)
    eg.lora_orthogonalize(u, out, steps=steps, coefficients=kw["abc"], eps=1e-3, scale=0.2)
    check(u, out, False, **kw)


def test_zero_and_broken_matrices_stay_alone():
    g = torch.Generator().manual_seed(7)
    u = torch.stack([matrix(16, 320, "noise", g) for _ in range(5)]).bfloat16().cuda()
    u[1] = 0.0
    u[3, 2, 5] = math.nan
    u[4, 2, 5] = math.inf
    out = torch.empty_like(u)
    eg.lora_orthogonalize(u, out)
    assert (out[1] == 0).all()
    assert torch.isnan(out[3].float()).all()
    assert not torch.isfinite(out[4].float()).any()
    check(u[[0, 2]], out[[0, 2]], False)


def test_in_place_leading_dimensions_and_another_stream():
    g = torch.Generator().manual_seed(11)
    u = torch.stack([matrix(24, 136, "noise", g) for _ in range(6)]).bfloat16().cuda().view(2, 3, 24, 136)
    out = torch.empty_like(u)
    eg.lora_orthogonalize(u, out)
    again = u.clone()
    ws = torch.full((eg.lora_orthogonalize_workspace(6, 24, 136),), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eg.lora_orthogonalize(again, again, workspace=ws)
    s.synchronize()
    assert torch.equal(out, again)
    check(u.view(6, 24, 136), out.view(6, 24, 136), False)


def test_nothing_beside_the_output_is_written():
    g = torch.Generator().manual_seed(13)
    u = matrix(23, 72, "noise", g)[None].float().cuda()
    full = torch.full((23 * 72 + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = full[32:32 + 23 * 72].view(1, 23, 72)
    eg.lora_orthogonalize(u, out)
    check(u, out, True)
    out.fill_(7.0)
    assert (full == 7.0).all()


def test_no_matrices():
    u = torch.empty((0, 16, 64), dtype=torch.bfloat16, device="cuda")
    eg.lora_orthogonalize(u, torch.empty_like(u))


def test_refusals():
    u = torch.zeros((2, 16, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(u)

    def bad(exc, u=u, out=out, **kw):
        with pytest.raises(exc):
            eg.lora_orthogonalize(u, out, **kw)
    bad(TypeError, u=u.half())
    bad(TypeError, out=out.float())
    bad(ValueError, u=u.cpu(), out=out.cpu())
    bad(ValueError, u=u.transpose(1, 2))
    bad(ValueError, out=out[:1])
    bad(ValueError, coefficients=(1.0, 2.0))
    bad(ValueError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    bad(eg.LoraError, steps=0)
    wide = torch.zeros((1, 136, 136), dtype=torch.bfloat16, device="cuda")
    bad(eg.LoraError, u=wide, out=torch.empty_like(wide))                 # both sides over 128
    odd = torch.zeros((1, 16, 60), dtype=torch.bfloat16, device="cuda")
    bad(eg.LoraError, u=odd, out=torch.empty_like(odd))                   # columns not a multiple of 8
    flat = torch.zeros(16 * 64 + 8, dtype=torch.bfloat16, device="cuda")[1:1 + 16 * 64].view(1, 16, 64)
    bad(eg.LoraError, u=flat, out=torch.empty((1, 16, 64), dtype=torch.bfloat16, device="cuda"))
