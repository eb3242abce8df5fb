"""lora_linear_backward as callers use it: dx written over dy or over x,
weights with room for more adapters than the metadata names, sums that are
exact (a lost or doubled token shows in any element), and norms."""
import math

import pytest
import torch

import expand_gemm_gb300 as eg
from test_gpu_linear_backward import LARGE, in_64_bits, make

pytestmark = pytest.mark.gpu

# T, H = sum of the widths, r, L, widths, runs: mma.sync and tcgen05 forms
SQUARE = [(5, 64, 8, 2, (64,), 1), (200, 136, 16, 3, (72, 64), 3), (700, 264, 32, 5, (264,), 7),
          (300, 1000, 40, 5, (523, 477), 30), (3500, 1288, 128, 4, (1024, 128, 136), 300),
          (5000, 1096, 64, 3, (1000, 96), 50)]


def grads(c):
    def blank(shape):
        return torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda")
    return dict(d_lora_a=[blank(a.shape) for a in c["A"]], d_lora_b=[blank(b.shape) for b in c["B"]],
                d_lora_bias=[blank(b.shape[:2]) for b in c["B"]])


def call(c, dy, x, dx, add, out, meta=None):
    if meta is None:
        meta = eg.LoRAKernelMeta.make(c["L"], c["x"].shape[0], "cuda")
        meta.prepare_tensors(c["ids"].cuda())
    eg.lora_linear_backward(dy, x, c["buf"].cuda(), [a.cuda() for a in c["A"]], [b.cuda() for b in c["B"]],
                            c["scale"], meta, dx=dx, add_inputs=add, **out)
    assert int(meta.error_word) == 0


@pytest.mark.parametrize("T,H,r,L,widths,runs", SQUARE)
@pytest.mark.parametrize("add", [True, False])
@pytest.mark.parametrize("over", ["dy", "x"])
def test_dx_in_place(over, add, T, H, r, L, widths, runs):
    """The same bits as with a dx of its own that held the same values."""
    assert sum(widths) == H
    c = make(T, H, r, L, widths, 61, runs=runs)
    dy, x = c["dy"].cuda(), c["x"].cuda()
    want, dx = grads(c), (dy if over == "dy" else x).clone()
    call(c, dy, x, dx, add, want)
    got = grads(c)
    call(c, dy, x, dy if over == "dy" else x, add, got)
    for k in want:
        for s, (u, v) in enumerate(zip(want[k], got[k])):
            assert torch.equal(u, v), (k, s)
    assert torch.equal(dx, dy if over == "dy" else x)


@pytest.mark.parametrize("T,H,r,widths", [(90, 72, 16, (40, 33)), (700, 264, 64, (264, 64)), (3500, 1288, 128, (136, 72))])
def test_weights_with_more_adapters_than_the_metadata(T, H, r, widths):
    """As lora_expand takes them: the rest have no tokens, so zero gradients."""
    named, spare = 3, 2
    c = make(T, H, r, named, widths, 67, runs=5)
    want = grads(c)
    call(c, c["dy"].cuda(), c["x"].cuda(), None, True, want)
    g = torch.Generator().manual_seed(1)
    meta = eg.LoRAKernelMeta.make(named, T, "cuda")
    meta.prepare_tensors(c["ids"].cuda())
    for k, n in (("A", spare), ("B", spare + 1)):
        c[k] = [torch.cat([w, torch.randn((n,) + w.shape[1:], generator=g).bfloat16()]) for w in c[k]]
    got = grads(c)
    dx = c["dx0"].cuda()
    call(c, c["dy"].cuda(), c["x"].cuda(), dx, True, got, meta)
    for k in want:
        for s, (u, v) in enumerate(zip(want[k], got[k])):
            assert torch.equal(u, v[:named]) and (v[named:] == 0).all(), (k, s)
    with pytest.raises(ValueError):                  # fewer adapters than the metadata
        few = {k: [w[:2].contiguous() for w in c[k]] for k in ("A", "B")}
        call(dict(c, **few), c["dy"].cuda(), c["x"].cuda(), None, True, {}, meta)


EXACT = [(1, 64, 8, 1, (64,), 1), (65, 136, 32, 2, (200,), 65), (700, 200, 48, 1, (130, 128), 700),
         (1300, 264, 16, 1, (1100,), 1300), (2100, 136, 24, 3, (75, 61), 1)] + [
         (T, H, r, L, w, runs) for T, H, r, L, w, runs in LARGE if len(w) <= 3]


@pytest.mark.parametrize("T,H,r,L,widths,runs", EXACT)
def test_exact_sums(T, H, r, L, widths, runs):
    """Small whole numbers: every product and sum is exact in the kernels'
    types (g below 256, sums below 2^24), so each output is the exact sum
    rounded to bf16 once."""
    c = make(T, H, r, L, widths, 71, runs=runs)
    g = torch.Generator().manual_seed(T + r)

    def whole(shape, low, high, share=1.0):
        v = torch.randint(low, high + 1, shape, generator=g).float()
        return v * (torch.rand(shape, generator=g) < share)
    c["dy"] = whole(c["dy"].shape, -1, 1).bfloat16()
    c["x"] = whole(c["x"].shape, -3, 3).bfloat16()
    c["buf"] = whole(c["buf"].shape, -4, 4)
    c["A"] = [whole(a.shape, -2, 2).bfloat16() for a in c["A"]]
    c["B"] = [whole(b.shape, -1, 1, 0.1).bfloat16() for b in c["B"]]
    c["dx0"] = whole(c["dx0"].shape, -8, 8).bfloat16()
    off = 0
    for s, w in enumerate(widths):
        top = (c["dy"][:, off:off + w].double().abs() @ c["B"][s].double().abs().amax(0)).max()
        assert top <= 256
        off += w
    ref, mag = in_64_bits(c, True)
    assert max(float(m.max()) for k in ("dA", "dB", "dbias") for m in mag[k]) < 2 ** 24
    out, dx = grads(c), c["dx0"].cuda()
    call(c, c["dy"].cuda(), c["x"].cuda(), dx, True, out)
    assert torch.equal(dx.cpu(), ref["dx"].bfloat16())
    for k, name in (("d_lora_a", "dA"), ("d_lora_b", "dB"), ("d_lora_bias", "dbias")):
        for s, (u, v) in enumerate(zip(out[k], ref[name])):
            assert torch.equal(u.cpu(), v.bfloat16()), (name, s, int((u.cpu() != v.bfloat16()).sum()))


@pytest.mark.parametrize("T,H,r,L,widths,runs", [(1200, 264, 16, 2, (1030, 8), 7)] + LARGE)
def test_norms(T, H, r, L, widths, runs):
    """Independent roundings (2^-9 of g or the buffer, and of the output) add
    up by their squares: the norm of the error is at most 2^-8 of the root of
    the summed squares of the output and of its products.  dbias is an fp32
    sum rounded once."""
    c = make(T, H, r, L, widths, 73, runs=runs)
    ref, mag = in_64_bits(c, False)
    out = grads(c)
    call(c, c["dy"].cuda(), c["x"].cuda(), None, True, out)
    for s, (u, v, m) in enumerate(zip(out["d_lora_bias"], ref["dbias"], mag["dbias"])):
        off = (u.double().cpu() - v).abs() - 2.0 ** -8 * v.abs() - 2.0 ** -12 * m
        assert (off <= 0).all(), ("dbias", s, float(off.max()))
    squares = [[torch.zeros_like(v) for v in ref[k]] for k in ("dA", "dB")]
    for a in range(L):
        at, off = (c["ids"] == a).nonzero()[:, 0], 0
        for s, w in enumerate(widths):
            dy = c["dy"][at, off:off + w].double()
            off += w
            g = c["scale"] * dy @ c["B"][s][a].double()
            squares[0][s][a] = (g * g).T @ c["x"][at].double() ** 2
            squares[1][s][a] = (dy * dy).T @ c["buf"][s, at].double() ** 2
    for k, name, sq in (("d_lora_a", "dA", squares[0]), ("d_lora_b", "dB", squares[1])):
        for s, (u, v, q) in enumerate(zip(out[k], ref[name], sq)):
            off = float(torch.linalg.norm(u.double().cpu() - v))
            assert off <= 2.0 ** -8 * math.sqrt(float((v * v).sum() + q.sum())), (name, s, off)


@pytest.mark.parametrize("T", [1, 2, 5, 20, 63, 64])
@pytest.mark.parametrize("H,r,L,widths,runs", [
    (264, 8, 1, (384,), 1), (136, 16, 5, (72, 131), 1), (512, 32, 2, (1500, 64), 9), (1000, 40, 4, (523, 75, 130), 3),
    (264, 64, 3, (256, 64), 20), (520, 128, 2, (1032, 72, 8), 50), (264, 96, 9, (136, 72, 64), 3), (72, 128, 64, (64,), 1),
    (264, 128, 2, (75, 64), 30)])
@pytest.mark.parametrize("add", [True, False])
def test_small_batches_round_once(add, H, r, L, widths, runs, T):
    """Up to 64 tokens g and the buffer enter the products with 16 bits: each
    output is the rounding to bf16 of a value within d = 2^-15 of the sum of
    magnitudes from the exact one (2^-16 of g or the buffer, and fp32 sums),
    so it is no further off than the exact one's own rounding and 2 d."""
    c = make(T, H, r, L, widths, 79 + T, none=0.1, runs=runs)
    out, dx = grads(c), c["dx0"].cuda()
    call(c, c["dy"].cuda(), c["x"].cuda(), dx, add, out)
    ref, mag = in_64_bits(c, add)
    for name, got in (("dx", [dx]), ("dA", out["d_lora_a"]), ("dB", out["d_lora_b"]), ("dbias", out["d_lora_bias"])):
        want, m = (ref[name], mag[name]) if name != "dx" else ([ref["dx"]], [mag["dx"]])
        for s, (u, v, w) in enumerate(zip(got, want, m)):
            off = (u.double().cpu() - v).abs() - (v.bfloat16().double() - v).abs() - 2.0 ** -14 * w - 1e-30
            assert (off <= 0).all(), (name, s, float(off.max()))
