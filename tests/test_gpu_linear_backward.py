"""lora_linear_backward against the gradients' formulas in 64 bits, and
against differences of the forward pass.

Tolerances, from the formats before any run: a term of a product is bf16 x
bf16, exact in fp32; g and the buffer are rounded to bf16 once (relative
2^-9 a term) before the second products; fp32 sums of n terms are off by at
most n 2^-24 of the sum of magnitudes (2^-12 covers the n here); outputs are
rounded to bf16 once.  Hence |out - ref| <= 2^-8 |ref| + 2^-8 m, m the same
sum over magnitudes (for products through g, over the magnitudes of g's own
terms only where g is cancelled: 2^-12 of those)."""
import math

import numpy as np
import pytest
import torch

import expand_gemm_gb300 as eg

pytestmark = pytest.mark.gpu


def make(T, H, r, L, widths, seed, none=0.2, runs=1, scale=0.5):
    g = torch.Generator().manual_seed(seed)
    ids = torch.randint(0, L, (T // runs + 1,), generator=g, dtype=torch.int32)
    ids[torch.rand(ids.shape, generator=g) < none] = -1
    ids = ids.repeat_interleave(runs)[:T].contiguous()

    def n(*shape, std=1.0):
        return (torch.randn(shape, generator=g) * std).bfloat16()
    return dict(ids=ids, x=n(T, H), dy=n(T, sum(widths), std=0.1), A=[n(L, r, H, std=0.1) for _ in widths],
                B=[n(L, w, r, std=0.1) for w in widths], buf=torch.randn((len(widths), T, r), generator=g),
                dx0=n(T, H), scale=scale, widths=list(widths), L=L)


def in_64_bits(c, add):
    """The gradients and their error scales (see above)."""
    dx = c["dx0"].double() if add else torch.zeros(c["dx0"].shape, dtype=torch.float64)
    out = dict(dx=dx, dA=[torch.zeros(a.shape, dtype=torch.float64) for a in c["A"]],
               dB=[torch.zeros(b.shape, dtype=torch.float64) for b in c["B"]],
               dbias=[torch.zeros(b.shape[:2], dtype=torch.float64) for b in c["B"]])
    mag = dict(dx=torch.zeros_like(dx), dA=[torch.zeros_like(v) for v in out["dA"]],
               dB=[torch.zeros_like(v) for v in out["dB"]], dbias=[torch.zeros_like(v) for v in out["dbias"]])
    for a in range(c["L"]):
        at = (c["ids"] == a).nonzero()[:, 0]
        if not len(at):
            continue
        x, off = c["x"][at].double(), 0
        for s, w in enumerate(c["widths"]):
            dy = c["dy"][at, off:off + w].double()
            off += w
            A, B, u = c["A"][s][a].double(), c["B"][s][a].double(), c["buf"][s, at].double()
            g = dy @ B
            gm = g.abs() + 2.0 ** -4 * (dy.abs() @ B.abs())
            out["dx"][at] += c["scale"] * (g @ A)
            mag["dx"][at] += c["scale"] * (gm @ A.abs())
            out["dA"][s][a] = c["scale"] * (g.T @ x)
            mag["dA"][s][a] = c["scale"] * (gm.T @ x.abs())
            out["dB"][s][a] = dy.T @ u
            mag["dB"][s][a] = dy.abs().T @ u.abs()
            out["dbias"][s][a] = dy.sum(0)
            mag["dbias"][s][a] = dy.abs().sum(0)
    return out, mag


def run(c, add=True, which=("dx", "dA", "dB", "dbias"), meta=None, **kw):
    dev = "cuda"
    T = c["x"].shape[0]
    if meta is None:
        meta = eg.LoRAKernelMeta.make(c["L"], max(T, 1), dev)
        meta.prepare_tensors(c["ids"].to(dev))

    def blank(shape):
        return torch.full(shape, math.nan, dtype=torch.bfloat16, device=dev)
    got = dict(dx=(c["dx0"].to(dev) if add else blank(c["dx0"].shape)) if "dx" in which else None,
               dA=[blank(a.shape) for a in c["A"]] if "dA" in which else None,
               dB=[blank(b.shape) for b in c["B"]] if "dB" in which else None,
               dbias=[blank(b.shape[:2]) for b in c["B"]] if "dbias" in which else None)
    eg.lora_linear_backward(c["dy"].to(dev), c["x"].to(dev), c["buf"].to(dev), [a.to(dev) for a in c["A"]],
                            [b.to(dev) for b in c["B"]], c["scale"], meta, dx=got["dx"], add_inputs=add,
                            d_lora_a=got["dA"], d_lora_b=got["dB"], d_lora_bias=got["dbias"], **kw)
    assert int(meta.error_word) == 0
    return got


def check(got, ref, what=""):
    out, mag = ref
    for k in ("dx", "dA", "dB", "dbias"):
        if got[k] is None:
            continue
        for i, (v, r, m) in enumerate(zip(*([t[k]] if k == "dx" else t[k] for t in (got, out, mag)))):
            v = v.double().cpu()
            assert torch.isfinite(v).all(), (what, k, i)
            off = (v - r).abs() - 2.0 ** -8 * r.abs() - 2.0 ** -8 * m - 1e-30
            assert (off <= 0).all(), (what, k, i, float(off.max()), int((off > 0).sum()), tuple(off.shape))


CASES = [
    # T, H, r, L, widths, length of the runs of one adapter
    (1, 8, 8, 1, (1,), 1), (1, 64, 16, 3, (64,), 1), (5, 72, 24, 2, (7, 9), 1), (63, 128, 8, 4, (128,), 1),
    (64, 256, 8, 4, (256,), 1), (65, 136, 32, 1, (200,), 65), (130, 264, 64, 5, (64, 192), 3),
    (257, 512, 128, 3, (256, 64, 72), 20), (300, 1000, 40, 5, (523, 75, 130), 30),
    (513, 392, 96, 7, (257,), 50), (200, 128, 16, 64, (96, 96), 1), (1000, 256, 128, 2, (384, 130), 400),
    (700, 200, 48, 1, (130, 128), 700), (256, 1032, 16, 8, (40, 40, 40, 40, 40, 40, 40, 40), 4),
    (90, 64, 8, 1024, (24,), 1), (3500, 264, 128, 4, (136, 72, 64), 300),
    (1300, 200, 64, 3, (64,) * 8, 40), (1300, 136, 128, 3, (64, 72, 80, 88, 8, 16, 24, 32), 1),
    (700, 136, 96, 2, (72,) * 5, 100), (700, 72, 64, 2, (72,) * 5, 3), (260, 64, 128, 1, (64,), 260),
    (5000, 64, 96, 3, (200, 520), 1)]


@pytest.mark.parametrize("T,H,r,L,widths,runs", CASES)
@pytest.mark.parametrize("add", [True, False])
def test_sizes(T, H, r, L, widths, runs, add):
    c = make(T, H, r, L, widths, T + H, runs=runs)
    check(run(c, add), in_64_bits(c, add))


# Slices of more than 1024 columns, whose g is summed by several blocks.
@pytest.mark.parametrize("T,H,r,L,widths,runs", [
    (1, 64, 8, 2, (1500,), 1), (130, 72, 8, 3, (1500, 1031), 1), (700, 64, 32, 5, (2100,), 7),
    (333, 136, 24, 4, (1100, 65, 3001), 1), (64, 64, 16, 1, (5000,), 64), (1200, 64, 16, 40, (1030, 8), 1)])
@pytest.mark.parametrize("add", [True, False])
def test_wide_slices(T, H, r, L, widths, runs, add):
    c = make(T, H, r, L, widths, T + H, runs=runs)
    check(run(c, add), in_64_bits(c, add))


# Large enough for every product to take the tensor-core kernels: tails of all
# kinds, tiles of one adapter's few tokens, g kept beside the stages and not.
LARGE = [
    (3500, 1400, 128, 4, (136, 72, 64), 300), (5000, 1096, 40, 3, (200, 520), 1), (5000, 1096, 128, 3, (200, 520), 1),
    (2600, 2056, 64, 3, (64,) * 8, 40), (2600, 2056, 128, 3, (64, 72, 80, 88, 8, 16, 24, 32), 1),
    (2600, 2056, 96, 2, (72,) * 5, 100), (4000, 1288, 72, 40, (328,), 7), (3900, 1288, 128, 2, (1000, 24), 1300)]


@pytest.mark.parametrize("T,H,r,L,widths,runs", LARGE)
@pytest.mark.parametrize("add", [True, False])
def test_large_sizes(T, H, r, L, widths, runs, add):
    c = make(T, H, r, L, widths, T + H, runs=runs)
    check(run(c, add), in_64_bits(c, add))


@pytest.mark.parametrize("which", [("dx",), ("dA",), ("dB",), ("dbias",), ("dA", "dbias"), ()])
def test_some_outputs_only(which):
    c = make(150, 136, 32, 4, (72, 131), 5)
    check(run(c, which=which), in_64_bits(c, True))


def test_no_adapters_and_no_tokens():
    c = make(100, 64, 16, 3, (72,), 7, none=2.0)
    assert (c["ids"] == -1).all()
    for add in (True, False):
        got = run(c, add)
        want = c["dx0"] if add else torch.zeros_like(c["dx0"])
        assert torch.equal(got["dx"].cpu(), want)
        for k in ("dA", "dB", "dbias"):
            assert (got[k][0] == 0).all(), k
    c = make(0, 64, 16, 3, (72,), 7)
    got = run(c)
    for k in ("dA", "dB", "dbias"):
        assert (got[k][0] == 0).all(), k


def test_tokens_without_an_adapter_reach_nothing():
    """NaN and infinities in their rows of dy, x and the buffer."""
    c = make(200, 136, 24, 3, (130, 62), 11, none=0.3)
    ref = {add: in_64_bits(c, add) for add in (True, False)}
    off = c["ids"] < 0
    c["x"][off] = math.nan
    c["dy"][off] = math.inf
    c["buf"][:, off] = math.nan
    for add in (True, False):
        check(run(c, add), ref[add])


def test_one_adapters_nan_stays_its_own():
    c = make(300, 136, 16, 4, (130,), 13)
    ref = in_64_bits(c, True)
    c["dy"][c["ids"] == 2] = math.nan
    got = run(c)
    keep = torch.tensor([0, 1, 3])
    pick = lambda d: dict(dx=d["dx"][(c["ids"] != 2).to(d["dx"].device)],  # noqa: E731
                          **{k: [v[keep.to(v.device)] for v in d[k]] for k in ("dA", "dB", "dbias")})
    check(pick(got), (pick(ref[0]), pick(ref[1])))
    assert torch.isnan(got["dA"][0][2].float()).all() and torch.isnan(got["dB"][0][2].float()).all()


def test_one_slices_nan_stays_its_own():
    """Slices begin off a 16-byte boundary: their neighbours' columns are not theirs."""
    c = make(100, 72, 16, 2, (61, 30, 37), 17)
    c["dy"][:, 61:91] = math.nan
    got = run(c, which=("dA", "dB", "dbias"))
    clean = dict(c, dy=torch.nan_to_num(c["dy"].float()).bfloat16())
    out, mag = in_64_bits(clean, True)
    pick = lambda d: dict(dx=None, **{k: [d[k][0], d[k][2]] for k in ("dA", "dB", "dbias")})  # noqa: E731
    check(pick(got), (dict(pick(out), dx=None), dict(pick(mag), dx=None)))


@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (5, 0), (16, 3)])
def test_strided_and_unaligned_rows(pad, shift):
    c = make(130, 136, 32, 3, (72, 131), 19)
    T = 130

    def spread(t, fill):
        w = t.shape[1]
        full = torch.full((T * (w + pad) + shift + 64,), fill, dtype=torch.bfloat16, device="cuda")
        v = full[shift:shift + T * (w + pad)].view(T, w + pad)[:, :w]
        v.copy_(t)
        return full, v
    meta = eg.LoRAKernelMeta.make(3, T, "cuda")
    meta.prepare_tensors(c["ids"].cuda())
    _, dy = spread(c["dy"], math.nan)
    _, x = spread(c["x"], math.nan)
    full, dx = spread(c["dx0"], 7.0)
    dA = [torch.empty_like(a, device="cuda") for a in c["A"]]
    dB = [torch.empty_like(b, device="cuda") for b in c["B"]]
    eg.lora_linear_backward(dy, x, c["buf"].cuda(), [a.cuda() for a in c["A"]], [b.cuda() for b in c["B"]],
                            c["scale"], meta, dx=dx, d_lora_a=dA, d_lora_b=dB)
    check(dict(dx=dx, dA=dA, dB=dB, dbias=None), in_64_bits(c, True))
    dx.fill_(7.0)
    assert (full == 7.0).all()


def test_same_bits_on_another_stream_and_workspace():
    c = make(700, 264, 64, 3, (200, 130), 23, runs=5)
    first = run(c)
    ws = torch.full((eg.lora_linear_backward_workspace(700, 264, c["widths"], 64, 3),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run(c, workspace=ws)
    s.synchronize()
    assert torch.equal(first["dx"], again["dx"])
    for k in ("dA", "dB", "dbias"):
        for u, v in zip(first[k], again[k]):
            assert torch.equal(u, v), k


def test_metadata_of_a_larger_batch_buffer():
    """max_num_tokens above the batch, and metadata used for another batch before."""
    c = make(90, 64, 16, 5, (72,), 29)
    meta = eg.LoRAKernelMeta.make(5, 400, "cuda")
    meta.prepare_tensors(torch.randint(-1, 5, (400,), dtype=torch.int32).cuda())
    meta.prepare_tensors(c["ids"].cuda())
    check(run(c, meta=meta), in_64_bits(c, True))


def test_gradients_against_differences():
    """Of f = <dy, layer(x, A, B, bias)> in 64 bits, along random directions."""
    c = make(60, 64, 16, 3, (40, 24), 31)
    g = torch.Generator().manual_seed(1)
    sc, ids = c["scale"], c["ids"].long()

    def forward(x, A, B, bias):
        total, off = 0.0, 0
        for s, w in enumerate(c["widths"]):
            for a in range(c["L"]):
                at = (ids == a).nonzero()[:, 0]
                y = sc * (x[at] @ A[s][a].T) @ B[s][a].T + bias[s][a]
                total = total + (c["dy"][at, off:off + w].double() * y).sum()
            off += w
        return float(total)
    x, A, B = c["x"].double(), [a.double() for a in c["A"]], [b.double() for b in c["B"]]
    bias = [torch.zeros(b.shape[:2], dtype=torch.float64) for b in B]
    for s in range(2):
        for t, a in enumerate(ids.tolist()):
            c["buf"][s, t] = (sc * (A[s][a] @ x[t])).float() if a >= 0 else 0.0
    got, (ref, mag) = run(c, add=False), in_64_bits(c, False)
    e = 1e-3
    for _ in range(3):
        d = [torch.randn(v.shape, generator=g, dtype=torch.float64) for v in [x] + A + B + bias]
        dx, dA, dB, db = d[0], d[1:3], d[3:5], d[5:7]

        def at(k):
            return forward(x + k * dx, [u + k * v for u, v in zip(A, dA)], [u + k * v for u, v in zip(B, dB)],
                           [u + k * v for u, v in zip(bias, db)])
        slope = (at(e) - at(-e)) / (2 * e)
        mine = float((got["dx"].double().cpu() * dx).sum())
        tol = float(((ref["dx"].abs() + mag["dx"]) * dx.abs()).sum())
        for k, ds in (("dA", dA), ("dB", dB), ("dbias", db)):
            for s in range(2):
                mine += float((got[k][s].double().cpu() * ds[s]).sum())
                tol += float(((ref[k][s].abs() + mag[k][s]) * ds[s].abs()).sum())
        assert abs(mine - slope) <= 2.0 ** -8 * tol + 1e-4 * abs(slope), (mine, slope, tol)


def test_refusals():
    c = make(20, 64, 16, 3, (40, 24), 37)
    meta = eg.LoRAKernelMeta.make(3, 20, "cuda")
    meta.prepare_tensors(c["ids"].cuda())
    ok = dict(dy=c["dy"].cuda(), x=c["x"].cuda(), buffer=c["buf"].cuda(), lora_a_stacked=[a.cuda() for a in c["A"]],
              lora_b_stacked=[b.cuda() for b in c["B"]], scale=0.5, meta=meta)

    def bad(exc, **kw):
        with pytest.raises(exc):
            eg.lora_linear_backward(**dict(ok, **kw))
    bf = dict(dtype=torch.bfloat16, device="cuda")
    bad(TypeError, dy=ok["dy"].float())
    bad(TypeError, buffer=ok["buffer"].bfloat16())
    bad(ValueError, x=ok["x"].cpu())
    bad(ValueError, dy=ok["dy"][:, :63])
    bad(ValueError, dy=ok["dy"][:19])
    bad(ValueError, buffer=ok["buffer"][:1])
    bad(ValueError, lora_b_stacked=ok["lora_b_stacked"][:1])
    bad(ValueError, lora_a_stacked=[a[:2].contiguous() for a in ok["lora_a_stacked"]])
    bad(ValueError, dx=torch.empty((20, 72), **bf))
    bad(ValueError, dx=torch.empty((1, 64), **bf).expand(20, 64))
    bad(ValueError, d_lora_a=[torch.empty((3, 16, 64), **bf)])
    bad(ValueError, d_lora_b=[torch.empty((3, 40, 8), **bf), None])
    bad(TypeError, d_lora_bias=[torch.empty((3, 40), device="cuda"), None])
    bad(ValueError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    small = eg.LoRAKernelMeta.make(3, 10, "cuda")
    bad(eg.LoraError, meta=small)                                   # more tokens than the metadata holds
    with pytest.raises(eg.LoraError):
        eg.lora_linear_backward_workspace(20, 64, [40], 12, 3)      # rank not a multiple of 8
