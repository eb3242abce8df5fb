"""lora_cross_entropy against the definition in 64 bits (computed here on the
CPU from the formulas), at sizes, masks and values where it can go wrong.

Tolerances, from the formats before any run: a product of bf16 values is
exact in fp32; a logit's sum of H products is off by at most about H 2^-24
of the sum of magnitudes m = sum |h W|, taken as 2^-18 m for the H used
here; a softmax term is off by that relative amount and rounded to bf16
once (2^-9); a gradient is rounded to bf16 once (2^-9).  Hence
  loss:         w (2^-17 max m + 2^-20 (1 + |lse|))
  hidden_grad:  2^-8 (|ref| + w sum_v p_v |W_v|) + 2^-17 max m times the same sum
  weight_grad:  2^-8 (|ref| + sum_t |w_t g_tv h_t|) + likewise.
"""
import math

import numpy as np
import pytest
import torch

import expand_gemm_gb300 as eg

pytestmark = pytest.mark.gpu


def make(T, H, V, seed, std=0.05, masked=0.2, sure=True):
    g = torch.Generator().manual_seed(seed)
    weight = (torch.randn((V, H), generator=g) * std).bfloat16()
    targets = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    hidden = torch.randn((T, H), generator=g)
    if sure:
        hidden += 20.0 * torch.rand((T, 1), generator=g) * weight[targets.long()].float()
    targets[torch.rand((T,), generator=g) < masked] = -100
    return hidden.bfloat16(), weight, targets, 0.25 + torch.rand((T,), generator=g)


def in_64_bits(hidden, weight, targets, token_weight):
    """Loss, logsumexp, gradients and the error scales of the docstring."""
    V = weight.shape[0]
    h, w = hidden.double(), weight.double()
    valid = (targets >= 0) & (targets < V)
    share = torch.where(valid, token_weight.double(), torch.zeros((), dtype=torch.float64))
    h = torch.where(valid[:, None], h, torch.zeros((), dtype=torch.float64))
    y = targets.long().clamp(0, V - 1)
    logits = h @ w.T
    mag = (h.abs() @ w.abs().T).amax(1)
    lse = torch.logsumexp(logits, 1)
    rows = torch.arange(h.shape[0], device=h.device)
    p = torch.exp(logits - lse[:, None])
    g = p.clone()
    g[rows, y] = 0.0
    g[rows, y] = -g.sum(1)                   # -(1 - p_y) without cancellation
    loss = share * torch.where(logits[rows, y] > lse - 1e-3, torch.log1p(-g[rows, y] / p[rows, y]),
                               lse - logits[rows, y])
    g = g * share[:, None]
    dh = g @ w
    dw = g.T @ h
    rel = 2.0 ** -17 * mag
    tol_loss = share * (2.0 ** -17 * mag + 2.0 ** -20 * (1 + lse.abs()))
    tol_dh = 2.0 ** -8 * dh.abs() + (2.0 ** -8 + rel)[:, None] * (g.abs() @ w.abs())
    tol_dw = 2.0 ** -8 * dw.abs() + (g.abs() * (2.0 ** -8 + rel)[:, None]).T @ h.abs()
    zero = torch.zeros((), dtype=torch.float64)
    ref = dict(loss=loss, lse=torch.where(valid, lse, zero), dh=dh, dw=dw, tol_loss=tol_loss,
               tol_lse=2.0 ** -17 * mag + 2.0 ** -20 * (1 + lse.abs()), tol_dh=tol_dh, tol_dw=tol_dw)
    return {k: v.cpu() for k, v in ref.items()}


def run(hidden, weight, targets, token_weight, head=True, dh=True, **kw):
    T, H = hidden.shape
    dev = "cuda"
    d = dict(loss=torch.full((T,), math.nan, device=dev), lse=torch.full((T,), math.nan, device=dev),
             dh=torch.full((T, H), math.nan, dtype=torch.bfloat16, device=dev) if dh else None,
             dw=torch.full(weight.shape, math.nan, dtype=torch.bfloat16, device=dev) if head else None,
             err=torch.full((1,), -1, dtype=torch.int32, device=dev))
    eg.lora_cross_entropy(hidden.to(dev) if not hidden.is_cuda else hidden, weight.to(dev), targets.to(dev),
                          d["loss"], token_weight=None if token_weight is None else token_weight.to(dev),
                          logsumexp=d["lse"], hidden_grad=d["dh"], weight_grad=d["dw"],
                          error_word=d["err"], **kw)
    return d


def check(got, ref, names=("loss", "lse", "dh", "dw")):
    for k in names:
        if got[k] is None:
            continue
        v = got[k].double().cpu()
        assert torch.isfinite(v).all(), k
        off = (v - ref[k]).abs() - ref["tol_" + k] - 1e-30
        assert (off <= 0).all(), (k, float(off.max()), int((off > 0).sum()), off.shape)


@pytest.mark.parametrize("T,H,V", [
    (1, 8, 1), (1, 64, 2), (1, 256, 1000), (2, 72, 255), (31, 64, 256), (64, 128, 257), (129, 200, 513),
    (255, 64, 1024), (256, 256, 1025), (257, 264, 2049), (300, 512, 4100), (700, 136, 3001)])
def test_sizes(T, H, V):
    a = make(T, H, V, 100 + T)
    check(run(*a), in_64_bits(*a))


@pytest.mark.parametrize("T,H,V", [(1, 8, 1), (1, 64, 2), (1, 4096, 1000), (2, 1032, 777), (2, 2056, 3000),
                                   (1, 8192, 500), (2, 8192, 1200), (1, 8200, 300), (3, 256, 900)])
@pytest.mark.parametrize("dh", [True, False])
def test_one_or_two_tokens(T, H, V, dh):
    a = make(T, H, V, 200 + H + T, std=0.1 if H < 2000 else 0.02, masked=0.0)
    check(run(*a, head=False, dh=dh), in_64_bits(*a))


@pytest.mark.parametrize("std", [3.0, 30.0])
def test_one_or_two_tokens_wide_logits_and_masks(std):
    for seed in range(4):
        hidden, weight, targets, share = make(2, 64, 1500, seed, std=std, masked=0.0, sure=False)
        check(run(hidden, weight, targets, share, head=False), in_64_bits(hidden, weight, targets, share))
        targets[seed % 2] = (-1, 1500)[seed // 2]
        hidden[seed % 2] = math.nan
        got = run(hidden, weight, targets, share, head=False)
        assert int(got["err"]) == seed // 2
        check(got, in_64_bits(torch.nan_to_num(hidden.float()).bfloat16(), weight, targets, share))
    targets[:] = -100
    got = run(hidden, weight, targets, share, head=False)
    for k in ("loss", "lse", "dh"):
        assert (got[k] == 0).all()


@pytest.mark.parametrize("head,dh", [(False, False), (False, True), (True, False)])
def test_without_some_gradients(head, dh):
    a = make(200, 128, 777, 3)
    check(run(*a, head=head, dh=dh), in_64_bits(*a))


@pytest.mark.parametrize("V,std", [(20000, 0.1), (17000, 3.0)])
def test_several_pieces(V, std):
    """More logits than one piece's scratch takes (2^27)."""
    a = make(8200, 64, V, 5, std=std)
    check(run(*a), in_64_bits(*(v.cuda() for v in a)))


@pytest.mark.parametrize("std", [3.0, 30.0])
def test_wide_logits(std):
    """Logits of tens to thousands: tiles leave the window around the reference."""
    a = make(130, 64, 1500, 7, std=std, sure=False)
    check(run(*a), in_64_bits(*a))


def test_low_logits():
    """Every logit far below zero, and the columns fall further from tile to tile."""
    T, H, V = 70, 64, 1100
    hidden = torch.ones((T, H)).bfloat16()
    weight = (-2.0 - torch.arange(V)[:, None] / 256.0 + 0.01 * torch.randn((V, H), generator=torch.Generator().manual_seed(1))).bfloat16()
    for w in (weight, weight.flip(0).contiguous()):
        a = (hidden, w, torch.arange(T, dtype=torch.int32) * 13, torch.ones(T))
        check(run(*a), in_64_bits(*a))


def test_sure_of_the_target():
    """1 - p_y down to 1e-20: the loss and the gradient keep their digits."""
    T, H, V = 40, 64, 600
    hidden, weight, targets, share = make(T, H, V, 9, std=0.02, masked=0.0, sure=False)
    weight[:, 0] = 0.0
    weight[targets.long(), 0] = 4.0
    targets = targets[:1].repeat(T)
    weight[:, 0] = 0.0
    weight[targets[0].long(), 0] = 4.0
    hidden[:, 0] = torch.linspace(0, 12, T).bfloat16()
    a = (hidden, weight, targets, share)
    check(run(*a), in_64_bits(*a))


def test_no_target_anywhere_and_no_tokens():
    hidden, weight, targets, share = make(50, 64, 300, 11)
    targets = torch.full_like(targets, -1)
    got = run(hidden, weight, targets, share)
    for k in ("loss", "lse", "dh", "dw"):
        assert (got[k] == 0).all(), k
    got = run(hidden[:0], weight, targets[:0], share[:0])
    assert (got["dw"] == 0).all() and got["loss"].numel() == 0


def test_rows_without_a_target_are_not_read():
    """NaN and infinity in masked rows reach no output."""
    hidden, weight, targets, share = make(300, 64, 700, 13, masked=0.4)
    ref = in_64_bits(hidden, weight, targets, share)
    hidden[targets < 0] = math.nan
    share[targets < 0] = math.inf
    hidden[(targets < 0).nonzero()[0]] = math.inf
    check(run(hidden, weight, targets, share), ref)


def test_targets_past_the_vocabulary_are_counted():
    hidden, weight, targets, share = make(90, 64, 500, 17, masked=0.0)
    targets[[3, 50, 89]] = 500
    targets[7] = 2 ** 31 - 1
    got = run(hidden, weight, targets, share)
    assert int(got["err"]) == 4
    check(got, in_64_bits(hidden, weight, targets, share))


def test_a_row_with_nan_stays_alone():
    hidden, weight, targets, share = make(64, 64, 400, 19, masked=0.0)
    ref = in_64_bits(hidden, weight, targets, share)
    hidden[5, 3] = math.nan
    got = run(hidden, weight, targets, share, head=False)
    assert torch.isnan(got["loss"][5]) and torch.isnan(got["dh"][5].float()).all()
    keep = torch.arange(64) != 5
    for k in ("loss", "lse", "dh"):
        v = got[k].double().cpu()[keep]
        assert ((v - ref[k][keep]).abs() <= ref["tol_" + k][keep] + 1e-30).all(), k


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (16, 1)])
def test_strided_and_unaligned_rows(pad, shift):
    hidden, weight, targets, share = make(70, 72, 300, 23)
    T, H = hidden.shape

    def spread(fill):
        full = torch.full((T * (H + pad) + shift + 64,), fill, dtype=torch.bfloat16, device="cuda")
        return full, full[shift:shift + T * (H + pad)].view(T, H + pad)[:, :H]
    _, h = spread(math.nan)
    h.copy_(hidden)
    full, dh = spread(7.0)
    loss = torch.empty(T, device="cuda")
    eg.lora_cross_entropy(h, weight.cuda(), targets.cuda(), loss, token_weight=share.cuda(), hidden_grad=dh)
    ref = in_64_bits(hidden, weight, targets, share)
    check(dict(loss=loss, dh=dh, lse=None, dw=None), ref)
    dh.fill_(7.0)
    assert (full == 7.0).all()            # nothing beside the rows was written


def test_same_inputs_same_bits_on_another_stream_and_workspace():
    a = make(300, 128, 2000, 29)
    first = run(*a)
    ws = torch.full((eg.lora_cross_entropy_workspace(300, 128, 2000, weight_grad=True),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        again = run(*a, workspace=ws)
    s.synchronize()
    for k in ("loss", "lse", "dh", "dw"):
        assert torch.equal(first[k], again[k]), k


def test_gradient_against_differences():
    """dh and dW of the loss's sum against central differences of the loss in 64 bits."""
    hidden, weight, targets, share = make(12, 64, 200, 31)
    got = run(hidden, weight, targets, share)
    ref = in_64_bits(hidden, weight, targets, share)
    g = torch.Generator().manual_seed(1)
    e = 1e-4
    for _ in range(3):
        dh, dw = (torch.randn(v.shape, generator=g, dtype=torch.float64) for v in (hidden, weight))
        up = in_64_bits(hidden.double() + e * dh, weight.double() + e * dw, targets, share)["loss"].sum()
        down = in_64_bits(hidden.double() - e * dh, weight.double() - e * dw, targets, share)["loss"].sum()
        slope = float(up - down) / (2 * e)
        mine = float((got["dh"].double().cpu() * dh).sum() + (got["dw"].double().cpu() * dw).sum())
        tol = float((ref["tol_dh"] * dh.abs()).sum() + (ref["tol_dw"] * dw.abs()).sum()) + 1e-5
        assert abs(mine - slope) <= tol, (mine, slope, tol)


def test_in_a_graph():
    a = make(100, 64, 500, 37)
    ref = in_64_bits(*a)
    h, w, t, s = (v.cuda() for v in a)
    loss, dh = torch.zeros(100, device="cuda"), torch.zeros_like(h)
    ws = torch.empty(eg.lora_cross_entropy_workspace(100, 64, 500), dtype=torch.uint8, device="cuda")
    eg.lora_cross_entropy(h, w, t, loss, token_weight=s, hidden_grad=dh, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        eg.lora_cross_entropy(h, w, t, loss, token_weight=s, hidden_grad=dh, workspace=ws)
    loss.zero_()
    dh.zero_()
    graph.replay()
    check(dict(loss=loss, dh=dh, lse=None, dw=None), ref)


def test_refusals():
    hidden, weight, targets, share = (v.cuda() for v in make(20, 64, 100, 41))
    loss = torch.zeros(20, device="cuda")
    ok = dict(hidden=hidden, weight=weight, targets=targets, loss=loss)

    def bad(exc, **kw):
        with pytest.raises(exc):
            eg.lora_cross_entropy(**dict(ok, **kw))
    bad(TypeError, hidden=hidden.float())
    bad(TypeError, weight=weight.half())
    bad(TypeError, targets=targets.long())
    bad(TypeError, loss=loss.bfloat16())
    bad(ValueError, hidden=hidden.cpu())
    bad(ValueError, hidden=hidden[:1].expand(20, 64))
    bad(ValueError, weight=weight[:, :32])
    bad(ValueError, weight=weight.T.contiguous().T)
    bad(ValueError, targets=targets[:19])
    bad(ValueError, loss=loss[:19])
    bad(ValueError, token_weight=share[:3])
    bad(ValueError, hidden_grad=torch.empty((20, 72), dtype=torch.bfloat16, device="cuda"))
    bad(ValueError, weight_grad=torch.empty((99, 64), dtype=torch.bfloat16, device="cuda"))
    bad(ValueError, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    ws = torch.empty(eg.lora_cross_entropy_workspace(20, 64, 100) + 8, dtype=torch.uint8, device="cuda")
    bad(eg.LoraError, workspace=ws[8:])                                       # not 256-byte aligned
    odd = torch.zeros((20, 60), dtype=torch.bfloat16, device="cuda")
    bad(eg.LoraError, hidden=odd, weight=odd)                                 # hidden size not a multiple of 8
    with pytest.raises(eg.LoraError):
        eg.lora_cross_entropy_workspace(-1, 64, 100)
