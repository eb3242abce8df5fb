"""lora_cross_entropy where values break or lie far out: NaN in valid rows and
in the head, a tile of the vocabulary that holds nothing but the target,
targets that are sure although their logit is negative, and logits beyond
1e9.  References in 64 bits; tolerances as in test_gpu_loss, or stated."""
import math

import pytest
import torch

import expand_gemm_gb300 as eg

from test_gpu_loss import check, in_64_bits, make, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dh", [True, False])
@pytest.mark.parametrize("where", ["row", "entry"])
@pytest.mark.parametrize("T", [1, 2, 3])
def test_nan_in_a_valid_row(T, where, dh):
    hidden, weight, targets, share = make(T, 256, 900, 51, masked=0.0)
    ref = in_64_bits(hidden, weight, targets, share)
    if where == "row":
        hidden[0] = math.nan
    else:
        hidden[0, 100] = math.nan
    got = run(hidden, weight, targets, share, head=False, dh=dh)
    assert torch.isnan(got["loss"][0]) and torch.isnan(got["lse"][0])
    assert got["dh"] is None or torch.isnan(got["dh"][0].float()).all()
    check({k: None if got[k] is None else got[k][1:] for k in ("loss", "lse", "dh")},
          {k: v[1:] for k, v in ref.items()}, ("loss", "lse", "dh"))


@pytest.mark.parametrize("T", [1, 2, 3, 70])
@pytest.mark.parametrize("rows", [slice(7, 8), slice(0, 128), slice(0, 900)])
def test_nan_in_the_head_reaches_every_token(T, rows):
    hidden, weight, targets, share = make(T, 64, 900, 53, masked=0.0)
    weight[rows] = math.nan
    got = run(hidden, weight, targets, share, head=False)
    for k in ("loss", "lse", "dh"):
        assert torch.isnan(got[k].float()).all(), k


@pytest.mark.parametrize("T", [1, 2, 3, 40])
def test_a_tile_of_nan_beside_tiles_far_below(T):
    """The other tiles take references of their own."""
    g = torch.Generator().manual_seed(55)
    weight = (-3.2 + 0.01 * torch.randn((512, 64), generator=g)).bfloat16()
    weight[:128] = math.nan
    targets = torch.full((T,), 300, dtype=torch.int32)
    got = run(torch.ones((T, 64)).bfloat16(), weight, targets, torch.ones(T), head=False)
    for k in ("loss", "lse", "dh"):
        assert torch.isnan(got[k].float()).all(), k


def test_one_column_whose_logit_is_nan():
    for T in (1, 2, 5):
        got = run(torch.full((T, 8), math.nan).bfloat16(), torch.ones((1, 8)).bfloat16(),
                  torch.zeros(T, dtype=torch.int32), torch.ones(T), head=False)
        assert torch.isnan(got["loss"]).all() and torch.isnan(got["dh"].float()).all()


@pytest.mark.parametrize("V", [129, 257, 1025])
@pytest.mark.parametrize("level", [-3.2, -0.8, 3.2])
@pytest.mark.parametrize("T", [3, 70])
def test_a_tile_that_holds_only_the_target(T, level, V):
    """The last column is the target and alone in its tile, the others lie
    about 64 level above zero."""
    g = torch.Generator().manual_seed(57)
    weight = (level + 0.02 * torch.randn((V, 64), generator=g)).bfloat16()
    a = (torch.ones((T, 64)).bfloat16(), weight, torch.full((T,), V - 1, dtype=torch.int32), torch.ones(T))
    check(run(*a), in_64_bits(*a))


@pytest.mark.parametrize("T", [1, 2, 40])
@pytest.mark.parametrize("others", [-30.0, -38.0])
def test_sure_of_a_target_with_a_negative_logit(T, others):
    """The loss is about the sum of the others' terms: its error is relative,
    that of the logits' difference (2^-17 of the sum of magnitudes) and a few
    roundings."""
    g = torch.Generator().manual_seed(59)
    H, V = 64, 600
    weight = (others / H + 0.002 * torch.randn((V, H), generator=g)).bfloat16()
    weight[11] = -(2.0 + torch.rand(H, generator=g)).bfloat16() / 32
    hidden = torch.ones((T, H)).bfloat16()
    targets = torch.full((T,), 11, dtype=torch.int32)
    ref = in_64_bits(hidden, weight, targets, torch.ones(T))
    assert (ref["loss"] < 1e-5).all() and (ref["loss"] > 1e-14).all()
    got = run(hidden, weight, targets, torch.ones(T), head=False)
    mag = (hidden.double().abs() @ weight.double().abs().T).amax(1)
    off = (got["loss"].double().cpu() - ref["loss"]).abs()
    assert (off <= ref["loss"] * (2.0 ** -17 * mag + 2.0 ** -19)).all(), (off / ref["loss"]).max()
    check(got, ref, ("lse", "dh"))


@pytest.mark.parametrize("T", [1, 2, 70])
@pytest.mark.parametrize("size", [2.0 ** 31, -2.0 ** 31, 2.0 ** 45, -2.0 ** 45, -2.0 ** 100])
def test_equal_logits_far_from_zero(T, size):
    """Every logit is exactly `size`: the loss is log V, the terms 1 / V."""
    H, V = 64, 700
    hidden = torch.zeros((T, H))
    weight = torch.zeros((V, H))
    hidden[:, 0] = abs(size) ** 0.5 if math.log2(abs(size)) % 2 == 0 else (abs(size) / 2) ** 0.5
    weight[:, 0] = size / hidden[0, 0]
    hidden[:, 1:] = 0.5
    hidden, weight = hidden.bfloat16(), weight.bfloat16()
    assert float(hidden[0, 0]) * float(weight[0, 0]) == size
    targets = torch.arange(T, dtype=torch.int32) * 9
    got = run(hidden, weight, targets, torch.ones(T), head=T > 2)
    assert ((got["loss"].double().cpu() - math.log(V)).abs() <= 2.0 ** -18).all(), got["loss"]
    # sum p W - W_y = 0 up to the terms' roundings, the other columns of W are zero
    dh = got["dh"].double().cpu()
    assert (dh[:, 0].abs() <= 2.0 ** -7 * abs(float(weight[0, 0]))).all() and (dh[:, 1:] == 0).all()
    if T > 2:
        want = (torch.full((V, T), 1.0 / V, dtype=torch.float64))
        want[targets.long(), torch.arange(T)] -= 1.0
        mag = want.abs() @ hidden.double().abs()
        want = want @ hidden.double()
        assert ((got["dw"].double().cpu() - want).abs() <= 2.0 ** -8 * (want.abs() + mag)).all()


@pytest.mark.parametrize("T", [1, 2, 3, 70])
@pytest.mark.parametrize("others", [0.0, 2.0 ** 30])
def test_an_infinite_target_logit(T, others):
    """Past fp32: logsumexp - logit is infinity - infinity, not a loss of 0."""
    hidden = torch.full((T, 64), 2.0 ** 100).bfloat16()
    weight = torch.full((300, 64), others).bfloat16()
    weight[5] = 2.0 ** 30
    got = run(hidden, weight, torch.full((T,), 5, dtype=torch.int32), torch.ones(T), head=False)
    assert torch.isnan(got["loss"]).all() and torch.isnan(got["dh"].float()).all()


@pytest.mark.parametrize("T", [1, 2, 3, 70])
def test_infinite_logits_of_other_columns(T):
    hidden = torch.full((T, 64), 2.0 ** 100).bfloat16()
    weight = torch.zeros((300, 64)).bfloat16()
    weight[200] = 2.0 ** 30
    got = run(hidden, weight, torch.full((T,), 5, dtype=torch.int32), torch.ones(T), head=False)
    assert (got["loss"] == math.inf).all()
    weight[200] = -2.0 ** 30                 # minus infinity: no term at all
    a = (hidden, weight, torch.full((T,), 5, dtype=torch.int32), torch.ones(T))
    got = run(*a, head=False)
    assert ((got["loss"] - math.log(299.0)).abs() <= 2.0 ** -18).all()
    assert torch.isfinite(got["dh"].float()).all()


@pytest.mark.parametrize("T", [1, 2, 300])
def test_hidden_grad_over_hidden(T):
    """The same bits as with a gradient of its own."""
    hidden, weight, targets, share = (v.cuda() for v in make(T, 264, 1025, 61, masked=0.3 if T > 2 else 0.0))
    want = [torch.empty_like(hidden), torch.empty_like(weight) if T > 2 else None, torch.empty(T, device="cuda")]
    eg.lora_cross_entropy(hidden, weight, targets, want[2], token_weight=share, hidden_grad=want[0], weight_grad=want[1])
    got = [hidden, torch.empty_like(weight) if T > 2 else None, torch.empty(T, device="cuda")]
    eg.lora_cross_entropy(hidden, weight, targets, got[2], token_weight=share, hidden_grad=hidden, weight_grad=got[1])
    for u, v in zip(want, got):
        assert u is None or torch.equal(u, v)


@pytest.mark.parametrize("T", [1, 2, 5, 16, 63, 64, 100, 127, 128])
@pytest.mark.parametrize("H,V,masked", [(72, 500, 0.0), (264, 2049, 0.3), (1000, 777, 0.0)])
def test_head_gradient_of_few_tokens_rounds_once(T, H, V, masked):
    """Up to 128 tokens the terms w (p - [y]) enter with 16 bits: dW is the
    rounding to bf16 of a value within d of the exact one, d = 2^-15 (16 bits,
    fp32 sums) and 2^-17 m (the logits) of the sum of magnitudes, so it is no
    further off than the exact one's own rounding and 2 d."""
    hidden, weight, targets, share = make(T, H, V, 67 + T, masked=masked)
    got = run(hidden, weight, targets, share)
    ref = in_64_bits(hidden, weight, targets, share)
    check(got, ref, ("loss", "lse", "dh"))
    h, w = hidden.double(), weight.double()
    valid = targets >= 0
    logits = h @ w.T
    g = torch.exp(logits - torch.logsumexp(logits, 1)[:, None])
    rows = torch.arange(T)[valid]
    y = targets[valid].long()
    g[rows, y] = 0.0
    g[rows, y] = -g[rows].sum(1)
    g = g.abs() * (share * valid)[:, None]
    d = (g * (2.0 ** -15 + 2.0 ** -17 * (h.abs() @ w.abs().T).amax(1))[:, None]).T @ h.abs()
    off = (got["dw"].double().cpu() - ref["dw"]).abs() - (ref["dw"].bfloat16().double() - ref["dw"]).abs() - 2 * d - 1e-30
    assert (off <= 0).all(), (float(off.max()), int((off > 0).sum()))
