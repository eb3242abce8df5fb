"""The training operators where element offsets pass 32 bits: weights,
gradients and stacks of more than 2^31 elements, and rows that lie 128 KB
apart.  The tolerances are those of the operators' own tests."""
import math

import pytest
import torch

import expand_gemm_gb300 as eg
import test_gpu_linear_backward as back
import test_gpu_loss as loss
import test_gpu_orthogonalize as ortho

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _randn(shape, std=1.0, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=dtype, device=DEV) * std


def _loss_in_chunks(hidden, weight, targets, tw, rows):
    """loss.in_64_bits over a vocabulary whose logits would not fit; dW's
    rows in `rows` only."""
    h, T = hidden.double(), len(targets)
    y = targets.long()
    chunks = [slice(i, min(i + 16384, weight.shape[0])) for i in range(0, weight.shape[0], 16384)]
    lse = torch.full((T,), -math.inf, dtype=torch.float64, device=DEV)
    mag = torch.zeros(T, dtype=torch.float64, device=DEV)
    for c in chunks:
        w = weight[c].double()
        lse = torch.logaddexp(lse, torch.logsumexp(h @ w.T, 1))
        mag = torch.maximum(mag, (h.abs() @ w.abs().T).amax(1))
    own = (h * weight[y].double()).sum(1)
    share = tw.double()
    dh, scale = torch.zeros_like(h), torch.zeros_like(h)
    for c in chunks:
        w = weight[c].double()
        g = torch.exp(h @ w.T - lse[:, None])
        at = ((y >= c.start) & (y < c.stop)).nonzero()[:, 0]
        g[at, y[at] - c.start] -= 1.0
        g *= share[:, None]
        dh += g @ w
        scale += g.abs() @ w.abs()
    rel = 2.0 ** -17 * mag
    ref = dict(loss=share * (lse - own), dh=dh, tol_loss=share * (rel + 2.0 ** -20 * (1 + lse.abs())),
               tol_dh=2.0 ** -8 * dh.abs() + (2.0 ** -8 + rel)[:, None] * scale)
    g = torch.exp(h @ weight[rows].double().T - lse[:, None])
    for j, r in enumerate(rows.tolist()):
        g[y == r, j] -= 1.0
    g *= share[:, None]
    ref["dw"] = g.T @ h
    ref["tol_dw"] = 2.0 ** -8 * ref["dw"].abs() + (g.abs() * (2.0 ** -8 + rel)[:, None]).T @ h.abs()
    return {k: v.cpu() for k, v in ref.items()}


@pytest.mark.parametrize("T,head", [(1, False), (130, True)])
def test_head_of_more_than_2_31_elements(T, head):
    V, H = 530003, 4096
    assert V * H > 2 ** 31
    weight, hidden = _randn((V, H), 0.02, seed=1), _randn((T, H), seed=2)
    targets = torch.randint(0, V, (T,), dtype=torch.int32, device=DEV)
    targets[-1] = V - 1
    tw = 0.5 + torch.rand(T, device=DEV)
    rows = torch.cat([torch.arange(64), torch.arange(V - 128, V), targets.cpu().long()]).unique().to(DEV)
    got = loss.run(hidden, weight, targets, tw, head=head)
    if head:
        got["dw"] = got["dw"][rows]
    loss.check(got, _loss_in_chunks(hidden, weight, targets, tw, rows), ("loss", "dh", "dw"))


def test_loss_of_rows_far_apart():
    T, H, V, ld = 33000, 64, 300, 65600
    assert T * ld > 2 ** 31
    big = torch.zeros((T, ld), dtype=torch.bfloat16, device=DEV)
    hidden, weight, targets, tw = loss.make(T, H, V, 3)
    big[:, 8:8 + H] = hidden.to(DEV)
    out = torch.empty(T, device=DEV)
    eg.lora_cross_entropy(big[:, 8:8 + H], weight.to(DEV), targets.to(DEV), out, token_weight=tw.to(DEV),
                          hidden_grad=big[:, 1000:1000 + H])
    ref = loss.in_64_bits(hidden, weight, targets, tw)
    loss.check(dict(loss=out, dh=big[:, 1000:1000 + H]), ref, ("loss", "dh"))
    assert torch.equal(big[:, 8:8 + H].cpu(), hidden)
    assert not big[:, 1000 + H:].any()


@pytest.mark.parametrize("r,H,n", [(128, 16400, 64), (128, 64, 16400), (32, 65600, 64), (32, 64, 65600)])
def test_adapters_of_more_than_2_31_elements(r, H, n):
    L, T, used = 1024, 200, [0, 511, 1023]
    assert L * r * max(H, n) > 2 ** 31
    c = back.make(T, H, r, 3, [n], 4, runs=20)
    a, b = _randn((L, r, H), 0.1, seed=5), _randn((L, n, r), 0.1, seed=6)
    a[used], b[used] = c["A"][0].to(DEV), c["B"][0].to(DEV)
    ids = torch.where(c["ids"] >= 0, torch.tensor(used, dtype=torch.int32)[c["ids"].clamp(min=0).long()],
                      torch.tensor(-1, dtype=torch.int32))
    meta = eg.LoRAKernelMeta.make(L, T, DEV)
    meta.prepare_tensors(ids.to(DEV))
    da, db = torch.full_like(a, math.nan), torch.full_like(b, math.nan)
    dbias = torch.full((L, n), math.nan, dtype=torch.bfloat16, device=DEV)
    dx = c["dx0"].to(DEV)
    eg.lora_linear_backward(c["dy"].to(DEV), c["x"].to(DEV), c["buf"].to(DEV), [a], [b], c["scale"], meta, dx=dx,
                            d_lora_a=[da], d_lora_b=[db], d_lora_bias=[dbias])
    assert int(meta.error_word) == 0
    back.check(dict(dx=dx, dA=[da[used]], dB=[db[used]], dbias=[dbias[used]]), back.in_64_bits(c, True))
    for g in (da, db, dbias):
        g[used] = 0.0
        assert not any(bool(part.any()) for part in g.split(64))


@pytest.mark.parametrize("r", [16, 128])
def test_gradients_of_rows_far_apart(r):
    T, H, n, ld = 33000, 64, 72, 65600
    assert T * ld > 2 ** 31
    big = torch.zeros((T, ld), dtype=torch.bfloat16, device=DEV)
    c = back.make(T, H, r, 3, [n], 7, runs=100)
    x, dy, dx = big[:, :H], big[:, 128:128 + n], big[:, 512:512 + H]
    x.copy_(c["x"])
    dy.copy_(c["dy"])
    dx.copy_(c["dx0"])
    meta = eg.LoRAKernelMeta.make(3, T, DEV)
    meta.prepare_tensors(c["ids"].to(DEV))
    da, db = torch.empty((3, r, H), dtype=torch.bfloat16, device=DEV), torch.empty((3, n, r), dtype=torch.bfloat16,
                                                                                   device=DEV)
    eg.lora_linear_backward(dy, x, c["buf"].to(DEV), [c["A"][0].to(DEV)], [c["B"][0].to(DEV)], c["scale"], meta,
                            dx=dx, d_lora_a=[da], d_lora_b=[db])
    back.check(dict(dx=dx, dA=[da], dB=[db], dbias=None), back.in_64_bits(c, True))
    assert not big[:, 512 + H:].any()


@pytest.mark.parametrize("count,rows,cols,f32", [(2048, 128, 8200, False), (1024, 65600, 32, True)])
def test_stacks_of_more_than_2_31_elements(count, rows, cols, f32):
    assert count * rows * cols > 2 ** 31
    u = _randn((count, rows, cols), 1e-3, torch.float32 if f32 else torch.bfloat16, seed=8)
    out = torch.empty((count, rows, cols), dtype=torch.bfloat16, device=DEV)
    eg.lora_orthogonalize(u, out)
    at = [0, count // 2, count - 1]
    ortho.check(u[at], out[at], f32)
