"""The operators that train a batch's adapters, as measured cases.

Three operators follow one another in a training step: the loss over the
vocabulary with its gradient (:func:`lora_cross_entropy`), the gradients of
many adapters of one linear layer (:func:`lora_linear_backward`), and the
orthogonalised update of stacked adapters (:func:`lora_orthogonalize`).
Where ``own`` is false ``run`` computes them in elementary torch operations
in 32 bits; where it is true it calls the framework.
"""
from functools import reduce
import math

import numpy as np
import torch

own = False

COEFFICIENTS = (3.4445, -4.7750, 2.0315)
EPS = 1e-7
STEPS = 5


def listed():
    return [
        # one position: the latency of a loss on a single sampled token (adapting on a stream)
        dict(name="loss_one", op="loss", tokens=1, hidden=4096, vocab=32000, masked=0.0, head=False),
        # the logits rows of a decode batch: 256 positions, hidden 4096, vocabulary 32000
        dict(name="loss_256", op="loss", tokens=256, hidden=4096, vocab=32000, masked=0.0, head=False),
        # a batch of prompts and answers: the prompts' third has no target
        dict(name="loss_8192", op="loss", tokens=8192, hidden=4096, vocab=32000, masked=0.33, head=False),
        # the head is trained too, sizes that fill no tile
        dict(name="loss_head_odd", op="loss", tokens=1031, hidden=1000, vocab=50021, masked=0.1, head=True),
        # the smallest layer with adapters: 64 tokens, rank 8, bias
        dict(name="back_tiny", op="backward", tokens=64, hidden=256, rank=8, loras=4, slices="256",
             ids="token", none=0.2, bias=True),
        # gate and up projections, per-token ids over 32 adapters, bias
        dict(name="back_mlp", op="backward", tokens=2048, hidden=4096, rank=32, loras=32,
             slices="11008,11008", ids="token", none=0.1, bias=True),
        # q, k and v of 16384 tokens in sequences, rank 128, ids by sequence over 64 adapters
        dict(name="back_large", op="backward", tokens=16384, hidden=8192, rank=128, loras=64,
             slices="8192,1024,1024", ids="sequence", none=0.2, bias=False),
        # sizes that fill no tile, slices that begin off a 16-byte boundary
        dict(name="back_odd", op="backward", tokens=1001, hidden=1000, rank=24, loras=5,
             slices="523,75,130", ids="sequence", none=0.1, bias=True),
        # the A factors of one layer's eight adapters
        dict(name="ortho_a_small", op="ortho", matrices=8, rows=16, cols=4096, f32=False),
        # the B factors of gate and up, from momentum in 32 bits
        dict(name="ortho_b_mlp", op="ortho", matrices=64, rows=11008, cols=32, f32=True),
        # the A factors of q, k and v of 64 adapters at rank 128
        dict(name="ortho_a_large", op="ortho", matrices=192, rows=128, cols=8192, f32=False),
        # odd counts and widths, from momentum in 32 bits
        dict(name="ortho_odd", op="ortho", matrices=5, rows=1003, cols=40, f32=True),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["loss", "backward", "ortho"])
    if op == "loss":
        head = rng.random() < 0.3
        return dict(op=op, tokens=_between(rng, 1, 5400), hidden=8 * _between(rng, 32, 512),
                    vocab=_between(rng, 1000, 21000 if head else 32000),
                    masked=rng.choice([0.0, 0.1, 0.33, 0.6]), head=head)
    if op == "backward":
        n = rng.choice([1, 2, 3])
        return dict(op=op, tokens=_between(rng, 1, 16384), hidden=8 * _between(rng, 32, 1024),
                    rank=rng.choice([8, 16, 24, 32, 64, 96, 128]), loras=_between(rng, 1, 64),
                    slices=",".join(str(_between(rng, 60, 10240 // n)) if rng.random() < 0.4
                                    else str(64 * _between(rng, 1, 160 // n)) for _ in range(n)),
                    ids=rng.choice(["token", "sequence"]), none=rng.choice([0.0, 0.1, 0.5]),
                    bias=rng.random() < 0.5)
    rank, wide = 8 * rng.choice([1, 2, 3, 4, 5, 8, 12, 16]), 8 * _between(rng, 16, 1376)
    rows, cols = (rank, wide) if rng.random() < 0.5 else (wide + rng.choice([0, 3]), rank)
    return dict(op=op, matrices=_between(rng, 1, 96), rows=rows, cols=cols, f32=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _slices(case):
    return [int(v) for v in case["slices"].split(",")]


def _ids(case, seed):
    """An adapter id per token (-1: none), uniform per token, or one per sequence by a
    Zipf law with exponent 1.1."""
    rng = np.random.Generator(np.random.PCG64(seed))
    T, L = case["tokens"], case["loras"]
    if case["ids"] == "token":
        ids = rng.integers(0, L, size=T)
        ids[rng.random(T) < case["none"]] = -1
        return ids.astype(np.int32)
    p = (np.arange(L) + 1.0) ** -1.1
    ends = np.cumsum(rng.integers(max(1, T // 64), max(2, T // 8) + 1, size=T))
    seq = np.searchsorted(ends, np.arange(T), side="right")
    by = rng.choice(L, size=T + 1, p=p / p.sum())
    by[rng.random(T + 1) < case["none"]] = -1
    return by[seq].astype(np.int32)


def _normal(g, shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).bfloat16()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"loss": _prepare_loss, "backward": _prepare_backward, "ortho": _prepare_ortho}[case["op"]](case, seed, g)


def _prepare_loss(case, seed, g):
    T, H, V = case["tokens"], case["hidden"], case["vocab"]
    weight = _normal(g, (V, H), 0.02)
    targets = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    # a trained model is sure of some tokens: part of the hidden states point at their target
    sure = 8.0 * torch.rand((T, 1), generator=g, device="cuda") * (4096 / H)
    hidden = (torch.randn((T, H), generator=g, device="cuda") + sure * weight[targets.long()].float()).bfloat16()
    masked = torch.rand((T,), generator=g, device="cuda") < case["masked"]
    targets[masked] = -100
    # each token's share of the batch's loss, scaled as a loss scaler does
    token_weight = 0.5 + torch.rand((T,), generator=g, device="cuda")
    state = dict(case=case, hidden=hidden, weight=weight, targets=targets, token_weight=token_weight)
    if own:
        import expand_gemm_gb300 as eg
        state.update(
            loss=torch.empty(T, device="cuda"), hidden_grad=torch.empty_like(hidden),
            weight_grad=torch.empty_like(weight) if case["head"] else None,
            workspace=torch.empty(eg.lora_cross_entropy_workspace(T, H, V, weight_grad=case["head"]),
                                  dtype=torch.uint8, device="cuda"))
    return state


def _prepare_backward(case, seed, g):
    T, H, r, L, widths = case["tokens"], case["hidden"], case["rank"], case["loras"], _slices(case)
    ids_host = _ids(case, seed)
    ids = torch.from_numpy(ids_host).cuda()
    x = _normal(g, (T, H))
    dy = _normal(g, (T, sum(widths)), 0.1)
    A = [_normal(g, (L, r, H), 0.02) for _ in widths]
    B = [_normal(g, (L, n, r), 0.02) for n in widths]
    scale = 0.5
    buffer = torch.zeros((len(widths), T, r), device="cuda")      # what the forward pass left
    for a in sorted(set(ids_host[ids_host >= 0].tolist())):
        at = (ids == a).nonzero()[:, 0]
        for s, w in enumerate(A):
            buffer[s, at] = scale * (x[at].float() @ w[a].float().T)
    state = dict(case=case, ids=ids, x=x, dy=dy, A=A, B=B, scale=scale, buffer=buffer)
    if own:
        import expand_gemm_gb300 as eg
        meta = eg.LoRAKernelMeta.make(L, T, "cuda")
        meta.prepare_tensors(ids)
        state.update(
            meta=meta, dx=torch.empty_like(x), dA=[torch.empty_like(a) for a in A],
            dB=[torch.empty_like(b) for b in B],
            dbias=[torch.empty((L, n), dtype=torch.bfloat16, device="cuda") for n in widths] if case["bias"] else None,
            workspace=torch.empty(eg.lora_linear_backward_workspace(T, H, widths, r, L),
                                  dtype=torch.uint8, device="cuda"))
    return state


def _prepare_ortho(case, seed, g):
    n, rows, cols = case["matrices"], case["rows"], case["cols"]
    # a gradient: a few strong directions over noise
    k = max(1, min(rows, cols) // 4)
    u = torch.randn((n, rows, k), generator=g, device="cuda") * torch.logspace(0, -1.5, k, device="cuda")
    update = u @ torch.randn((n, k, cols), generator=g, device="cuda")
    update = 1e-3 * (update + 0.3 * torch.randn(update.shape, generator=g, device="cuda"))
    update = update if case["f32"] else update.bfloat16()
    state = dict(case=case, update=update)
    if own:
        import expand_gemm_gb300 as eg
        state.update(out=torch.empty(update.shape, dtype=torch.bfloat16, device="cuda"),
                     workspace=torch.empty(eg.lora_orthogonalize_workspace(n, rows, cols),
                                           dtype=torch.uint8, device="cuda"))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"loss": _own_loss, "backward": _own_backward, "ortho": _own_ortho}[op](state)
    return {"loss": _plain_loss, "backward": _plain_backward, "ortho": _plain_ortho}[op](state)


def _own_loss(s):
    import expand_gemm_gb300 as eg
    eg.lora_cross_entropy(s["hidden"], s["weight"], s["targets"], s["loss"], token_weight=s["token_weight"],
                          hidden_grad=s["hidden_grad"], weight_grad=s["weight_grad"], workspace=s["workspace"])
    return {"loss": s["loss"], "hidden_grad": s["hidden_grad"], "weight_grad": s["weight_grad"]}


def _own_backward(s):
    import expand_gemm_gb300 as eg
    eg.lora_linear_backward(s["dy"], s["x"], s["buffer"], s["A"], s["B"], s["scale"], s["meta"], dx=s["dx"],
                            add_inputs=False, d_lora_a=s["dA"], d_lora_b=s["dB"], d_lora_bias=s["dbias"],
                            workspace=s["workspace"])
    return {"dx": s["dx"], "dA": s["dA"], "dB": s["dB"], "dbias": s["dbias"]}


def _own_ortho(s):
    import expand_gemm_gb300 as eg
    eg.lora_orthogonalize(s["update"], s["out"], workspace=s["workspace"])
    return {"out": s["out"]}


def _plain_loss(s):
    h, w, t, share = s["hidden"].float(), s["weight"].float(), s["targets"].long(), s["token_weight"]
    valid = t >= 0
    at = t.clamp(min=0)[:, None]
    share = torch.where(valid, share, torch.zeros_like(share))
    logits = h @ w.T
    top = logits.amax(1, keepdim=True)
    e = torch.exp(logits - top)
    total = e.sum(1, keepdim=True)
    loss = share * (torch.log(total) + top - logits.gather(1, at))[:, 0]
    grad = e / total
    grad.scatter_add_(1, at, torch.full_like(total, -1.0))
    grad *= share[:, None]
    return {"loss": loss, "hidden_grad": (grad @ w).bfloat16(),
            "weight_grad": (grad.T @ h).bfloat16() if s["case"]["head"] else None}


def _plain_backward(s):
    """Tokens are laid out by adapter, each adapter's run padded to whole blocks of 64 rows, so that
    every product is one batched product over blocks."""
    case, ids, widths, block = s["case"], s["ids"].long(), _slices(s["case"]), 64
    T, H, r, L = case["tokens"], case["hidden"], case["rank"], case["loras"]
    blocks = T // block + L + 1
    key = torch.where(ids < 0, torch.full_like(ids, L), ids)
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(L + 1, device=ids.device)).sum(0)
    first = torch.cumsum(counts, 0) - counts
    padded = (counts + block - 1) // block
    begin = torch.cumsum(padded, 0) - padded
    place = begin[key[order]] * block + torch.arange(T, device=ids.device) - first[key[order]]
    # tokens without an adapter all go to one row that is left zero
    spare = blocks * block
    place = torch.where(key[order] < L, place, torch.full_like(place, spare))

    def laid(v):
        out = torch.zeros((spare + 1, v.shape[1]), device=v.device)
        out[place] = v[order].float()
        return out[:spare].view(blocks, block, -1)

    owner = (torch.arange(blocks, device=ids.device)[:, None] >= (begin + padded)[None, :L]).sum(1).clamp(max=L - 1)
    member = (owner[None, :] == torch.arange(L, device=ids.device)[:, None]).float()

    def joined(v):                                  # the blocks of an adapter, summed
        return (member @ v.reshape(blocks, -1)).view(L, *v.shape[1:])

    x = laid(s["x"])
    dys = [laid(v) for v in torch.split(s["dy"], widths, 1)]
    us = [laid(u) for u in s["buffer"]]
    gs = [dy @ b.float()[owner] for dy, b in zip(dys, s["B"])]
    dx = s["scale"] * sum(g @ a.float()[owner] for g, a in zip(gs, s["A"]))
    dA = [(s["scale"] * joined(g.transpose(1, 2) @ x)).bfloat16() for g in gs]
    dB = [joined(dy.transpose(1, 2) @ u).bfloat16() for dy, u in zip(dys, us)]
    dbias = [joined(dy.sum(1)).bfloat16() for dy in dys] if case["bias"] else None
    flat = torch.cat([dx.view(spare, H), torch.zeros((1, H), device=ids.device)])
    out = torch.empty((T, H), dtype=torch.bfloat16, device=ids.device)
    out[order] = flat[place].bfloat16()
    return {"dx": out, "dA": dA, "dB": dB, "dbias": dbias}


def _plain_ortho(s):
    a, b, c = COEFFICIENTS
    x = s["update"].float()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + EPS)

    def step(x, _):
        gram = x @ x.transpose(1, 2)
        return a * x + (b * gram + c * (gram @ gram)) @ x

    x = reduce(step, range(STEPS), x)
    x = x.transpose(1, 2) if tall else x
    return {"out": x.bfloat16().contiguous()}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] == "loss":
        T, H, V = case["tokens"], case["hidden"], case["vocab"]
        n = max(1.0, T * (1 - case["masked"]))
        return {"bytes": n * H * 2 + T * H * 2 + V * H * 2 * (2 if case["head"] else 1) + T * 12,
                "flops": (6.0 if case["head"] else 4.0) * n * H * V}
    if case["op"] == "backward":
        H, r, L, widths = case["hidden"], case["rank"], case["loras"], _slices(case)
        ids = _ids(case, 1)
        n, d, S, N = int((ids >= 0).sum()), len(set(ids[ids >= 0].tolist())), len(widths), sum(widths)
        factors = S * r * H * 2 + N * r * 2
        return {"bytes": n * (H + N) * 2 + case["tokens"] * H * 2 + n * S * r * 4 + (d + L) * factors + (L * N * 2 if case["bias"] else 0) + 4,
                "flops": 4.0 * n * r * (N + S * H) + 1}
    n, size, r = case["matrices"], case["rows"] * case["cols"], min(case["rows"], case["cols"])
    return {"bytes": n * size * (6 if case["f32"] else 4), "flops": 3.0 * n * size * r}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    return {"loss": _exact_loss, "backward": _exact_backward, "ortho": _exact_ortho}[case["op"]](state)


def _exact_loss(s):
    T = s["hidden"].shape[0]
    w = s["weight"].double()
    loss = torch.zeros(T, dtype=torch.float64, device="cuda")
    dh = torch.zeros(s["hidden"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros_like(w) if s["case"]["head"] else None
    for at in (s["targets"] >= 0).nonzero()[:, 0].split(2048):
        h, y, share = s["hidden"][at].double(), s["targets"][at].long(), s["token_weight"][at].double()
        p = h @ w.T
        lse = torch.logsumexp(p, 1)
        rows = torch.arange(len(at), device="cuda")
        loss[at] = share * (lse - p[rows, y])
        p = torch.exp(p - lse[:, None]) * share[:, None]
        p[rows, y] -= share
        dh[at] = p @ w
        if dw is not None:
            dw += p.T @ h
    return {"loss": loss, "hidden_grad": dh, "weight_grad": dw}


def _exact_backward(s):
    case, widths = s["case"], _slices(s["case"])
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dA = [torch.zeros(a.shape, dtype=torch.float64, device="cuda") for a in s["A"]]
    dB = [torch.zeros(b.shape, dtype=torch.float64, device="cuda") for b in s["B"]]
    dbias = [torch.zeros(b.shape[:2], dtype=torch.float64, device="cuda") for b in s["B"]]
    for a in range(case["loras"]):
        at = (s["ids"] == a).nonzero()[:, 0]
        x, start = s["x"][at].double(), 0
        for k, n in enumerate(widths):
            dy = s["dy"][at, start:start + n].double()
            start += n
            g = dy @ s["B"][k][a].double()
            dx[at] += s["scale"] * (g @ s["A"][k][a].double())
            dA[k][a] = s["scale"] * (g.T @ x)
            dB[k][a] = dy.T @ s["buffer"][k, at].double()
            dbias[k][a] = dy.sum(0)
    return {"dx": dx, "dA": dA, "dB": dB, "dbias": dbias if case["bias"] else None}


def _exact_ortho(s):
    a, b, c = COEFFICIENTS
    out = []
    for m in s["update"]:
        x = m.double() if m.shape[0] <= m.shape[1] else m.double().T
        x = x / (torch.linalg.norm(x) + EPS)
        for _ in range(STEPS):
            gram = x @ x.T
            x = a * x + b * (gram @ x) + c * (gram @ (gram @ x))
        out.append(x if m.shape[0] <= m.shape[1] else x.T)
    return {"out": torch.stack(out)}
