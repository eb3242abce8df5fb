"""The operators of the layers under the adapters, as measured cases.

Adapters are served and trained over frozen layers.  Four operators deal with
those layers and with what their training leaves: the product of a mixture of
experts (:func:`lora_expert_linear`, with weights in bf16 or in microscaled 4
bits), its gradients (:func:`lora_expert_linear_backward`), the quantisation
of weights to 4 bits and back (:func:`lora_quantize_mxfp4`,
:func:`lora_dequantize_mxfp4`) and the clipping of gradients by their norm,
for all tensors together or for every adapter (:func:`lora_clip_gradients`).
Where ``own`` is false ``run`` computes them in elementary torch operations in
32 bits; where it is true it calls the framework.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 32                       # elements that share a scale
EPS = 1e-6


def listed():
    return [
        # one token decoded: two of eight experts, the latency of reading their weights
        dict(name="expert_one", op="expert", tokens=1, fan=2, experts=8, hidden=4096, width=4096, none=0.0, skew=0.0, four=False),
        # a decode batch of 256 tokens, two of sixteen experts each
        dict(name="expert_decode", op="expert", tokens=256, fan=2, experts=16, hidden=4096, width=4096, none=0.0, skew=0.5, four=False),
        # prompts: 8192 tokens through the gate or up projection, experts used unevenly
        dict(name="expert_prefill", op="expert", tokens=8192, fan=2, experts=16, hidden=4096, width=11008, none=0.0, skew=0.7, four=False),
        # sizes that fill no tile, half of the experts on another device
        dict(name="expert_odd", op="expert", tokens=333, fan=3, experts=5, hidden=1000, width=523, none=0.5, skew=1.0, four=False),
        # a decode batch over frozen experts in 4 bits
        dict(name="four_decode", op="expert", tokens=32, fan=4, experts=32, hidden=4096, width=11008, none=0.0, skew=0.3, four=True),
        # prompts over one frozen dense layer in 4 bits (one expert), as adapters are trained over
        dict(name="four_dense", op="expert", tokens=4096, fan=1, experts=1, hidden=4096, width=4096, none=0.1, skew=0.0, four=True),
        # a training batch: gradients of the hidden states and of all experts
        dict(name="back_large", op="backward", tokens=4096, fan=2, experts=8, hidden=4096, width=4096, none=0.0, skew=0.5, four=False, weight=True),
        # sizes that fill no tile, rows without an expert
        dict(name="back_odd", op="backward", tokens=1001, fan=1, experts=5, hidden=1000, width=523, none=0.2, skew=1.0, four=False, weight=True),
        # one projection's weights, from 32 bits
        dict(name="quant_small", op="quantize", matrices=1, rows=1003, cols=1024, f32=True),
        # the experts of one layer
        dict(name="quant_layer", op="quantize", matrices=8, rows=4096, cols=4096, f32=False),
        # the gradients of one layer's adapters, a norm for each adapter
        dict(name="clip_layer", op="clip", adapters=8, each=True, layers=1, hidden=4096, rank=16, kinds=3, f32=False, level=1.0),
        # the gradients of a whole model's adapters, one norm
        dict(name="clip_model", op="clip", adapters=8, each=False, layers=32, hidden=4096, rank=32, kinds=7, f32=False, level=3.0),
    ]


def _between(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["expert", "expert", "backward", "quantize", "clip"])
    if op in ("expert", "backward"):
        while True:
            four = rng.random() < (0.5 if op == "expert" else 0.25)
            experts = rng.choice([1, 2, 3, 5, 8, 16, 24, 32, 64])
            hidden = 32 * _between(rng, 2, 256) if four else 8 * _between(rng, 8, 1024)
            width = _between(rng, 40, 11008)
            if rng.random() < 0.6:
                width = max(64, width // 64 * 64)
            case = dict(op=op, tokens=_between(rng, 1, 8192), fan=rng.randint(1, min(4, experts)), experts=experts, hidden=hidden,
                        width=width, none=rng.choice([0.0, 0.0, 0.1, 0.5]), skew=rng.choice([0.0, 0.5, 1.0]), four=four)
            if op == "backward":
                case["weight"] = not four and rng.random() < 0.6
            rows = case["tokens"] * case["fan"]
            if rows * hidden * width <= 2.0e11 and experts * hidden * width <= 4.0e8 and rows * (hidden + width) <= 2.0e8:
                return case
    if op == "quantize":
        return dict(op=op, matrices=_between(rng, 1, 12), rows=_between(rng, 20, 3000), cols=32 * _between(rng, 2, 112), f32=rng.random() < 0.5)
    return dict(op=op, adapters=_between(rng, 1, 24), each=rng.random() < 0.6, layers=_between(rng, 1, 16), hidden=8 * _between(rng, 16, 512),
                rank=rng.choice([8, 16, 24, 32]), kinds=rng.randint(1, 7), f32=rng.random() < 0.4, level=rng.choice([0.3, 1.0, 3.0]))


# ---------------------------------------------------------------- inputs

def _ids(case, seed):
    """An expert id per row (token t has rows t fan .. t fan + fan - 1, all of different experts;
    -1: none).  The experts' popularity is log-normal with deviation `skew`."""
    rng = np.random.Generator(np.random.PCG64(seed))
    T, E, k = case["tokens"], case["experts"], case["fan"]
    liking = case["skew"] * rng.standard_normal(E) + rng.gumbel(size=(T, E))
    ids = np.argsort(-liking, axis=1)[:, :k].reshape(-1).astype(np.int32)
    ids[rng.random(T * k) < case["none"]] = -1
    return ids


def _normal(g, shape, std=1.0):
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    for part in out.view(-1).split(1 << 28):                  # in pieces: 32 bits of a large stack take space
        part.copy_(torch.randn(part.shape, generator=g, device="cuda") * std)
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"expert": _prepare_expert, "backward": _prepare_expert, "quantize": _prepare_quantize,
            "clip": _prepare_clip}[case["op"]](case, seed, g)


def _prepare_expert(case, seed, g):
    T, k, E, H, N = (case[n] for n in ("tokens", "fan", "experts", "hidden", "width"))
    ids = torch.from_numpy(_ids(case, seed)).cuda()
    x = _normal(g, (T, H))
    weight, scale = _normal(g, (E, N, H), H ** -0.5), None
    if case["four"]:
        weight, scale = _plain_encode(weight)                 # frozen: held in 4 bits from then on
    state = dict(case=case, ids=ids, x=x, weight=weight, scale=scale)
    if case["op"] == "backward":
        state["dy"] = _normal(g, (T * k, N), 0.1)
    if own:
        import expand_gemm_gb300 as eg
        meta = eg.LoRAKernelMeta.make(E, T * k, "cuda")
        if case["op"] == "expert":
            need = eg.lora_expert_linear_workspace(T * k, H, N, E, quantized=case["four"])
            state.update(y=torch.zeros((T * k, N), dtype=torch.bfloat16, device="cuda"))
        else:
            meta.prepare_tensors(ids)                         # the forward pass's
            need = eg.lora_expert_linear_backward_workspace(T * k, H, N, E, fan_out=k, hidden_grad=True,
                                                            weight_grad=case["weight"], quantized=case["four"])
            state.update(dx=torch.empty_like(x),
                         dw=torch.empty((E, N, H), dtype=torch.bfloat16, device="cuda") if case["weight"] else None)
        state.update(meta=meta, workspace=torch.empty(need, dtype=torch.uint8, device="cuda"))
    return state


def _prepare_quantize(case, seed, g):
    shape = (case["matrices"], case["rows"], case["cols"])
    weight = torch.randn(shape, generator=g, device="cuda") * case["cols"] ** -0.5
    # some columns are much larger than others, as in trained weights
    weight *= torch.exp(0.7 * torch.randn((1, 1, case["cols"]), generator=g, device="cuda"))
    weight = weight if case["f32"] else weight.bfloat16()
    state = dict(case=case, weight=weight)
    if own:
        state.update(codes=torch.empty((*shape[:2], shape[2] // 2), dtype=torch.uint8, device="cuda"),
                     scales=torch.empty((*shape[:2], shape[2] // BLOCK), dtype=torch.uint8, device="cuda"),
                     values=torch.empty_like(weight))
    return state


def _prepare_clip(case, seed, g):
    L, H, r = case["adapters"], case["hidden"], case["rank"]
    shapes = [(L, r, H), (L, H, r)] * (case["layers"] * case["kinds"])
    size = L * r * H
    # one buffer holds all gradients, as a training program lays them out
    flat = torch.empty(size * len(shapes), dtype=torch.float32 if case["f32"] else torch.bfloat16, device="cuda")
    grads = [v.view(shape) for v, shape in zip(flat.split(size), shapes)]
    # adapters learn at different paces: some are clipped, others are not
    pace = torch.exp(torch.randn((L, 1, 1), generator=g, device="cuda"))
    for v in grads:
        v.copy_(1e-3 * pace * torch.randn(v.shape, generator=g, device="cuda"))
    groups = L if case["each"] else 1
    # what the norm is without differences of pace
    usual = 1e-3 * math.sqrt(flat.numel() / groups)
    state = dict(case=case, grads=grads, groups=groups, max_norm=usual / case["level"])
    if own:
        import expand_gemm_gb300 as eg
        out = torch.empty_like(flat)
        state.update(out=out, norms=torch.empty(groups, device="cuda"),
                     handle=eg.LoRAGradients.make(grads, groups, out=[v.view(n) for v, n in zip(out.split(size), shapes)]))
    return state


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["case"]["op"]
    if own:
        return {"expert": _own_expert, "backward": _own_backward, "quantize": _own_quantize, "clip": _own_clip}[op](state)
    return {"expert": _plain_expert, "backward": _plain_backward, "quantize": _plain_quantize, "clip": _plain_clip}[op](state)


def _own_expert(s):
    import expand_gemm_gb300 as eg
    s["meta"].prepare_tensors(s["ids"])
    eg.lora_expert_linear(s["x"], s["weight"], s["y"], s["meta"], weight_scale=s["scale"], workspace=s["workspace"])
    return {"y": s["y"]}


def _own_backward(s):
    import expand_gemm_gb300 as eg
    eg.lora_expert_linear_backward(s["dy"], s["x"], s["weight"], s["meta"], weight_scale=s["scale"], dx=s["dx"],
                                   d_weight=s["dw"], workspace=s["workspace"])
    return {"dx": s["dx"], "dw": s["dw"]}


def _own_quantize(s):
    import expand_gemm_gb300 as eg
    eg.lora_quantize_mxfp4(s["weight"], s["codes"], s["scales"])
    eg.lora_dequantize_mxfp4(s["codes"], s["scales"], s["values"])
    return {"values": s["values"]}


def _own_clip(s):
    import expand_gemm_gb300 as eg
    eg.lora_clip_gradients(s["handle"], s["max_norm"], s["norms"], eps=EPS)
    return {"norms": s["norms"], "grads": s["out"]}


def _power(exponent):
    """2 ** exponent in 32 bits, exactly (rounded from 64)."""
    return torch.exp2(exponent.double()).float()


def _plain_scales(w):
    """The blocks' scale exponents floor(log2 max) - 2, at least -127."""
    top = w.view(*w.shape[:-1], -1, BLOCK).abs().amax(-1)
    exponent = torch.frexp(top).exponent - 3                  # frexp's mantissa lies in [0.5, 1)
    return torch.where(top > 0, exponent, torch.full_like(exponent, -127)).clamp(min=-127)


def _plain_elements(w, exponent):
    """The blocks' elements over their scale, rounded to the eight magnitudes (ties to the even code)."""
    v = w.view(*w.shape[:-1], -1, BLOCK) * _power(-exponent)[..., None]
    a = v.abs()
    a = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2)))
    return torch.copysign(a.clamp(max=6.0), v)


def _plain_encode(weight):
    """Codes (two to a byte, the even element in the low half) and scale bytes of a stack of weights."""
    codes = torch.empty((*weight.shape[:-1], weight.shape[-1] // 2), dtype=torch.uint8, device=weight.device)
    scales = torch.empty((*weight.shape[:-1], weight.shape[-1] // BLOCK), dtype=torch.uint8, device=weight.device)
    for m, w in enumerate(weight):
        exponent = _plain_scales(w.float())
        v = _plain_elements(w.float(), exponent).view(w.shape)
        a = v.abs()
        code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
        code += 8 * torch.signbit(v).to(torch.uint8)
        codes[m] = code[..., ::2] + 16 * code[..., 1::2]
        scales[m] = (exponent + 127).to(torch.uint8)
    return codes, scales


def _plain_weight(s, e):
    """The weights of expert e in 32 bits."""
    w = s["weight"][e]
    if not s["case"]["four"]:
        return w.float()
    code = torch.stack((w % 16, w // 16), -1).view(w.shape[0], -1).int()
    m = (code % 8).float()
    m = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    m = torch.where(code >= 8, -m, m)
    exponent = s["scale"][e].int() - 127
    return (m.view(w.shape[0], -1, BLOCK) * _power(exponent)[..., None]).view(w.shape[0], -1)


def _plain_expert(s):
    case = s["case"]
    y = torch.zeros((s["ids"].shape[0], case["width"]), dtype=torch.bfloat16, device=s["x"].device)
    for e in range(case["experts"]):
        at = (s["ids"] == e).nonzero()[:, 0]
        y[at] = (s["x"][at // case["fan"]].float() @ _plain_weight(s, e).T).bfloat16()
    return {"y": y}


def _plain_backward(s):
    case = s["case"]
    dx = torch.zeros((s["ids"].shape[0], case["hidden"]), device=s["x"].device)
    dw = torch.empty(s["weight"].shape, dtype=torch.bfloat16, device=s["x"].device) if case["weight"] else None
    for e in range(case["experts"]):
        at = (s["ids"] == e).nonzero()[:, 0]
        dy = s["dy"][at].float()
        dx[at] = dy @ _plain_weight(s, e)
        if dw is not None:
            dw[e] = (dy.T @ s["x"][at // case["fan"]].float()).bfloat16()
    return {"dx": dx.view(case["tokens"], case["fan"], -1).sum(1).bfloat16(), "dw": dw}


def _plain_quantize(s):
    w = s["weight"].float()
    exponent = _plain_scales(w)
    values = (_plain_elements(w, exponent) * _power(exponent)[..., None]).view(w.shape)
    return {"values": values.to(s["weight"].dtype)}


def _plain_clip(s):
    # the sums in 64 bits: a model's gradients are hundreds of millions of terms
    total = sum(v.view(s["groups"], -1).float().square().sum(1, dtype=torch.float64) for v in s["grads"])
    norms = total.sqrt()
    factor = (s["max_norm"] / (norms + EPS)).clamp(max=1.0).float()
    clipped = [(v.view(s["groups"], -1).float() * factor[:, None]).to(v.dtype).view(-1) for v in s["grads"]]
    return {"norms": norms.float(), "grads": torch.cat(clipped)}


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    if case["op"] in ("expert", "backward"):
        T, k, E, H, N = (case[n] for n in ("tokens", "fan", "experts", "hidden", "width"))
        ids = _ids(case, 1)
        n, d = int((ids >= 0).sum()), len(set(ids[ids >= 0].tolist()))
        weights = d * N * H * (0.53125 if case["four"] else 2.0)
        if case["op"] == "expert":
            return {"bytes": T * H * 2 + weights + n * N * 2 + T * k * 4, "flops": 2.0 * n * N * H + 1}
        more = case["weight"]
        return {"bytes": n * N * 2 + weights + T * H * 2 + (T * H * 2 + E * N * H * 2 if more else 0) + T * k * 4,
                "flops": (4.0 if more else 2.0) * n * N * H + 1}
    if case["op"] == "quantize":
        n = case["matrices"] * case["rows"] * case["cols"]
        size = 4 if case["f32"] else 2
        # the weights read, 4 bits and scales written, then these read and the values written
        return {"bytes": n * (2 * size + 2 * 0.53125), "flops": 4.0 * n}
    n = case["adapters"] * case["layers"] * case["kinds"] * 2 * case["hidden"] * case["rank"]
    return {"bytes": n * 2 * (4 if case["f32"] else 2), "flops": 3.0 * n}


# ---------------------------------------------------------------- in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"expert": _exact_expert, "backward": _exact_backward, "quantize": _exact_quantize,
            "clip": _exact_clip}[case["op"]](s)


def _exact_power(exponent):
    """2 ** exponent: the device's power may be off by its last bit, which decides ties."""
    return torch.tensor([2.0 ** e for e in range(-130, 131)], dtype=torch.float64, device="cuda")[exponent.long() + 130]


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_weight(s, e):
    if not s["case"]["four"]:
        return s["weight"][e].double()
    grid = torch.tensor(_E2M1 + [-v for v in _E2M1], dtype=torch.float64, device="cuda")
    byte = s["weight"][e].long()
    out = torch.empty((byte.shape[0], 2 * byte.shape[1]), dtype=torch.float64, device="cuda")
    out[:, 0::2] = grid[byte & 15]
    out[:, 1::2] = grid[byte >> 4]
    return out * _exact_power(s["scale"][e].long() - 127).repeat_interleave(BLOCK, 1)


def _exact_expert(s):
    case = s["case"]
    tokens = torch.arange(case["tokens"], device="cuda").repeat_interleave(case["fan"])
    y = torch.zeros((len(tokens), case["width"]), dtype=torch.float64, device="cuda")
    for e in range(case["experts"]):
        mine = s["ids"] == e
        if bool(mine.any()):
            y[mine] = s["x"][tokens[mine]].double() @ _exact_weight(s, e).T
    return {"y": y}


def _exact_backward(s):
    case = s["case"]
    tokens = torch.arange(case["tokens"], device="cuda").repeat_interleave(case["fan"])
    dx = torch.zeros(s["x"].shape, dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["weight"].shape, dtype=torch.float64, device="cuda") if case["weight"] else None
    for e in range(case["experts"]):
        mine = s["ids"] == e
        if bool(mine.any()):
            dy = s["dy"][mine].double()
            dx.index_add_(0, tokens[mine], dy @ _exact_weight(s, e))
            if dw is not None:
                dw[e] = dy.T @ s["x"][tokens[mine]].double()
    return {"dx": dx, "dw": dw}


def _exact_quantize(s):
    out = torch.empty(s["weight"].shape, dtype=torch.float64, device="cuda")
    for m, w in enumerate(s["weight"]):
        v = w.double().view(w.shape[0], -1, BLOCK)
        top = v.abs().amax(2, keepdim=True)
        exponent = torch.full_like(top, -127.0)
        # the largest power of two that is not above the block's largest magnitude, over four
        for e in range(-127, 126):
            exponent = torch.where(top >= 2.0 ** (e + 2), torch.full_like(top, float(e)), exponent)
        power = _exact_power(exponent)
        a = v.abs() / power
        best, off = torch.zeros_like(a), a.clone()
        for code, value in list(enumerate(_E2M1))[1:]:
            away = (a - value).abs()
            better = (away < off) | ((away == off) & (code % 2 == 0))
            best, off = torch.where(better, torch.full_like(a, value), best), torch.where(better, away, off)
        out[m] = (torch.where(v < 0, -best, best) * power).view(w.shape)
    return {"values": out}


def _exact_clip(s):
    groups = s["groups"]
    norms = torch.zeros(groups, dtype=torch.float64, device="cuda")
    for v in s["grads"]:
        d = v.double().reshape(groups, -1)
        norms += (d * d).sum(1)
    norms = norms ** 0.5
    factor = torch.minimum(torch.ones_like(norms), s["max_norm"] / (norms + EPS))
    return {"norms": norms, "grads": torch.cat([(v.double().reshape(groups, -1) * factor[:, None]).reshape(-1) for v in s["grads"]])}
