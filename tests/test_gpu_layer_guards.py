"""Stray-write checks of the layers under the adapters: every tensor that their
entry points write, and the end of their workspaces, sits between guard values
that must be the same afterwards; and on the debug-checks build, metadata that
point outside the batch are reported in bit 29 of the error word instead of being
used.  Each corrupted index lands in memory that the tensors really have."""
import json
import os
import subprocess
import sys

import pytest
import torch

import expand_gemm_gb300 as eg
from test_gpu_expert import inputs, meta_of
from test_gpu_training_guards import Guards

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# tokens, fan out, experts, hidden, width: gathered, in tiles of 16, 32 and 64 rows, by a table, on pairs
LAYERS = [(1, 2, 4, 320, 129), (5, 1, 3, 544, 75), (18, 2, 3, 544, 523), (40, 2, 3, 1024, 1500), (150, 2, 300, 96, 200),
          (700, 1, 2, 992, 523), (1100, 2, 3, 96, 264)]


@pytest.mark.parametrize("size", LAYERS, ids=str)
@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("add", [False, True])
def test_expert_linear_and_its_gradients(size, four, add):
    tokens, fan, E, H, N = size
    ids, x, (w, scale), _, dy = inputs(*size, 0.2, four=four)
    meta, rows = meta_of(ids, E), tokens * fan
    g = Guards()
    y, dx, dw = g.of((rows, N), torch.bfloat16, 0.5), g.of((tokens, H), torch.bfloat16, 0.5), g.of((E, N, H), torch.bfloat16)
    ws = g.of((eg.lora_expert_linear_workspace(rows, H, N, E, quantized=four),), torch.uint8)
    back = g.of((eg.lora_expert_linear_backward_workspace(rows, H, N, E, fan_out=fan, weight_grad=True, quantized=four),),
                torch.uint8)
    eg.lora_expert_linear(x, w, y, meta, weight_scale=scale, add_inputs=add, workspace=ws)
    eg.lora_expert_linear_backward(dy, x, w, meta, weight_scale=scale, dx=dx, add_inputs=add, d_weight=dw, workspace=back)
    assert int(meta.error_word) == 0 and g.intact()
    assert all(bool(torch.isfinite(t.float()).all()) for t in (y, dx, dw))


@pytest.mark.parametrize("rows, cols", [(1, 32), (3, 96), (129, 1024), (1003, 4096)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mxfp4(rows, cols, dtype):
    g = Guards()
    w = torch.randn(rows, cols, device="cuda").to(dtype)
    codes, scales = g.of((rows, cols // 2), torch.uint8), g.of((rows, cols // 32), torch.uint8)
    out = g.of((rows, cols), dtype)
    eg.lora_quantize_mxfp4(w, codes, scales)
    eg.lora_dequantize_mxfp4(codes, scales, out)
    assert g.intact() and bool(torch.isfinite(out).all())


@pytest.mark.parametrize("count, groups", [(1, 1), (3, 5), (70, 2), (1030, 3)])
@pytest.mark.parametrize("max_norm", [1e-3, 1e9])
@pytest.mark.parametrize("apart", [False, True])
def test_clip_gradients(count, groups, max_norm, apart):
    g = Guards()
    kinds = [torch.bfloat16 if i % 2 else torch.float32 for i in range(count)]
    shapes = [(groups, 3 + i % 7, 5 + 40 * (i % 3)) for i in range(count)]
    grads = [g.of(s, d, torch.randn(s, device="cuda").to(d)) for s, d in zip(shapes, kinds)]
    out = [g.of(s, d) for s, d in zip(shapes, kinds)] if apart else None
    norms = g.of((groups,), torch.float32)
    eg.lora_clip_gradients(eg.LoRAGradients.make(grads, groups, out=out), max_norm, norms)
    assert g.intact() and all(bool(torch.isfinite(t).all()) for t in (out or grads) + [norms])


# The child process: runs on the debug-checks build (LORA_PUNICA_LIBRARY).
_CHILD = r'''
import json, os, sys
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, os.path.join(sys.argv[1], "tests"))
import torch
import expand_gemm_gb300 as eg
from test_gpu_expert import inputs
from test_gpu_layer_guards import LAYERS
from test_gpu_training_guards import Guards
out = {"library": os.path.basename(eg.library()._name)}
ROWS = 64               # rows of x, y, dy and dx past the batch

def run(corrupt, size, four):
    tokens, fan, E, H, N = size
    R = tokens * fan
    ids, x0, (w, scale), _, dy0 = inputs(tokens, fan, E, H, N, 0.0, four=four)
    g = Guards()
    def spare(t, n, fill):              # the first n rows of n + ROWS
        full = g.of((n + ROWS, t.shape[1]), t.dtype, fill)
        full[:n].copy_(t)
        return full, full[:n]
    (_, x), (_, dy) = spare(x0, tokens, 1.0), spare(dy0, R, 1.0)
    ally, y = spare(torch.zeros_like(dy0), R, 7.0)
    alldx, dx = spare(torch.zeros_like(x0), tokens, 7.0)
    alldw = g.of((E + 1, N, H), torch.bfloat16, 7.0)
    weight = g.like(torch.cat([w, w[:1]]))[:E]
    scales = None if scale is None else g.like(torch.cat([scale, scale[:1]]))[:E]
    ws = g.of((eg.lora_expert_linear_workspace(R, H, N, E, quantized=four),), torch.uint8)
    back = g.of((eg.lora_expert_linear_backward_workspace(R, H, N, E, fan_out=fan, weight_grad=True, quantized=four),), torch.uint8)
    meta = eg.LoRAKernelMeta.make(E, R + ROWS, "cuda")
    meta.prepare_tensors(ids)
    meta.token_indices_sorted_by_lora_ids[R:] = R + 5
    torch.cuda.synchronize()
    n = int((meta.num_tokens_per_lora > 0).sum().item())
    if corrupt == "row":
        meta.token_indices_sorted_by_lora_ids[R // 2] = R + 3
    elif corrupt == "expert":
        meta.active_lora_ids[n - 1] = E
    elif corrupt == "segment":
        meta.num_tokens_per_lora[n - 1] += 8
        meta.lora_token_start_loc[n] += 8
    torch.cuda.synchronize()
    words = []
    for call in (0, 1):
        meta.error_word.zero_()
        if call == 0:
            eg.lora_expert_linear(x, weight, y, meta, weight_scale=scales, workspace=ws)
        else:
            eg.lora_expert_linear_backward(dy, x, weight, meta, weight_scale=scales, dx=dx, d_weight=alldw[:E], workspace=back)
        torch.cuda.synchronize()
        words.append(int(meta.error_word.item()))
    clean = g.intact() and bool((ally[R:] == 7.0).all()) and bool((alldx[tokens:] == 7.0).all()) and bool((alldw[E] == 7.0).all())
    return {"words": words, "intact": clean}

for k, size in enumerate(LAYERS):
    for four in (False, True):
        for corrupt in ("none", "row", "expert", "segment"):
            out["%d/%s/%s" % (k, four, corrupt)] = run(corrupt, size, four)
print(json.dumps(out))
'''


def test_debug_build_reports_metadata_outside_the_batch():
    from expand_gemm_gb300.build import build
    lib = build(debug=True)
    env = dict(os.environ, LORA_PUNICA_LIBRARY=lib)
    r = subprocess.run([sys.executable, "-c", _CHILD, ROOT], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout + r.stderr
    res = json.loads(r.stdout.strip().splitlines()[-1])
    assert res.pop("library") == "liblora_punica_debug.so"
    for key, v in res.items():
        assert v["intact"], key
        for word in v["words"]:
            assert word == (0 if key.endswith("/none") else 1 << 29), (key, word)
