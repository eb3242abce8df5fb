"""Stray-write checks of the training entry points: every tensor that they
write, and the end of the workspace, sits between guard values that must be
the same afterwards; and on the debug-checks build, metadata that points
outside the batch is reported in bit 29 of the error word instead of being
used.  As in test_gpu_guards, each corrupted index lands in memory that the
tensors really have."""
import json
import math
import os
import subprocess
import sys

import pytest
import torch

import expand_gemm_gb300 as eg
from test_gpu_linear_backward import make as make_layer
from test_gpu_loss import make as make_loss

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BAND = 4096             # elements before and after


class Guards:
    """Tensors inside bands of one value."""

    def __init__(self):
        self.full = []

    def like(self, t, fill=None):
        return self.of(t.shape, t.dtype, t if fill is None else fill)

    def of(self, shape, dtype, fill=math.nan):
        n = math.prod(shape)
        mark = 0xA5 if dtype is torch.uint8 else 7
        full = torch.full((n + 2 * BAND,), mark, dtype=dtype, device="cuda")
        at = full[BAND:BAND + n].view(*shape)
        if isinstance(fill, torch.Tensor):
            at.copy_(fill)
        elif dtype is not torch.uint8:
            at.fill_(fill if dtype.is_floating_point else -1)
        self.full.append((full, n, mark))
        return at

    def intact(self):
        return all(bool((f[:BAND] == mark).all()) and bool((f[BAND + n:] == mark).all()) for f, n, mark in self.full)


LAYERS = [(5, 72, 24, 2, (7, 9), 1), (300, 1000, 40, 5, (523, 75, 130), 30), (700, 264, 16, 3, (200, 64), 7),
          (3500, 1288, 128, 4, (136, 72, 64), 300), (5000, 1096, 64, 3, (200, 520), 1),
          (2600, 2056, 128, 3, (64, 72, 80, 88, 8, 16, 24, 32), 1)]


@pytest.mark.parametrize("T,H,r,L,widths,runs", LAYERS)
@pytest.mark.parametrize("add", [True, False])
def test_linear_backward(T, H, r, L, widths, runs, add):
    c = make_layer(T, H, r, L, widths, 81, runs=runs)
    meta = eg.LoRAKernelMeta.make(L, T, "cuda")
    meta.prepare_tensors(c["ids"].cuda())
    g = Guards()
    dx = g.like(c["dx0"])
    dA, dB = [g.like(a, math.nan) for a in c["A"]], [g.like(b, math.nan) for b in c["B"]]
    dbias = [g.of(b.shape[:2], torch.bfloat16) for b in c["B"]]
    ws = g.of((eg.lora_linear_backward_workspace(T, H, widths, r, L),), torch.uint8)
    eg.lora_linear_backward(c["dy"].cuda(), c["x"].cuda(), c["buf"].cuda(), [a.cuda() for a in c["A"]],
                            [b.cuda() for b in c["B"]], c["scale"], meta, dx=dx, add_inputs=add, d_lora_a=dA,
                            d_lora_b=dB, d_lora_bias=dbias, workspace=ws)
    assert int(meta.error_word) == 0 and g.intact()
    for t in [dx] + dA + dB + dbias:
        assert torch.isfinite(t.float()).all()


@pytest.mark.parametrize("T,H,V", [(1, 64, 1000), (2, 1032, 777), (3, 72, 129), (255, 264, 1025), (257, 1000, 2049),
                                   (700, 136, 3001)])
@pytest.mark.parametrize("head", [True, False])
def test_cross_entropy(T, H, V, head):
    hidden, weight, targets, share = make_loss(T, H, V, 83)
    g = Guards()
    loss, lse = g.of((T,), torch.float32), g.of((T,), torch.float32)
    dh, err = g.like(hidden, math.nan), g.of((1,), torch.int32)
    dw = g.like(weight, math.nan) if head else None
    ws = g.of((eg.lora_cross_entropy_workspace(T, H, V, weight_grad=head),), torch.uint8)
    eg.lora_cross_entropy(hidden.cuda(), weight.cuda(), targets.cuda(), loss, token_weight=share.cuda(), logsumexp=lse,
                          hidden_grad=dh, weight_grad=dw, error_word=err, workspace=ws)
    assert int(err) == 0 and g.intact()
    for t in (loss, lse, dh, dw):
        assert t is None or torch.isfinite(t.float()).all()


@pytest.mark.parametrize("f32", [True, False])
@pytest.mark.parametrize("steps", [5, 8])
@pytest.mark.parametrize("count,rows,cols", [(3, 9, 136), (5, 1003, 16), (2, 40, 2048), (3, 520, 72), (2, 127, 1032),
                                             (2, 1500, 128)])
def test_orthogonalize(count, rows, cols, steps, f32):
    u = 1e-3 * torch.randn((count, rows, cols), generator=torch.Generator().manual_seed(85))
    g = Guards()
    out, err = g.of(u.shape, torch.bfloat16), g.of((1,), torch.int32)
    err.zero_()
    ws = g.of((eg.lora_orthogonalize_workspace(count, rows, cols),), torch.uint8)
    eg.lora_orthogonalize((u if f32 else u.bfloat16()).cuda(), out, steps=steps, error_word=err, workspace=ws)
    assert int(err) == 0 and g.intact() and torch.isfinite(out.float()).all()


# The child process: runs on the debug-checks build (LORA_PUNICA_LIBRARY).
_CHILD = r'''
import json, os, sys
sys.path.insert(0, sys.argv[1])
sys.path.insert(0, os.path.join(sys.argv[1], "tests"))
import math, torch
import expand_gemm_gb300 as eg
from test_gpu_training_guards import BAND, Guards, make_layer
out = {"library": os.path.basename(eg.library()._name)}
ROWS = 64               # rows of x, dy, dx and the buffer past the batch

def run(corrupt, which, T, H, r, L, widths, runs):
    c = make_layer(T, H, r, L, widths, 87, runs=runs)
    S = len(widths)
    g = Guards()

    def spare(t, fill):                 # the first T rows of T + ROWS
        full = g.of((T + ROWS,) + tuple(t.shape[1:]), t.dtype, fill)
        full[:T].copy_(t)
        return full[:T]
    x, dy, dx = spare(c["x"], 1.0), spare(c["dy"], 1.0), spare(c["dx0"], 7.0)
    buf = g.of((S, T, r), torch.float32, c["buf"])      # bands on both sides
    A = [g.like(torch.cat([a, torch.ones_like(a[:1])]))[:L] for a in c["A"]]
    B = [g.like(torch.cat([b, torch.ones_like(b[:1])]))[:L] for b in c["B"]]
    dA = [g.of((L + 1,) + tuple(a.shape[1:]), torch.bfloat16, 7.0)[:L] for a in c["A"]]
    dB = [g.of((L + 1,) + tuple(b.shape[1:]), torch.bfloat16, 7.0)[:L] for b in c["B"]]
    dbias = [g.of((L + 1, b.shape[1]), torch.bfloat16, 7.0)[:L] for b in c["B"]]
    meta = eg.LoRAKernelMeta.make(L, T + ROWS, "cuda")
    meta.prepare_tensors(c["ids"].cuda())
    meta.token_indices_sorted_by_lora_ids[T:] = T + 5
    torch.cuda.synchronize()
    if corrupt == "token":
        k = int(meta.lora_token_start_loc[1].item())
        meta.token_indices_sorted_by_lora_ids[k + 1] = T + 3
    elif corrupt == "lora":
        meta.active_lora_ids[1] = L
    elif corrupt == "segment":
        n = int((meta.num_tokens_per_lora > 0).sum().item())
        meta.num_tokens_per_lora[n - 1] += 8
        meta.lora_token_start_loc[n] += 8
    torch.cuda.synchronize()
    meta.error_word.zero_()
    eg.lora_linear_backward(dy, x, buf, A, B, c["scale"], meta, dx=dx if "dx" in which else None,
                            d_lora_a=dA if "dA" in which else None, d_lora_b=dB if "dB" in which else None,
                            d_lora_bias=dbias if "dB" in which else None)
    torch.cuda.synchronize()
    clean = g.intact()
    for t in [dx] + dA + dB + dbias:    # and the spare rows and adapters
        full = [f for f, n, mark in g.full if f.data_ptr() + 2 * BAND == t.data_ptr()][0]
        clean = clean and bool((full[BAND + t.numel():] == 7.0).all())
    return {"error_word": int(meta.error_word.item()), "intact": clean}

SIZES = {"mma": (700, 264, 32, 6, (128, 64), 60), "whole": (130, 72, 16, 4, (40, 33), 3),
         "tcgen05": (3500, 1288, 128, 6, (136, 72, 64), 300), "rank64": (5000, 1096, 64, 6, (200, 520), 40)}
for name, size in SIZES.items():
    for corrupt in ("none", "token", "lora", "segment"):
        for which in ("dx,dA,dB", "dx", "dA", "dB"):
            out["%s/%s/%s" % (name, which, corrupt)] = run(corrupt, which, *size)
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
        assert bool(v["error_word"] & (1 << 29)) == (not key.endswith("/none")), key
