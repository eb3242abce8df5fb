"""Host-side checks of the entry points of the layers under the adapters (no
GPU needed): bad arguments are refused before anything is launched, and the
workspaces' sizes hold what they must."""
import ctypes

import pytest

from test_abi_training import ALIGN, NULL, PTR, SIZE, TOKENS, WORKSPACE, _meta, lib  # noqa: F401

META_FIELDS = ["token_lora_mapping", "token_indices_sorted_by_lora_ids", "num_tokens_per_lora", "lora_token_start_loc",
               "active_lora_ids", "no_lora_flag", "error_word"]


def _forward(lib, meta=None, **kw):  # noqa: F811
    a = dict(x=PTR, x_ld=64, rows=8, fan=2, K=64, w=PTR, scale=None, N=48, y=PTR, y_ld=48, ws=PTR, ws_bytes=1 << 40)
    a.update(kw)
    m = ctypes.byref(_meta()) if meta is None else meta
    return lib.lora_expert_linear(a["x"], a["x_ld"], a["rows"], a["fan"], a["K"], a["w"], a["scale"], a["N"], a["y"],
                                  a["y_ld"], 0, m, a["ws"], a["ws_bytes"], None)


BAD = [(dict(rows=-2), SIZE), (dict(fan=0), SIZE), (dict(rows=7), SIZE), (dict(K=0), SIZE), (dict(K=60), ALIGN),
       (dict(K=72, x_ld=72, scale=PTR), ALIGN), (dict(N=0), SIZE), (dict(rows=66), TOKENS), (dict(x_ld=63), SIZE),
       (dict(w=None), NULL), (dict(x=None), NULL), (dict(ws=None), NULL), (dict(w=PTR + 8), ALIGN),
       (dict(scale=PTR + 4), ALIGN), (dict(ws=PTR + 64), ALIGN), (dict(ws_bytes=0), WORKSPACE)]


@pytest.mark.parametrize("bad, status", BAD + [(dict(y=None), NULL), (dict(y_ld=47), SIZE)])
def test_expert_linear_refuses(lib, bad, status):  # noqa: F811
    assert _forward(lib, **bad) == status


def _backward(lib, meta=None, **kw):  # noqa: F811
    a = dict(dy=PTR, dy_ld=48, rows=8, fan=2, x=PTR, x_ld=64, K=64, w=PTR, scale=None, N=48, dx=PTR, dx_ld=64,
             dw=PTR, ws=PTR, ws_bytes=1 << 40)
    a.update(kw)
    m = ctypes.byref(_meta()) if meta is None else meta
    return lib.lora_expert_linear_backward(a["dy"], a["dy_ld"], a["rows"], a["fan"], a["x"], a["x_ld"], a["K"], a["w"],
                                           a["scale"], a["N"], a["dx"], a["dx_ld"], 0, a["dw"], m, a["ws"],
                                           a["ws_bytes"], None)


@pytest.mark.parametrize("bad, status", BAD + [(dict(dy=None), NULL), (dict(dy_ld=47), SIZE), (dict(dx_ld=63), SIZE),
                                               (dict(dw=PTR + 8), ALIGN)])
def test_expert_linear_backward_refuses(lib, bad, status):  # noqa: F811
    assert _backward(lib, **bad) == status


@pytest.mark.parametrize("field", META_FIELDS)
def test_incomplete_metadata_is_refused(lib, field):  # noqa: F811
    m = _meta(null_field=field)
    assert _forward(lib, meta=ctypes.byref(m)) == NULL
    assert _backward(lib, meta=ctypes.byref(m)) == NULL


def test_null_metadata_is_refused(lib):  # noqa: F811
    assert _forward(lib, meta=ctypes.POINTER(type(_meta()))()) == NULL


def test_nothing_asked_for_is_nothing_done(lib):  # noqa: F811
    assert _forward(lib, rows=0, x=None, y=None) == 0
    assert _backward(lib, dx=None, dw=None) == 0
    assert _backward(lib, rows=0, dy=None, x=None, dw=None) == 0


def test_expert_workspaces(lib):  # noqa: F811
    size, back = lib.lora_expert_linear_workspace, lib.lora_expert_linear_backward_workspace
    assert size(-1, 64, 48, 4, 0) == SIZE and size(8, 64, 0, 4, 0) == SIZE and size(8, 64, 48, 0, 0) == SIZE
    assert size(8, 64, 48, 1025, 0) == SIZE and size(8, 60, 48, 4, 0) == ALIGN and size(8, 72, 48, 4, 1) == ALIGN
    assert back(9, 2, 64, 48, 4, 1, 1, 0) == SIZE and back(8, 0, 64, 48, 4, 1, 1, 0) == SIZE
    need = size(8, 64, 48, 4, 0)
    assert need > 0 and _forward(lib, ws_bytes=need - 1) == WORKSPACE
    need = back(8, 2, 64, 48, 4, 1, 1, 0)
    assert need > 0 and _backward(lib, ws_bytes=need - 1) == WORKSPACE


def test_an_expert_workspace_holds_every_smaller_batch(lib):  # noqa: F811
    rows = sorted({0, 2, 4, 8, 16, 62, 64, 66, 126, 128, 130, 254, 256, 258, 510, 512, 514, 1022, 1024, 1026, 2048, 4096,
                   8190, 8192, 16384, 32768, 100000})
    for K, N, E in ((4096, 4096, 8), (64, 24, 1024), (4096, 11008, 1), (1024, 75, 64)):
        for four in (0, 1):
            sizes = [lib.lora_expert_linear_workspace(r, K, N, E, four) for r in rows]
            assert sizes == sorted(sizes) and sizes[0] > 0
            for fan in (1, 2):
                full = [lib.lora_expert_linear_backward_workspace(r, fan, K, N, E, 1, 1, four) for r in rows]
                assert full == sorted(full) and full[0] > 0
                # ... and calls that ask for fewer gradients
                for grads in ((0, 0), (1, 0), (0, 1)):
                    some = [lib.lora_expert_linear_backward_workspace(r, fan, K, N, E, *grads, four) for r in rows]
                    assert some == sorted(some) and all(a <= b for a, b in zip(some, full))


@pytest.mark.parametrize("bad, status", [
    (dict(n=-32), SIZE), (dict(n=33), SIZE), (dict(v=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL),
    (dict(v=PTR + 8), ALIGN), (dict(codes=PTR + 8), ALIGN)])
@pytest.mark.parametrize("f32", [0, 1])
def test_mxfp4_refuses(lib, bad, status, f32):  # noqa: F811
    a = dict(v=PTR, n=64, codes=PTR, scales=PTR)
    a.update(bad)
    assert lib.lora_quantize_mxfp4(a["v"], f32, a["n"], a["codes"], a["scales"], None) == status
    assert lib.lora_dequantize_mxfp4(a["codes"], a["scales"], a["n"], a["v"], f32, None) == status


def test_mxfp4_of_nothing(lib):  # noqa: F811
    assert lib.lora_quantize_mxfp4(None, 0, 0, None, None, None) == 0
    assert lib.lora_dequantize_mxfp4(None, None, 0, None, 0, None) == 0


def _clip(lib, **kw):  # noqa: F811
    a = dict(grads=(PTR, PTR), out=None, sizes=(8, 16), f32=(0, 1), groups=4, max_norm=1.0, eps=1e-6, norms=PTR,
             ws=PTR, ws_bytes=1 << 40)
    a.update(kw)
    n = a.get("n", len(a["sizes"] or ()))

    def array(kind, v):
        return None if v is None else (kind * max(1, len(v)))(*v)
    return lib.lora_clip_gradients(array(ctypes.c_void_p, a["grads"]), array(ctypes.c_void_p, a["out"]),
                                   array(ctypes.c_int64, a["sizes"]), array(ctypes.c_int32, a["f32"]), n, a["groups"],
                                   a["max_norm"], a["eps"], a["norms"], a["ws"], a["ws_bytes"], None)


NAN = float("nan")


@pytest.mark.parametrize("bad, status", [
    (dict(n=-1), SIZE), (dict(groups=0), SIZE), (dict(max_norm=-1.0), SIZE), (dict(max_norm=NAN), SIZE),
    (dict(eps=-1.0), SIZE), (dict(eps=NAN), SIZE), (dict(sizes=(8, -1)), SIZE), (dict(sizes=(1 << 46, 8)), SIZE),
    (dict(norms=None), NULL), (dict(ws=None), NULL), (dict(grads=None), NULL), (dict(grads=(PTR, None)), NULL),
    (dict(out=(None, PTR)), NULL), (dict(sizes=None, n=2), NULL), (dict(f32=None), NULL),
    (dict(grads=(PTR + 1, PTR)), ALIGN), (dict(grads=(PTR, PTR + 2)), ALIGN), (dict(out=(PTR, PTR + 2)), ALIGN),
    (dict(ws=PTR + 128), ALIGN), (dict(ws_bytes=0), WORKSPACE)])
def test_clip_refuses(lib, bad, status):  # noqa: F811
    assert _clip(lib, **bad) == status


def test_clip_workspace(lib):  # noqa: F811
    assert lib.lora_clip_gradients_workspace(0) == SIZE
    sizes = [lib.lora_clip_gradients_workspace(g) for g in (1, 2, 8, 64, 1024, 100000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    assert _clip(lib, groups=64, ws_bytes=sizes[3] - 1) == WORKSPACE
