"""Host-side checks of the training entry points of the C ABI (no GPU
needed): bad arguments are refused before anything is launched, and the
workspaces' sizes hold what they must."""
import ctypes

import pytest

NULL, SIZE, ALIGN, RANK, SLICES, TOKENS, WIDTH, WORKSPACE = -1, -2, -3, -4, -5, -6, -7, -10
PTR = 0x100000          # never read on the host


@pytest.fixture(scope="module")
def lib():
    from expand_gemm_gb300.build import build as pkg_build
    from expand_gemm_gb300 import _lib
    pkg_build()
    return _lib.load()


def _meta(max_loras=4, max_tokens=64, null_field=None):
    from expand_gemm_gb300 import _lib
    names = [f for f, _ in _lib.LoraMetaC._fields_[:7]]
    return _lib.LoraMetaC(*[0 if f == null_field else PTR * (i + 1) for i, f in enumerate(names)],
                          max_loras, max_tokens)


def test_the_workspace_status_has_a_string(lib):
    assert lib.lora_status_string(WORKSPACE) not in (b"", b"unknown status")


# ------------------------------------------------------------ the loss

def _loss(lib, **kw):
    a = dict(hidden=PTR, T=8, H=64, ld=64, weight=PTR, V=100, targets=PTR, tw=None, loss=PTR, lse=None,
             dh=None, dh_ld=64, dw=None, err=None, ws=PTR, ws_bytes=1 << 40)
    a.update(kw)
    return lib.lora_cross_entropy(a["hidden"], a["T"], a["H"], a["ld"], a["weight"], a["V"], a["targets"], a["tw"],
                                  a["loss"], a["lse"], a["dh"], a["dh_ld"], a["dw"], a["err"], a["ws"],
                                  a["ws_bytes"], None)


@pytest.mark.parametrize("bad, status", [
    (dict(T=-1), SIZE), (dict(H=0, ld=64), SIZE), (dict(V=0), SIZE), (dict(ld=63), SIZE),
    (dict(dh=PTR, dh_ld=63), SIZE), (dict(H=60), ALIGN), (dict(weight=None), NULL), (dict(ws=None), NULL),
    (dict(hidden=None), NULL), (dict(targets=None), NULL), (dict(loss=None), NULL),
    (dict(weight=PTR + 2), ALIGN), (dict(dw=PTR + 8), ALIGN), (dict(ws=PTR + 16), ALIGN),
    (dict(ws_bytes=0), WORKSPACE)])
def test_cross_entropy_refuses(lib, bad, status):
    assert _loss(lib, **bad) == status


def test_cross_entropy_workspace(lib):
    size = lib.lora_cross_entropy_workspace
    assert size(-1, 64, 100, 1, 0) == SIZE and size(8, 60, 100, 1, 0) == SIZE and size(8, 64, 0, 1, 0) == SIZE
    need = size(8, 64, 100, 1, 1)
    assert need > 0
    assert _loss(lib, dh=PTR, dw=PTR, ws_bytes=need - 1) == WORKSPACE
    # the scratch of a piece is bounded: the logits of a long batch over a
    # large vocabulary would be 32 GB in bf16
    assert size(131072, 4096, 128000, 1, 1) < 6 << 30
    assert size(0, 64, 100, 1, 0) >= 0


# ------------------------------------------------------------ the gradients

def _back(lib, meta=None, **kw):
    a = dict(dy=PTR, dy_ld=96, T=8, x=PTR, H=64, x_ld=64, buf=PTR, a=(PTR, PTR), b=(PTR, PTR), n=(64, 32), r=16,
             dx=None, dx_ld=64, da=None, db=None, dbias=None, ws=PTR, ws_bytes=1 << 40)
    a.update(kw)
    S = a.get("S", len(a["n"]))

    def ptrs(v):
        return None if v is None else (ctypes.c_void_p * max(1, len(v)))(*v)
    sizes = None if a["n"] is None else (ctypes.c_int32 * max(1, len(a["n"])))(*a["n"])
    m = ctypes.byref(_meta()) if meta is None else meta
    return lib.lora_linear_backward(a["dy"], a["dy_ld"], a["T"], a["x"], a["H"], a["x_ld"], a["buf"], ptrs(a["a"]),
                                    ptrs(a["b"]), sizes, S, a["r"], 1.0, a["dx"], a["dx_ld"], 1, ptrs(a["da"]),
                                    ptrs(a["db"]), ptrs(a["dbias"]), m, a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad, status", [
    (dict(S=0), SLICES), (dict(S=9), SLICES), (dict(r=12), RANK), (dict(r=0), RANK), (dict(r=136), RANK),
    (dict(T=-1), SIZE), (dict(H=0), SIZE), (dict(T=65), TOKENS), (dict(H=60), ALIGN), (dict(dy=None), NULL),
    (dict(x=None), NULL), (dict(buf=None), NULL), (dict(ws=None), NULL), (dict(a=(PTR, None)), NULL),
    (dict(b=(None, PTR)), NULL), (dict(a=None), NULL), (dict(n=(64, 0)), SIZE), (dict(dy_ld=95), WIDTH),
    (dict(x_ld=63), SIZE), (dict(dx=PTR, dx_ld=63), SIZE), (dict(a=(PTR, PTR + 8)), ALIGN),
    (dict(b=(PTR + 2, PTR)), ALIGN), (dict(da=(PTR + 8, None)), ALIGN), (dict(db=(None, PTR + 8)), ALIGN),
    (dict(buf=PTR + 4), ALIGN), (dict(ws=PTR + 128), ALIGN), (dict(ws_bytes=0), WORKSPACE)])
def test_linear_backward_refuses(lib, bad, status):
    assert _back(lib, **bad) == status


@pytest.mark.parametrize("field", ["token_indices_sorted_by_lora_ids", "num_tokens_per_lora", "lora_token_start_loc",
                                   "active_lora_ids", "no_lora_flag", "error_word"])
def test_linear_backward_refuses_incomplete_metadata(lib, field):
    assert _back(lib, meta=ctypes.byref(_meta(null_field=field))) == NULL


def test_linear_backward_workspace(lib):
    size = lib.lora_linear_backward_workspace
    n = (ctypes.c_int32 * 2)(64, 32)
    assert size(8, 64, None, 2, 16, 4) == NULL
    assert size(-1, 64, n, 2, 16, 4) == SIZE and size(8, 60, n, 2, 16, 4) == SIZE
    assert size(8, 64, n, 2, 16, 0) == SIZE and size(8, 64, n, 2, 16, 1025) == SIZE
    assert size(8, 64, n, 0, 16, 4) == SLICES and size(8, 64, n, 2, 20, 4) == RANK
    need = size(8, 64, n, 2, 16, 4)
    assert need > 0
    assert _back(lib, ws_bytes=need - 1) == WORKSPACE
    assert size(1000, 64, n, 2, 16, 4) > size(8, 64, n, 2, 16, 4)


# ------------------------------------------------------------ the update

def _ortho(lib, **kw):
    a = dict(u=PTR, f32=0, count=2, rows=16, cols=64, steps=5, out=PTR, err=None, ws=PTR, ws_bytes=1 << 40)
    a.update(kw)
    return lib.lora_orthogonalize(a["u"], a["f32"], a["count"], a["rows"], a["cols"], a["steps"], 3.4445, -4.775,
                                  2.0315, 1e-7, 1.0, a["out"], a["err"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("bad, status", [
    (dict(count=-1), SIZE), (dict(rows=0), SIZE), (dict(cols=0), SIZE), (dict(rows=136, cols=200), SIZE),
    (dict(steps=0), SIZE), (dict(u=None), NULL), (dict(out=None), NULL), (dict(ws=None), NULL),
    (dict(u=PTR + 2), ALIGN), (dict(out=PTR + 8), ALIGN), (dict(ws=PTR + 16), ALIGN),
    (dict(ws_bytes=0), WORKSPACE)])
def test_orthogonalize_refuses(lib, bad, status):
    assert _ortho(lib, **bad) == status


def test_orthogonalize_workspace(lib):
    size = lib.lora_orthogonalize_workspace
    assert size(2, 0, 64) == SIZE and size(-1, 16, 64) == SIZE
    need = size(2, 16, 64)
    assert need > 0
    assert _ortho(lib, ws_bytes=need - 1) == WORKSPACE
    assert _ortho(lib, count=0, u=None, out=None) == 0
