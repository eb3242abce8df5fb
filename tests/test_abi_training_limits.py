"""Host-side checks of the training entry points' limits (no GPU needed)."""
import pytest

from test_abi_training import SIZE, WORKSPACE, _ortho, lib  # noqa: F401


@pytest.mark.parametrize("count", [65535, 65536, 70001, 1 << 20])
def test_orthogonalize_takes_any_count(lib, count):  # noqa: F811
    assert _ortho(lib, count=count, rows=8, cols=8, ws_bytes=0) == WORKSPACE
    need = lib.lora_orthogonalize_workspace(count, 8, 8)
    assert need > 0
    assert _ortho(lib, count=count, rows=8, cols=8, ws_bytes=need - 1) == WORKSPACE
