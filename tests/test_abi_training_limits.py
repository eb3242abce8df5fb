"""Host-side checks of the training entry points' limits (no GPU needed)."""
import pytest

from test_abi_training import SIZE, WORKSPACE, _ortho, lib  # noqa: F401


@pytest.mark.parametrize("count", [65535, 65536, 70001, 1 << 20])
def test_orthogonalize_takes_any_count(lib, count):  # noqa: F811
    assert _ortho(lib, count=count, rows=8, cols=8, ws_bytes=0) == WORKSPACE
    need = lib.lora_orthogonalize_workspace(count, 8, 8)
    assert need > 0
    assert _ortho(lib, count=count, rows=8, cols=8, ws_bytes=need - 1) == WORKSPACE


def test_orthogonalize_workspace_holds_a_matrix_in_fp32(lib):  # noqa: F811
    """A long run of steps iterates on X itself, at least a matrix at a time."""
    for rows, cols in ((8, 200008), (128, 8192), (11008, 32), (1, 8)):
        assert lib.lora_orthogonalize_workspace(1, rows, cols) >= rows * cols * 4
    assert lib.lora_orthogonalize_workspace(1, 136, 200) == SIZE
