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


def test_a_workspace_holds_every_smaller_batch(lib):  # noqa: F811
    """A training loop sizes its workspace once, for its largest batch."""
    import ctypes
    import random
    rng = random.Random(3)
    tokens = sorted({0, 1, 2, 3, 63, 64, 65, 100, 128, 129, 255, 256, 257, 512, 513, 768, 1024, 4096, 4097, 4352, 8192} |
                    {rng.randrange(1, 20000) for _ in range(60)})
    for hidden, widths, rank, loras in ((4096, (4096,), 16, 4), (8192, (8192, 1024, 1024), 128, 64), (64, (24,), 8, 1024),
                                        (4096, (1024, 72), 40, 64)):
        n = (ctypes.c_int32 * len(widths))(*widths)
        sizes = [lib.lora_linear_backward_workspace(t, hidden, n, len(widths), rank, loras) for t in tokens]
        assert sizes == sorted(sizes) and sizes[0] > 0, (hidden, widths, rank)
    for hidden, vocab in ((4096, 32000), (4096, 1000), (64, 50021), (8192, 128000), (16384, 500)):
        full = None
        for grads in ((0, 0), (1, 0), (0, 1), (1, 1)):
            full = [lib.lora_cross_entropy_workspace(t, hidden, vocab, *grads) for t in tokens]
            assert full == sorted(full) and full[0] > 0, (hidden, vocab, grads)
        # ... and calls that ask for fewer gradients
        for grads in ((0, 0), (1, 0), (0, 1)):
            assert all(lib.lora_cross_entropy_workspace(t, hidden, vocab, *grads) <= f for t, f in zip(tokens, full))
