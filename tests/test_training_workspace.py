"""The cross entropy backward pass's workspace, by its size function: dz of a
piece of the vocabulary (256 MB, or 4096 columns where that is more), its column
sums, and the fp32 slabs of dx and dW; nothing that grows with rows x classes."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from video_vit_encoder_gb300 import build
    build.build()
    import video_vit_encoder_gb300 as jg
    return jg.load()


@pytest.mark.parametrize("dtype,plane", [(0, 6), (1, 2), (2, 2)])
@pytest.mark.parametrize("rows", [1, 300, 10922, 32768, 73728, 1 << 20])
@pytest.mark.parametrize("dim,vocab", [(64, 1000), (1024, 50021), (1024, 131072), (768, 1 << 20)])
def test_bound(lib, rows, dim, vocab, dtype, plane):
    up = (lambda n, k: -(-n // k) * k)
    held = up(rows, 256) if plane == 6 else rows
    # a row's dz of one class more than fits is a piece of 256 columns more
    columns = min(up(vocab, 256), max(4096, (256 << 20) // (plane * held)) + 256)
    dz = plane * held * columns
    sums = 4 * up(rows, 32) // 32 * columns
    slabs = 16 * 4 * (up(rows, 256) + up(columns, 256)) * up(dim, 8)
    if rows * dim > 4 * 76 * 65536:   # more tiles than K is split for: one slab
        slabs = 4 * (up(rows, 256) + 16 * up(columns, 256)) * up(dim, 8)
    copies = 6 * (up(rows, 64) + up(vocab, 64)) * up(dim, 8) if plane == 6 else 0
    got = lib.jepa_linear_ce_workspace_bytes(rows, dim, vocab, dtype, 1)
    assert 0 < got <= dz + sums + slabs + copies + 4096
    if rows * vocab * plane > 1 << 31 and rows <= 32768 // (plane // 2):
        assert got < (256 << 20) + sums + slabs + copies + 4096


def test_many_rows_take_more_than_256_mb(lib):
    """The documented 8 GB for 2^20 rows in 16 bits, three times that in fp32."""
    assert lib.jepa_linear_ce_workspace_bytes(1 << 20, 64, 100000, 2, 1) >= 8 << 30
    assert lib.jepa_linear_ce_workspace_bytes(1 << 20, 64, 100000, 0, 1) >= 24 << 30
