"""Workspace sizes of the gather's gradient, which show the sizes of its pieces, on the host."""
import ctypes

import pytest

import embedding_table_gather_amd as etg


def _up(n, a=256):
    return -(-n // a) * a


def _size(n, d, dtype=etg.BF16, V=1000):
    L, h = etg.lib(), ctypes.c_void_p()
    assert L.etg_table_create(ctypes.c_void_p(0x10000), dtype, V, d, ctypes.byref(h)) == 0
    size = L.etg_embed_gather_grad_workspace(h, n)
    L.etg_table_destroy(h)
    return size


# positions to a piece: 8 up to 1,024 ids, 16 up to 4,096; keys, order and two rows of f32 partial
# sums per piece
@pytest.mark.parametrize("n,d,piece", [(1, 64, 8), (8, 64, 8), (9, 64, 8), (100, 64, 8), (628, 896, 8),
                                       (1024, 65536, 8), (1025, 64, 16), (4096, 64, 16), (4096, 65536, 16),
                                       (4097, 64, 32), (8192, 768, 32)])
def test_pieces_of_few_ids(n, d, piece):
    assert _size(n, d) == 2 * _up(4 * n) + _up(-(-n // piece) * 2 * d * 4)


# longer pieces only where the partial sums would pass 256 MiB
def test_pieces_at_the_limit_of_the_partial_sums():
    for n, d, piece in ((32768, 32768, 32), (32769, 32768, 64), (32768, 65536, 64), (100000, 65536, 224),
                        (65536, 32768, 64), (65537, 32768, 96)):
        tile = 1024 if n <= 65536 else 4096
        pieces = -(-n // piece)
        want = 4 * _up(4 * n) + _up(-(-n // tile) * 4096) + _up(pieces * 2 * d * 4)
        assert _size(n, d) == want, (n, d)
        assert pieces * 2 * d * 4 <= 256 << 20
