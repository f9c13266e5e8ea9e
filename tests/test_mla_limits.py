"""The latent attention's size limits, where a product of sizes passes 64 bits."""
import pytest

from test_mla_args import EINVAL, attend, cache, lib  # noqa: F401


@pytest.mark.parametrize("ps,page,n", [((1 << 31) - 1, 65536, 1 << 24), (1 << 30, 65536, 1 << 25), ((1 << 31) - 1, 65536, (1 << 31) - 1),
                                       (1 << 30, 1024, 1 << 20), ((1 << 31) - 1, 16, 16)])
def test_attend_tiles(lib, ps, page, n):  # noqa: F811
    """More tiles of 128 tokens over all sequences than an int holds, also where their number times n_seq passes 2^63."""
    assert attend(lib, cache(page_size=page, n_pages=1), ps=ps, n=n, H=1) == EINVAL
    assert b"pages_stride" in lib.coli_last_error()
