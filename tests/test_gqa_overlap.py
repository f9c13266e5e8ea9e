"""Steps whose outputs lie in their queries: in place without weights, refused where queries would be read after they were overwritten."""
import pytest

from test_gqa_args import A, BF16, EINVAL, F32, I64, attend, lib  # noqa: F401

ROWS = 2 * 16                                             # the arguments' 2 sequences of 16 heads, dim 128


@pytest.mark.parametrize("kw", [
    dict(weigh=1), dict(weigh=1, dq=F32, do=F32), dict(dq=F32), dict(do=F32), dict(out=A + 16), dict(q=A + 16), dict(weigh=1, out=A + ROWS * 256 - 16),
    dict(weigh=1, q=A + ROWS * 256 - 16), dict(dq=F32, out=A + ROWS * 512 - 16), dict(out=A + (1 << 20), lse=A), dict(out=A + (1 << 20), lse=A + ROWS * 256 - 4),
    dict(out=A + (1 << 20), q=A + ROWS * 4 - 16, lse=A)])
def test_refused(lib, kw):  # noqa: F811
    assert attend(lib, **kw) == EINVAL
    assert b"q" in lib.coli_last_error()


@pytest.mark.parametrize("kw", [
    dict(), dict(dq=F32, do=F32), dict(weigh=1, out=A + ROWS * 256), dict(weigh=1, q=A + ROWS * 256), dict(weigh=1, dq=F32, out=A + ROWS * 512),
    dict(out=A + (1 << 20), lse=A + ROWS * 256), dict(out=A + (1 << 20), q=A + ROWS * 4, lse=A)])
def test_not_refused(lib, kw):  # noqa: F811
    """The injected failure stands behind the checks."""
    lib.coli_set_fail_after(I64(0))
    try:
        assert attend(lib, **kw) == -6
    finally:
        lib.coli_set_fail_after(I64(-1))
