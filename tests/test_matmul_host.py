"""Refusals of the 8-bit matrix product, on the host: every call below is turned
down by its argument checks, before any CUDA call.  No GPU."""
import pytest

from test_step_host import INVALID, UNSUPPORTED, lib  # noqa: F401


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(m=-1)), (INVALID, dict(n=-1)), (INVALID, dict(k=0)), (INVALID, dict(k=-16)), (INVALID, dict(dt=2)),
    (INVALID, dict(a=None)), (INVALID, dict(sa=None)), (INVALID, dict(b=None)), (INVALID, dict(sb=None)), (INVALID, dict(out=None)),
    (INVALID, dict(a=0x100008)), (INVALID, dict(b=0x300004)), (INVALID, dict(out=0x600008)), (INVALID, dict(sa=0x200002)),
    (INVALID, dict(sb=0x400001)), (INVALID, dict(bias=0x500002)), (INVALID, dict(out=0x100000)), (INVALID, dict(out=0x300010)),
    (INVALID, dict(bias=0x600010)), (INVALID, dict(sa=0x600100)), (INVALID, dict(out=0x400000)),
    (UNSUPPORTED, dict(k=100)), (UNSUPPORTED, dict(k=8)), (UNSUPPORTED, dict(m=(1 << 30) + 1)), (UNSUPPORTED, dict(n=(1 << 30) + 1)),
    (UNSUPPORTED, dict(k=1 << 31)), (UNSUPPORTED, dict(m=1 << 30, n=1 << 30)), (0, dict(m=0)), (0, dict(n=0, out=None)),
])
def test_refusals(lib, want, kw):  # noqa: F811
    a = dict(a=0x100000, sa=0x200000, b=0x300000, sb=0x400000, bias=0x500000, m=64, n=256, k=512, out=0x600000, dt=0)
    a.update(kw)
    assert lib.fp8kv_block_matmul(*a.values(), None) == want
