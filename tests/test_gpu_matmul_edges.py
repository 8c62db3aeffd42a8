"""The matrix product of e4m3 codes where its kernels end and where K is long:
calls directly behind each other.  Definition, tolerance and inputs are those of
test_gpu_matmul."""
import pytest
import torch

import fp8_quantized_kv_gb300 as fk
from test_gpu_matmul import check, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


def test_kernels_that_follow_a_pair_of_ctas():
    """Pairs of CTAs end while the next kernel starts on their SMs, with barriers of its
    own at other places of shared memory: 256 and 128 columns a tile, half tiles, one block
    of K (fewer than any ring has places), clusters that split K.  Every result stays what
    it was alone, on one stream and on two."""
    shapes = [(300, 2304, 128), (1000, 6144, 512), (64, 1024, 1024), (600, 4608, 640), (129, 256, 16), (30, 2048, 2048),
              (4000, 2560, 256), (128, 6144, 384), (200, 1000, 1408), (900, 4609, 272)]
    sets = [make(*s, seed=9) for s in shapes]
    want = [fk.fp8kv_block_matmul(*s[:4]) for s in sets]
    for w, s in zip(want, sets):
        check(w, *s[:4])
    outs = [[torch.empty_like(w) for w in want] for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in outs]
    torch.cuda.synchronize()
    for turn in range(40):
        for k, (out, st) in enumerate(zip(outs, streams)):
            for o in out:
                o.fill_(7)
        torch.cuda.synchronize()
        for i in range(len(sets)):
            for k, (out, st) in enumerate(zip(outs, streams[:1 + turn % 2])):
                j = (i * (3 if k else 1) + turn) % len(sets)
                fk.fp8kv_block_matmul(*sets[j][:4], out=out[j], stream=st)
        torch.cuda.synchronize()
        for out in outs[:1 + turn % 2]:
            assert all(torch.equal(o, w) for o, w in zip(out, want))
    assert fk.fp8kv_get_device_error() == 0
