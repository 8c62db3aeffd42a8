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


@pytest.mark.parametrize("M", [3, 12, 20, 64, 100, 200])
@pytest.mark.parametrize("N,K", [(4096, 14336), (1000, 8192), (2050, 14224)])
def test_long_k(M, N, K):
    """Dozens of blocks of K in a CTA's share: every ring goes round several times, and
    the scales of the next blocks take the place of those before."""
    a, sa, b, sb, bias = make(M, N, K, seed=M + K, spread=5.0)
    check(fk.fp8kv_block_matmul(a, sa, b, sb, out_dtype=torch.float32), a, sa, b, sb)
    check(fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias), a, sa, b, sb, bias)


@pytest.mark.parametrize("M", [8, 20, 64])
def test_long_k_and_many_columns(M):
    """So many columns that no share of K is split off: 64 blocks one after the other."""
    a, sa, b, sb, _ = make(M, 28672, 8192, seed=M, spread=5.0)
    check(fk.fp8kv_block_matmul(a, sa, b, sb, out_dtype=torch.float32), a, sa, b, sb)


@pytest.mark.parametrize("M", [20, 100, 300])
def test_long_k_each_block_has_its_scales(M):
    """Ones everywhere: the sum of the pairs of scales, exactly (powers of two, 112 blocks)."""
    N, K, kb = 300, 14336, 112
    a, b = (torch.full((r, K), 0x38, dtype=torch.uint8, device="cuda") for r in (M, N))
    g = torch.Generator(device="cuda").manual_seed(2)
    sa = torch.exp2(torch.randint(-3, 4, (M, kb), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-3, 4, (3, kb), generator=g, device="cuda").float())
    out = fk.fp8kv_block_matmul(a, sa, b, sb, out_dtype=torch.float32)
    want = 128 * (sa.double() @ sb.double().T).repeat_interleave(128, 1)[:, :N]
    assert fk.fp8kv_get_device_error() == 0 and torch.equal(out.double(), want)
