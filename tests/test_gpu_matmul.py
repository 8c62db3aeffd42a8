"""Matrix product of e4m3 codes with a scale for each block of 128
(fp8kv_block_matmul) against the definition in 64 bits.

Tolerance, per element (derived, not fitted).  With S = sum over all blocks of
|sa sb| sum |a||b|: a block's 128 products of codes are exact, their fp32 sum is at
most 128 2^-23 of their absolute sum off (the tensor core may truncate); the
product of two scales is rounded once (2^-24), and each of the KB sums of blocks
once (2^-24 of what has been summed, below S; the shares of a cluster and the bias
add at most 9 more).  So |out - exact| <= S (2^-16 + 2^-23 + (KB + 9) 2^-24) +
2^-24 |bias|, and a bf16 output adds its rounding, 2^-8 of the value."""
import pytest
import torch

import fp8_quantized_kv_gb300 as fk

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clear_device_error():
    fk.fp8kv_get_device_error(clear=True)
    yield


def values(codes):
    return codes.view(torch.float8_e4m3fn).double()


def make(M, N, K, seed, spread=0.0):
    """Random codes (no NaN) of all sizes, scales that differ by 2^spread either way."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kb = -(-K // 128)
    a, b = (torch.randint(0, 256, (r, K), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8) for r in (M, N))
    for t in (a, b):
        t[(t & 0x7F) == 0x7F] = 0x31
    sa, sb = ((0.5 + torch.rand(s, generator=g, device="cuda")) * torch.exp2(spread * (2 * torch.rand(s, generator=g, device="cuda") - 1))
              for s in ((M, kb), (-(-N // 128), kb)))
    return a, sa, b, sb, torch.randn(N, generator=g, device="cuda") * 1000


def definition(a, sa, b, sb):
    """fp64 product and the sum of its absolute terms."""
    N, K = b.shape
    wa = sa.double().repeat_interleave(128, 1)[:, :K]
    wb = sb.double().repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    x, w = values(a) * wa, values(b) * wb
    return x @ w.T, x.abs() @ w.abs().T


def check(out, a, sa, b, sb, bias=None):
    want, size = definition(a, sa, b, sb)
    tol = size * (2.0 ** -16 + 2.0 ** -23 + (sa.shape[1] + 9) * 2.0 ** -24)
    if bias is not None:
        want = want + bias.double()
        tol = tol + 2.0 ** -24 * bias.double().abs()
    if out.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    assert fk.fp8kv_get_device_error() == 0
    assert torch.isfinite(out).all()
    worst = ((out.double() - want).abs() - tol).max().item()
    assert worst <= 0, f"past the tolerance by {worst:.3e}"


@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 128, 129, 200, 300])
@pytest.mark.parametrize("N,K", [(1, 16), (7, 128), (130, 144), (128, 1024), (392, 400), (1000, 640), (2304, 2064)])
def test_sizes(M, N, K):
    """Single rows to several tiles, short last blocks, odd widths."""
    a, sa, b, sb, bias = make(M, N, K, seed=M + N, spread=3.0)
    check(fk.fp8kv_block_matmul(a, sa, b, sb, out_dtype=torch.float32), a, sa, b, sb)
    check(fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias), a, sa, b, sb, bias)


@pytest.mark.parametrize("M,N,K", [(640, 4608, 896), (1500, 2560, 2048), (997, 4609, 272), (2100, 1111, 512), (5000, 6144, 384),
                                   (12, 5003, 272), (100, 6144, 272), (128, 9001, 128), (600, 2568, 16),
                                   (4100, 1217, 144), (2600, 2056, 400), (20000, 250, 160)])
def test_many_rows(M, N, K):
    """Several tiles a CTA, ragged at both ends, last waves cut into half tiles; few rows beside many columns."""
    a, sa, b, sb, bias = make(M, N, K, seed=M, spread=8.0)
    check(fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias, out_dtype=torch.float32), a, sa, b, sb, bias)
    check(fk.fp8kv_block_matmul(a, sa, b, sb), a, sa, b, sb)


@pytest.mark.parametrize("M", [3, 50, 100, 700])
def test_each_block_has_its_scales(M):
    """Ones everywhere: the result is the sum of the pairs of scales, exactly for powers of two."""
    N, K = 300, 1408
    a, b = (torch.full((r, K), 0x38, dtype=torch.uint8, device="cuda") for r in (M, N))
    g = torch.Generator(device="cuda").manual_seed(1)
    sa = torch.exp2(torch.randint(-3, 4, (M, 11), generator=g, device="cuda").float())
    sb = torch.exp2(torch.randint(-3, 4, (3, 11), generator=g, device="cuda").float())
    out = fk.fp8kv_block_matmul(a, sa, b, sb, out_dtype=torch.float32)
    want = 128 * (sa.double() @ sb.double().T).repeat_interleave(128, 1)[:, :N]
    assert fk.fp8kv_get_device_error() == 0 and torch.equal(out.double(), want)


@pytest.mark.parametrize("M", [5, 12, 50, 600])
def test_not_finite(M):
    """NaN codes and infinite or NaN scales reach the rows and columns that they belong to, and no others."""
    N, K = 260, 384
    a, sa, b, sb, _ = make(M, N, K, seed=3)
    a[2, 200], b[131, 5] = 0x7F, 0xFF
    sa[4, 1] = float("inf")
    out = fk.fp8kv_block_matmul(a, sa, b, sb, out_dtype=torch.float32)
    assert fk.fp8kv_get_device_error() == 0
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[2], bad[4], bad[:, 131] = True, True, True
    assert not bool(torch.isfinite(out[bad]).any()) and bool(torch.isfinite(out[~bad]).all())
    sb[1, 2] = float("nan")
    out = fk.fp8kv_block_matmul(a, sa, b, sb)
    bad[:, 128:256] = True
    assert not bool(torch.isfinite(out[bad]).any()) and bool(torch.isfinite(out[~bad]).all())


@pytest.mark.parametrize("M", [1, 40, 128, 500])
def test_zero_scales(M):
    """All-zero rows as the quantiser leaves them: scale 0, codes 0."""
    x = torch.randn(M, 512, device="cuda").to(torch.bfloat16)
    x[0] = 0
    x[:, 128:256] = 0
    codes, sa = fk.fp8kv_quantize(x.view(M, 4, 128))
    b = torch.randint(0, 127, (256, 512), device="cuda", dtype=torch.int32).to(torch.uint8)
    sb = torch.rand(2, 4, device="cuda")
    out = fk.fp8kv_block_matmul(codes.view(M, 512), sa, b, sb, out_dtype=torch.float32)
    check(out, codes.view(M, 512), sa, b, sb)
    assert not bool(out[0].any())


def test_writes_nothing_else():
    """Rows in front of and behind the output stay as they were."""
    for M, N in ((3, 250), (130, 129), (700, 2000)):
        a, sa, b, sb, _ = make(M, N, 256, seed=5)
        for dt in (torch.bfloat16, torch.float32):
            room = torch.full((M * N + 64 * 8,), 7.0, dtype=dt, device="cuda")
            fk.fp8kv_block_matmul(a, sa, b, sb, out=room[256:256 + M * N].view(M, N))
            assert bool((room[:256] == 7).all()) and bool((room[256 + M * N:] == 7).all())


@pytest.mark.parametrize("M", [8, 100, 900])
def test_repeats_and_graphs(M):
    """The same bits at every call, on another stream and from a replayed graph with other inputs."""
    N, K = 1300, 1664
    a, sa, b, sb, bias = make(M, N, K, seed=6)
    out = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    first = fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias)
    for _ in range(20):
        assert torch.equal(fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias), first)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    again = fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias, stream=other)
    other.synchronize()
    assert torch.equal(again, first)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fk.fp8kv_block_matmul(a, sa, b, sb, bias=bias, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first)
    new = make(M, N, K, seed=7)
    for t, u in zip((a, sa, b, sb, bias), new):
        t.copy_(u)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, fk.fp8kv_block_matmul(*new[:4], bias=new[4])) and fk.fp8kv_get_device_error() == 0


def test_two_streams_at_once():
    """Calls that overlap on the GPU share nothing."""
    sets = [make(*s, seed=8) for s in ((60, 1000, 2048), (900, 1500, 1024))]
    want = [fk.fp8kv_block_matmul(*s[:4]) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(10):
        got = [fk.fp8kv_block_matmul(*s[:4], stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
