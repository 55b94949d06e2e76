"""The 8-bit matrix product against the float64 product of the values its
operands stand for.

Tolerance, per element, relative to S = sum |terms|: products of two e4m3
values are exact in float32; the tensor cores may lose up to 2^-23 of a block's
partial sum in each of its 128 additions (2^-16 S); each of the G blocks then
costs three roundings of 2^-24.  bf16 output adds one rounding, 2^-8."""
import numpy as np
import pytest
import torch

from oracle import head_ops as ref

pytestmark = pytest.mark.gpu

flce = pytest.importorskip("lm_head_linear_flce_gb300")

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def operands(M, V, K, seed=0, spread=1.0):
    """Random bytes with scales that vary over orders of magnitude."""
    g = torch.Generator().manual_seed(seed)

    def q(r, c):
        v = torch.randn(r, c, generator=g) * 120
        return v.clamp(-448, 448).to(torch.float8_e4m3fn).cuda()

    def s(r):
        return (torch.exp(spread * torch.randn(r, -(-K // 128), generator=g)) * 1e-3).cuda()
    return q(M, K), s(M), q(V, K), s(-(-V // 128))


def check(y, a, sa, b, sb, out):
    want, mag = ref.matmul_fp8(f64(a), f64(sa), f64(b), f64(sb))
    G = sa.shape[-1]
    tol = (2.0 ** -16 + 3 * (G + 1) * 2.0 ** -24) * mag
    if out == BF:
        tol = tol + 1.01 * 2.0 ** -8 * np.abs(want)
    err = np.abs(f64(y) - want)
    assert y.dtype == out and (err <= tol).all(), (err - tol).max()


SHAPES = [(1, 1, 16), (1, 128, 128), (1, 1000, 4096), (2, 129, 144), (16, 300, 256), (17, 257, 384),
          (31, 5000, 272), (32, 130, 1024), (33, 127, 2064), (64, 513, 640), (65, 512, 128),
          (100, 1000, 1040), (127, 2000, 512), (128, 700, 1552), (129, 300, 400), (200, 999, 1024),
          (255, 257, 256), (256, 256, 384), (257, 1025, 272), (512, 3000, 512), (700, 40, 3584),
          (5, 40000, 128), (3, 20, 8192), (1, 8, 65536)]


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("M,V,K", SHAPES)
def test_matches_the_float64_product(M, V, K, out):
    a, sa, b, sb = operands(M, V, K, seed=M + V + K)
    y = flce.matmul_fp8(a, sa, b, sb, out_dtype=out)
    assert y.shape == (M, V)
    check(y, a, sa, b, sb, out)


# several tiles for every CTA or pair, of each kind of tile
@pytest.mark.parametrize("M,V,K", [(60, 20003, 144), (90, 20001, 160), (300, 20099, 272),
                                   (250, 39001, 144), (130, 10007, 400), (1000, 9001, 128)])
def test_many_tiles(M, V, K):
    a, sa, b, sb = operands(M, V, K, 5, 1.0)
    for out in (BF, F32):
        check(flce.matmul_fp8(a, sa, b, sb, out_dtype=out), a, sa, b, sb, out)


def test_every_number_of_rows():
    # each padding of the rows, filled, one below and one above; rows of 144 bytes
    g = torch.Generator().manual_seed(3)
    V, K = 259, 144
    b, sb = flce.quantize_fp8(torch.randn(V, K, generator=g).cuda())
    x = torch.randn(70, K, generator=g).cuda()
    whole = flce.quantize_fp8(x, block_rows=1)
    want, mag = ref.matmul_fp8(f64(whole[0]), f64(whole[1]), f64(b), f64(sb))
    for M in range(1, 71):
        y = f64(flce.matmul_fp8(whole[0][:M], whole[1][:M], b, sb, out_dtype=F32))
        assert y.shape == (M, V)
        assert (np.abs(y - want[:M]) <= 2.0 ** -15 * mag[:M]).all(), M


@pytest.mark.parametrize("M", [1, 7, 40, 90, 300, 1100])
def test_every_scale_reaches_its_block(M):
    """Exact case: operands of ones, scales powers of two that name their place;
    sums of a few such are exact in float32."""
    V, K = 700, 144 + 128
    G = -(-K // 128)
    a = torch.ones(M, K).to(torch.float8_e4m3fn).cuda()
    b = torch.ones(V, K).to(torch.float8_e4m3fn).cuda()
    sa = (2.0 ** -(torch.arange(M)[:, None] % 5 + 2.0 * torch.arange(G))).cuda()
    sb = (2.0 ** (torch.arange(-(-V // 128))[:, None] + 1.0 * torch.arange(G))).cuda()
    want, _ = ref.matmul_fp8(f64(a), f64(sa), f64(b), f64(sb))
    assert np.array_equal(f64(flce.matmul_fp8(a, sa, b, sb, out_dtype=F32)), want)


def test_small_integers_are_exact():
    """Integers up to 8 in magnitude: every partial sum is exact in float32."""
    g = torch.Generator().manual_seed(3)
    for M, V, K in ((1, 300, 512), (20, 200, 1040), (129, 256, 2048), (600, 520, 640)):
        a = torch.randint(-8, 9, (M, K), generator=g).float()
        b = torch.randint(-8, 9, (V, K), generator=g).float()
        G = -(-K // 128)
        y = flce.matmul_fp8(a.to(torch.float8_e4m3fn).cuda(), torch.ones(M, G, device="cuda"),
                            b.to(torch.float8_e4m3fn).cuda(),
                            torch.ones(-(-V // 128), G, device="cuda"), out_dtype=F32)
        assert torch.equal(y.cpu(), a @ b.t())


def test_large_product_spot_rows():
    M, V, K = 1500, 20000, 1024
    a, sa, b, sb = operands(M, V, K, seed=9)
    y = flce.matmul_fp8(a, sa, b, sb)
    rows = torch.tensor([0, 1, 127, 128, 255, 256, 700, 1279, 1280, 1499], device="cuda")
    check(y[rows], a.view(torch.uint8)[rows].view(a.dtype), sa[rows], b, sb, BF)


def test_shapes_strides_and_views():
    a, sa, b, sb = operands(12, 300, 256, seed=4)
    want = flce.matmul_fp8(a, sa, b, sb, out_dtype=F32)
    y = flce.matmul_fp8(a.view(3, 4, 256), sa.view(3, 4, 2), b, sb, out_dtype=F32)
    assert y.shape == (3, 4, 300) and torch.equal(y.view(12, 300), want)
    wide = torch.zeros(12, 304, dtype=torch.uint8, device="cuda")
    for lo in (0, 16, 7):  # 7: copied, its rows are not 16-byte aligned
        v = wide[:, lo:lo + 256]
        v.copy_(a.view(torch.uint8))
        y = flce.matmul_fp8(v.view(torch.float8_e4m3fn), sa, b, sb, out_dtype=F32)
        assert torch.equal(y, want)
    y = flce.matmul_fp8(a, sa.t().contiguous().t(), b, sb.t().contiguous().t(), out_dtype=F32)
    assert torch.equal(y, want)
    e = flce.matmul_fp8(a[:0], sa[:0], b, sb)
    assert e.shape == (0, 300)


@pytest.mark.parametrize("M", [2, 50, 400])
def test_non_finite_values_stay_in_their_row_and_column(M):
    a, sa, b, sb = operands(M, 260, 256, seed=5)
    av = a.float()
    av[1, 3] = float("nan")
    a2 = av.to(torch.float8_e4m3fn)
    y = flce.matmul_fp8(a2, sa, b, sb)
    y0 = flce.matmul_fp8(a, sa, b, sb)
    assert torch.isnan(y[1]).all()
    keep = [m for m in range(M) if m != 1]
    assert torch.equal(y[keep], y0[keep])
    sb2 = sb.clone()
    sb2[2, 1] = float("inf")
    y = flce.matmul_fp8(a, sa, b, sb2)
    assert torch.equal(y[:, :256], y0[:, :256]) and not torch.isfinite(y[:, 256:]).any()


def test_writes_stay_inside_and_repeat_bit_for_bit():
    from lm_head_linear_flce_gb300 import head_ops
    for M, V, K in ((3, 301, 256), (40, 1000, 1024), (300, 777, 384)):
        for out in (BF, F32):
            a, sa, b, sb = operands(M, V, K, seed=6)
            ldy = V + 3
            buf = torch.full((M + 2, ldy), 7.0, dtype=out, device="cuda")
            head_ops._call("flce_matmul_fp8", a.get_device(), a.data_ptr(), K, sa.data_ptr(),
                           b.data_ptr(), K, sb.data_ptr(), M, V, K, buf[1:].data_ptr(), ldy,
                           head_ops._DTYPE[out])
            y = flce.matmul_fp8(a, sa, b, sb, out_dtype=out)
            assert torch.equal(buf[1:M + 1, :V], y)
            buf[1:M + 1, :V] = 7
            assert (buf == 7).all()


def test_side_stream_and_graph():
    a, sa, b, sb = operands(5, 3000, 1024, seed=7)
    want = flce.matmul_fp8(a, sa, b, sb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y = flce.matmul_fp8(a, sa * 1, b, sb)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(y, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = flce.matmul_fp8(a, sa, b, sb)
    sa.mul_(2)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want * 2)


def test_refusals():
    a, sa, b, sb = operands(4, 100, 256)
    for call in (lambda: flce.matmul_fp8(a.float(), sa, b, sb),
                 lambda: flce.matmul_fp8(a, sa[:3], b, sb),
                 lambda: flce.matmul_fp8(a, sa, b, sb[:, :1]),
                 lambda: flce.matmul_fp8(a[:, :128], sa, b, sb),
                 lambda: flce.matmul_fp8(a, sa.double(), b, sb),
                 lambda: flce.matmul_fp8(a, sa, b, sb, out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(flce.FlceError):  # K is not a multiple of 16
        flce.matmul_fp8(a[:, :200], sa, b[:, :200], sb)


# each kernel: rows of every padding, whole K and split; tiles of 128 and 256
# columns on a CTA, and on a pair
TIMEOUTS = [(5, 45000, 640), (20, 45000, 640), (40, 45000, 640), (5, 1000, 1024), (64, 1000, 1024),
            (100, 4000, 640), (100, 45000, 640), (256, 45000, 640)]


def stopped(M, V, K, out, stop_after, limit_ns):
    """The product of CTAs that stop loading after `stop_after` blocks, in a
    buffer of ones with a row and three columns to spare."""
    from lm_head_linear_flce_gb300 import head_ops
    a, sa, b, sb = operands(M, V, K, seed=8)
    buf = torch.ones(M + 1, V + 3, dtype=out, device="cuda")
    head_ops._call("flce_selftest_matmul_fp8_timeout", a.get_device(), stop_after, limit_ns,
                   a.data_ptr(), K, sa.data_ptr(), b.data_ptr(), K, sb.data_ptr(), M, V, K,
                   buf.data_ptr(), V + 3, head_ops._DTYPE[out])
    torch.cuda.synchronize()
    assert (buf[M] == 1).all() and (buf[:, V:] == 1).all()
    return buf[:M, :V], (a, sa, b, sb)


@pytest.mark.parametrize("stop_after", [0, 1, 3])
@pytest.mark.parametrize("M,V,K", TIMEOUTS)
def test_a_wait_that_runs_out_ends_the_kernel(M, V, K, stop_after):
    for out in (BF, F32):
        y, op = stopped(M, V, K, out, stop_after, 20_000_000)
        # the next product is right
        check(flce.matmul_fp8(*op, out_dtype=out)[:, :257], op[0], op[1],
              op[2].view(torch.uint8)[:257].view(op[2].dtype), op[3][:3], out)


@pytest.mark.parametrize("M,V,K", TIMEOUTS)
def test_a_short_limit_leaves_nothing_in_flight(M, V, K):
    """Kernels that give up at once, right before one that takes their place on
    the SMs: its stages are its own."""
    for stop_after in (0, 1, 2, 3, 4):
        y, op = stopped(M, V, K, F32, stop_after, 1)
        for _ in range(2):
            check(flce.matmul_fp8(*op, out_dtype=F32)[:, :257], op[0], op[1],
                  op[2].view(torch.uint8)[:257].view(op[2].dtype), op[3][:3], F32)


@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("stop_after", [0, 1, 5])
@pytest.mark.parametrize("M,V,K", TIMEOUTS + [(5, 1000, 1104), (64, 1000, 1104), (33, 700, 2064)])
def test_what_is_not_complete_is_nan(M, V, K, stop_after, out):
    """Every element is NaN or right, where parts of a split K are complete and
    others are not too, and where a CTA gives up in its second tile."""
    y, (a, sa, b, sb) = stopped(M, V, K, out, stop_after, 20_000_000)
    gone = torch.isnan(y)
    want = flce.matmul_fp8(a, sa, b, sb, out_dtype=out)  # (checked by the tests above)
    assert torch.equal(y[~gone], want[~gone])
    G, tiles = -(-K // 128), -(-V // 128)
    split = M <= 64 and 2 * tiles <= 304 and 2 <= G
    if stop_after == 0:
        assert gone.all()
    elif split:  # parts of 1 block, or of 1 and 2: complete or not, the same for every tile
        parts = max(p for p in (1, 2, 4, 8) if p * tiles <= 304 and p <= G)
        assert gone.all() if -(-G // parts) > stop_after else not gone.any()
    elif stop_after < G:
        assert gone.all()
    elif V == 45000:  # the first tiles are complete, the next are not
        assert gone.any() and not gone.all()
    else:
        assert not gone.any()


# (V, K): more tiles of V than places for them, so that a CTA goes on to a second
# one; and fewer, but too many to split K.  Blocks of K that fill neither the
# stages nor the accumulators evenly.
@pytest.mark.parametrize("V,K", [(40003, 400), (39001, 912), (30000, 656)])
def test_few_rows_on_a_vocabulary(V, K):
    a, sa, b, sb = operands(48, V, K, seed=V)
    want, mag = ref.matmul_fp8(f64(a), f64(sa), f64(b), f64(sb))
    G = sa.shape[-1]
    tol = (2.0 ** -16 + 3 * (G + 1) * 2.0 ** -24) * mag
    for M in (1, 16, 17, 32, 33, 48):
        for out in (BF, F32):
            y = f64(flce.matmul_fp8(a[:M], sa[:M], b, sb, out_dtype=out))
            t = tol[:M] + (1.01 * 2.0 ** -8 * np.abs(want[:M]) if out == BF else 0)
            assert (np.abs(y - want[:M]) <= t).all(), (M, out)
