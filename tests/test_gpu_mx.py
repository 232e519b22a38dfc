"""Microscaled 4-bit quantization and products against the fp64 oracle.

Tolerances. Quantization is compared bit for bit. A product sums exact terms
in fp32: a chain through K has at most K / 32 matrix instructions, each adding
at most 32 or 128 products, and the partial sums of at most 16 waves; with B
the sum of the terms' magnitudes every addition loses at most 2^-23 of B, so
|y - ref| <= (K / 32 + 160) * 2^-23 * B before the one rounding to y's type
(2^-11 or 2^-8 of |y|, and half of fp16's smallest step).
"""

import numpy as np
import pytest

from oracle import mx

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
HALF = [torch.float16, torch.bfloat16]
ALL = [torch.float32, *HALF]


@pytest.fixture(scope="module")
def lutq():
    import weight_only_lut_amd as m
    m.load_library()
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    return m


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def unit(dtype):
    return 2.0 ** -11 if dtype == torch.float16 else 2.0 ** -8


def close(y, ref, B, K, dtype):
    bound = (K / 32 + 160) * 2.0 ** -23 * B
    bound = bound + unit(dtype) * (np.abs(ref) + bound) + (2.0 ** -25 if dtype == torch.float16 else 0)
    bad = np.abs(f64(y) - ref) > bound
    assert not bad.any(), (int(bad.sum()), float((np.abs(f64(y) - ref) / np.maximum(bound, 1e-300)).max()))


def values(rng, shape, spread):
    """Normal values over `spread` octaves, with zeros and powers of two among them."""
    x = rng.standard_normal(shape) * 2.0 ** rng.integers(-spread, spread + 1, shape)
    x[rng.random(shape) < 0.05] = 0.0
    return x


def weights(rng, N, K):
    """Codes of every value and scales of a few octaves, as a quantizer leaves them."""
    return rng.integers(0, 256, (N, K // 2)).astype(np.uint8), rng.integers(118, 124, (N, K // 32)).astype(np.uint8)


# ---- quantization ----------------------------------------------------------------

@pytest.mark.parametrize("rule", ["floor", "ceil"])
@pytest.mark.parametrize("dtype", ALL)
@pytest.mark.parametrize("rows,K", [(1, 32), (1, 2048), (3, 96), (2, 8224), (37, 1056), (0, 64), (5, 0)])
def test_quantize_matches_the_oracle(lutq, rows, K, dtype, rule):
    x = torch.from_numpy(values(np.random.default_rng(rows * 7 + K), (rows, K), 6)).to(dtype)
    c, s = lutq.mx_quantize(x.cuda(), rule=rule)
    oc, os_ = mx.quantize(f64(x), rule)
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)
    for out in ALL:
        v = lutq.mx_dequantize(c, s, out)
        assert torch.equal(v.cpu(), torch.from_numpy(mx.dequantize(oc, os_)).to(out))


@pytest.mark.parametrize("rule", ["floor", "ceil"])
def test_quantize_halfway_cases_and_extremes(lutq, rule):
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.999])
    blocks = []
    for e in (-149, -140, -127, -126, -30, 0, 30, 120, 125):
        v = np.zeros(32)
        m = np.concatenate((mids, np.nextafter(mids.astype(np.float32), np.float32(0)),
                            np.nextafter(mids.astype(np.float32), np.float32(9))))
        v[:len(m)] = m * 2.0 ** e * np.where(np.arange(len(m)) % 2, -1, 1)
        blocks.append(v)
    blocks += [np.full(32, 3.4e38), np.full(32, -0.0), np.zeros(32)]
    x = np.concatenate(blocks)[None].astype(np.float32)
    c, s = lutq.mx_quantize(dev(x), rule=rule)
    oc, os_ = mx.quantize(x, rule)
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)


@pytest.mark.parametrize("dtype", ALL)
def test_quantize_nan_and_inf_blocks(lutq, dtype):
    x = torch.randn(4, 128)
    x[0, 5], x[1, 40], x[2, 127], x[3, 64] = float("nan"), float("inf"), float("-inf"), float("nan")
    x = x.to(dtype)
    c, s = lutq.mx_quantize(x.cuda())
    oc, os_ = mx.quantize(f64(x))
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)
    assert (s.cpu() == 255).sum() == 4
    assert torch.isnan(lutq.mx_dequantize(c, s, dtype).cpu()).sum() == 4 * 32


@pytest.mark.parametrize("dtype", ALL)
def test_quantize_strided_rows(lutq, dtype):
    x = torch.randn(70, 512, dtype=torch.float32).to(dtype).cuda()
    view = x[:, 64:160]
    c, s = lutq.mx_quantize(view)
    oc, os_ = mx.quantize(f64(view))
    assert np.array_equal(s.cpu().numpy(), os_) and np.array_equal(c.cpu().numpy(), oc)
    with pytest.raises(lutq.LutqError) as e:      # a row start that is not 16-byte aligned
        lutq.mx_quantize(x[:, 1:33])
    assert e.value.code == -4


def test_quantize_many_strided_rows(lutq):
    """More rows than one grid dimension holds."""
    x = torch.randn(70001, 64, device="cuda")
    c, s = lutq.mx_quantize(x[:, :32])
    oc, os_ = lutq.mx_quantize(x[:, :32].contiguous())
    assert torch.equal(c, oc) and torch.equal(s, os_)


def test_quantize_past_32_bit_offsets(lutq):
    rows, K = 2 ** 17 + 1, 2 ** 14 + 32      # over 2^31 values
    x = torch.zeros(rows, K, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.arange(K, device="cuda") % 13 - 6
    x[rows // 2, 7] = 3.0
    c, s = lutq.mx_quantize(x)
    v = lutq.mx_dequantize(c, s)
    want_c, want_s = mx.quantize(f64(x[-1:]))
    assert np.array_equal(c[-1:].cpu().numpy(), want_c) and np.array_equal(s[-1:].cpu().numpy(), want_s)
    assert float(v[rows // 2, 7]) == 3.0 and int(v[:-1].count_nonzero()) == 1
    assert np.array_equal(f64(v[-1:]), mx.dequantize(want_c, want_s))


# ---- products ----------------------------------------------------------------------

PATHS = ["stream", "tile"]


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("N,K", [(16, 32), (33, 160), (300, 672), (272, 1024)])
def test_identity_activations_return_the_weights(lutq, N, K, dtype, path):
    """x = I: every weight comes out once, exactly, from every place of the layout."""
    c, s = weights(np.random.default_rng(N + K), N, K)
    y = lutq.mx_matmul(torch.eye(K, dtype=dtype, device="cuda"), lutq.mx_pack(dev(c), dev(s)), path=path)
    assert np.array_equal(f64(y), mx.dequantize(c, s).T)


SHAPES = [(1, 1, 32), (1, 1024, 1024), (2, 17, 96), (5, 130, 4128), (16, 64, 256), (17, 48, 288), (31, 77, 992),
          (33, 100, 2048), (64, 16, 64), (65, 200, 544), (127, 257, 160), (300, 530, 1056), (513, 31, 128)]


@pytest.mark.parametrize("path", ["auto", *PATHS])
@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul(lutq, M, N, K, dtype, path):
    rng = np.random.default_rng(M * 31 + N + K)
    c, s = weights(rng, N, K)
    x = torch.from_numpy(values(rng, (M, K), 3)).to(dtype)
    y = lutq.mx_matmul(x.cuda(), lutq.mx_pack(dev(c), dev(s)), path=path)
    close(y, *mx.matmul(f64(x), mx.dequantize(c, s)), K, dtype)


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_matmul_of_two_4_bit_operands(lutq, M, N, K, dtype):
    rng = np.random.default_rng(M * 37 + N + K)
    c, s = weights(rng, N, K)
    x = torch.from_numpy(values(rng, (M, K), 3)).float().cuda()
    xc, xs = lutq.mx_quantize(x)
    y = lutq.mx_matmul((xc, xs), lutq.mx_pack(dev(c), dev(s)), dtype=dtype)
    xv = mx.dequantize(xc.cpu().numpy(), xs.cpu().numpy())
    close(y, *mx.matmul(xv, mx.dequantize(c, s)), K, dtype)


# enough tiles to fill the device, for each of the large shapes, with ragged edges; wide
# results whose rows are not a multiple of 16 bytes; and few tiles with a long K
LARGE = [(2043, 8184, 160), (4220, 7928, 96), (2053, 8200, 224), (2050, 8189, 96), (4090, 4088, 288),
         (520, 1000, 4128), (200, 130, 14336), (1030, 2056, 1056)]


@pytest.mark.parametrize("dtype", HALF)
@pytest.mark.parametrize("M,N,K", LARGE)
def test_matmul_large(lutq, M, N, K, dtype):
    rng = np.random.default_rng(M + N + K)
    c, s = weights(rng, N, K)
    W, w = lutq.mx_pack(dev(c), dev(s)), mx.dequantize(c, s)
    x = torch.from_numpy(values(rng, (M, K), 3)).to(dtype).cuda()
    y = lutq.mx_matmul(x, W)
    close(y, *mx.matmul(f64(x), w), K, dtype)
    assert torch.equal(y, lutq.mx_matmul(x, W))
    xc, xs = lutq.mx_quantize(x)
    y = lutq.mx_matmul((xc, xs), W, dtype=dtype)
    close(y, *mx.matmul(mx.dequantize(xc.cpu().numpy(), xs.cpu().numpy()), w), K, dtype)
    assert torch.equal(y, lutq.mx_matmul((xc, xs), W, dtype=dtype))


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", HALF)
def test_matmul_scales_far_apart(lutq, dtype, path):
    """Blocks within 2^36 of their row's largest enter exactly; rows may be anywhere;
    a zero block's scale does not matter."""
    rng = np.random.default_rng(8)
    N, K = 48, 256
    c, s = weights(rng, N, K)
    s[:] = rng.integers(0, 37, s.shape) + rng.integers(60, 160, (N, 1))
    s[5] = 0
    c[7, 16:32] &= 0x88
    s[7, 1] = 254
    c[9] = 0
    W = lutq.mx_pack(dev(c), dev(s))
    w = mx.dequantize(c, s)
    x = torch.eye(K, dtype=dtype, device="cuda")
    with np.errstate(over="ignore"):
        want = torch.from_numpy(w.T).to(torch.float32).to(dtype)
    got = lutq.mx_matmul(x, W, path=path).cpu()
    assert torch.equal(got, want)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("dtype", HALF)
def test_matmul_nan_blocks_and_nan_activations(lutq, dtype, path):
    """A NaN block makes its row's outputs NaN and no other; so does a NaN activation its row's."""
    rng = np.random.default_rng(9)
    c, s = weights(rng, 40, 160)
    s[3, 4] = s[20, 0] = 255
    x = torch.randn(7, 160, dtype=torch.float32).to(dtype)
    x[2, 159] = float("nan")
    y = lutq.mx_matmul(x.cuda(), lutq.mx_pack(dev(c), dev(s)), path=path).cpu()
    want = torch.zeros(7, 40, dtype=torch.bool)
    want[2] = want[:, 3] = want[:, 20] = True
    assert torch.equal(torch.isnan(y), want)
    xc, xs = lutq.mx_quantize(x.cuda())
    assert torch.equal(torch.isnan(lutq.mx_matmul((xc, xs), lutq.mx_pack(dev(c), dev(s))).cpu()), want)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("M", [1, 20, 200])
def test_matmul_reads_and_writes_nothing_else(lutq, M, path):
    """NaN around strided rows of x is not read; y around the output is not written."""
    rng = np.random.default_rng(M)
    N, K = 45, 224
    c, s = weights(rng, N, K)
    W = lutq.mx_pack(dev(c), dev(s))
    wide = torch.full((M, K + 32), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 16:16 + K] = torch.randn(M, K, device="cuda").to(torch.bfloat16)
    x = wide[:, 16:16 + K]
    buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
    y = lutq.mx_matmul(x, W, path=path, out=buf[32:32 + M * N].view(M, N))
    assert bool((buf[:32] == 7).all()) and bool((buf[32 + M * N:] == 7).all())
    close(y, *mx.matmul(f64(x), mx.dequantize(c, s)), K, torch.bfloat16)


@pytest.mark.parametrize("M", [3, 70, 600])
def test_matmul_into_an_8_byte_aligned_output(lutq, M):
    rng = np.random.default_rng(M)
    N, K = 264, 320
    c, s = weights(rng, N, K)
    W = lutq.mx_pack(dev(c), dev(s))
    x = torch.randn(M, K, device="cuda").half()
    buf = torch.full((M * N + 8,), 7.0, dtype=torch.float16, device="cuda")
    for src in (x, lutq.mx_quantize(x)):
        y = lutq.mx_matmul(src, W, dtype=torch.float16, out=buf[4:4 + M * N].view(M, N))
        assert torch.equal(y, lutq.mx_matmul(src, W, dtype=torch.float16))
        assert bool((buf[:4] == 7).all()) and bool((buf[4 + M * N:] == 7).all())
    with pytest.raises(lutq.LutqError) as e:
        lutq.mx_matmul(x, W, out=buf[2:2 + M * N].view(M, N))
    assert e.value.code == -4


@pytest.mark.parametrize("M,N,K", [(0, 16, 64), (4, 0, 64), (4, 16, 0)])
def test_matmul_empty(lutq, M, N, K):
    W = lutq.mx_pack(torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda"),
                     torch.zeros((N, K // 32), dtype=torch.uint8, device="cuda"))
    x = torch.ones((M, K), dtype=torch.float16, device="cuda")
    assert not lutq.mx_matmul(x, W).any()
    assert not lutq.mx_matmul(lutq.mx_quantize(x), W).any()


@pytest.mark.parametrize("dtype", HALF)
def test_packed_offsets_past_32_bits(lutq, dtype):
    """Weights of over 2^32 bytes: one-hot activations read the first and last block of the last rows."""
    N, K = 2 ** 18 + 5, 2 ** 15 + 32
    c = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.full((N, K // 32), 127, dtype=torch.uint8, device="cuda")
    rng = np.random.default_rng(3)
    tail, _ = weights(rng, 21, K)
    c[-21:] = dev(tail)
    W = lutq.mx_pack(c, s)
    del c
    at = [0, 31, 32, K - 33, K - 1]
    x = torch.zeros((len(at), K), dtype=dtype, device="cuda")
    for i, k in enumerate(at):
        x[i, k] = 1
    w = mx.dequantize(tail, s[-21:].cpu().numpy())
    for path in PATHS:
        y = lutq.mx_matmul(x, W, path=path)
        assert np.array_equal(f64(y[:, -21:]), w[:, at].T) and not y[:, :-21].any()
    y = lutq.mx_matmul(lutq.mx_quantize(x), W)
    assert np.array_equal(f64(y[:, -21:]), w[:, at].T) and not y[:, :-21].any()


def test_graph_replays_and_streams(lutq):
    """Captured products replay the eager bits, with eager work between replays;
    work on a side stream uses that stream."""
    rng = np.random.default_rng(4)
    c, s = weights(rng, 200, 512)
    W = lutq.mx_pack(dev(c), dev(s))
    x1, x2 = (torch.randn(m, 512, device="cuda").to(torch.float16) for m in (3, 150))

    def work():
        return (lutq.mx_matmul(x1, W), lutq.mx_matmul(x2, W), lutq.mx_matmul(lutq.mx_quantize(x2), W))
    eager = [t.clone() for t in work()]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        out = work()
    for _ in range(4):
        for t in out:
            t.fill_(9)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        work()
        torch.cuda.synchronize()
        for a, b in zip(out, eager):
            assert torch.equal(a, b)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x3 = x1 * 2
        y3 = lutq.mx_matmul(x3, W)
    side.synchronize()
    assert torch.equal(y3, lutq.mx_matmul(x1 * 2, W))


@pytest.mark.parametrize("M", [1, 40, 150, 700])
@pytest.mark.parametrize("four_bit", [False, True])
def test_rows_of_any_width_are_whole_and_nothing_past_them_is_written(lutq, M, four_bit):
    # the same rows of weights, one to eight cut off: the same outputs, bit for bit
    rng = torch.Generator(device="cuda").manual_seed(M)
    K, wide = 512, 1008
    codes, scales = lutq.mx_quantize(torch.randn(wide, K, generator=rng, device="cuda"))
    x = torch.randn(M, K, generator=rng, device="cuda").to(torch.bfloat16)
    x = lutq.mx_quantize(x) if four_bit else x
    full = lutq.mx_matmul(x, lutq.mx_pack(codes, scales))
    for N in range(wide - 8, wide):
        buf = torch.full((M * N + 64,), 7.0, dtype=torch.bfloat16, device="cuda")
        lutq.mx_matmul(x, lutq.mx_pack(codes[:N].contiguous(), scales[:N].contiguous()),
                       out=buf[:M * N].view(M, N))
        assert torch.equal(buf[:M * N].view(M, N), full[:, :N]), N
        assert torch.all(buf[M * N:] == 7.0), N


@pytest.mark.parametrize("M", [1, 6, 13, 29, 70])
def test_4_bit_rows_with_scales_far_apart_and_a_nan(lutq, M):
    # every code under scales from 2^-127 to 2^63, one row with a NaN block
    rng = np.random.default_rng(M)
    N, K = 50, 416
    c, s = weights(rng, N, K)
    xc = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
    xs = np.array([0, 3, 90, 127, 190], np.uint8)[rng.integers(0, 5, (M, K // 32))]
    if M > 1:
        xs[M // 2, 5] = 255
    y = lutq.mx_matmul((dev(xc), dev(xs)), lutq.mx_pack(dev(c), dev(s)))
    ref, B = mx.matmul(mx.dequantize(xc, xs), mx.dequantize(c, s))
    if M > 1:
        assert torch.all(torch.isnan(y[M // 2]))
    rows = [m for m in range(M) if M == 1 or m != M // 2]
    close(y[rows], ref[rows], B[rows], K, torch.bfloat16)
