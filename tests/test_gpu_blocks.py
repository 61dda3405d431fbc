"""Block-scaled FP8 on the GPU: the quantisers bit for bit against FP32
arithmetic on the CPU, the product against float64 with the tolerance of
tests/block_ref.py and exactly where every sum is a small integer."""
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def m(gpu):
    import nvfp4_moe_skinny_amd as m
    return m


def _randn(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g) * std


def _spread_values(seed, *shape):
    """Unit values with large columns, a zero block, -0, tiny and huge rows."""
    x = _randn(seed, *shape)
    x[..., ::61] *= 50
    flat = x.reshape(-1, shape[-1])
    n = flat.shape[0]
    if n > 2:
        flat[1, :128] = 0
        flat[1, ::7] = -0.0
    if n > 4:
        flat[2] *= 1e-37   # amax below the floor in places
        flat[3] *= 1e36
        flat[4] = 2.0 ** -149
    return x


def _same_codes(got, want):
    """Equal code bytes; a NaN code may have either sign."""
    got, want = got.cpu(), want
    nan = (want & 0x7F) == 0x7F
    assert torch.equal(got[~nan], want[~nan])
    assert ((got[nan] & 0x7F) == 0x7F).all()


@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (1, 128), (3, 144), (16, 2048), (17, 1936), (130, 512),
                                 (1000, 240), (5, 65536), (4099, 32)])
def test_quantize_rows_bit_exact(m, gpu, M, K, typ):
    x = _spread_values(M * 7 + K, M, K).to(TYPES[typ])
    codes, scales = ref.quantize_f32(x.float(), (1,))
    q = m.fp8_quantize_rows(x.to(gpu))
    torch.cuda.synchronize()
    _same_codes(q.codes, codes)
    assert torch.equal(q.scales.cpu(), scales.t())


def test_quantize_rows_every_rounding(m, gpu):
    """A block whose scale is 1 (amax 448): every E4M3 midpoint, its FP32
    neighbours and every E4M3 value, both signs."""
    v = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (v[1:] + v[:-1]) / 2
    inf = torch.tensor(float("inf"))
    vals = torch.cat([v, mid, torch.nextafter(mid, inf), torch.nextafter(mid, -inf)])
    vals = torch.cat([vals, -vals])
    n = ref.nblk(vals.numel()) + 8
    x = torch.zeros(n, 128)
    x[:, 0] = 448.0
    take = vals[: n * 127]
    pad = torch.zeros(n * 127)
    pad[: take.numel()] = take
    x[:, 1:] = pad.view(n, 127)
    codes, scales = ref.quantize_f32(x, (1,))
    assert (scales == 1.0).all()
    q = m.fp8_quantize_rows(x.to(gpu))
    torch.cuda.synchronize()
    _same_codes(q.codes, codes)


@pytest.mark.parametrize("typ", ["bf16", "f32"])
def test_quantize_rows_not_finite(m, gpu, typ):
    x = _randn(3, 6, 400)
    x[0, 5] = float("inf")
    x[1, 200] = float("nan")
    x[2, 399] = -float("inf")
    x[3, 130] = float("nan")
    x[3, 131] = float("inf")
    x = x.to(TYPES[typ])
    q = m.fp8_quantize_rows(x.to(gpu))
    torch.cuda.synchronize()
    codes, scales = ref.quantize_f32(x.float(), (1,))
    s = q.scales.cpu().t()
    bad = ~torch.isfinite(scales)
    assert torch.equal(~torch.isfinite(s), bad)
    assert bad.tolist() == [[True, False, False, False], [False, True, False, False],
                            [False, False, False, True], [False, True, False, False],
                            [False] * 4, [False] * 4]
    ok = ~bad[:, ref.idx(400)]
    assert torch.equal(q.codes.cpu()[ok], codes[ok])
    # every product of such a row is NaN, the other rows' are finite
    w = m.fp8_quantize_blocks(_randn(4, 40, 400).to(gpu))
    y = m.fp8_block_gemm(q, w).cpu()
    assert torch.isnan(y[:4]).all() and torch.isfinite(y[4:]).all()


def test_quantize_rows_strided(m, gpu):
    x = _randn(5, 37, 1024).to(torch.bfloat16).to(gpu)
    part = x[:, 256:256 + 240]
    a, b = m.fp8_quantize_rows(part), m.fp8_quantize_rows(part.contiguous())
    torch.cuda.synchronize()
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    with pytest.raises(m.NVFP4MoEError):  # rows not 16-byte aligned
        m.fp8_quantize_rows(torch.zeros((4, 257), dtype=torch.bfloat16, device=gpu)[:, :256])


@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 16), (4, 512), (33, 1936), (1024, 512), (3, 4096)])
def test_quantize_rows_swiglu(m, gpu, M, K, typ):
    """FP32 silu is within 2^-20 of the value for |a| <= 30: exp's argument
    scaling |a| u, exp and the quotient a few u each ((30 + 8) 2^-24 < 2^-18.7
    doubled for the correlated scale). The code is off by half an E4M3 step of
    the exact v / scale: 2^-4 of the value, or 2^-10 in the subnormal range."""
    u = (_randn(M + K, M, 2 * K) * 4).to(TYPES[typ])
    q = m.fp8_quantize_rows(u.to(gpu), swiglu=True)
    torch.cuda.synchronize()
    a, b = u.double()[:, :K], u.double()[:, K:]
    v = a * torch.sigmoid(a) * b
    eps = 2.0 ** -17
    amax = ref.block_amax(v, (1,)).clamp_min(ref.AMAX_MIN)
    s = q.scales.cpu().double().t()
    assert ((s - amax / 448).abs() <= eps * amax / 448).all()
    sf = s[:, ref.idx(K)]
    got = ref.dequant_rows(q)
    tol = (2.0 ** -4 + eps) * v.abs() + sf * 2.0 ** -10 * (1 + eps)
    assert ((got - v).abs() <= tol).all()


@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("G,N,K", [(1, 1, 16), (2, 130, 272), (3, 128, 128), (1, 257, 2048),
                                   (9, 5, 48), (1, 16, 65536), (4, 1000, 1936)])
def test_quantize_blocks_bit_exact(m, gpu, G, N, K, typ):
    x = _spread_values(G + N + K, G, N, K).to(TYPES[typ])
    codes, scales = ref.quantize_f32(x.float(), (1, 2))
    q = m.fp8_quantize_blocks(x.to(gpu))
    torch.cuda.synchronize()
    _same_codes(q.codes, codes)
    assert torch.equal(q.scales.cpu(), scales)


def _quantized(m, gpu, seed, M, N, K):
    x = m.fp8_quantize_rows(_randn(seed, M, K).to(gpu))
    w = m.fp8_quantize_blocks((_randn(seed + 1, 1, N, K) * K ** -0.5).to(gpu))
    return x, w


GEMM_SHAPES = [(1, 1, 16), (1, 5120, 2048), (2, 130, 128), (4, 64, 2048), (15, 17, 144),
               (16, 2048, 4096), (17, 100, 272), (33, 257, 640), (64, 512, 512), (100, 1, 1936),
               (129, 384, 1024), (333, 1000, 1936), (700, 640, 256), (1, 3, 65536),
               (1025, 1280, 384), (513, 129, 16)]


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", GEMM_SHAPES)
def test_block_gemm(m, gpu, M, N, K, out):
    x, w = _quantized(m, gpu, M + N + K, M, N, K)
    y = m.fp8_block_gemm(x, w, out_dtype=TYPES[out])
    torch.cuda.synchronize()
    x64, w64 = ref.dequant_rows(x), ref.dequant_blocks(w)[0]
    r, mag = ref.gemm_f64(x64, w64)
    cut = ref.fp8_cut(x64, w64, gpu) if out == "bf16" else 0
    ref.assert_close(y, r, ref.gemm_tol(r, mag, K, out == "bf16", cut), (M, N, K))
    again = m.fp8_block_gemm(x, w, out_dtype=TYPES[out])
    assert torch.equal(y, again)


@pytest.mark.parametrize("M,N,K", GEMM_SHAPES + [(2048, 1024, 1536), (300, 5000, 400)])
def test_block_gemm_integers_exact(m, gpu, M, N, K):
    """Codes of integers up to 4 and scales that are powers of two: every sum
    is an integer times a power of two below 2^24, so FP32 holds it exactly and
    any element multiplied with a wrong partner or scale shows."""
    g = torch.Generator().manual_seed(M * N + K)
    xi = torch.randint(-4, 5, (M, K), generator=g).float()
    wi = torch.randint(-4, 5, (1, N, K), generator=g).float()
    xs = 2.0 ** torch.randint(0, 3, (ref.nblk(K), M), generator=g).float()
    ws = 2.0 ** torch.randint(0, 3, (1, ref.nblk(N), ref.nblk(K)), generator=g).float()
    if K > 16384:
        xs, ws = torch.ones_like(xs), torch.ones_like(ws)
    u8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)
    x, w = m.Fp8Rows(u8(xi), xs), m.Fp8Blocks(u8(wi), ws)
    r, mag = ref.gemm_f64(ref.dequant_rows(x), ref.dequant_blocks(w)[0])
    assert mag.max() < 2 ** 24
    dev = lambda q, t: t(q.codes.to(gpu), q.scales.to(gpu))
    xd, wd = dev(x, m.Fp8Rows), dev(w, m.Fp8Blocks)
    assert torch.equal(m.fp8_block_gemm(xd, wd, out_dtype=torch.float32).cpu().double(), r)
    # products of integers up to 4 are multiples of 2^-13 of the largest: none is cut
    assert torch.equal(m.fp8_block_gemm(xd, wd).cpu(), r.to(torch.bfloat16))


@pytest.mark.parametrize("K", [16, 144, 272, 400, 8320])
@pytest.mark.parametrize("M,N", [(2176, 4112), (2300, 4000), (5000, 1300), (300, 33000),
                                 (9000, 1300)])
def test_block_gemm_more_tiles_than_blocks(m, gpu, M, N, K):
    """Blocks that take several tiles in turn, with one to four k steps and with
    more than 64: integers up to 4 (8320 products of at most 16: exact in FP32)."""
    g = torch.Generator(device=gpu).manual_seed(M + N + K)
    u8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device=gpu).float()
    p2 = lambda *s: 2.0 ** torch.randint(0, 2, s, generator=g, device=gpu).float()
    x = m.Fp8Rows(u8(ints(M, K)), p2(ref.nblk(K), M))
    w = m.Fp8Blocks(u8(ints(1, N, K)), p2(1, ref.nblk(N), ref.nblk(K)))
    want = torch.mm(ref.dequant_rows(x).to(gpu), ref.dequant_blocks(w)[0].to(gpu).t().contiguous())
    assert want.abs().max() < 2 ** 24
    out = torch.full((M + 1, N + 3), 7.0, dtype=torch.bfloat16, device=gpu)
    m.fp8_block_gemm(x, w, out=out[:M, :N])
    assert torch.equal(out[:M, :N], want.to(torch.bfloat16))
    assert (out[M] == 7.0).all() and (out[:, N:] == 7.0).all()
    assert torch.equal(m.fp8_block_gemm(x, w, out_dtype=torch.float32).double(), want)


def test_block_gemm_nan_codes_stay_in_their_row_and_column(m, gpu):
    for M, N, K in ((5, 70, 272), (300, 400, 272)):
        x, w = _quantized(m, gpu, 9, M, N, K)
        x.codes[3, 270] = 0x7F
        w.codes[0, 60, 5] = 0xFF
        y = m.fp8_block_gemm(x, w, out_dtype=torch.float32).cpu()
        bad = torch.isnan(y)
        want = torch.zeros_like(bad)
        want[3] = True
        want[:, 60] = True
        assert torch.equal(bad, want)


@pytest.mark.parametrize("M,N", [(3, 50), (200, 300), (600, 130)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_block_gemm_strided_out_leaves_the_rest(m, gpu, M, N, out):
    x, w = _quantized(m, gpu, 21, M, N, 512)
    base = torch.full((M, N + 13), 7.0, dtype=TYPES[out], device=gpu)
    y = m.fp8_block_gemm(x, w, out_dtype=TYPES[out], out=base[:, 5:5 + N])
    plain = m.fp8_block_gemm(x, w, out_dtype=TYPES[out])
    torch.cuda.synchronize()
    assert torch.equal(y, plain) and torch.equal(base[:, 5:5 + N], plain)
    assert (base[:, :5] == 7).all() and (base[:, 5 + N:] == 7).all()


def test_no_rows(m, gpu):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=gpu)
    q = m.fp8_quantize_rows(z(0, 256))
    assert q.codes.shape == (0, 256) and q.scales.shape == (2, 0)
    w = m.fp8_quantize_blocks(z(1, 40, 256))
    assert m.fp8_block_gemm(q, w).shape == (0, 40)
    assert m.fp8_quantize_blocks(z(0, 40, 256)).codes.shape == (0, 40, 256)
    torch.cuda.synchronize()


def test_other_stream(m, gpu):
    x = _randn(31, 64, 1024).to(torch.bfloat16).to(gpu)
    w = m.fp8_quantize_blocks(_randn(32, 256, 1024).to(gpu))
    a = m.fp8_block_gemm(m.fp8_quantize_rows(x), w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    b = m.fp8_block_gemm(m.fp8_quantize_rows(x, stream=st), w, stream=st)
    st.synchronize()
    assert torch.equal(a, b)


def test_offsets_past_32_bits(m, gpu):
    """Rows and results whose offsets pass 2^31 elements and 2^32 bytes: the last
    rows are those of a call on them alone."""
    g = torch.Generator(device=gpu).manual_seed(3)
    M, K = 270000, 8192
    x = torch.empty((M, K), dtype=torch.bfloat16, device=gpu)
    x[:-7].fill_(1.0)
    x[-7:] = torch.randn((7, K), generator=g, device=gpu).to(torch.bfloat16)
    q, q7 = m.fp8_quantize_rows(x), m.fp8_quantize_rows(x[-7:])
    assert torch.equal(q.codes[-7:], q7.codes) and torch.equal(q.scales[:, -7:], q7.scales)
    assert torch.equal(q.codes[0], m.fp8_quantize_rows(x[:1]).codes[0])
    # the codes as operand: 2.2 GB of x; then 2.3e9 results
    w = m.fp8_quantize_blocks(torch.randn((1, 40, K), generator=g, device=gpu))
    y = m.fp8_block_gemm(q, w, out_dtype=torch.float32)
    y7 = m.fp8_block_gemm(q7, w, out_dtype=torch.float32)
    x64, w64 = ref.dequant_rows(q7), ref.dequant_blocks(w)[0]
    r, mag = ref.gemm_f64(x64, w64)
    for got in (y[-7:], y7):
        ref.assert_close(got, r, ref.gemm_tol(r, mag, K, False))
    del q, x, y
    M, N, K = 140000, 16400, 128
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device=gpu).to(torch.float8_e4m3fn)
    xc, wc = ints(M, K), ints(1, N, K)
    ones = lambda *s: torch.ones(s, device=gpu)
    y = m.fp8_block_gemm(m.Fp8Rows(xc.view(torch.uint8), ones(1, M)),
                         m.Fp8Blocks(wc.view(torch.uint8), ones(1, ref.nblk(N), 1)))
    for rows in (slice(0, 5), slice(M // 2, M // 2 + 5), slice(M - 5, M)):
        want = torch.mm(xc[rows].double(), wc[0].double().t().contiguous())
        assert torch.equal(y[rows], want.to(torch.bfloat16))
    # a weight of 4.9 GB
    G, N, K = 300, 4000, 2048
    wb = torch.empty((G, N, K), dtype=torch.bfloat16, device=gpu)
    wb[:-1].fill_(1.0)
    wb[-1] = torch.randn((N, K), generator=g, device=gpu).to(torch.bfloat16)
    q, q1 = m.fp8_quantize_blocks(wb), m.fp8_quantize_blocks(wb[-1])
    assert torch.equal(q.codes[-1:], q1.codes) and torch.equal(q.scales[-1:], q1.scales)
