"""Products grouped by expert and the combine on the GPU against float64, the
chain they form, and the chain captured in a HIP graph."""
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def m(gpu):
    import nvfp4_moe_skinny_amd as m
    return m


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def _ids(seed, M, E, k, how):
    """Distinct experts per row: spread evenly, or crowded on a few."""
    g = torch.Generator().manual_seed(seed)
    score = torch.rand((M, E), generator=g)
    if how == "skewed":
        score = score + 3.0 / (1 + torch.arange(E)) ** 0.5
    elif how == "one":  # every row chooses the same k experts
        score = torch.rand((1, E), generator=g).expand(M, E)
    return score.topk(k, 1).indices


def _operands(m, gpu, seed, typ, rows, E, N, K):
    """(x, w) for the call and their float64 values."""
    x, w = _randn(seed, rows, K), _randn(seed + 1, E, N, K) * K ** -0.5
    if typ == "fp8":
        xq, wq = m.fp8_quantize_rows(x.to(gpu)), m.fp8_quantize_blocks(w.to(gpu))
        return xq, wq, ref.dequant_rows(xq), ref.dequant_blocks(wq)
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    return x.to(gpu), w.to(gpu), x.double(), w.double()


def _check(m, gpu, typ, M, E, k, N, K, how, per_pair, out, seed=0):
    ids = _ids(seed + M + E, M, E, k, how)
    r = ref.routing_of(m, ids, E, gpu)
    x, w, x64, w64 = _operands(m, gpu, seed + N + K, typ, M * k if per_pair else M, E, N, K)
    y = m.moe_grouped_gemm(x, r, w, out_dtype=TYPES[out])
    torch.cuda.synchronize()
    cut_on = gpu if (typ, out) == ("fp8", "bf16") else None
    want, mag, cut = ref.grouped_f64(x64, w64, ids, per_pair, cut_on)
    ref.assert_close(y, want, ref.gemm_tol(want, mag, K, out == "bf16", cut),
                     (typ, M, E, k, N, K, how))
    assert torch.equal(y, m.moe_grouped_gemm(x, r, w, out_dtype=TYPES[out]))


@pytest.mark.parametrize("typ,out", [("fp8", "bf16"), ("fp8", "f32"), ("bf16", "bf16"),
                                     ("bf16", "f32")])
@pytest.mark.parametrize("M,E,k,N,K,how,per_pair", [
    (1, 1, 1, 1, 16, "even", False), (1, 256, 8, 64, 2048, "even", False),
    (4, 64, 8, 100, 512, "even", True), (16, 64, 8, 48, 272, "skewed", False),
    (40, 16, 3, 130, 144, "even", False), (100, 8, 2, 257, 400, "one", True),
    (256, 32, 8, 128, 256, "skewed", False), (300, 5, 5, 96, 640, "even", False),
    (64, 300, 4, 33, 128, "even", True), (1, 600, 8, 20, 64, "even", False),
    (513, 3, 1, 320, 160, "skewed", True), (257, 1, 1, 200, 1024, "even", False),
    (700, 4, 2, 256, 512, "one", False)])
def test_grouped(m, gpu, typ, out, M, E, k, N, K, how, per_pair):
    _check(m, gpu, typ, M, E, k, N, K, how, per_pair, out)


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
@pytest.mark.parametrize("M,N,K", [(24, 40, 144), (900, 260, 272)])
def test_grouped_integers_exact(m, gpu, typ, M, N, K):
    """Small integers and power-of-two scales: every FP32 sum is exact."""
    E, k = 6, 2
    g = torch.Generator().manual_seed(M)
    ids = _ids(M, M, E, k, "skewed")
    xi = torch.randint(-4, 5, (M, K), generator=g).float()
    wi = torch.randint(-4, 5, (E, N, K), generator=g).float()
    r = ref.routing_of(m, ids, E, gpu)
    if typ == "fp8":
        u8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).to(gpu)
        p2 = lambda *s: (2.0 ** torch.randint(0, 3, s, generator=g).float()).to(gpu)
        x = m.Fp8Rows(u8(xi), p2(ref.nblk(K), M))
        w = m.Fp8Blocks(u8(wi), p2(E, ref.nblk(N), ref.nblk(K)))
        x64, w64 = ref.dequant_rows(x), ref.dequant_blocks(w)
    else:
        x, w = xi.to(torch.bfloat16).to(gpu), wi.to(torch.bfloat16).to(gpu)
        x64, w64 = xi.double(), wi.double()
    y = m.moe_grouped_gemm(x, r, w, out_dtype=torch.float32)
    want = ref.grouped_f64(x64, w64, ids, False)[0]
    assert torch.equal(y.cpu().double(), want)
    assert torch.equal(m.moe_grouped_gemm(x, r, w).cpu(), want.to(torch.bfloat16))


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
@pytest.mark.parametrize("K", [16, 144, 272, 400])
@pytest.mark.parametrize("M,E,k,N,how", [
    (600, 300, 4, 260, "even"), (1500, 200, 4, 260, "skewed"), (2000, 40, 4, 520, "even"),
    (4000, 300, 4, 260, "skewed"), (4100, 8, 2, 1300, "even"), (3000, 4, 2, 2100, "skewed")])
def test_grouped_more_tiles_than_blocks(m, gpu, typ, K, M, E, k, N, how):
    """Blocks that take several tiles in turn, of every tile shape, with one k
    step and more, up to 300 slots (a wave holds 256 at a time): exact integers."""
    g = torch.Generator(device=gpu).manual_seed(M + N + K)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device=gpu).float()
    p2 = lambda *s: 2.0 ** torch.randint(0, 3, s, generator=g, device=gpu).float()
    ids = _ids(M, M, E, k, how)
    r = ref.routing_of(m, ids, E, gpu)
    if typ == "fp8":
        u8 = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8)
        x = m.Fp8Rows(u8(ints(M, K)), p2(ref.nblk(K), M))
        w = m.Fp8Blocks(u8(ints(E, N, K)), p2(E, ref.nblk(N), ref.nblk(K)))
        x64, w64 = ref.dequant_rows(x).to(gpu), ref.dequant_blocks(w).to(gpu)
    else:
        x, w = ints(M, K).to(torch.bfloat16), ints(E, N, K).to(torch.bfloat16)
        x64, w64 = x.double(), w.double()
    want = torch.empty((M * k, N), dtype=torch.float64, device=gpu)
    flat = ids.reshape(-1).to(gpu)
    for e in range(E):
        p = (flat == e).nonzero().reshape(-1)
        want[p] = torch.mm(x64[p // k], w64[e].t().contiguous())
    assert want.abs().max() < 2 ** 24
    assert torch.equal(m.moe_grouped_gemm(x, r, w, out_dtype=torch.float32).double(), want)
    assert torch.equal(m.moe_grouped_gemm(x, r, w), want.to(torch.bfloat16))


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
@pytest.mark.parametrize("M", [6, 400])
def test_grouped_local_experts_only(m, gpu, typ, M):
    """A rank that passes some experts' slots: other pairs' rows stay as they
    were; a slot of an expert out of range and a pair out of range are skipped."""
    E, k, N, K = 12, 4, 70, 272
    ids = _ids(M, M, E, k, "even")
    r = ref.routing_of(m, ids, E, gpu)
    x, w, x64, w64 = _operands(m, gpu, M, typ, M, E, N, K)
    want, mag, _ = ref.grouped_f64(x64, w64, ids, False)
    tol = ref.gemm_tol(want, mag, K, False)
    active, off = r.active.cpu().tolist(), r.active_offsets.cpu().tolist()
    pairs = r.pairs.cpu().tolist()
    n = int(r.n_active)
    keep = n // 2
    act2 = list(active)
    act2[1] = E        # an expert that does not exist
    pairs2 = list(pairs)
    pairs2[off[0]] = M * k + 3  # a pair that does not exist
    pairs2[off[0] + 1] = -1
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=gpu)
    r2 = m.Routing(r.ids, r.w, r.counts, r.offsets, i32(pairs2), i32(act2), r.active_offsets,
                   i32([keep]))
    done = [pairs[i] for s in range(keep) if s != 1 for i in range(off[s], off[s + 1])
            if i not in (off[0], off[0] + 1)]
    out = torch.full((M * k, N), 5.0, device=gpu)
    y = m.moe_grouped_gemm(x, r2, w, out_dtype=torch.float32, out=out).cpu().double()
    rest = torch.ones(M * k, dtype=torch.bool)
    rest[done] = False
    assert rest.any() and not rest.all()
    assert (y[rest] == 5.0).all()
    ref.assert_close(y[~rest], want[~rest], tol[~rest])
    # nothing active at all
    r2.n_active.zero_()
    out.fill_(5.0)
    assert (m.moe_grouped_gemm(x, r2, w, out_dtype=torch.float32, out=out) == 5.0).all()


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
@pytest.mark.parametrize("M", [2, 60, 3000])
def test_grouped_offsets_out_of_order(m, gpu, typ, M):
    """Offsets and counts outside their range are taken as the nearer end, a slot
    that ends before it starts is empty; rows around y stay as they were."""
    E, k, N, K = 9, 2, 260, 272
    ids = _ids(M, M, E, k, "even")
    r = ref.routing_of(m, ids, E, gpu)
    x, w, x64, w64 = _operands(m, gpu, M, typ, M, E, N, K)
    R, half = M * k, M * k // 2
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=gpu)
    pairs = torch.randperm(R, generator=torch.Generator().manual_seed(M)).int().to(gpu)
    big = 2 ** 31 - 1
    # slot 0: [0, half) of expert 3; 1: empty; 2: [0, 0) after the clamp; 3: empty;
    # 4: [half, R) of expert 5; 5: [R, R); the others end before they start
    off = i32(-7, half, 0, -big, half, big, R + 1, half, 0, -1)
    active = i32(3, 4, 6, 7, 5, 1, 2, 8, 0)
    # slot 3 would be [0, half) as well: an expert that does not exist drops it
    active[3] = -2
    r2 = m.Routing(r.ids, r.w, r.counts, r.offsets, pairs, active, off, i32(big))
    buf = torch.full((R + 2, N + 8), 5.0, device=gpu)
    m.moe_grouped_gemm(x, r2, w, out_dtype=torch.float32, out=buf[1:-1, :N])
    torch.cuda.synchronize()
    y = buf.cpu().double()
    assert (y[0] == 5.0).all() and (y[-1] == 5.0).all() and (y[:, N:] == 5.0).all()
    p = pairs.cpu().long()
    for part, slot, e in ((p[:half], 0, 3), (p[half:], 4, 5)):
        if slot >= min(E, R):  # (four pairs have at most four slots)
            assert (y[1:-1, :N][part] == 5.0).all()
            continue
        want, mag = ref.gemm_f64(x64[part // k], w64[e])
        ref.assert_close(y[1:-1, :N][part], want, ref.gemm_tol(want, mag, K, False))
    r2.n_active.fill_(-big)
    buf.fill_(5.0)
    m.moe_grouped_gemm(x, r2, w, out_dtype=torch.float32, out=buf[1:-1, :N])
    assert (buf == 5.0).all()


@pytest.mark.parametrize("M", [3, 300])
def test_grouped_bf16_infinity_and_nan(m, gpu, M):
    """An infinite or NaN weight reaches its own column of its own expert only;
    the partial last step (16 of 64 columns) adds no NaN."""
    E, k, N, K = 4, 2, 50, 80
    ids = _ids(M, M, E, k, "even")
    r = ref.routing_of(m, ids, E, gpu)
    x, w, x64, w64 = _operands(m, gpu, M, "bf16", M, E, N, K)
    x = x.abs() + 1
    e0 = int(ids[0, 0])
    w[e0, 7, 64] = float("inf")
    w[e0, 9, 0] = float("nan")
    y = m.moe_grouped_gemm(x, r, w, out_dtype=torch.float32).cpu()
    hit = ids.reshape(-1) == e0
    assert (y[hit][:, 7] == float("inf")).all() and torch.isnan(y[hit][:, 9]).all()
    y[:, 7] = 0
    y[:, 9] = 0
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
@pytest.mark.parametrize("M", [5, 260])
def test_grouped_strided_out(m, gpu, typ, M):
    E, k, N, K = 8, 2, 129, 256
    ids = _ids(M, M, E, k, "even")
    r = ref.routing_of(m, ids, E, gpu)
    x, w, _, _ = _operands(m, gpu, M, typ, M, E, N, K)
    base = torch.full((M * k, N + 6), 3.0, dtype=torch.bfloat16, device=gpu)
    y = m.moe_grouped_gemm(x, r, w, out=base[:, 3:3 + N])
    plain = m.moe_grouped_gemm(x, r, w)
    assert torch.equal(y, plain)
    assert (base[:, :3] == 3).all() and (base[:, 3 + N:] == 3).all()


def test_no_rows(m, gpu):
    z = lambda *s, t=torch.bfloat16: torch.zeros(s, dtype=t, device=gpu)
    ids = torch.zeros((0, 2), dtype=torch.int64)
    r = ref.routing_of(m, ids, 4, gpu)
    assert m.moe_grouped_gemm(z(0, 32), r, z(4, 8, 32)).shape == (0, 8)
    assert m.moe_combine(z(0, 8), z(0, 2, t=torch.float32)).shape == (0, 8)
    torch.cuda.synchronize()


# ---- combine --------------------------------------------------------------------------

def _combine_tol(y, w, shared, residual, H):
    """k multiply-adds and two additions, half a step each, then BF16."""
    M, k = w.shape
    terms = w.double().unsqueeze(2) * y.double().view(M, k, H)
    val, mag = terms.sum(1), terms.abs().sum(1)
    for t in (shared, residual):
        if t is not None:
            val, mag = val + t.double(), mag + t.double().abs()
    t = (k + 2) * ref.U * mag
    return val, t + ref.BF16_HALF_STEP * (val.abs() + t)


@pytest.mark.parametrize("typ", ["bf16", "f32"])
@pytest.mark.parametrize("shared,residual", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("M,k,H", [(1, 1, 1), (1, 8, 2048), (16, 8, 2048), (7, 3, 100),
                                   (33, 5, 257), (1000, 2, 66), (300, 8, 512)])
def test_combine(m, gpu, M, k, H, typ, shared, residual):
    y = _randn(M + H, M * k, H).to(TYPES[typ])
    w = torch.softmax(_randn(k, M, k), 1)
    s = _randn(1, M, H).to(TYPES[typ]) if shared else None
    r = _randn(2, M, H).to(torch.bfloat16) if residual else None
    dev = lambda t: None if t is None else t.to(gpu)
    out = m.moe_combine(dev(y), dev(w), shared=dev(s), residual=dev(r))
    val, tol = _combine_tol(y, w, s, r, H)
    ref.assert_close(out, val, tol)


def test_combine_in_place_unaligned_and_weight_zero(m, gpu):
    M, k, H = 20, 4, 64
    y = _randn(1, M * k, H).to(gpu)
    w = torch.softmax(_randn(2, M, k), 1).to(gpu)
    res = _randn(3, M, H).to(torch.bfloat16).to(gpu)
    want = m.moe_combine(y, w, residual=res)
    inout = res.clone()
    m.moe_combine(y, w, residual=inout, out=inout)
    assert torch.equal(inout, want)
    # rows that start two bytes off: the scalar form, same order, same bits
    buf = torch.zeros(M * H + 1, dtype=torch.bfloat16, device=gpu)
    off = buf[1:].view(M, H)
    off.copy_(res)
    assert torch.equal(m.moe_combine(y, w, residual=off), want)
    # weight 0: NaN or infinity in y does not matter
    w2 = w.clone()
    w2[:, 1] = 0
    w2[5] = 0
    clean, dirty = y.clone().view(M, k, H), y.clone().view(M, k, H)
    clean[:, 1] = 0
    clean[5] = 0
    dirty[:, 1] = float("nan")
    dirty[5] = float("inf")
    a = m.moe_combine(dirty.view(M * k, H), w2, residual=res)
    assert torch.equal(a, m.moe_combine(clean.view(M * k, H), w2, residual=res))
    assert torch.equal(a[5], res[5])


# ---- the chain ------------------------------------------------------------------------

def _chain_inputs(m, gpu, seed, M, E, k, H, I):
    bf = lambda *s, std=1.0: (_randn(seed + sum(s), *s) * std).to(torch.bfloat16).to(gpu)
    return dict(x=bf(M, H), logits=_randn(seed, M, E).to(gpu),
                gu=m.fp8_quantize_blocks(bf(E, 2 * I, H, std=H ** -0.5)),
                dn=m.fp8_quantize_blocks(bf(E, H, I, std=I ** -0.5)),
                sgu=m.fp8_quantize_blocks(bf(1, 2 * I, H, std=H ** -0.5)),
                sdn=m.fp8_quantize_blocks(bf(1, H, I, std=I ** -0.5)))


def _chain(m, d, k):
    """One MoE block on FP8 experts with a shared expert and a residual."""
    r = m.moe_route_topk(d["logits"], k)
    xq = m.fp8_quantize_rows(d["x"])
    u = m.moe_grouped_gemm(xq, r, d["gu"], out_dtype=torch.float32)
    h = m.fp8_quantize_rows(u, swiglu=True)
    y = m.moe_grouped_gemm(h, r, d["dn"], out_dtype=torch.float32)
    su = m.fp8_block_gemm(xq, d["sgu"], out_dtype=torch.float32)
    sh = m.fp8_quantize_rows(su, swiglu=True)
    sy = m.fp8_block_gemm(sh, d["sdn"], out_dtype=torch.float32)
    out = m.moe_combine(y, r.w, shared=sy, residual=d["x"])
    return dict(r=r, xq=xq, u=u, h=h, y=y, su=su, sh=sh, sy=sy, out=out)


@pytest.mark.parametrize("M,E,k,H,I", [(1, 256, 8, 2048, 512), (4, 64, 8, 512, 144),
                                       (64, 16, 4, 272, 96), (900, 8, 2, 256, 128)])
def test_chain(m, gpu, M, E, k, H, I):
    """Every step of the block against float64 on that step's own inputs."""
    d = _chain_inputs(m, gpu, 77, M, E, k, H, I)
    c = _chain(m, d, k)
    torch.cuda.synchronize()
    ids = c["r"].ids.cpu().long()
    f = lambda q: ref.dequant_rows(q)
    for x, w, y, K, pp in ((c["xq"], d["gu"], c["u"], H, False),
                           (c["h"], d["dn"], c["y"], I, True)):
        want, mag, _ = ref.grouped_f64(f(x), ref.dequant_blocks(w), ids, pp)
        ref.assert_close(y, want, ref.gemm_tol(want, mag, K, False))
    for x, w, y, K in ((c["xq"], d["sgu"], c["su"], H), (c["sh"], d["sdn"], c["sy"], I)):
        want, mag = ref.gemm_f64(f(x), ref.dequant_blocks(w)[0])
        ref.assert_close(y, want, ref.gemm_tol(want, mag, K, False))
    codes, scales = ref.quantize_f32(d["x"].cpu().float(), (1,))
    assert torch.equal(c["xq"].codes.cpu(), codes)
    val, tol = _combine_tol(c["y"].cpu(), c["r"].w.cpu(), c["sy"].cpu(), d["x"].cpu(), H)
    ref.assert_close(c["out"], val, tol)
    # the whole block against float64 weights and rows, no step rounded but the
    # codes: quantising x and h moves each by at most 2^-4 of the value
    u64, _, _ = ref.grouped_f64(d["x"].cpu().double(), ref.dequant_blocks(d["gu"]), ids, False)
    rel = (c["u"].cpu().double() - u64).norm() / u64.norm()
    assert rel <= 2.0 ** -4


def test_chain_in_a_graph(m, gpu):
    """Two chains captured one after the other share one memory pool; every
    replay, with eager work between, gives the eager results of the inputs then
    in place."""
    sizes = dict(M=24, E=16, k=4, H=512, I=128)
    d = _chain_inputs(m, gpu, 5, **sizes)
    sets = [_chain_inputs(m, gpu, 100 + i, **sizes) for i in range(3)]
    eager = [_chain(m, dict(d, x=s["x"], logits=s["logits"]), 4)["out"].clone() for s in sets]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        _chain(m, d, 4)
    st.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
    with torch.cuda.stream(st):
        for g in graphs:
            with torch.cuda.graph(g, stream=st):
                outs.append(_chain(m, d, 4)["out"])
    torch.cuda.synchronize()
    for rep in range(4):
        s = sets[rep % 3]
        d["x"].copy_(s["x"])
        d["logits"].copy_(s["logits"])
        for g, o in zip(graphs, outs):
            o.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(o, eager[rep % 3]), rep
        assert torch.equal(_chain(m, d, 4)["out"], eager[rep % 3])


def test_two_streams_at_once(m, gpu):
    """The calls keep no state: the same chain on two streams at once."""
    sizes = dict(M=40, E=8, k=2, H=384, I=128)
    d = [_chain_inputs(m, gpu, s, **sizes) for s in (1, 2)]
    want = [_chain(m, v, 2)["out"].clone() for v in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_chain(m, d[i], 2)["out"])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
@pytest.mark.parametrize("M", [2, 400])
def test_offsets_past_32_bits(m, gpu, typ, M):
    """Experts whose weights lie past 2^32 bytes, and pairs whose results do."""
    E, k, N, K = 1000, 4, 4608, 1024 if typ == "fp8" else 512
    g = torch.Generator(device=gpu).manual_seed(M)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device=gpu)
    if typ == "fp8":
        codes = lambda *s: ints(*s).to(torch.float8_e4m3fn).view(torch.uint8)
        w = m.Fp8Blocks(codes(1, N, K).repeat(E, 1, 1),
                        torch.ones((E, N // 128, K // 128), device=gpu))
        w.scales *= 2.0 ** (torch.arange(E, device=gpu) % 5).view(E, 1, 1)
        x = m.Fp8Rows(codes(M, K), torch.ones((K // 128, M), device=gpu))
        w64 = lambda e: ref.e4m3_values(w.codes[e]).to(gpu) * 2.0 ** (e % 5)
        x64 = ref.e4m3_values(x.codes).to(gpu)
        assert w.codes.numel() > 2 ** 32
    else:
        w = ints(1, N, K).to(torch.bfloat16).repeat(E, 1, 1)
        w *= (2.0 ** (torch.arange(E, device=gpu) % 5)).to(torch.bfloat16).view(E, 1, 1)
        x = ints(M, K).to(torch.bfloat16)
        w64, x64 = (lambda e: w[e].double()), x.double()
        assert w.numel() * 2 > 2 ** 32
    ids = E - 1 - _ids(M, M, 40, k, "even")
    r = ref.routing_of(m, ids, E, gpu)
    y = torch.zeros((M * k, 1500000 if M == 400 else N), dtype=torch.bfloat16, device=gpu)[:, :N]
    m.moe_grouped_gemm(x, r, w, out=y)
    flat = ids.reshape(-1).to(gpu)
    for e in sorted(set(ids.reshape(-1).tolist())):
        p = (flat == e).nonzero().reshape(-1)
        want = torch.mm(x64[p // k], w64(e).t().contiguous())
        assert torch.equal(y[p], want.to(torch.bfloat16)), e


def test_combine_offsets_past_32_bits(m, gpu):
    M, k, H = 70000, 8, 4096
    g = torch.Generator(device=gpu).manual_seed(1)
    y = torch.empty((M * k, H), dtype=torch.bfloat16, device=gpu).fill_(1.0)
    y[-5 * k:] = torch.randn((5 * k, H), generator=g, device=gpu).to(torch.bfloat16)
    w = torch.rand((M, k), generator=g, device=gpu)
    out = m.moe_combine(y, w)
    assert torch.equal(out[-5:], m.moe_combine(y[-5 * k:], w[-5:].contiguous()))
    assert torch.equal(out[:5], m.moe_combine(y[:5 * k], w[:5].contiguous()))


@pytest.mark.parametrize("typ", ["fp8", "bf16"])
def test_large_products_in_graphs_on_two_streams(m, gpu, typ):
    """Two graphs of products with more tiles than blocks, replayed at once on two
    streams with new routing and rows each time, against eager calls."""
    M, E, k, N, K = 1200, 64, 4, 1100, 400
    x, w, _, _ = _operands(m, gpu, 5, typ, M, E, N, K)
    r = ref.routing_of(m, _ids(0, M, E, k, "even"), E, gpu)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs, outs = [], []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        out = torch.zeros((M * k, N), dtype=torch.bfloat16, device=gpu)
        with torch.cuda.stream(s):
            m.moe_grouped_gemm(x, r, w, out=out)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            m.moe_grouped_gemm(x, r, w, out=out)
        graphs.append(g)
        outs.append(out)
    for rep in range(4):
        how = ("skewed", "even", "one", "skewed")[rep]
        new = ref.routing_of(m, _ids(rep + 1, M, E, k, how), E, gpu)
        for a, b in zip((r.pairs, r.active, r.active_offsets, r.n_active),
                        (new.pairs, new.active, new.active_offsets, new.n_active)):
            a.copy_(b)
        xc = x.codes if typ == "fp8" else x
        xc.copy_(xc.roll(rep + 1, 0))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = m.moe_grouped_gemm(x, r, w)
        for o in outs:
            assert torch.equal(o, want), rep
