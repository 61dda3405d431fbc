"""Cases of the FP8 block-scaled and expert-grouped operators: what is timed, the
operators' plain forms in elementary torch operations, and their values in 64 bits.

Formats. A block-scaled FP8 matrix of rows is E4M3 codes [M][K] with an FP32 scale
per 128 consecutive elements of a row, scales [ceil(K/128)][M]; a block-scaled FP8
weight is codes [G][N][K] with an FP32 scale per 128 x 128 block, scales
[G][ceil(N/128)][ceil(K/128)]. Quantising takes a = max(amax, 2^-117) of each block:
scale = a / 448, code = E4M3 nearest to v * (448 / a).

Operators (field "op"):
  rows     quantise rows (swiglu: of silu(first half) * second half)
  blocks   quantise weights
  gemm     block-scaled FP8 product of rows and one weight
  grouped  products grouped by expert: y[p] = W_expert(p) x[p / k] (x: the token
           rows) or W_expert(p) x[p] (x: one row per (row, slot) pair)
  combine  out[m] = sum_j w[m][j] y[m k + j] + shared[m] + residual[m]
"""
import math

import torch

own = False

BLOCK = 128
AMAX_MIN = 2.0 ** -117


def listed():
    return [
        # one speculative-decode step's rows of the 2048-wide model: launch latency
        dict(name="rows decode M=4", op="rows", M=4, K=2048, swiglu=False, type="bf16"),
        # a 1024-token chunk's gate_up outputs (8 experts a token) on their way into down
        dict(name="rows swiglu M=8192", op="rows", M=8192, K=512, swiglu=True, type="bf16"),
        # one output projection 4096 -> 2048 quantised at load time
        dict(name="blocks o_proj", op="blocks", G=1, N=2048, K=4096, type="bf16"),
        # the gate_up matrices of a layer's 256 experts quantised at load time
        dict(name="blocks 256 experts", op="blocks", G=256, N=1024, K=2048, type="bf16"),
        # plain decode of one token: query/key/value projection 2048 -> 5120
        dict(name="gemm qkv M=1", op="gemm", M=1, N=5120, K=2048, out="bf16"),
        # odd sizes: rows of a ragged batch, a last block of 16 columns, FP32 logits
        dict(name="gemm ragged M=333", op="gemm", M=333, N=1000, K=1936, out="f32"),
        # prefill of 8192 tokens: the same projection, bound by arithmetic
        dict(name="gemm qkv M=8192", op="gemm", M=8192, N=5120, K=2048, out="bf16"),
        # one token and three drafted ones through gate_up: few rows, many experts
        dict(name="grouped gate_up M=4", op="grouped", type="fp8", M=4, E=256, k=8, N=1024, K=2048,
             x="tokens", routing="uniform", out="bf16"),
        # BF16 down projections of a 1024-token chunk under skewed routing: ragged groups
        dict(name="grouped down M=1024 bf16", op="grouped", type="bf16", M=1024, E=256, k=8, N=2048,
             K=512, x="pairs", routing="zipf", out="bf16"),
        # prefill of 8192 tokens through gate_up: 256 rows an expert, bound by arithmetic
        dict(name="grouped gate_up M=8192", op="grouped", type="fp8", M=8192, E=256, k=8, N=1024,
             K=2048, x="tokens", routing="uniform", out="bf16"),
        # the M = 16 step's combine with its shared expert and residual
        dict(name="combine M=16", op="combine", M=16, k=8, H=2048, type="f32", shared=True,
             residual=True),
        # a prefill chunk's combine
        dict(name="combine M=4096", op="combine", M=4096, k=8, H=2048, type="bf16", shared=False,
             residual=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rows", "blocks", "gemm", "gemm", "grouped", "grouped", "combine"])
    if op == "rows":
        return dict(op=op, M=_log_int(rng, 1, 16384), K=16 * _log_int(rng, 1, 256),
                    swiglu=rng.random() < 0.5, type=rng.choice(["bf16", "f32"]))
    if op == "blocks":
        return dict(op=op, G=_log_int(rng, 1, 64), N=_log_int(rng, 1, 4096),
                    K=16 * _log_int(rng, 1, 128), type=rng.choice(["bf16", "f32"]))
    if op == "gemm":
        return dict(op=op, M=_log_int(rng, 1, 8192), N=_log_int(rng, 1, 5120),
                    K=16 * _log_int(rng, 1, 128), out=rng.choice(["bf16", "f32"]))
    if op == "grouped":
        routing = rng.choice(["uniform", "zipf"])
        E = _log_int(rng, 8, 256)
        return dict(op=op, type=rng.choice(["fp8", "bf16"]),
                    M=_log_int(rng, 1, 4096 if routing == "uniform" else 1024), E=E,
                    k=rng.randint(1, 8), N=_log_int(rng, 16, 2048), K=16 * _log_int(rng, 2, 64),
                    x=rng.choice(["tokens", "pairs"]), routing=routing,
                    out=rng.choice(["bf16", "f32"]))
    return dict(op=op, M=_log_int(rng, 1, 4096), k=rng.randint(1, 8), H=_log_int(rng, 16, 4096),
                type=rng.choice(["bf16", "f32"]), shared=rng.random() < 0.5,
                residual=rng.random() < 0.5)


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _blocks(n):
    return -(-n // BLOCK)


# ---- plain forms, FP32 ---------------------------------------------------------------

def _pad_blocks(v, *dims):
    """v with each of `dims` split into (blocks, 128), zeros past the end."""
    for d in sorted(dims, reverse=True):
        n = v.shape[d]
        extra = _blocks(n) * BLOCK - n
        if extra:
            shape = list(v.shape)
            shape[d] = extra
            v = torch.cat([v, v.new_zeros(shape)], d)
        v = v.unflatten(d, (_blocks(n), BLOCK))
    return v


def _scale_of(amax):
    """amax of a block -> (scale, factor onto codes), each one FP32 division."""
    a = amax.clamp_min(AMAX_MIN)
    c = torch.full_like(a, 448.0)
    return a / c, c / a


def _spread(s, n, dim):
    return s.repeat_interleave(BLOCK, dim).narrow(dim, 0, n)


def _quantize_rows(x, swiglu):
    v = x.float()
    if swiglu:
        a, b = v.chunk(2, 1)
        v = a / (1.0 + torch.exp(-a)) * b
    K = v.shape[1]
    s, f = _scale_of(_pad_blocks(v, 1).abs().amax(2))
    codes = (v * _spread(f, K, 1)).to(torch.float8_e4m3fn)
    return codes, s.t().contiguous()


def _quantize_blocks(x):
    v = x.float()
    G, N, K = v.shape
    s, f = _scale_of(_pad_blocks(v, 1, 2).abs().amax((2, 4)))
    codes = (v * _spread(_spread(f, N, 1), K, 2)).to(torch.float8_e4m3fn)
    return codes, s


def _rows_f32(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * _spread(scales.t(), codes.shape[1], 1)


def _weight_f32(codes, scales):
    return codes.view(torch.float8_e4m3fn).float() * _spread(
        _spread(scales, codes.shape[1], 1), codes.shape[2], 2)


def _grouped(s):
    x = _rows_f32(*s["x"]) if s["type"] == "fp8" else s["x"][0].float()
    ids, pairs, offsets = s["ids"], s["pairs"], s["offsets"]
    R, E, div = pairs.numel(), offsets.numel() - 1, s["div"]
    if R <= 64:  # few rows: each pair's own matrix
        e = ids.reshape(-1).long()
        w = _weight_f32(s["w"][0][e], s["w"][1][e]) if s["type"] == "fp8" else s["w"][0][e].float()
        rows = torch.arange(R, device=x.device) // div
        return torch.bmm(w, x[rows].unsqueeze(2)).squeeze(2).to(s["out"])
    # many rows: every expert's rows padded to the largest group
    w = _weight_f32(*s["w"]) if s["type"] == "fp8" else s["w"][0].float()
    e = ids.reshape(-1)[pairs.long()].long()
    at = torch.arange(R, device=x.device) - offsets.long()[e]
    xp = x.new_zeros((E, s["most"], x.shape[1]))
    xp[e, at] = x[pairs.long() // div]
    yp = torch.bmm(w, xp.transpose(1, 2).contiguous())
    y = torch.empty((R, w.shape[1]), dtype=torch.float32, device=x.device)
    y[pairs.long()] = yp.transpose(1, 2)[e, at]
    return y.to(s["out"])


def _combine(s):
    M, k = s["w"].shape
    v = (s["y"].float().view(M, k, -1) * s["w"].unsqueeze(2)).sum(1)
    if s["shared"] is not None:
        v = v + s["shared"].float()
    if s["residual"] is not None:
        v = v + s["residual"].float()
    return v.to(torch.bfloat16)


def _values(codes):
    return codes if codes.dtype == torch.float8_e4m3fn else codes.view(torch.float8_e4m3fn)


# ---- inputs ---------------------------------------------------------------------------

def _routing(M, E, k, how, g, dev):
    """Top-k ids and softmax weights of random logits, and the pairs grouped by expert."""
    k = min(k, E)
    logits = torch.randn((M, E), generator=g, device=dev)
    if how == "zipf":  # expert popularity ~ rank^-1.1 through Gumbel noise
        rank = torch.randperm(E, generator=g, device=dev).float() + 1
        u = torch.rand((M, E), generator=g, device=dev).clamp(1e-7, 1 - 1e-7)
        logits = -1.1 * rank.log() - torch.log(-torch.log(u))
    top, ids = logits.topk(k, 1)
    counts = torch.bincount(ids.reshape(-1), minlength=E)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    pairs = torch.sort(ids.reshape(-1), stable=True).indices
    used = counts > 0
    n = used.sum().reshape(1)
    order = torch.sort((~used).to(torch.int32), stable=True).indices
    slot = torch.arange(E, device=dev)
    active = torch.where(slot < n, order, torch.full_like(order, -1))
    slot1 = torch.arange(E + 1, device=dev)
    act_off = torch.where(slot1 < n, offsets[torch.cat([order, order[:1]])],
                          torch.full_like(slot1, M * k))
    i32 = lambda t: t.to(torch.int32)
    return dict(ids=i32(ids), rw=torch.softmax(top, 1), counts=i32(counts), offsets=i32(offsets),
                pairs=i32(pairs), active=i32(active), active_offsets=i32(act_off),
                n_active=i32(n), most=int(counts.max()))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    randn = lambda *shape, type="bf16", std=1.0: torch.randn(
        shape, generator=g, device=dev, dtype=_TYPES[type]) * std
    op = case["op"]
    s = {"op": op}
    if op == "rows":
        # activations of unit scale with a few large channels
        cols = case["K"] * (2 if case["swiglu"] else 1)
        x = randn(case["M"], cols, type=case["type"])
        x[:, ::61] *= 12
        s.update(x=x, swiglu=case["swiglu"])
    elif op == "blocks":
        s.update(x=randn(case["G"], case["N"], case["K"], type=case["type"], std=0.02))
    elif op == "gemm":
        s.update(x=_u8(_quantize_rows(randn(case["M"], case["K"]), False)),
                 w=_u8(_quantize_blocks(randn(1, case["N"], case["K"], std=case["K"] ** -0.5))),
                 out=_TYPES[case["out"]])
    elif op == "grouped":
        M, E, K = case["M"], case["E"], case["K"]
        r = _routing(M, E, case["k"], case["routing"], g, dev)
        k = r["ids"].shape[1]
        x = randn(M if case["x"] == "tokens" else M * k, K)
        w = randn(E, case["N"], K, std=K ** -0.5)
        s.update(r, type=case["type"], div=k if case["x"] == "tokens" else 1,
                 out=_TYPES[case["out"]])
        if case["type"] == "fp8":
            s.update(x=_u8(_quantize_rows(x, False)), w=_u8(_quantize_blocks(w)))
        else:
            s.update(x=(x,), w=(w,))
    else:
        M, k, H = case["M"], case["k"], case["H"]
        s.update(y=randn(M * k, H, type=case["type"]),
                 w=torch.softmax(torch.randn((M, k), generator=g, device=dev), 1),
                 shared=randn(M, H, type=case["type"]) if case["shared"] else None,
                 residual=randn(M, H) if case["residual"] else None)
    return s


def _u8(q):
    return q[0].view(torch.uint8), q[1]


# ---- one pass -------------------------------------------------------------------------

def run(s):
    op = s["op"]
    if own:
        import nvfp4_moe_skinny_amd as m
        if op == "rows":
            q = m.fp8_quantize_rows(s["x"], swiglu=s["swiglu"])
            return {"codes": _values(q.codes), "scales": q.scales}
        if op == "blocks":
            q = m.fp8_quantize_blocks(s["x"])
            return {"codes": _values(q.codes), "scales": q.scales}
        if op == "gemm":
            return m.fp8_block_gemm(m.Fp8Rows(*s["x"]), m.Fp8Blocks(*s["w"]), out_dtype=s["out"])
        if op == "grouped":
            r = m.Routing(s["ids"], s["rw"], s["counts"], s["offsets"], s["pairs"], s["active"],
                          s["active_offsets"], s["n_active"])
            if s["type"] == "fp8":
                return m.moe_grouped_gemm(m.Fp8Rows(*s["x"]), r, m.Fp8Blocks(*s["w"]),
                                          out_dtype=s["out"])
            return m.moe_grouped_gemm(s["x"][0], r, s["w"][0], out_dtype=s["out"])
        return m.moe_combine(s["y"], s["w"], shared=s["shared"], residual=s["residual"])
    if op == "rows":
        codes, scales = _quantize_rows(s["x"], s["swiglu"])
        return {"codes": _values(codes), "scales": scales}
    if op == "blocks":
        codes, scales = _quantize_blocks(s["x"])
        return {"codes": _values(codes), "scales": scales}
    if op == "gemm":
        return torch.mm(_rows_f32(*s["x"]), _weight_f32(*s["w"])[0].t()).to(s["out"])
    if op == "grouped":
        return _grouped(s)
    return _combine(s)


# ---- work -----------------------------------------------------------------------------

def _touched(case):
    """Expected number of experts with at least one row."""
    M, E, k = case["M"], case["E"], min(case["k"], case["E"])
    if case["routing"] == "uniform":
        return E * (1 - (1 - k / E) ** M)
    p = [(r + 1) ** -1.1 for r in range(E)]
    t = sum(p)
    return sum(1 - (1 - min(1.0, k * v / t)) ** M for v in p)


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "rows":
        M, K = case["M"], case["K"]
        n = 2 if case["swiglu"] else 1
        return {"bytes": M * K * (n * size[case["type"]] + 1) + 4 * M * _blocks(K),
                "flops": M * K * (8 if case["swiglu"] else 3)}
    if op == "blocks":
        G, N, K = case["G"], case["N"], case["K"]
        return {"bytes": G * N * K * (size[case["type"]] + 1) + 4 * G * _blocks(N) * _blocks(K),
                "flops": 3 * G * N * K}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K + 4 * M * _blocks(K) + N * K + 4 * _blocks(N) * _blocks(K)
                + M * N * size[case["out"]], "flops": 2 * M * N * K}
    if op == "grouped":
        M, N, K, k = case["M"], case["N"], case["K"], min(case["k"], case["E"])
        R = M * k
        el = 1 if case["type"] == "fp8" else 2
        rows = M if case["x"] == "tokens" else R
        b = _touched(case) * N * K * el + rows * K * el + R * N * size[case["out"]] + 4 * R
        if case["type"] == "fp8":
            b += 4 * rows * _blocks(K) + 4 * _touched(case) * _blocks(N) * _blocks(K)
        return {"bytes": b, "flops": 2 * R * N * K}
    M, k, H = case["M"], case["k"], case["H"]
    el = size[case["type"]]
    b = M * k * H * el + 4 * M * k + 2 * M * H
    b += (M * H * el if case["shared"] else 0) + (2 * M * H if case["residual"] else 0)
    return {"bytes": b, "flops": 2 * M * k * H}


# ---- 64 bits --------------------------------------------------------------------------

def _e4m3_f64(v):
    """E4M3 nearest to each value of v (|v| <= 464), ties to even: steps of
    2^(e-3) in [2^e, 2^(e+1)), of 2^-9 below 2^-6, at most 448."""
    e = torch.frexp(v.abs())[1].to(torch.float64) - 1
    step = torch.exp2(e.clamp_min(-6.0) - 3)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _block_index(n, dev):
    return torch.arange(n, device=dev) // BLOCK


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("rows", "blocks"):
        v = s["x"].double()
        dev = v.device
        if op == "rows":
            if s["swiglu"]:
                h = v.shape[1] // 2
                v = v[:, :h] * torch.sigmoid(v[:, :h]) * v[:, h:]
            M, K = v.shape
            kb = _block_index(K, dev)
            a = torch.zeros((M, _blocks(K)), dtype=torch.float64, device=dev)
            a.scatter_reduce_(1, kb.expand(M, K), v.abs(), "amax")
            a = a.clamp_min(AMAX_MIN)
            return {"codes": _e4m3_f64(v * 448 / a[:, kb]), "scales": (a / 448).t().contiguous()}
        G, N, K = v.shape
        nb, kb = _block_index(N, dev), _block_index(K, dev)
        a = torch.zeros((G, N, _blocks(K)), dtype=torch.float64, device=dev)
        a.scatter_reduce_(2, kb.expand(G, N, K), v.abs(), "amax")
        b = torch.zeros((G, _blocks(N), _blocks(K)), dtype=torch.float64, device=dev)
        b.scatter_reduce_(1, nb.view(1, N, 1).expand(G, N, _blocks(K)), a, "amax")
        b = b.clamp_min(AMAX_MIN)
        return {"codes": _e4m3_f64(v.mul_(448 / b[:, nb][:, :, kb])), "scales": b / 448}
    if op == "combine":
        M, k = s["w"].shape
        y = torch.bmm(s["w"].double().unsqueeze(1), s["y"].double().view(M, k, -1)).squeeze(1)
        for t in (s["shared"], s["residual"]):
            if t is not None:
                y = y + t.double()
        return y
    fp8 = op == "gemm" or s["type"] == "fp8"

    def wide(codes, row_scale):
        if not fp8:
            return codes.double()
        kb = _block_index(codes.shape[-1], codes.device)
        return codes.view(torch.float8_e4m3fn).double() * row_scale.double()[..., kb]

    x = wide(s["x"][0], s["x"][1].t() if fp8 else None)

    def weight(e):
        w = s["w"][0][e]
        nb = _block_index(w.shape[0], w.device)
        return wide(w, s["w"][1][e][nb] if fp8 else None)

    if op == "gemm":
        return x @ weight(0).t()
    pairs = s["pairs"].long()
    y = torch.empty((pairs.numel(), s["w"][0].shape[1]), dtype=torch.float64, device=x.device)
    off = s["offsets"].tolist()
    for e in range(len(off) - 1):
        p = pairs[off[e]:off[e + 1]]
        if p.numel():
            y[p] = x[p // s["div"]] @ weight(e).t()
    return y
