// blockgemm.hpp - products of token rows with weights [N][K] on the matrix
// cores, dense or grouped by expert, two operand types:
//   FP8   E4M3 codes with an FP32 scale per 128 columns of a token row
//         (xs[b][row]) and per 128 x 128 block of a weight (ws[n / 128][b]):
//         y = sum_b (xs ws) sum_{k in b} x w
//   BF16  y = sum_k x w
// FP32 sums, y rounded once (BF16) or not at all (FP32).
//
// A k step is 128 bytes of each row: one scale block of FP8, 64 columns of
// BF16. A block's sum starts from zero and its result times xs ws is added to
// the FP32 sum, so no scale is rounded into an operand. Two instructions
// multiply codes:
//   v_mfma_f32_16x16x32_bf16 on codes decoded to BF16 (exact): FP32 sums in
//     the full sense (measured: an addend counts down to 2^-24 of the largest
//     term). Used where the result is FP32, and for few rows, where reading
//     the weights is what takes the time.
//   v_mfma_f32_16x16x128_f8f6f4 on the codes: twice the rate and no decoding,
//     but inside it the products of a group of 16 are cut to multiples of
//     2^-13 of the largest one's power of two before they are added (measured).
//     Products of E4M3 values have 8 bits, so only those below 2^-5 of the
//     largest lose anything: about 10^-4 of a result's size on normal data,
//     a twentieth of the BF16 rounding (2^-9 on average) that follows. Used
//     for many rows when the result is BF16.
// Which k values an instruction's lanes hold is free as long as both operands
// agree: lane l holds row l % 16, bytes 16 g .. 16 g + 15 and 64 + 16 g .. + 15
// of the step (g = l / 16), so four lanes read 64 contiguous bytes of a row.
// Weights are the A operand and token rows the B operand: a lane's results
// are four consecutive n of one token, so xs is one value per lane and y is
// stored four elements at a time.
//
// Grouped: position i of `pairs` belongs to slot s with active_offsets[s] <= i
// < active_offsets[s + 1] and expert active[s]; pair p = pairs[i] reads x row
// p / div and writes y row p. Tiles hold rows of one slot only.
#pragma once

#include <utility>

#include "block8.hpp"
#include "fp8.hpp"

namespace nvfp4moe {

typedef __bf16 bg_bf16x8 __attribute__((ext_vector_type(8)));
typedef float bg_f32x4 __attribute__((ext_vector_type(4)));
typedef int bg_i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStepBytes = 128;

// f(0), ..., f(N - 1) with the index a constant expression: arrays indexed by
// it are registers from the start (indexed by the counter of a loop that is
// unrolled later, the compiler moved one of them to LDS).
template <typename F, int... I>
__device__ __forceinline__ void static_for(F& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F f) {
  static_for(f, std::make_integer_sequence<int, N>{});
}

struct BlockGemmParams {
  const uint8_t* x;   // [Mx][row_bytes]
  const float* xs;    // FP8: [KB][Mx]
  const uint8_t* w;   // [E][N][row_bytes]
  const float* ws;    // FP8: [E][NB][KB]
  void* y;            // [rows][ldy]
  const int32_t* pairs;
  const int32_t* active;
  const int32_t* active_offsets;
  const int32_t* n_active;
  int64_t ldy;
  int64_t Mx;         // rows of x
  int64_t w_mat_bytes;
  int R;              // rows of y (dense: M)
  int div;            // pairs per x row
  int slots;          // min(E, R)
  int E;
  int N;
  int NB, KB;         // scale blocks (BF16: KB = k steps of 64)
  int row_bytes;      // K in bytes, a multiple of 16
};

// The two 16-byte pieces of a row's k step that a lane holds.
struct Frag {
  uint4 lo, hi;
};

__device__ __forceinline__ void keep(uint4& v, uint32_t mask) {
  v.x &= mask;
  v.y &= mask;
  v.z &= mask;
  v.w &= mask;
}

// Zeroes the pieces whose mask is 0 (those past K in the last step).
__device__ __forceinline__ void mask_frag(Frag& f, uint32_t lo, uint32_t hi) {
  keep(f.lo, lo);
  keep(f.hi, hi);
}

enum class Mma {
  kBf16,      // BF16 operands
  kFp8Exact,  // E4M3 codes decoded to BF16
  kFp8,       // E4M3 codes
};

// A lane's part of an operand as the instructions take it.
template <Mma MODE>
struct Operand {  // BF16 operands
  bg_bf16x8 v[2];
  __device__ __forceinline__ void set(const Frag& f) {
    v[0] = __builtin_bit_cast(bg_bf16x8, f.lo);
    v[1] = __builtin_bit_cast(bg_bf16x8, f.hi);
  }
};

__device__ __forceinline__ bg_bf16x8 decode8_e4m3(uint32_t w0, uint32_t w1) {
  const bf16x2 a = fp8_pair_bf16(w0, false), b = fp8_pair_bf16(w0, true);
  const bf16x2 c = fp8_pair_bf16(w1, false), d = fp8_pair_bf16(w1, true);
  return bg_bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

template <>
struct Operand<Mma::kFp8Exact> {
  bg_bf16x8 v[4];
  __device__ __forceinline__ void set(const Frag& f) {
    v[0] = decode8_e4m3(f.lo.x, f.lo.y);
    v[1] = decode8_e4m3(f.lo.z, f.lo.w);
    v[2] = decode8_e4m3(f.hi.x, f.hi.y);
    v[3] = decode8_e4m3(f.hi.z, f.hi.w);
  }
};

template <>
struct Operand<Mma::kFp8> {
  bg_i32x8 v;
  __device__ __forceinline__ void set(const Frag& f) {
    v = bg_i32x8{(int)f.lo.x, (int)f.lo.y, (int)f.lo.z, (int)f.lo.w,
                 (int)f.hi.x, (int)f.hi.y, (int)f.hi.z, (int)f.hi.w};
  }
};

// The sum over one scale block.
template <Mma MODE>
__device__ __forceinline__ bg_f32x4 block_mma(const Operand<MODE>& a, const Operand<MODE>& b) {
  bg_f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (MODE == Mma::kFp8) {
    t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, t, 0, 0, 0, 0, 0,
                                                         0);  // E4M3 x E4M3, no scale operand
  } else {
#pragma unroll
    for (int i = 0; i < (int)(sizeof(a.v) / sizeof(a.v[0])); ++i)
      t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], t, 0, 0, 0);
  }
  return t;
}

__device__ __forceinline__ void scale_into(const bg_f32x4& t, float s, bg_f32x4& acc) {
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r] = fmaf(t[r], s, acc[r]);
}

// acc += (A B) * s over one k step (BF16 operands: s is 1 and not applied).
template <Mma MODE>
__device__ __forceinline__ void step_mma(const Operand<MODE>& a, const Operand<MODE>& b, float s,
                                         bg_f32x4& acc) {
  if constexpr (MODE == Mma::kBf16) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], acc, 0, 0, 0);
  } else {
    scale_into(block_mma<MODE>(a, b), s, acc);
  }
}

// Rows of one tile.
struct RowTile {
  int e;     // expert (0 when dense)
  int row0;  // position in pairs (dense: first row)
  int rows;  // rows of the tile, 0 = nothing to do
};

// Four slots of the lane: rows and tiles of BM rows in each. Every value read
// from memory is put in range, so no contents of the arrays can send a load or
// a store out of x, w or y.
template <int BM>
struct SlotTiles {
  int off[5], e[4], n[4];
  int sum;

  __device__ __forceinline__ void load(const BlockGemmParams& p, int base, int lane) {
    const int na = min(max(p.n_active[0], 0), p.slots);
#pragma unroll
    for (int j = 0; j < 5; ++j) off[j] = p.active_offsets[min(base + 4 * lane + j, p.slots)];
#pragma unroll
    for (int j = 0; j < 4; ++j) e[j] = p.active[min(base + 4 * lane + j, p.slots - 1)];
#pragma unroll
    for (int j = 0; j < 5; ++j) off[j] = min(max(off[j], 0), p.R);
    sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int rows = max(off[j + 1] - off[j], 0);
      const bool live = base + 4 * lane + j < na && (unsigned)e[j] < (unsigned)p.E;
      n[j] = live ? (rows + BM - 1) / BM : 0;
      sum += n[j];
    }
  }
};

__device__ __forceinline__ int wave_inclusive_sum(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int t = __shfl_up(v, d);
    v += lane >= d ? t : 0;
  }
  return v;
}

// Tiles of BM rows in all slots (the whole wave active); first: the slots 0 .. 255.
template <int BM>
__device__ __forceinline__ int count_tiles(const BlockGemmParams& p, const SlotTiles<BM>& first,
                                           int lane) {
  int total = __builtin_amdgcn_readlane(wave_inclusive_sum(first.sum, lane), 63);
  for (int base = 256; base < p.slots; base += 256) {
    SlotTiles<BM> st;
    st.load(p, base, lane);
    total += __builtin_amdgcn_readlane(wave_inclusive_sum(st.sum, lane), 63);
  }
  return total;
}

// The slot that holds row tile t of the slots' tiles in slot order.
struct SlotAt {
  int e, start, end;  // expert, its positions in pairs
  int tiles, rel;     // its row tiles, t among them
};

// (t uniform, below count_tiles; the whole wave active)
template <int BM>
__device__ __forceinline__ SlotAt find_slot(const BlockGemmParams& p, const SlotTiles<BM>& first,
                                            int t, int lane) {
  for (int base = 0; base < p.slots; base += 256) {
    SlotTiles<BM> st = first;
    if (base > 0) st.load(p, base, lane);
    const int incl = wave_inclusive_sum(st.sum, lane);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (t < total) {
      int rel = t - (incl - st.sum);  // < 0: an earlier lane's, >= sum: a later one's
      const unsigned long long hit = __ballot(rel >= 0 && rel < st.sum);
      SlotAt s = {0, 0, 0, 1, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (rel >= 0 && rel < st.n[j]) s = {st.e[j], st.off[j], st.off[j + 1], st.n[j], rel};
        rel -= st.n[j];
      }
      const int src = (int)__builtin_ctzll(hit);
      s.e = __builtin_amdgcn_readlane(s.e, src);
      s.start = __builtin_amdgcn_readlane(s.start, src);
      s.end = __builtin_amdgcn_readlane(s.end, src);
      s.tiles = __builtin_amdgcn_readlane(s.tiles, src);
      s.rel = __builtin_amdgcn_readlane(s.rel, src);
      return s;
    }
    t -= total;
  }
  return {0, 0, 0, 1, 0};
}

// A block's work: a row tile and the first of its weight rows.
struct Work {
  RowTile t;
  int n0;
};

// The block's tiles. Blocks are handed to the eight XCDs in turn (block b to
// XCD b % 8), each with its own L2, so XCD x gets the consecutive part
// [x T / 8, (x + 1) T / 8) of the T tiles, and its blocks take those in turn; a
// block past its XCD's part has none. The order is slot by slot, a slot (or the
// dense rows) in bands of eight row tiles: within a band all row tiles of one
// column of weight rows, then the next column. The blocks that an XCD runs at a
// time then share row tiles and weight rows about equally, and read an expert's
// weights together (bands across slots cut at every eighth row tile, and half an
// expert's weights came again: grouped gate_up at M = 8192 read 955 MB, this way
// 800 to 870; every byte once: 554).
// T counts at most the tiles that `limit` (the host's bound) allows, whatever
// off holds.
template <int BN, int BM, bool GROUPED>
struct BlockTiles {
  static constexpr int kBand = 8;
  int m_tiles, n_tiles;
  uint32_t q, end;
  // first: the slots 0 .. 255 (grouped; also in next)
  __device__ __forceinline__ BlockTiles(const BlockGemmParams& p, const SlotTiles<BM>& first,
                                        int n_tiles, uint32_t limit, int lane)
      : n_tiles(n_tiles) {
    if constexpr (GROUPED) {
      m_tiles = min((uint32_t)count_tiles<BM>(p, first, lane), limit / (uint32_t)n_tiles);
    } else {
      m_tiles = (p.R + BM - 1) / BM;
    }
    const uint32_t tiles = (uint32_t)m_tiles * (uint32_t)n_tiles;  // at most limit, < 2^31
    const uint32_t x = blockIdx.x & 7;
    q = tiles / 8 * x + tiles % 8 * x / 8 + (blockIdx.x >> 3);
    end = tiles / 8 * (x + 1) + tiles % 8 * (x + 1) / 8;
  }
  // The next tile; no rows: there is none.
  __device__ __forceinline__ Work next(const BlockGemmParams& p, const SlotTiles<BM>& first,
                                       int lane) {
    Work w = {{0, 0, 0}, 0};
    if (q >= end) return w;
    SlotAt slot = {0, 0, p.R, m_tiles, 0};
    uint32_t at = q;  // among the slot's tiles
    if constexpr (GROUPED) {
      const uint32_t t = q / (uint32_t)n_tiles;
      slot = find_slot<BM>(p, first, (int)t, lane);
      at = q - (t - (uint32_t)slot.rel) * (uint32_t)n_tiles;
    }
    const uint32_t per_band = kBand * (uint32_t)n_tiles;
    const uint32_t band = at / per_band, in = at - band * per_band;
    const uint32_t rows = min((uint32_t)kBand, (uint32_t)slot.tiles - band * kBand);
    const uint32_t n = in / rows;
    const int row0 = slot.start + (int)(band * kBand + (in - n * rows)) * BM;
    w.n0 = (int)n * BN;
    w.t = {slot.e, row0, min(slot.end - row0, BM)};
    q += gridDim.x >> 3;
    return w;
  }
};

// y row of row i of a tile; -1 for rows past the tile's last or a pair index
// out of range.
template <bool GROUPED>
__device__ __forceinline__ int y_row(const BlockGemmParams& p, const RowTile& t, int i) {
  if (i >= t.rows) return -1;
  if constexpr (!GROUPED) return t.row0 + i;
  const int v = p.pairs[t.row0 + i];
  return (unsigned)v < (unsigned)p.R ? v : -1;
}

// x row of row i of a tile; rows past the last read the last one again.
template <bool GROUPED>
__device__ __forceinline__ int x_row(const BlockGemmParams& p, const RowTile& t, int i) {
  const int c = t.row0 + min(i, t.rows - 1);
  if constexpr (!GROUPED) return c;
  const int v = p.pairs[c];
  return (unsigned)v < (unsigned)p.R ? v / p.div : 0;
}

__device__ __forceinline__ void store_y(uint16_t* y, float v) { *y = f32_to_bf16_rne(v); }
__device__ __forceinline__ void store_y(float* y, float v) { *y = v; }

// ---- few rows: operands straight to registers, K split over the waves -----------------
//
// One block per (row tile of 16 MT rows, 16 NT weight rows); wave v takes k
// steps v, v + W, ... and the W partial tiles are added in LDS in wave order.
// Bound: the latency of one read of the weights (M = 1, 2048 -> 5120, 10.5 MB:
// 5.6 us, 1.9 TB/s, of which a launch with nothing to read takes 2; 2048 -> 1024
// of eight experts, 16.8 MB: 6.5 us, 2.6 TB/s), so the chip needs many short
// blocks: 16 weight rows a block (32: 5.8 us, and 8.5 against 5.8 at N = 2048,
// K = 4096), four waves (eight: 5.6, with 16.8 MB 7.0 against 6.5).
constexpr int kDirectWaves = 4;

template <Mma MODE, bool GROUPED, int NT, int MT, int U, typename Y>
__global__ void __launch_bounds__(kDirectWaves * 64) direct_gemm_kernel(BlockGemmParams p,
                                                                        int n_tiles,
                                                                        uint32_t limit) {
  constexpr int BN = 16 * NT, BM = 16 * MT, W = kDirectWaves;
  constexpr bool FP8 = MODE != Mma::kBf16;
  __shared__ float red[W][BM][BN + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  SlotTiles<BM> slots;
  if constexpr (GROUPED) slots.load(p, 0, lane);
  const Work work =
      BlockTiles<BN, BM, GROUPED>(p, slots, n_tiles, limit, lane).next(p, slots, lane);
  const RowTile t = work.t;
  const int n0 = work.n0;
  if (t.rows <= 0) return;
  const int c = lane & 15, g = lane >> 4;

  const uint8_t* wr[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
    wr[i] = p.w + t.e * p.w_mat_bytes + (int64_t)min(n0 + 16 * i + c, p.N - 1) * p.row_bytes;
  const uint8_t* xr[MT];
  const float* xsr[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    const int64_t row = x_row<GROUPED>(p, t, 16 * j + c);
    xr[j] = p.x + row * p.row_bytes;
    xsr[j] = p.xs + row;
  }
  const float* wsr = nullptr;
  if constexpr (FP8) wsr = p.ws + ((int64_t)t.e * p.NB + n0 / kBlock8) * p.KB;

  bg_f32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = {0.0f, 0.0f, 0.0f, 0.0f};

  for (int kb0 = wave; kb0 < p.KB; kb0 += W * U) {
    Frag a[U][NT], b[U][MT];
    float xs[U][MT], ws[U];
    // every load is issued; steps past the last read the last one's bytes and
    // are not multiplied, pieces past K the step's first piece and are zeroed
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(kb0 + u * W, p.KB - 1);
      const int base = kb * kStepBytes;
      const int o0 = base + 16 * g < p.row_bytes ? base + 16 * g : base;
      const int o1 = base + 64 + 16 * g < p.row_bytes ? base + 64 + 16 * g : base;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        a[u][i].lo = load_stream(reinterpret_cast<const uint4*>(wr[i] + o0));
        a[u][i].hi = load_stream(reinterpret_cast<const uint4*>(wr[i] + o1));
      }
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        b[u][j].lo = *reinterpret_cast<const uint4*>(xr[j] + o0);
        b[u][j].hi = *reinterpret_cast<const uint4*>(xr[j] + o1);
        if constexpr (FP8) xs[u][j] = xsr[j][kb * p.Mx];
      }
      if constexpr (FP8) ws[u] = wsr[kb];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = kb0 + u * W;
      if (kb >= p.KB) break;
      const int base = kb * kStepBytes;
      if (base + kStepBytes > p.row_bytes) {  // the last step, partly past K
        const uint32_t k0 = base + 16 * g < p.row_bytes ? ~0u : 0u;
        const uint32_t k1 = base + 64 + 16 * g < p.row_bytes ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i < NT; ++i) mask_frag(a[u][i], k0, k1);
#pragma unroll
        for (int j = 0; j < MT; ++j) mask_frag(b[u][j], k0, k1);
      }
      Operand<MODE> ao[NT];
#pragma unroll
      for (int i = 0; i < NT; ++i) ao[i].set(a[u][i]);
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const float s = FP8 ? xs[u][j] * ws[u] : 1.0f;
        Operand<MODE> bo;
        bo.set(b[u][j]);
#pragma unroll
        for (int i = 0; i < NT; ++i) step_mma<MODE>(ao[i], bo, s, acc[i][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) red[wave][16 * j + c][16 * i + 4 * g + r] = acc[i][j][r];
  __syncthreads();
  for (int o = threadIdx.x; o < BM * BN; o += W * 64) {
    const int m = o / BN, n = o % BN;
    float v = red[0][m][n];
#pragma unroll
    for (int q = 1; q < W; ++q) v += red[q][m][n];
    const int yr = y_row<GROUPED>(p, t, m);
    if (yr >= 0 && n0 + n < p.N) store_y(static_cast<Y*>(p.y) + yr * p.ldy + n0 + n, v);
  }
}

// ---- many rows: operands staged in LDS --------------------------------------------------
//
// A block multiplies tiles of BM rows and BN weight rows, wave tiles of
// BN / WVN x BM / WVM. A k step of the BN + BM rows (128 bytes each, and the x
// scales) is copied to one of S LDS stages by direct loads, 16 bytes a lane,
// S - 1 steps ahead of its products. Piece c of row r lies at piece
// c ^ (r % 8) of the row's 128 bytes, so lanes that read the same piece of
// neighbouring rows hit different banks (no bank conflict counted in the
// loop); a copy's lanes are contiguous in LDS, so the exchange is made on the
// global side (eight lanes still read one row's whole 128 bytes).
//
// Order within step k, for a wave with NT rows of MT product tiles: its first
// operands (two weight and MT x operands, the scales) are already in
// registers; weight operand i + 2 is read while row i is multiplied, and the
// copies of step k + S - 1 go out between the products, into the stage of step
// k - 1; before the last row, one barrier: step k + 1 is complete and nobody
// reads this stage any more; during the last row the first operands of step
// k + 1 replace those just used. So the matrix cores have work across the
// barrier (with the barrier between the steps and the operands read after it:
// grouped gate_up 2048 -> 1024 at M = 4 15.0 us, this way 13.0), and a copy has
// more than a step to arrive (with two stages and one step: M = 16 53 us,
// this way 44). Three stages; four where a tile a CU is all there is (beside the
// choice of tiles).
//
// With more tiles than the chip holds at once (MANY), a CU's worth of blocks
// takes them in turn: the last two steps of a tile copy the first two of the
// next one, whose pairs and scales were looked up a tile earlier, so only the
// results stand between two tiles (one tile a block: M = 8192, 2048 -> 5120
// 98.6 us, this way 93.6; grouped gate_up, E = 256, M = 8192 265 and 241).
//
// What bounds large products (M = 8192, 2048 -> 5120: 90 to 97 us by the card's
// clock, 1.77 to 1.9 PFLOP/s, 46 % of the cycles matrix instructions): LDS. A
// 256 x 128 step is 48 direct loads of 1 KB, about 24 clocks of the LDS each
// beside reads, and 128 KB of operand reads at about 230 bytes a clock, 0.86 us
// of the step's 1.1; its matrix instructions alone take 0.67 (through registers
// and LDS stores it took the same time; 256 x 256 tiles have a third fewer
// bytes, but only two stages fit: 93.7 with one tile a block). Grouped products
// of some hundred rows an expert (M = 8192: 239 us, 1.15 PFLOP/s): a quarter of
// the tiles' rows are empty, and every step's weights come from HBM, two steps
// ahead and no more, for that is what LDS holds (eight experts of 8192 rows, the
// same products: 176 us). With few rows a slot the bytes of the weights
// are the bound (M = 256 98 us, 5.5 TB/s).
typedef __attribute__((address_space(3))) void lds_void;
typedef const __attribute__((address_space(1))) void global_void;

// The lane's 16 (4) bytes at src to dst + 16 (4) * lane; dst is wave-uniform.
__device__ __forceinline__ void copy16_to_lds(const uint8_t* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((global_void*)src, (lds_void*)dst, 16, 0, 0);
}
__device__ __forceinline__ void copy4_to_lds(const void* src, uint8_t* dst) {
  __builtin_amdgcn_global_load_lds((global_void*)src, (lds_void*)dst, 4, 0, 0);
}

// All of the wave's requests but the N newest loads are done, then those of
// every wave of the block.
template <int N>
__device__ __forceinline__ void arrive() {
  static_assert(N >= 0 && N < 64, "");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

template <Mma MODE, bool GROUPED, int BN, int BM, int WVN, int WVM, int S>
struct Tiled {
  static constexpr bool FP8 = MODE != Mma::kBf16;
  static constexpr int kWaves = WVN * WVM, kThreads = kWaves * 64;
  static constexpr int WN = BN / WVN, WM = BM / WVM, NT = WN / 16, MT = WM / 16;
  // copies per wave and step: weight rows, x rows, x scales of the wave's rows
  static constexpr int LA = BN / 8 / kWaves, LB = BM / 8 / kWaves;
  static constexpr int LS = FP8 ? (WM + 63) / 64 : 0;
  static constexpr int kCopies = LA + LB + LS;
  static constexpr int kScales = (BN + BM) * kStepBytes;  // where a stage's scales start
  static constexpr int kStageBytes = kScales + kWaves * LS * 256;
  static_assert(LA * 8 * kWaves == BN && LB * 8 * kWaves == BM, "rows split evenly over the waves");
  static_assert(kBlock8 % WN == 0, "a wave's weight rows share a scale block");
  static_assert(NT % 2 == 0, "the first weight operand of a step is always a[0]");
  // copies that may be on their way when the next step is to be complete
  static constexpr int kLater = (S - 2) * kCopies;
  static_assert(S * kStageBytes <= 160 * 1024, "the stages fit the LDS");

  // What a lane copies: byte offsets of its rows (weights: from the tile's
  // first row; x: from the tile's first row, or of any row when gathered),
  // and the x rows whose scales it copies.
  struct Rows {
    uint32_t a[LA];
    uint64_t b[LB];  // dense: below 2^32
    uint32_t s[LS ? LS : 1];
  };

  // The step that is being copied: bases plus the step's offset, and the
  // lane's piece of its rows (past K: the step's first piece, zeroed after the
  // read from LDS). After the last step the last one is copied again.
  struct Cursor {
    const uint8_t *w, *x;
    const float* xs;
    uint32_t o;
    int step;
    __device__ __forceinline__ void set_piece(const BlockGemmParams& p, int piece) {
      o = step * kStepBytes + 16 * piece < p.row_bytes ? 16 * piece : 0;
    }
    __device__ __forceinline__ void advance(const BlockGemmParams& p, int piece) {
      const int more = step + 1 < p.KB ? 1 : 0;  // no branch: the compiler would move the
      step += more;                              // scaling of the products behind it
      w += more * kStepBytes;
      x += more * kStepBytes;
      if constexpr (FP8) xs += more * p.Mx;
      set_piece(p, piece);
    }
  };

  // Copy i of the cursor's step into a stage.
  template <int i>
  static __device__ __forceinline__ void copy(const Rows& r, const Cursor& c, int wave,
                                              uint8_t* stage) {
    if constexpr (i < LA) {
      copy16_to_lds(c.w + (uint32_t)(r.a[i] + c.o), stage + (i * kWaves + wave) * 1024);
    } else if constexpr (i < LA + LB) {
      constexpr int j = i - LA;
      copy16_to_lds(c.x + (GROUPED ? r.b[j] + c.o : (uint32_t)((uint32_t)r.b[j] + c.o)),
                    stage + BN * kStepBytes + (j * kWaves + wave) * 1024);
    } else {
      constexpr int j = i - LA - LB;
      copy4_to_lds(c.xs + r.s[j], stage + kScales + (wave * LS + j) * 256);
    }
  }

  // A wave's place in a stage.
  struct Place {
    int w, x, s;  // byte offsets of the lane's first weight row, x row and scale
    int lo;       // the lane's first piece of a row (the second: lo ^ 64)
    __device__ __forceinline__ Place(int wave, int wn, int wm, int lane) {
      const int c = lane & 15, g = lane >> 4;
      w = (wn + c) * kStepBytes;
      x = (BN + wm + c) * kStepBytes;
      s = kScales + wave * LS * 256 + 4 * c;
      lo = 16 * (g ^ (c & 7));
    }
  };

  static __device__ __forceinline__ Frag read(const uint8_t* row, int lo) {
    Frag f;
    f.lo = *reinterpret_cast<const uint4*>(row + lo);
    f.hi = *reinterpret_cast<const uint4*>(row + (lo ^ 64));
    return f;
  }

  // The first operands of a step.
  struct First {
    Frag a[2], b[MT];
    float xs[MT];
    template <int j>
    __device__ __forceinline__ void read_b(const uint8_t* stage, const Place& at) {
      b[j] = read(stage + at.x + 16 * j * kStepBytes, at.lo);
    }
    __device__ __forceinline__ void read_a(const uint8_t* stage, const Place& at) {
      a[0] = read(stage + at.w, at.lo);
      a[1] = read(stage + at.w + 16 * kStepBytes, at.lo);
    }
    __device__ __forceinline__ void read_xs(const uint8_t* stage, const Place& at) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
        xs[j] = FP8 ? *reinterpret_cast<const float*>(stage + at.s + 64 * j) : 1.0f;
    }
  };

  // One step, held by cur: its products, ahead(i) (copy i of the step
  // S - 1 further on) between them, and the first operands of the next step, held by
  // other. MASK: the step may end past K (k0, k1: masks of the lane's pieces). LAST:
  // no step follows, so there are no copies, barrier and first operands.
  // FP8: a tile's block sum is scaled into the result two instructions later,
  // while the matrix cores work on (the scheduling barriers keep that order:
  // left alone, the compiler moves the scaling next to its product and waits
  // there).
  template <bool MASK, bool LAST, typename Ahead>
  static __device__ __forceinline__ void step(const uint8_t* cur, const uint8_t* other,
                                              const Place& at, First& f, float ws, uint32_t k0,
                                              uint32_t k1, bg_f32x4 (&acc)[NT][MT], Ahead ahead) {
    Frag a[3];  // rows i, i + 1 and i + 2 at i mod 3
    a[0] = f.a[0];
    a[1] = f.a[1];
    Operand<MODE> b[MT];
    float s[MT];
    if constexpr (MASK) {
      mask_frag(a[0], k0, k1);
      mask_frag(a[1], k0, k1);
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      if constexpr (MASK) mask_frag(f.b[j], k0, k1);
      b[j].set(f.b[j]);
      s[j] = f.xs[j] * ws;
    }
    auto weights_ahead = [&](auto row) {
      a[row % 3] = read(cur + at.w + 16 * row * kStepBytes, at.lo);
      if constexpr (MASK) mask_frag(a[row % 3], k0, k1);
    };
    if constexpr (MODE == Mma::kFp8) {
      constexpr int kLag = 3;
      bg_f32x4 t[kLag + 1];
      static_for<NT * MT>([&](auto qc) {
        constexpr int q = qc, i = q / MT, j = q % MT, d = q - kLag;
        if constexpr (!LAST && i == NT - 1 && j == 0) arrive<kLater>();
        Operand<MODE> ao;
        ao.set(a[i % 3]);
        t[q % (kLag + 1)] = block_mma<MODE>(ao, b[j]);
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (j == 0 && i + 2 < NT) weights_ahead(std::integral_constant<int, i + 2>{});
        if constexpr (!LAST && i == NT - 1) {
          if constexpr (j == 0) f.read_a(other, at);
          f.template read_b<j>(other, at);
          if constexpr (j == MT - 1) f.read_xs(other, at);
        }
        if constexpr (d >= 0) scale_into(t[d % (kLag + 1)], s[d % MT], acc[d / MT][d % MT]);
        if constexpr (!LAST && i < NT - 1)
          static_for<kCopies>([&](auto v) {
            if constexpr (v * (NT - 1) * MT / kCopies == q) ahead(v);
          });
        __builtin_amdgcn_sched_barrier(0);
      });
#pragma unroll
      for (int d = NT * MT - kLag; d < NT * MT; ++d)
        scale_into(t[d % (kLag + 1)], s[d % MT], acc[d / MT][d % MT]);
    } else {
      // several instructions per tile and step: those of a row of tiles in
      // turn, so that none waits for the one before it
      constexpr int kParts = (int)(sizeof(Operand<MODE>::v) / sizeof(bg_bf16x8));
      static_for<NT>([&](auto ic) {
        constexpr int i = ic;
        if constexpr (!LAST && i == NT - 1) arrive<kLater>();
        Operand<MODE> ao;
        ao.set(a[i % 3]);
        bg_f32x4 t[MT];
#pragma unroll
        for (int j = 0; j < MT; ++j) t[j] = FP8 ? bg_f32x4{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j];
#pragma unroll
        for (int e = 0; e < kParts; ++e)
#pragma unroll
          for (int j = 0; j < MT; ++j)
            t[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ao.v[e], b[j].v[e], t[j], 0, 0, 0);
        if constexpr (i + 2 < NT) weights_ahead(std::integral_constant<int, i + 2>{});
        if constexpr (!LAST && i == NT - 1) {
          f.read_a(other, at);
          static_for<MT>([&](auto j) { f.template read_b<j>(other, at); });
          f.read_xs(other, at);
        }
        if constexpr (!LAST && i < NT - 1)
          static_for<kCopies>([&](auto v) {
            if constexpr (v * (NT - 1) / kCopies == i) ahead(v);
          });
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          if constexpr (FP8)
            scale_into(t[j], s[j], acc[i][j]);
          else
            acc[i][j] = t[j];
        }
      });
    }
  }

  // A step of a wave whose rows all lie past the tile's last: its copies only,
  // and in a tile's last step (MASK) the first operands of what follows.
  template <bool MASK, bool LAST, typename Ahead>
  static __device__ __forceinline__ void idle(const uint8_t* other, const Place& at, First& f,
                                              Ahead ahead) {
    if constexpr (LAST) return;
    static_for<kCopies>([&](auto v) { ahead(v); });
    arrive<kLater>();
    if constexpr (MASK) {
      f.read_a(other, at);
      static_for<MT>([&](auto j) { f.template read_b<j>(other, at); });
      f.read_xs(other, at);
    }
  }
};

__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, v2{(__bf16)a, (__bf16)b});  // RNE, one instruction
}

// Four consecutive results in y's type.
__device__ __forceinline__ void pack4(const bg_f32x4& v, uint16_t* dst) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
}
__device__ __forceinline__ void pack4(const bg_f32x4& v, float* dst) {
  *reinterpret_cast<bg_f32x4*>(dst) = v;
}

template <Mma MODE, bool GROUPED, int BN, int BM, int WVN, int WVM, int S>
struct TiledLds {
  using T = Tiled<MODE, GROUPED, BN, BM, WVN, WVM, S>;
  static constexpr int kScaleRows = T::FP8 ? (BN + kBlock8 - 1) / kBlock8 : 0;
  static constexpr int kScaleBytes = kScaleRows * 256;
  static constexpr int kPairBytes = GROUPED ? (BM + 63) / 64 * 256 : 0;
  static constexpr int kPairs = S * T::kStageBytes;           // the pairs of three tiles
  static constexpr int kScales = kPairs + 3 * kPairBytes;     // and 64 weight scales a row
  static constexpr int kSlots = kScales + 3 * kScaleBytes;
  static constexpr int kBytes = kSlots + (GROUPED ? 64 * (int)sizeof(SlotTiles<BM>) : 0);
  // blocks a CU holds: by LDS, and at least 128 registers a lane
  static constexpr int kPerCu = 160 * 1024 / kBytes < 16 / T::kWaves ? 160 * 1024 / kBytes
                                                                    : 16 / T::kWaves;
  static constexpr int kWavesPerSimd = kPerCu * T::kWaves / 4;
  static_assert(kPerCu >= 1, "fits the LDS");
};

template <Mma MODE, bool GROUPED, int BN, int BM, int WVN, int WVM, int S, bool MANY, typename Y>
__global__ void __launch_bounds__(WVN* WVM * 64,
                                  (TiledLds<MODE, GROUPED, BN, BM, WVN, WVM, S>::kWavesPerSimd))
    tiled_gemm_kernel(BlockGemmParams p, int n_tiles, uint32_t limit) {
  using T = Tiled<MODE, GROUPED, BN, BM, WVN, WVM, S>;
  using L = TiledLds<MODE, GROUPED, BN, BM, WVN, WVM, S>;
  static_assert(!MANY || S == 3, "a tile starts two steps before the last one ends");
  __shared__ __align__(1024) uint8_t stages[L::kBytes];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  SlotTiles<BM> slots;
  if constexpr (GROUPED) slots.load(p, 0, lane);
  BlockTiles<BN, BM, GROUPED> tiles(p, slots, n_tiles, limit, lane);
  Work work = tiles.next(p, slots, lane);
  if (work.t.rows <= 0) return;

  const int piece = (lane & 7) ^ (lane >> 3);
  const int wn = (wave % WVN) * T::WN, wm = (wave / WVN) * T::WM;
  const typename T::Place at(wave, wn, wm, lane);
  const bool aligned16 = (p.ldy % (16 / (int)sizeof(Y)) |
                          (int64_t)((uintptr_t)p.y % 16)) == 0;  // rows of y start on 16 bytes

  // The lane, for what is worked out once a tile: taken out of the loop, as the
  // compiler would from the plain variable, it holds registers that the products
  // need, and each reload from scratch would wait for every copy and store.
  auto lane_here = [&] {
    int l = lane;
    asm volatile("" : "+v"(l));
    return l;
  };
  // What a tile's copies need to know before the first one: its pairs and the
  // first 64 steps' weight scales, one a lane of the first waves; later in LDS.
  int32_t pair_lane = 0;
  float scale_lane = 1.0f;
  auto look_up = [&](const Work& k) {
    if (k.t.rows <= 0) return;
    const int l = lane_here();
    if constexpr (GROUPED)
      if (wave < (BM + 63) / 64)
        pair_lane = p.pairs[k.t.row0 + min(wave * 64 + l, k.t.rows - 1)];
    if constexpr (T::FP8)
      if (wave < L::kScaleRows)
        scale_lane = p.ws[((int64_t)k.t.e * p.NB + min(k.n0 / kBlock8 + wave, p.NB - 1)) * p.KB +
                          min(l, p.KB - 1)];
  };
  auto keep_pairs = [&](int third) {
    const int l = lane_here();
    if constexpr (GROUPED)
      if (wave < (BM + 63) / 64)
        reinterpret_cast<int32_t*>(stages + L::kPairs + third * L::kPairBytes)[wave * 64 + l] =
            pair_lane;
  };
  auto keep_scales = [&](int third) {
    const int l = lane_here();
    if constexpr (T::FP8)
      if (wave < L::kScaleRows)
        reinterpret_cast<float*>(stages + L::kScales + third * L::kScaleBytes)[wave * 64 + l] =
            scale_lane;
  };
  auto pair = [&](int third, int i) {
    return reinterpret_cast<const int*>(stages + L::kPairs + third * L::kPairBytes)[i];
  };
  auto source_row = [&](const Work& k, int third, int i) -> uint32_t {  // x row of row i
    if constexpr (!GROUPED) return k.t.row0 + min(i, k.t.rows - 1);
    const int v = pair(third, i);
    return (unsigned)v < (unsigned)p.R ? v / p.div : 0;
  };
  typename T::Cursor c;
  typename T::Rows rows;
  auto enter = [&](const Work& k, int third) {  // the copies go on with this tile
    const int l = lane_here();
    c.w = p.w + k.t.e * p.w_mat_bytes + (int64_t)k.n0 * p.row_bytes;
    c.x = GROUPED ? p.x : p.x + (int64_t)k.t.row0 * p.row_bytes;
    c.xs = p.xs;
    c.step = 0;
    c.set_piece(p, piece);
#pragma unroll
    for (int j = 0; j < T::LA; ++j) {
      const int n = min((j * T::kWaves + wave) * 8 + (l >> 3), p.N - 1 - k.n0);
      rows.a[j] = (uint32_t)n * (uint32_t)p.row_bytes;
    }
#pragma unroll
    for (int j = 0; j < T::LB; ++j) {
      const int r = (j * T::kWaves + wave) * 8 + (l >> 3);
      if constexpr (GROUPED)
        rows.b[j] = (uint64_t)source_row(k, third, r) * (uint32_t)p.row_bytes;
      else
        rows.b[j] = (uint32_t)min(r, k.t.rows - 1) * (uint32_t)p.row_bytes;
    }
#pragma unroll
    for (int j = 0; j < T::LS; ++j)
      rows.s[j] = source_row(k, third, wm + 64 * j + (l & (T::WM < 64 ? T::WM - 1 : 63)));
  };

  auto one_more = [&] {
    const int l = lane_here();
    SlotTiles<BM> st;
    if constexpr (GROUPED) __builtin_memcpy(&st, stages + L::kSlots + l * sizeof(st), sizeof(st));
    return tiles.next(p, st, l);
  };

  const float* wsr = nullptr;  // the wave's row of weight scales, 64 of them one a lane
  float ws_lanes = 1.0f;
  auto scales_of = [&](const Work& k, int third) {
    if constexpr (T::FP8) {
      wsr = p.ws + ((int64_t)k.t.e * p.NB + min((k.n0 + wn) / kBlock8, p.NB - 1)) * p.KB;
      ws_lanes = reinterpret_cast<const float*>(stages + L::kScales + third * L::kScaleBytes +
                                                wn / kBlock8 * 256)[lane_here()];
    }
  };
  auto ws_of = [&](int kb) {
    if (T::FP8 && kb > 0 && (kb & 63) == 0) {
      ws_lanes = wsr[min(kb + lane, p.KB - 1)];
      // (a use: the wait for this load stays here, instead of one for
      // everything outstanding in every step)
      asm volatile("" : "+v"(ws_lanes));
    }
    return T::FP8 ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(ws_lanes), kb & 63))
                  : 1.0f;
  };

  bg_f32x4 acc[T::NT][T::MT];
  typename T::First f;
  // Some of the wave's rows are the tile's; a wave without any leaves the
  // products to the others (grouped gate_up, E = 256, M = 2048, 64 rows a slot:
  // 131.5 us, this way 127).
  bool busy = true;
  auto step = [&](auto mask, auto last, int kb, uint32_t k0, uint32_t k1,
                  const uint8_t* __restrict__ cur, const uint8_t* __restrict__ next,
                  uint8_t* __restrict__ fill) {
    auto copies = [&](auto v) { T::template copy<v>(rows, c, wave, fill); };
    if (!MANY || WVM == 1 || busy)
      T::template step<mask, last>(cur, next, at, f, ws_of(kb), k0, k1, acc, copies);
    else
      T::template idle<mask, last>(next, at, f, copies);
    c.advance(p, piece);
  };
  auto after = [](uint32_t stage) {
    stage += T::kStageBytes;
    return stage == S * T::kStageBytes ? 0u : stage;
  };
  // While a tile's steps run, the next one's pairs and scales are in LDS, and
  // from the last but one step on its copies are made; the one after that is
  // looked up in the last step, and put into LDS before the results, where the
  // wave waits for its copies anyway. With one or two steps a tile starts afresh.
  uint32_t cur = 0, fill = (S - 1) * T::kStageBytes;
  auto start = [&](const Work& k, int third) {
    enter(k, third);
    cur = 0;
    fill = (S - 1) * T::kStageBytes;
    static_for<S - 1>([&](auto q) {
      static_for<T::kCopies>(
          [&](auto v) { T::template copy<v>(rows, c, wave, stages + q * T::kStageBytes); });
      c.advance(p, piece);
    });
  };
  look_up(work);
  keep_pairs(0);
  if constexpr (GROUPED) arrive<63>();
  start(work, 0);
  keep_scales(0);
  Work ahead = {{0, 0, 0}, 0}, next = ahead;
  if constexpr (MANY) ahead = tiles.next(p, slots, lane);
  if (MANY && ahead.t.rows > 0) {
    look_up(ahead);
    keep_pairs(1);
    keep_scales(1);
    next = tiles.next(p, slots, lane);
    // a lane's slots stay in LDS, for the registers are the products'
    if (GROUPED && wave == 0)
      __builtin_memcpy(stages + L::kSlots + lane * sizeof(slots), &slots, sizeof(slots));
  }
  int third = 0;  // of the looked up
  bool first = true, flowing = false;  // flowing: the tile's first operands are in registers
  for (;;) {
    arrive<63>();  // what was kept is in LDS, and the last results are out of it
    scales_of(work, third);
    const int third1 = third == 2 ? 0 : third + 1;
    if (!flowing) {
      if (!first) {
        arrive<0>();  // copies that nothing needed
        start(work, third);
      }
      first = false;
      arrive<T::kLater>();
      f.read_a(stages, at);
      static_for<T::MT>([&](auto j) { f.template read_b<j>(stages, at); });
      f.read_xs(stages, at);
    }
    flowing = MANY && ahead.t.rows > 0 && p.KB > 2;
    busy = wm < work.t.rows;
#pragma unroll
    for (int i = 0; i < T::NT; ++i)
#pragma unroll
      for (int j = 0; j < T::MT; ++j) acc[i][j] = {0.0f, 0.0f, 0.0f, 0.0f};
    asm volatile("" : "+v"(c.o));  // a use: no wait for a load of it in the loop
#pragma unroll 1
    for (int kb = 0; kb + 1 < p.KB; ++kb) {
      if (flowing && kb + 2 == p.KB) enter(ahead, third1);
      step(std::false_type{}, std::false_type{}, kb, ~0u, ~0u, stages + cur, stages + after(cur),
           stages + fill);
      cur = after(cur);
      fill = after(fill);
    }
    if constexpr (MANY) look_up(next);
    {
      const int g = lane_here() >> 4, base = (p.KB - 1) * kStepBytes;
      const uint32_t k0 = base + 16 * g < p.row_bytes ? ~0u : 0u;
      const uint32_t k1 = base + 64 + 16 * g < p.row_bytes ? ~0u : 0u;
      step(std::true_type{}, std::bool_constant<!MANY>{}, p.KB - 1, k0, k1, stages + cur,
           stages + after(cur), stages + fill);
    }
    Work later = ahead;
    if constexpr (MANY) {
      keep_pairs(third1 == 2 ? 0 : third1 + 1);
      keep_scales(third1 == 2 ? 0 : third1 + 1);
      later = one_more();
    } else {
      arrive<0>();  // the stage's reads are done; also copies that nothing needed
    }

    // The results, 16 token rows at a time through the wave's part of the stage
    // that the last step has left: a lane holds four n of one row, and the 16
    // rows of one store would take 32 bytes each; read back, eight or more lanes
    // write one row's consecutive 16-byte pieces.
    constexpr int kRow = T::WN * (int)sizeof(Y) + 16, kPieces = T::WN * (int)sizeof(Y) / 16;
    constexpr int kPer = 16 / (int)sizeof(Y);  // elements of a piece
    static_assert(T::kWaves * 16 * kRow <= T::kStageBytes, "the exchange fits a stage");
    const int l = lane_here();
    uint8_t* ex = stages + cur + wave * 16 * kRow;
#pragma unroll
    for (int j = 0; j < T::MT; ++j) {
      if (wm + 16 * j >= work.t.rows) break;
#pragma unroll
      for (int i = 0; i < T::NT; ++i)
        pack4(acc[i][j], reinterpret_cast<Y*>(ex + (l & 15) * kRow) + 16 * i + 4 * (l >> 4));
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int q = l; q < 16 * kPieces; q += 64) {
        const int r = wm + 16 * j + q / kPieces, n = work.n0 + wn + (q % kPieces) * kPer;
        const uint4 v =
            *reinterpret_cast<const uint4*>(ex + q / kPieces * kRow + (q % kPieces) * 16);
        if (r >= work.t.rows || n >= p.N) continue;
        int64_t yr = work.t.row0 + r;
        if constexpr (GROUPED) {
          yr = pair(third, r);
          if ((uint64_t)yr >= (uint64_t)p.R) continue;
        }
        Y* dst = static_cast<Y*>(p.y) + yr * p.ldy + n;
        if (aligned16 && n + kPer <= p.N) {
          *reinterpret_cast<uint4*>(dst) = v;
        } else {
          Y el[kPer];
          __builtin_memcpy(el, &v, 16);
#pragma unroll
          for (int e = 0; e < kPer; ++e)
            if (n + e < p.N) dst[e] = el[e];
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (!MANY || ahead.t.rows <= 0) break;
    cur = after(cur);
    fill = after(fill);
    work = ahead;
    ahead = next;
    next = later;
    third = third1;
  }
  if constexpr (MANY) arrive<0>();  // copies that nothing needed
}

}  // namespace nvfp4moe
