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

#include "block8.hpp"
#include "fp8.hpp"

namespace nvfp4moe {

typedef __bf16 bg_bf16x8 __attribute__((ext_vector_type(8)));
typedef float bg_f32x4 __attribute__((ext_vector_type(4)));
typedef int bg_i32x8 __attribute__((ext_vector_type(8)));

constexpr int kStepBytes = 128;

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

// acc += (A B) * s over one k step (BF16 operands: s is 1 and not applied).
template <Mma MODE>
__device__ __forceinline__ void step_mma(const Operand<MODE>& a, const Operand<MODE>& b, float s,
                                         bg_f32x4& acc) {
  if constexpr (MODE == Mma::kBf16) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], acc, 0, 0, 0);
  } else {
    bg_f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (MODE == Mma::kFp8) {
      t = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, t, 0, 0, 0, 0, 0,
                                                           0);  // E4M3 x E4M3, no scale operand
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], t, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = fmaf(t[r], s, acc[r]);
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

// Row tile t of the slots' tiles in slot order (t uniform; the whole wave active).
template <int BM>
__device__ __forceinline__ RowTile find_tile(const BlockGemmParams& p, int t, int lane) {
  RowTile r = {0, 0, 0};
  for (int base = 0; base < p.slots; base += 256) {
    SlotTiles<BM> st;
    st.load(p, base, lane);
    const int incl = wave_inclusive_sum(st.sum, lane);
    const int total = __builtin_amdgcn_readlane(incl, 63);
    if (t < total) {
      int rel = t - (incl - st.sum);  // < 0: an earlier lane's, >= sum: a later one's
      const unsigned long long hit = __ballot(rel >= 0 && rel < st.sum);
      int e = 0, row0 = 0, rows = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (rel >= 0 && rel < st.n[j]) {
          e = st.e[j];
          row0 = st.off[j] + rel * BM;
          rows = min(st.off[j + 1] - row0, BM);
        }
        rel -= st.n[j];
      }
      const int src = (int)__builtin_ctzll(hit);
      r.e = __builtin_amdgcn_readlane(e, src);
      r.row0 = __builtin_amdgcn_readlane(row0, src);
      r.rows = __builtin_amdgcn_readlane(rows, src);
      return r;
    }
    t -= total;
  }
  return r;
}

template <int BM, bool GROUPED>
__device__ __forceinline__ RowTile row_tile(const BlockGemmParams& p, int t, int lane) {
  if constexpr (GROUPED) {
    return find_tile<BM>(p, t, lane);
  } else {
    const int row0 = t * BM;
    return {0, row0, min(p.R - row0, BM)};
  }
}

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
constexpr int kDirectWaves = 4;

template <Mma MODE, bool GROUPED, int NT, int MT, int U, typename Y>
__global__ void __launch_bounds__(kDirectWaves * 64) direct_gemm_kernel(BlockGemmParams p,
                                                                        int n_tiles) {
  constexpr int BN = 16 * NT, BM = 16 * MT, W = kDirectWaves;
  constexpr bool FP8 = MODE != Mma::kBf16;
  __shared__ float red[W][BM][BN + 1];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = (int)(blockIdx.x / (unsigned)n_tiles);
  const int n0 = (int)(blockIdx.x % (unsigned)n_tiles) * BN;
  const RowTile t = row_tile<BM, GROUPED>(p, tile, lane);
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
        const uint4 z = make_uint4(0, 0, 0, 0);
        const bool k0 = base + 16 * g < p.row_bytes, k1 = base + 64 + 16 * g < p.row_bytes;
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          a[u][i].lo = k0 ? a[u][i].lo : z;
          a[u][i].hi = k1 ? a[u][i].hi : z;
        }
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          b[u][j].lo = k0 ? b[u][j].lo : z;
          b[u][j].hi = k1 ? b[u][j].hi : z;
        }
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

}  // namespace nvfp4moe
