// fp4q_linear_many.h -- products of many rows of activations with a 4-bit
// weight: y = x W^T, h = SiLU(x Wg^T) * (x Wu^T) and dx = dy W, in tiles.
//
// A workgroup computes BM rows of activations by BN outputs in stages of 64 of
// the contraction.  A stage's activations go to LDS as bf16 (fp32 ones as three
// planes of pieces), its weights as the codes they are, an eighth of the bytes
// of x: each wave turns the codes that it needs into bf16 in registers.  Loads of
// a stage are in flight while the one before it is multiplied.
//
// v_mfma_f32_16x16x32_bf16, weights as the left operand, so that a lane ends up
// with consecutive outputs of one row.  The order of the contraction inside a
// stage is free:
//  - y = x W^T (contraction over k): lane group g = lane / 16 takes k = 16 g .. +
//    15 of the stage, 8 bytes of codes with one scale, in two instructions.
//  - dx = dy W (contraction over the weight's rows): a lane needs 8 rows' codes
//    of one column.  It reads those of FN neighbouring columns (2 bytes for 4) of
//    each of the rows, whose scales differ, converts them row by row, and pairs
//    neighbouring rows' values: instruction j then takes columns FN r + j, r =
//    lane mod 16, and a lane's outputs are consecutive columns again.
//
// One wave has all BM rows of its columns, so that no code is converted twice in a
// workgroup; two workgroups of 4 waves a CU overlap one's conversions with the
// other's products.  (A workgroup of 8 waves on 256 x 256, which converted twice
// (forward) or four times (back): dx of 1024 rows, k and n 8192, NVFP4 392 us.)
#pragma once

#include <type_traits>

#include "fp4q_ffn.h"

namespace fp4q {

constexpr int kStage = 64;
enum ManyMode { kForward = 0, kGated = 1, kTransposed = 2 };

// What a launch of the tile kernel adds to the call: how the contraction is
// parted, and where parts go.
struct ManyArgs {
  LinearLaunch l;
  int tiles_m, tiles_n, ntiles;
  int splits, stages, per_split;   // stages of the contraction, of one part
};

template <int FMT, int XT, int MODE, int BM, int BN, int WM, int WN>
struct ManyTile {
  static constexpr int kThreads = 64 * WM * WN, kWavesM = WM;
  static constexpr int TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  static constexpr int P = kPieces<XT>;
  static constexpr int kBlock = FMT == 0 ? 32 : 16;
  static constexpr bool kT = MODE == kTransposed;
  static constexpr int kXBytes = P * BM * 2 * kStage;
  // codes: rows of 32 bytes; transposed, rows of BN / 2 with a pad each 8 rows
  // that spreads the 4 lane groups' reads over the banks
  static constexpr int kWPitch = kT ? BN / 2 : kStage / 2;
  static constexpr int kColBytes = FN / 2;               // transposed: codes of a lane's columns in a row
  static constexpr int kWBytes = kT ? kStage * kWPitch + kStage / 8 * 64 : BN * kWPitch;
  // scales: by row; transposed, by block of columns, a byte for each row
  static constexpr int kSPitch = kT ? kStage + 8 : kStage / kBlock;
  static constexpr int kSBytes = kT ? BN / kBlock * kSPitch : BN * kSPitch;
  static constexpr int kBuf = (kXBytes + kWBytes + kSBytes + 15) / 16 * 16;
  static constexpr int kXPer = BM * 8 / kThreads;                                // 8-element pieces a thread
  static constexpr int kWPer = (kT ? kStage * (BN / 32) : BN * 2) / kThreads;    // 16-byte pieces
  static_assert(kXPer * kThreads == BM * 8 && kWPer >= 1, "whole pieces");
  static_assert(!kT || FN == 2 || FN == 4, "a lane takes 2 or 4 neighbouring columns");
  static_assert(MODE != kGated || FN % 2 == 0, "both factors in a wave");
};

// Where in LDS the 16-byte chunk `chunk` of a row's 8 lies, by the row: 16 rows'
// reads of one chunk meet all banks.
__device__ __forceinline__ int x_chunk(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// acc += a stage's products, from its buffer in LDS.
// (half: of its first or second 32 of the contraction alone, or both, -1.)
template <class T, int FMT>
__device__ __forceinline__ void many_multiply(const uint8_t* buf, f32x4_t (&acc)[T::FN][T::FM], int wm, int wn, int r,
                                              int g, float power, int half = -1) {
  constexpr int P = T::P, FM = T::FM, FN = T::FN, BM = T::TM * T::kWavesM;
  const uint8_t* bw = buf + T::kXBytes;
  const uint8_t* bs = bw + T::kWBytes;
#pragma unroll
  for (int i = 0; i < (half < 0 ? 2 : 1); ++i) {
    const int t = half < 0 ? i : half;
    u32x4_t wf[FN];
    if constexpr (T::kT) {
      // (hidden, as one addition to the buffer's address: more, and the compiler no
      // longer tells which loads into LDS the reads have to wait for, and waits for all)
      int c0 = T::kXBytes + (32 * t + 8 * g) * T::kWPitch + (4 * t + g) * 64 + wn * (T::TN / 2) + T::kColBytes * r;
      asm volatile("" : "+v"(c0));
      const u32x2_t sb = *reinterpret_cast<const u32x2_t*>(
          bs + ((wn * T::TN + FN * r) / T::kBlock) * T::kSPitch + 32 * t + 8 * g);
#pragma unroll
      for (int i = 0; i < 8; i += 2) {     // rows i and i + 1 of this lane's 8
        uint32_t ca, cb;
        if constexpr (FN == 4) {
          ca = *reinterpret_cast<const uint16_t*>(buf + (c0 + i * T::kWPitch));
          cb = *reinterpret_cast<const uint16_t*>(buf + (c0 + (i + 1) * T::kWPitch));
        } else {
          ca = buf[c0 + i * T::kWPitch];
          cb = buf[c0 + (i + 1) * T::kWPitch];
        }
        const uint32_t sw = i < 4 ? sb.x : sb.y;
        const float sa = scale_operand<FMT>((sw >> (8 * (i & 3))) & 0xFFu);
        const float sc = scale_operand<FMT>((sw >> (8 * (i & 3) + 8)) & 0xFFu);
        uint32_t o[FN];
        weight_pairs<FMT, FN>(ca, sa, cb, sc, power, o);
#pragma unroll
        for (int j = 0; j < FN; ++j) wf[j][i >> 1] = o[j];
      }
    } else {
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        const int row = wn * T::TN + 16 * n + r;
        const uint32_t c = *reinterpret_cast<const uint32_t*>(bw + row * T::kWPitch + 8 * g + 4 * t);
        const uint32_t s = bs[row * T::kSPitch + (FMT == 0 ? g >> 1 : g)];
        wf[n] = weights8<FMT>(c, scale_operand<FMT>(s), power);
      }
    }
    // this lane's 8 of the contraction: chunk 4 t + g where groups take runs of
    // 8 (transposed), 2 g + t where they take runs of 16
    const int chunk = T::kT ? 4 * t + g : 2 * g + t;
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const int row = wm * T::TM + 16 * m + r;
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const u32x4_t xf = *reinterpret_cast<const u32x4_t*>(buf + (p * BM + row) * 128 + x_chunk(row, chunk) * 16);
#pragma unroll
        for (int n = 0; n < FN; ++n) acc[n][m] = mfma16(wf[n], xf, acc[n][m]);
      }
    }
  }
}

// The sums to where they belong: outputs, or parts of sums.
template <class T, int FMT, int MODE>
__device__ __forceinline__ void many_results(const ManyArgs& a, const f32x4_t (&acc)[T::FN][T::FM], int64_t m0, int64_t o0,
                                             int wm, int wn, int r, int g) {
  constexpr int FM = T::FM, FN = T::FN;
  const LinearLaunch& l = a.l;
  const int64_t K = l.w.k, half = l.w.n / 2;
  const int64_t cols = T::kT ? K : l.w.n;               // of the sums
  // 4 consecutive outputs, or the first `count`
  auto put4 = [&](void* to, int64_t at, f32x4_t v, int count, int bf16) {
    if (bf16) {
      __bf16* o = static_cast<__bf16*>(to) + at;
      if (count >= 4) {
        store_any(o, u32x2_t{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)});
      } else {
        for (int i = 0; i < count; ++i) o[i] = (__bf16)v[i];
      }
    } else {
      float* o = static_cast<float*>(to) + at;
      if (count >= 4) {
        store_any(o, v);
      } else {
        for (int i = 0; i < count; ++i) o[i] = v[i];
      }
    }
  };
  const float tensor = FMT == 1 ? tensor_rest(tensor_scale(l.w.g)) : 1.0f;
#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int64_t row = m0 + wm * T::TM + 16 * m + r;
    if (row >= l.rows) continue;
    if constexpr (T::kT) {
      // columns FN (4 g + i) + j of the wave's: 4 FN consecutive ones a lane, by fours
#pragma unroll
      for (int q = 0; q < FN; ++q) {
        const int64_t k = o0 + wn * T::TN + FN * 4 * g + 4 * q;
        if (k >= K) continue;                           // (K is a multiple of 8)
        const f32x4_t v = {acc[(4 * q) % FN][m][4 * q / FN], acc[(4 * q + 1) % FN][m][(4 * q + 1) / FN],
                           acc[(4 * q + 2) % FN][m][(4 * q + 2) / FN], acc[(4 * q + 3) % FN][m][(4 * q + 3) / FN]};
        if (a.splits > 1) store_any(l.partials + ((int64_t)blockIdx.y * l.rows + row) * cols + k, v);
        else put4(l.out, row * K + k, v * tensor, 4, l.out_bf16);
      }
    } else {
#pragma unroll
      for (int n = 0; n < (MODE == kGated ? FN / 2 : FN); ++n) {
        const int64_t side = MODE == kGated ? half : l.w.n;
        const int64_t col = o0 + wn * (MODE == kGated ? T::TN / 2 : T::TN) + 16 * n + 4 * g;
        const int count = (int)min(side - col, (int64_t)4);
        if (count <= 0) continue;
        f32x4_t v = acc[n][m], u = acc[MODE == kGated ? n + FN / 2 : n][m];
        if (a.splits > 1) {
          float* o = l.partials + ((int64_t)blockIdx.y * l.rows + row) * cols + col;
          for (int i = 0; i < count; ++i) o[i] = v[i];
          if constexpr (MODE == kGated)
            for (int i = 0; i < count; ++i) o[half + i] = u[i];
          continue;
        }
        v *= tensor;
        if constexpr (MODE == kGated) {
          u *= tensor;
          if (l.products) {
            put4(l.products, row * l.w.n + col, v, count, l.products_bf16);
            put4(l.products, row * l.w.n + half + col, u, count, l.products_bf16);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
          put4(l.out, row * half + col, v, count, l.out_bf16);
        } else {
          if (l.bias) {
            for (int i = 0; i < count; ++i)
              v[i] += l.out_bf16 ? (float)static_cast<const __bf16*>(l.bias)[col + i]
                                 : static_cast<const float*>(l.bias)[col + i];
          }
          put4(l.out, row * l.w.n + col, v, count, l.out_bf16);
        }
      }
    }
  }
}

template <int FMT, int XT, int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void many_kernel(ManyArgs a) {
  using T = ManyTile<FMT, XT, MODE, BM, BN, WM, WN>;
  constexpr int kElem = XT == kXF32 ? 4 : XT == kXBF16 ? 2 : 1;
  constexpr int P = T::P, FM = T::FM, FN = T::FN;
  __shared__ __align__(16) uint8_t s_buf[2][T::kBuf];
  const LinearLaunch& l = a.l;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;

  // workgroup w runs on XCD w mod 8: each XCD walks a contiguous range of tiles,
  // in groups of 4 tile rows column by column, so that its L2 serves both sides
  const int w = blockIdx.x, per = (a.ntiles + 7) / 8;
  const int tile = (w % 8) * per + w / 8;
  if (tile >= a.ntiles || w / 8 >= per) return;
  const int group = tile / (4 * a.tiles_n), first = group * 4;
  const int gsize = min(a.tiles_m - first, 4), in_g = tile - group * 4 * a.tiles_n;
  const int64_t m0 = (int64_t)(first + in_g % gsize) * BM;
  const int64_t half = l.w.n / 2;
  const int64_t o0 = (int64_t)(in_g / gsize) * (MODE == kGated ? BN / 2 : BN);   // first output column

  const int64_t K = l.w.k, srow = K / T::kBlock;
  const int64_t len = T::kT ? l.w.n : K;                // of the contraction
  const int s0 = blockIdx.y * a.per_split, s1 = min(a.stages, s0 + a.per_split);
  const float power = FMT == 1 ? tensor_power(tensor_scale(l.w.g)) : 1.0f;

  // ---- loads of a stage: global memory to registers, registers to LDS
  uint32_t xr[T::kXPer][XT == kXF32 ? 8 : XT == kXBF16 ? 4 : 3];
  u32x4_t wr[T::kWPer];
  uint32_t wsr[T::kWPer];
  auto load_x = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < T::kXPer; ++i) {
      const int q = tid + i * T::kThreads, row = q >> 3;
      const int64_t kk = at + (q & 7) * 8, m = min(m0 + row, l.rows - 1);
      const uint8_t* p = static_cast<const uint8_t*>(l.x) + (m * l.x_stride + kk) * kElem;
      if (kk + 8 <= len) {
        if constexpr (XT == kXF32) {
          const u32x4_t v = load_any<u32x4_t>(p), u = load_any<u32x4_t>(p + 16);
          xr[i][0] = v.x; xr[i][1] = v.y; xr[i][2] = v.z; xr[i][3] = v.w;
          xr[i][4] = u.x; xr[i][5] = u.y; xr[i][6] = u.z; xr[i][7] = u.w;
        } else if constexpr (XT == kXBF16) {
          const u32x4_t v = load_any<u32x4_t>(p);
          xr[i][0] = v.x; xr[i][1] = v.y; xr[i][2] = v.z; xr[i][3] = v.w;
        } else {
          const u32x2_t v = load_any<u32x2_t>(p);
          xr[i][0] = v.x; xr[i][1] = v.y;
          xr[i][2] = l.x_scales[m * (K / 32) + (kk >> 5)];
        }
      } else {   // the end of a row; only rows of gradients end inside a piece
#pragma unroll
        for (int e = 0; e < (XT == kXF32 ? 8 : XT == kXBF16 ? 4 : 3); ++e) xr[i][e] = 0u;
        if constexpr (XT == kXF32) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (kk + e < len) xr[i][e] = load_any<uint32_t>(p + 4 * e);
        } else if constexpr (XT == kXBF16) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (kk + e < len) xr[i][e >> 1] |= (uint32_t)load_any<uint16_t>(p + 2 * e) << (16 * (e & 1));
        }
      }
    }
  };
  auto load_w = [&](int64_t at) {
#pragma unroll
    for (int i = 0; i < T::kWPer; ++i) {
      const int q = tid + i * T::kThreads;
      wr[i] = u32x4_t{0u, 0u, 0u, 0u};
      wsr[i] = 0u;
      int64_t n, k;
      if constexpr (T::kT) {
        n = at + q / (BN / 32);
        k = o0 + (q % (BN / 32)) * 32;
        if (n >= l.w.n) continue;                       // rows that the contraction does not have
      } else {
        const int row = q >> 1;
        k = at + (q & 1) * 32;
        if constexpr (MODE == kGated) {
          const int f = (row % T::TN) / 16;
          n = min(o0 + (row / T::TN) * (T::TN / 2) + (f % (FN / 2)) * 16 + (row & 15), half - 1) + (f >= FN / 2 ? half : 0);
        } else {
          n = min(o0 + row, l.w.n - 1);
        }
      }
      const uint8_t* c = l.w.codes + n * (K / 2) + (k >> 1);
      const uint8_t* s = l.w.scales + n * srow + k / T::kBlock;
      if (k + 32 <= K) {
        wr[i] = load_any<u32x4_t>(c);
        wsr[i] = FMT == 0 ? *s : load_any<uint16_t>(s);
      } else if (FMT == 1 && k + 16 <= K) {
        const u32x2_t v = load_any<u32x2_t>(c);
        wr[i].x = v.x;
        wr[i].y = v.y;
        wsr[i] = *s;
      }
    }
  };
  auto commit = [&](uint8_t* buf) {
    uint8_t* bw = buf + T::kXBytes;
    uint8_t* bs = bw + T::kWBytes;
#pragma unroll
    for (int i = 0; i < T::kXPer; ++i) {
      const int q = tid + i * T::kThreads, row = q >> 3, ch = x_chunk(row, q & 7);
      u32x4_t o[P];
      if constexpr (XT == kXF32) split8(xr[i], o);
      else if constexpr (XT == kXBF16) o[0] = u32x4_t{xr[i][0], xr[i][1], xr[i][2], xr[i][3]};
      else o[0] = e4m3_values8(u32x2_t{xr[i][0], xr[i][1]}, xr[i][2]);
#pragma unroll
      for (int p = 0; p < P; ++p) *reinterpret_cast<u32x4_t*>(buf + (p * BM + row) * 128 + ch * 16) = o[p];
    }
#pragma unroll
    for (int i = 0; i < T::kWPer; ++i) {
      const int q = tid + i * T::kThreads;
      if constexpr (T::kT) {
        const int n = q / (BN / 32), pc = q % (BN / 32);
        *reinterpret_cast<u32x4_t*>(bw + n * T::kWPitch + (n >> 3) * 64 + pc * 16) = wr[i];
        if constexpr (FMT == 0) {
          bs[pc * T::kSPitch + n] = (uint8_t)wsr[i];
        } else {
          bs[2 * pc * T::kSPitch + n] = (uint8_t)wsr[i];
          bs[(2 * pc + 1) * T::kSPitch + n] = (uint8_t)(wsr[i] >> 8);
        }
      } else {
        *reinterpret_cast<u32x4_t*>(bw + q * 16) = wr[i];
        if constexpr (FMT == 0) bs[q] = (uint8_t)wsr[i];
        else *reinterpret_cast<uint16_t*>(bs + 2 * q) = (uint16_t)wsr[i];
      }
    }
  };

  f32x4_t acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  if (s0 < s1) {
    load_x((int64_t)s0 * kStage);
    load_w((int64_t)s0 * kStage);
    commit(s_buf[0]);
    __syncthreads();
    for (int s = s0; s < s1; ++s) {
      const int b = (s - s0) & 1;
      if (s + 1 < s1) {
        load_x((int64_t)(s + 1) * kStage);
        load_w((int64_t)(s + 1) * kStage);
      }
      many_multiply<T, FMT>(s_buf[b], acc, wm, wn, r, g, power);
      if (s + 1 < s1) commit(s_buf[b ^ 1]);
      __syncthreads();
    }
  }

  many_results<T, FMT, MODE>(a, acc, m0, o0, wm, wn, r, g);
}

// ----------------------------------------------------------------------------
// The same tile for bf16 rows that are whole 16-byte pieces and stages.  x and
// codes go straight into LDS, into a ring of three buffers, two stages ahead.
// NW = 4: waves as above, two workgroups on a CU.  NW = 8: four waves side by side
// twice, each four with one half of a stage's contraction, so that every SIMD has
// two waves on one tile and still no code is converted twice; at the end the two
// fours exchange halves of their rows' sums.  Measured, k and n 8192, us, NVFP4 /
// MXFP4 (at 1024 rows there is a tile a CU, at 2048 two):
//   rows   direction    many_kernel   NW = 4      NW = 8
//   1024   forward      182 / 155     206 / 144   138 / 129
//   2048   forward      282 / 244     282 / 235   273 / 251
//   1024   gradient     196 / 178     207 / 188   137 / 120
//   2048   gradient     272 / 248     236 / 218   271 / 236
// so four waves where every CU has two workgroups.  (NVFP4 forward has not the
// registers for that: its eight scales a lane spill.)  The conversion bounds it: a
// wave's 8 codes cost 4 conversions, 8 multiplications (NVFP4) and 4 joins of bf16
// pairs for the 8 matrix instructions (64 of the matrix unit's clocks) that use them.
typedef __attribute__((address_space(3))) void lds_void_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const uint8_t* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), (short)0,
                                           (int)(bytes < 0x7FFFFFFF ? bytes : 0x7FFFFFFF), 0x00020000);
}
// Until at most N loads are on their way, and every LDS access is done.
template <int N>
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

template <int FMT, int MODE, int NW>
__global__ __launch_bounds__(64 * NW, 2) void ring_kernel(ManyArgs a) {
  constexpr int BM = 128, BN = 256;
  static_assert(BN / 2 == kRingFactorRows, "what ring_scales_fit counts");
  using T = ManyTile<FMT, kXBF16, MODE, BM, BN, 1, 4>;
  constexpr int XL = 16 / NW, WL = 8 / NW;                      // a wave's loads of a stage
  // separate objects, so that reads of one are not ordered after loads into others
  __shared__ __align__(16) uint8_t s_b0[T::kBuf];
  __shared__ __align__(16) uint8_t s_b1[T::kBuf];
  __shared__ __align__(16) uint8_t s_b2[T::kBuf];
  const LinearLaunch& l = a.l;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, wn = wave & 3, part = wave >> 2;

  const int w = blockIdx.x, per = (a.ntiles + 7) / 8;
  const int tile = (w % 8) * per + w / 8;
  if (tile >= a.ntiles || w / 8 >= per) return;
  const int group = tile / (4 * a.tiles_n), first = group * 4;
  const int gsize = min(a.tiles_m - first, 4), in_g = tile - group * 4 * a.tiles_n;
  const int64_t m0 = (int64_t)(first + in_g % gsize) * BM;
  const int64_t half = l.w.n / 2;
  const int64_t o0 = (int64_t)(in_g / gsize) * (MODE == kGated ? BN / 2 : BN);
  const int64_t K = l.w.k, kb = K / 2, srow = K / T::kBlock;
  const int s0 = blockIdx.y * a.per_split, s1 = min(a.stages, s0 + a.per_split);
  const float power = FMT == 1 ? tensor_power(tensor_scale(l.w.g)) : 1.0f;

  f32x4_t acc[T::FN][T::FM];
#pragma unroll
  for (int n = 0; n < T::FN; ++n)
#pragma unroll
    for (int m = 0; m < T::FM; ++m) acc[n][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // Offsets within a tile are below 2^31 (rows of at most 2^22 elements); rows past
  // the ends read the last one, columns past the end what lies there (zeros past
  // the plane's), and their results are not stored.
  const uint8_t* x = static_cast<const uint8_t*>(l.x) + m0 * l.x_stride * 2;
  int x_off[4], w_off[2];                           // XL and WL of them
#pragma unroll
  for (int i = 0; i < XL; ++i) {                    // 8 rows of x a load, 128 bytes each
    const int row = (wave * XL + i) * 8 + (lane >> 3);
    x_off[i] = (int)((min(m0 + row, l.rows - 1) - m0) * l.x_stride * 2) + x_chunk(row, lane & 7) * 16;
  }
  // row of the weight that local row i is (of the forward directions), from its side's first
  auto w_row = [&](int i) {
    if constexpr (MODE == kGated) return min(o0 + (i >> 6) * 32 + (i & 31), half - 1) - o0;
    else return min(o0 + i, l.w.n - 1) - o0;
  };
  auto w_side = [&](int i) { return MODE == kGated && (i & 32) ? o0 + half : o0; };
  // 32 rows' 32 bytes a load, or 8 rows' 128
#pragma unroll
  for (int i = 0; i < WL; ++i) {
    if constexpr (T::kT) w_off[i] = (int)(((wave * WL + i) * 8 + (lane >> 3)) * kb) + (lane & 7) * 16;
    else w_off[i] = (int)(w_row((wave * WL + i) * 32 + (lane >> 1)) * kb) + (lane & 1) * 16;
  }
  auto issue = [&](int st, uint8_t* buf) {
    const __amdgpu_buffer_rsrc_t xb = buffer_of(x + (int64_t)st * (kStage * 2), 0x7FFFFFFF);
#pragma unroll
    for (int i = 0; i < XL; ++i)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(xb, (lds_void_t*)(buf + (wave * XL + i) * 1024), 16, x_off[i], 0, 0, 0);
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int piece = wave * WL + i;
      const int64_t at = T::kT ? (int64_t)st * kStage * kb + o0 / 2 : w_side(piece * 32) * kb + (int64_t)st * (kStage / 2);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(l.w.codes + at, l.w.n * kb - at),
                                               (lds_void_t*)(buf + T::kXBytes + piece * (T::kT ? 1024 + 64 : 1024)), 16,
                                               w_off[i], 0, 0, 0);
    }
  };
  // Scales go through a register: a thread has a row's, or a half of them, and
  // transposed a fourth or an eighth, which it puts to the places of their blocks.
  constexpr int kBlocks = T::kT ? BN / T::kBlock : kStage / T::kBlock;          // a row's in a stage
  constexpr int kThreadsRow = T::kT ? NW : NW / 4;
  constexpr int kHave = kBlocks / kThreadsRow;                                  // 1, 2 or 4 bytes
  using scale_t = typename std::conditional<kHave == 1, uint8_t,
                                            typename std::conditional<kHave == 2, uint16_t, uint32_t>::type>::type;
  const int s_row = tid / kThreadsRow, s_col = tid % kThreadsRow * kHave;
  int s_off;                                        // from the tile's first scale (transposed: the stage's)
  if constexpr (T::kT) {
    // (K is a multiple of 64: all are there or none, and then the row's first ones stand in)
    s_off = s_row * (int)srow + (o0 / T::kBlock + s_col < srow ? s_col : 0);
  } else {
    s_off = (int)((w_side(s_row) - o0 + w_row(s_row)) * srow) + s_col;
  }
  auto load_scales = [&](int st) {
    const uint8_t* p = l.w.scales + (T::kT ? (int64_t)st * kStage * srow + o0 / T::kBlock
                                           : o0 * srow + (int64_t)st * (kStage / T::kBlock));
    return (uint32_t)load_any<scale_t>(p + s_off);
  };
  auto store_scales = [&](uint8_t* buf, uint32_t v) {
    uint8_t* bs = buf + T::kXBytes + T::kWBytes;
    if constexpr (T::kT) {
#pragma unroll
      for (int i = 0; i < kHave; ++i) bs[(s_col + i) * T::kSPitch + s_row] = (uint8_t)(v >> (8 * i));
    } else {
      *reinterpret_cast<scale_t*>(bs + tid * kHave) = (scale_t)v;
    }
  };
  // As the block-scaled kernel's step: wait until only the loads of the step before
  // are on their way, which are the next stage's, meet, ask for the stage after the
  // next, which goes where the one before lay, and multiply.  Scales are written
  // there before: beside a stage that is on its way the write would wait for it.
  // They are asked for three steps ahead, each position of the ring's into a register
  // of its own, and first in their step, so that nothing waits for them.  The order of
  // loads is fixed, and there is no branch, so that all counts are exact; after the
  // loop nobody takes the scales that are asked for, the compiler leaves those loads
  // out, and a step has one less on its way.
  auto step = [&](int st, const uint8_t* cur, uint8_t* fill, uint32_t& sc, auto looped) {
    wait_loads<XL + WL + (decltype(looped)::value ? 1 : 0)>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    store_scales(fill, sc);
    sc = load_scales(min(st + 5, s1 - 1));
    __builtin_amdgcn_sched_barrier(0);
    issue(min(st + 2, s1 - 1), fill);
    __builtin_amdgcn_sched_barrier(0);
    // (the lane's part of the addresses is made anew each time: kept for three
    // buffers, it would take more registers than there are)
    int rr = r, gg = g;
    asm volatile("" : "+v"(rr), "+v"(gg));
    if constexpr (NW == 8) {
      many_multiply<T, FMT>(cur, acc, 0, wn, rr, gg, power, part);
    } else {
      many_multiply<T, FMT>(cur, acc, 0, wn, rr, gg, power, 0);
      __builtin_amdgcn_sched_barrier(0);            // (or both halves' operands would be held at once)
      many_multiply<T, FMT>(cur, acc, 0, wn, rr, gg, power, 1);
    }
  };
  if (s0 < s1) {
    store_scales(s_b0, load_scales(s0));
    store_scales(s_b1, load_scales(min(s0 + 1, s1 - 1)));
    uint32_t sc0 = load_scales(min(s0 + 2, s1 - 1)), sc1 = load_scales(min(s0 + 3, s1 - 1));
    __builtin_amdgcn_sched_barrier(0);
    issue(s0, s_b0);
    __builtin_amdgcn_sched_barrier(0);
    uint32_t sc2 = load_scales(min(s0 + 4, s1 - 1));
    __builtin_amdgcn_sched_barrier(0);
    issue(min(s0 + 1, s1 - 1), s_b1);
    const std::true_type looped;
    const std::false_type last;
    int st = s0;
    for (; st + 3 <= s1; st += 3) {
      step(st, s_b0, s_b2, sc0, looped);
      step(st + 1, s_b1, s_b0, sc1, looped);
      step(st + 2, s_b2, s_b1, sc2, looped);
    }
    if (st < s1) step(st, s_b0, s_b2, sc0, last);
    if (st + 1 < s1) step(st + 1, s_b1, s_b0, sc1, last);
  }

  wait_loads<0>();                                  // (the last stage, asked for again, is on its way to the ring)
  if constexpr (NW == 4) {
    many_results<T, FMT, MODE>(a, acc, m0, o0, 0, wn, r, g);
  } else {
    // The first four waves take rows 0 to 63, the others 64 to 127: each gives the
    // other its sums of them, 8 KiB at a time.
    using H = ManyTile<FMT, kXBF16, MODE, BM / 2, BN, 1, 4>;
    f32x4_t mine[H::FN][H::FM];
    auto region = [&](int i) {
      uint8_t* buf = i < 3 ? s_b0 : i < 6 ? s_b1 : s_b2;
      return reinterpret_cast<f32x4_t*>(buf + i % 3 * 8192) + lane;
    };
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < T::FN; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          region(wave)[(n * 2 + m) * 64] = part ? acc[n][2 * q + m] : acc[n][4 + 2 * q + m];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < T::FN; ++n)
#pragma unroll
        for (int m = 0; m < 2; ++m)
          mine[n][2 * q + m] = (part ? acc[n][4 + 2 * q + m] : acc[n][2 * q + m]) + region(wave ^ 4)[(n * 2 + m) * 64];
    }
    many_results<H, FMT, MODE>(a, mine, m0 + 64 * part, o0, 0, wn, r, g);
  }
}

// Whether rows are whole stages and offsets small enough, and whether the pieces of
// them are aligned.  (Parts of the contraction go by the sizes alone, and rows whose
// pieces lie between words then go through many_kernel in the same parts.)
inline bool ring_sizes(const LinearLaunch& l) {
  return l.x_type == kXBF16 && l.w.k > 0 && l.w.k % kStage == 0 && l.w.n % (l.transposed ? kStage : 1) == 0 &&
         l.w.k <= 1 << 22 && ring_scales_fit(l.gated, l.w.n, l.w.k);
}
inline bool ring_fits(const LinearLaunch& l) {
  return ring_sizes(l) && l.x_stride % 8 == 0 && l.x_stride <= 1 << 22 && reinterpret_cast<uintptr_t>(l.x) % 16 == 0 &&
         reinterpret_cast<uintptr_t>(l.w.codes) % 16 == 0;
}

template <int FMT, int MODE, int NW>
hipError_t launch_ring(const ManyArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((ring_kernel<FMT, MODE, NW>), dim3((a.ntiles + 7) / 8 * 8, a.splits), dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

template <int FMT, int XT, int MODE, int BM, int BN, int WM, int WN>
hipError_t launch_many_t(const ManyArgs& a, hipStream_t s) {
  using T = ManyTile<FMT, XT, MODE, BM, BN, WM, WN>;
  hipLaunchKernelGGL((many_kernel<FMT, XT, MODE, BM, BN, WM, WN>), dim3((a.ntiles + 7) / 8 * 8, a.splits),
                     dim3(T::kThreads), 0, s, a);
  return hipGetLastError();
}

// Instances, by format and direction (fp4q_linear_many_*.hip); `size`: 0 the
// small tiles, 1 the large ones.
struct ManySize {
  int bm, bn;
};
hipError_t launch_many_mx(const ManyArgs& a, int size, hipStream_t s);
hipError_t launch_many_nv(const ManyArgs& a, int size, hipStream_t s);
hipError_t launch_many_back_mx(const ManyArgs& a, int size, hipStream_t s);
hipError_t launch_many_back_nv(const ManyArgs& a, int size, hipStream_t s);
hipError_t launch_mx8(const ManyArgs& a, hipStream_t s);   // tiles of 256 x 256

// Tiles: large ones where there are enough of them.  fp32 activations take three
// times the LDS and half the rows.
constexpr ManySize many_size(int x_type, int size) {
  return size == 0 ? ManySize{64, 128} : x_type == kXF32 ? ManySize{64, 256} : ManySize{128, 256};
}

template <int FMT, int XT, int MODE>
hipError_t launch_many_size(const ManyArgs& a, int size, hipStream_t s) {
  if (size == 0) return launch_many_t<FMT, XT, MODE, 64, 128, 1, 4>(a, s);
  constexpr int BM = many_size(XT, 1).bm;
  if constexpr (XT == kXBF16) {
    if (ring_fits(a.l)) {
      if constexpr (FMT == 0 || MODE == kTransposed) {
        if ((int64_t)a.ntiles * a.splits >= 2 * device_cu_count()) return launch_ring<FMT, MODE, 4>(a, s);
      }
      return launch_ring<FMT, MODE, 8>(a, s);
    }
  }
  return launch_many_t<FMT, XT, MODE, BM, 256, 1, 4>(a, s);
}

}  // namespace fp4q
