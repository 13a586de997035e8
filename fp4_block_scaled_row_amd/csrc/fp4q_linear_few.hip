// fp4q_linear_few.hip -- y = x W^T and h = SiLU(x Wg^T) * (x Wu^T) for few rows
// of x: a stream over the 4-bit weight.
//
// A workgroup of 8 waves takes 16 NT rows of the weight (a gated call half of
// them from each factor) and all rows of x.  Chunks of CH k go round the waves, so
// that together they read 4 CH contiguous bytes of each row, D chunks a wave in
// flight; the waves' sums meet in LDS.  Nothing crosses workgroups, so the order
// of sums is fixed.
//
// Codes are loaded as they lie, neighbouring lanes 16 neighbouring bytes (whole
// 128-byte lines of 8 rows with CH 256), and change lanes through a scratch of
// the wave's own in LDS.  Loaded into the lanes that multiply them, 16 rows over
// neighbouring lanes, they cost the load unit a lookup a lane: 16 bytes a clock
// and CU, which bounded calls of 17 rows and more.
//
// x goes to LDS as bf16 (fp32 as three planes of pieces, MXFP8 as its values).
// Short and few rows all lie there, converted once a workgroup (WHOLE).  Else each
// wave brings its own chunk of all rows, as it does its codes, with D chunks of
// both in flight and no barrier: no other wave of the workgroup needs it.  (With
// parts of x that all waves waited for, 24 rows of k 8192 by n 8192 took 20.9 us.)
// Reading x in the lanes that multiply it took the load unit's time too: a load of
// 16 bytes a lane costs it 16 clocks at least even where all lanes want one line.
// Workgroups of an XCD begin at different chunks: rows are often a power of two
// apart, and what all of them read at once would lie in few of the L2's channels
// (28.3 us for 20.9 there).
//
// v_mfma_f32_16x16x32_bf16 with weights as the left operand: lane l holds row l
// mod 16 and k = 32 (l / 16) .. + 31 of each 128 of a chunk, 16 bytes of codes,
// which four instructions take eight at a time; x is read from LDS in the same
// order.  The result has 4 consecutive weight rows of one x row in a lane.
#include "fp4q_ffn.h"

namespace fp4q {
namespace {

constexpr int kFewWaves = 8;
constexpr int kFewThreads = 64 * kFewWaves;

// Eight elements of x on their way from memory to LDS.
template <int XT>
struct XPiece {
  uint32_t w[XT == kXF32 ? 8 : XT == kXBF16 ? 4 : 3];
};

// The piece at element `at` of x; MXFP8's scale is byte `scale_at`.
template <int XT>
__device__ __forceinline__ void load_piece(const LinearLaunch& l, int64_t at, int64_t scale_at, XPiece<XT>& d) {
  if constexpr (XT == kXE4M3) {
    const u32x2_t v = load_any<u32x2_t>(static_cast<const uint8_t*>(l.x) + at);
    d.w[0] = v.x;
    d.w[1] = v.y;
    d.w[2] = l.x_scales[scale_at];
  } else {
    const uint8_t* p = static_cast<const uint8_t*>(l.x) + at * (XT == kXF32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < (int)(sizeof(d.w) / 4); i += 4) {
      const u32x4_t v = load_any<u32x4_t>(p + 4 * i);
      d.w[i] = v.x; d.w[i + 1] = v.y; d.w[i + 2] = v.z; d.w[i + 3] = v.w;
    }
  }
}
template <int XT>
__device__ __forceinline__ void no_piece(XPiece<XT>& d) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(d.w) / 4); ++i) d.w[i] = 0u;
}

// ... and into LDS: planes `plane` bytes apart.
template <int XT>
__device__ __forceinline__ void store_piece(const XPiece<XT>& d, uint8_t* to, int plane) {
  u32x4_t o[kPieces<XT>];
  if constexpr (XT == kXF32) split8(d.w, o);
  else if constexpr (XT == kXBF16) o[0] = u32x4_t{d.w[0], d.w[1], d.w[2], d.w[3]};
  else o[0] = e4m3_values8(u32x2_t{d.w[0], d.w[1]}, d.w[2]);
#pragma unroll
  for (int p = 0; p < kPieces<XT>; ++p) *reinterpret_cast<u32x4_t*>(to + p * plane) = o[p];
}

// What a wave has in flight of a chunk.  Codes: CH / 32 lanes hold a row's, 16
// bytes each, a load takes 2048 / CH rows; four lanes hold a row's scales.  x
// (XR rows, 0 where LDS has it whole): CH / 8 lanes hold a row's.
template <int FMT, int XT, int CH, int NT, int XR>
struct FewRing {
  static constexpr int kRowScales = CH / (FMT == 0 ? 32 : 16);        // bytes
  static constexpr int kXLoads = XR * (CH / 8) / 64;
  u32x4_t c[NT][CH / 128];
  uint32_t s[NT];
  XPiece<XT> x[kXLoads > 0 ? kXLoads : 1];
};

// Scratch of a wave: a tile's codes, rows of CH / 2 bytes whose 16-byte pieces are
// exchanged so that 16 rows' reads of one piece meet all banks, and its scales.
template <int CH>
constexpr int kScratch = 16 * CH / 2 + 256;
template <int CH>
__device__ __forceinline__ int scratch_at(int row, int piece) {
  return row * (CH / 2) + (piece ^ (CH == 256 ? row >> 1 : row >> 2)) * 16;
}
// What a wave's lanes wrote to LDS before is what they read after (they execute
// together: only the compiler has to keep the order).
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Codes are read once.  Whole lines are not kept in the caches (k 28672 by n 8192,
// one row: 23.7 us for 27.3); a line that two waves take half of each is, for the
// second one (24 rows of k 8192 by n 8192: 14.9 us for 17.4).
typedef u32x4_t u32x4_any_t __attribute__((aligned(1)));
template <int CH>
__device__ __forceinline__ u32x4_t load_codes(const uint8_t* p) {
  if constexpr (CH == 256) return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any_t*>(p));
  else return load_any<u32x4_t>(p);
}

// `B` bytes (1, 2 or 4) as a word.
template <int B>
__device__ __forceinline__ uint32_t load_small(const uint8_t* p) {
  if constexpr (B == 1) return *p;
  else if constexpr (B == 2) return load_any<uint16_t>(p);
  else return load_any<uint32_t>(p);
}

// Where in LDS the waves' scratch begins: behind x (WHOLE).
struct FewArgs {
  LinearLaunch l;
  int log_kp, scratch;         // WHOLE: x lies in rows of 2^log_kp elements
};

template <int FMT, int XT, int MT, int NT, int CH, int D, bool GATED, bool WHOLE>
__global__ __launch_bounds__(kFewThreads) void few_kernel(FewArgs a) {
  constexpr int kHalves = GATED ? 2 : 1;
  constexpr int kSide = NT / kHalves;            // tiles of each factor
  constexpr int P = kPieces<XT>;
  constexpr int kScales = CH / (FMT == 0 ? 32 : 16);
  constexpr int XR = WHOLE ? 0 : 16 * MT;
  extern __shared__ __align__(16) uint8_t s_x[];
  const LinearLaunch& l = a.l;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t K = l.w.k, half = l.w.n / kHalves;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kSide);
  const int64_t srow = K / (FMT == 0 ? 32 : 16);
  const int rows = (int)l.rows;

  // ---- x in LDS: rows of `pitch` bytes (16 rows' pieces meet all banks), planes
  constexpr int kChunkPitch = 2 * CH + 16;
  const int kp = WHOLE ? 1 << a.log_kp : CH;
  const int pitch = WHOLE ? 2 * kp + 16 : kChunkPitch, plane = WHOLE ? rows * pitch : XR * kChunkPitch;
  uint8_t* xs = WHOLE ? s_x : s_x + a.scratch + wave * (kScratch<CH> + P * XR * kChunkPitch) + kScratch<CH>;

  // ---- weights; rows past the end read the last one, and their results are not stored
  using Ring = FewRing<FMT, XT, CH, NT, XR>;
  constexpr int kLoads = CH / 128, kLanes = CH / 32, kLane = Ring::kRowScales / 4;   // (scale bytes a lane)
  uint8_t* scratch = s_x + a.scratch + wave * (kScratch<CH> + P * XR * kChunkPitch);
  const int piece_at = lane % kLanes;
  const uint8_t *wc[NT][kLoads], *ws[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    auto row = [&](int i) { return min(n0 + 16 * (t % kSide) + i, half - 1) + (t / kSide) * half; };
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      wc[t][i] = l.w.codes + row(lane / kLanes + i * (64 / kLanes)) * (K / 2) + 16 * piece_at;
    ws[t] = l.w.scales + row(lane >> 2) * srow + (lane & 3) * kLane;
  }
  // this lane's piece of a row of x, and the rows that it loads; rows past the last read it
  constexpr int kXLanes = CH / 8;
  const int x_piece = lane % kXLanes;
  int64_t x_at[Ring::kXLoads > 0 ? Ring::kXLoads : 1];
  auto x_row = [&](int i) { return min((int64_t)(i * (64 / kXLanes) + lane / kXLanes), l.rows - 1); };
#pragma unroll
  for (int i = 0; i < Ring::kXLoads; ++i) x_at[i] = x_row(i) * l.x_stride + 8 * x_piece;
  auto x_scale = [&](int i, int64_t k) { return XT == kXE4M3 ? x_row(i) * (K / 32) + (k >> 5) : 0; };

  const int whole = (int)(K / CH), chunks = (int)((K + CH - 1) / CH);
  auto load = [&](int c, Ring& d) {           // a whole chunk
#pragma unroll
    for (int i = 0; i < Ring::kXLoads; ++i)
      load_piece<XT>(l, x_at[i] + (int64_t)c * CH, x_scale(i, (int64_t)c * CH + 8 * x_piece), d.x[i]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) d.c[t][i] = load_codes<CH>(wc[t][i] + (int64_t)c * (CH / 2));
      d.s[t] = load_small<kLane>(ws[t] + (int64_t)c * kScales);
    }
  };
  auto load_end = [&](int c, Ring& d) {       // the chunk that the rows end in, zeros behind them
#pragma unroll
    for (int i = 0; i < Ring::kXLoads; ++i) {
      const int64_t k = (int64_t)c * CH + 8 * x_piece;             // (K is a multiple of 8)
      if (k < K) load_piece<XT>(l, x_at[i] + (int64_t)c * CH, x_scale(i, k), d.x[i]);
      else no_piece<XT>(d.x[i]);
    }
    const int64_t k0 = (int64_t)c * CH, v = K - k0 - 32 * piece_at;    // v: what this lane's 32 codes have of them
    const int have = (int)(K - k0) / (FMT == 0 ? 32 : 16) - (lane & 3) * kLane;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        d.c[t][i] = u32x4_t{0u, 0u, 0u, 0u};
        const uint8_t* p = wc[t][i] + k0 / 2;
        if (v >= 32) {
          d.c[t][i] = load_any<u32x4_t>(p);
        } else if (v >= 16) {
          const u32x2_t w = load_any<u32x2_t>(p);
          d.c[t][i].x = w.x;
          d.c[t][i].y = w.y;
        }
      }
      d.s[t] = 0u;
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (i < have) d.s[t] |= (uint32_t)ws[t][(int64_t)c * kScales + i] << (8 * i);
    }
  };
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  int xrow[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) xrow[m] = (WHOLE ? min(16 * m + r, rows - 1) : 16 * m + r) * pitch + 64 * g;
  auto multiply = [&](int c, const Ring& d) {
    // from the lanes that loaded them to those that multiply them
#pragma unroll
    for (int i = 0; i < Ring::kXLoads; ++i)
      store_piece<XT>(d.x[i], xs + (i * (64 / kXLanes) + lane / kXLanes) * pitch + 16 * x_piece, plane);
    u32x4_t wv[NT][kLoads];
    uint32_t sv[NT][kLoads];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        *reinterpret_cast<u32x4_t*>(scratch + scratch_at<CH>(lane / kLanes + i * (64 / kLanes), piece_at)) = d.c[t][i];
      uint8_t* ss = scratch + 16 * CH / 2;
      if constexpr (kLane == 1) ss[lane] = (uint8_t)d.s[t];
      else if constexpr (kLane == 2) *reinterpret_cast<uint16_t*>(ss + 2 * lane) = (uint16_t)d.s[t];
      else *reinterpret_cast<uint32_t*>(ss + 4 * lane) = d.s[t];
      wave_order();
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        wv[t][i] = *reinterpret_cast<const u32x4_t*>(scratch + scratch_at<CH>(r, 4 * i + g));
      // scales of this lane's 32 of each 128: a byte (MX), or two (NV)
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const uint8_t* sr = ss + r * Ring::kRowScales + (FMT == 0 ? 4 * i + g : 8 * i + 2 * g);
        sv[t][i] = FMT == 0 ? *sr : *reinterpret_cast<const uint16_t*>(sr);
      }
      wave_order();
    }
    const uint8_t* x = xs + (WHOLE ? ((unsigned)c * CH & (unsigned)(kp - 1)) * 2 : 0u);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4_t xf[MT][P];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = 0; p < P; ++p)
            xf[m][p] = *reinterpret_cast<const u32x4_t*>(x + xrow[m] + p * plane + 256 * i + 16 * j);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const uint32_t s = FMT == 0 ? sv[t][i] : sv[t][i] >> (8 * (j >> 1));   // (of NV's two the first for 0 and 1)
          const u32x4_t wf = weights8<FMT>(wv[t][i][j], scale_operand<FMT>(s & 0xFFu));
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = 0; p < P; ++p) acc[t][m] = mfma16(wf, xf[m][p], acc[t][m]);
        }
      }
  };

  // The wave's chunks are number wave, wave + 8, ... from the workgroup's first:
  // the first D are asked for, then each step asks for the one D further on.
  const int turn = WHOLE || whole == 0 ? 0 : (int)((blockIdx.x >> 3) * kFewWaves % (unsigned)whole);
  auto chunk_of = [&](int i) {                // (the end chunk stays the last)
    return i >= whole ? i : i + turn < whole ? i + turn : i + turn - whole;
  };
  Ring ring[D];
  auto load_one = [&](int i, Ring& d) {
    if (i < whole) load(chunk_of(i), d);
    else if (i < chunks) load_end(i, d);
  };
#pragma unroll
  for (int i = 0; i < D; ++i) load_one(wave + i * kFewWaves, ring[i]);
  if constexpr (WHOLE) {
    const int pieces = rows << (a.log_kp - 3);
    for (int q = tid; q < pieces; q += kFewThreads) {
      const int row = q >> (a.log_kp - 3), k = (q & ((kp >> 3) - 1)) * 8;
      if (k >= chunks * CH) continue;          // (no chunk reads there)
      XPiece<XT> d;
      if (k < K) load_piece<XT>(l, row * l.x_stride + k, XT == kXE4M3 ? row * (K / 32) + (k >> 5) : 0, d);
      else no_piece<XT>(d);
      store_piece<XT>(d, s_x + row * pitch + 2 * k, plane);
    }
    __syncthreads();
  }
  int c = wave;
  // without a branch, as long as what is asked for is whole chunks
  for (; c + (2 * D - 1) * kFewWaves < whole; c += D * kFewWaves) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      multiply(chunk_of(c + i * kFewWaves), ring[i]);
      load(chunk_of(c + (D + i) * kFewWaves), ring[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  for (; c < chunks; c += D * kFewWaves) {
#pragma unroll
    for (int i = 0; i < D; ++i) {
      if (c + i * kFewWaves < chunks) multiply(chunk_of(c + i * kFewWaves), ring[i]);
      load_one(c + (D + i) * kFewWaves, ring[i]);
    }
  }

  // ---- the sums of a wave's tiles, to where x was
  __syncthreads();
  float* s_sum = reinterpret_cast<float*>(s_x);      // [wave][tile][lane][4]
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *reinterpret_cast<f32x4_t*>(s_sum + ((wave * NT * MT + t * MT + m) * 64 + lane) * 4) = acc[t][m];
  __syncthreads();

  // element (row of x, weight row) of the joined sums
  const float tensor = FMT == 1 ? *l.w.g : 1.0f;
  auto sum = [&](int t, int m, int n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w)
      s += s_sum[((w * NT * MT + t * MT + (m >> 4)) * 64 + (m & 15) + 16 * (n >> 2)) * 4 + (n & 3)];
    return s * tensor;
  };
  auto put = [&](void* to, int64_t at, float v, int bf16) {
    if (bf16) static_cast<__bf16*>(to)[at] = (__bf16)v;
    else static_cast<float*>(to)[at] = v;
  };
  constexpr int kCols = 16 * kSide;
  for (int e = tid; e < rows * kCols; e += kFewThreads) {
    const int m = e / kCols, nn = e % kCols;
    const int64_t n = n0 + nn;
    if (n >= half) continue;
    float v = sum(nn >> 4, m, nn & 15);
    if constexpr (GATED) {
      const float u = sum(kSide + (nn >> 4), m, nn & 15);
      if (l.products) {
        put(l.products, m * l.w.n + n, v, l.products_bf16);
        put(l.products, m * l.w.n + half + n, u, l.products_bf16);
      }
      v = v * sigmoid(v) * u;
    } else if (l.bias) {
      v += l.out_bf16 ? (float)static_cast<const __bf16*>(l.bias)[n] : static_cast<const float*>(l.bias)[n];
    }
    put(l.out, m * half + n, v, l.out_bf16);
  }
}

template <int FMT, int XT, int MT, int NT, int CH, int D, bool GATED, bool WHOLE>
hipError_t launch_t(const LinearLaunch& l, int log_kp, hipStream_t s) {
  constexpr int P = kPieces<XT>;
  const int64_t n = GATED ? l.w.n / 2 : l.w.n;
  const int64_t per = 16 * (GATED ? NT / 2 : NT);
  const size_t x = WHOLE ? (size_t)P * l.rows * ((2 << log_kp) + 16) : 0;
  const size_t lds = x + (size_t)kFewWaves * (kScratch<CH> + (WHOLE ? 0 : P * 16 * MT * (2 * CH + 16)));
  const size_t sums = (size_t)kFewWaves * NT * MT * 1024;
  const FewArgs a = {l, log_kp, (int)x};
  hipLaunchKernelGGL((few_kernel<FMT, XT, MT, NT, CH, D, GATED, WHOLE>), dim3((unsigned)((n + per - 1) / per)),
                     dim3(kFewThreads), lds > sums ? lds : sums, s, a);
  return hipGetLastError();
}

// Two tiles a workgroup, which share what is read of x (24 rows of k 8192 by n
// 8192: 14.9 us; four tiles 23, one 21), one where two would leave CUs without
// work; one chunk in flight (two: 15.9 us; the other waves' loads hide the rest).
template <int FMT, int XT, bool GATED>
hipError_t launch_m(const LinearLaunch& l, hipStream_t s) {
  // all of x in LDS where 64 KiB hold it (and one tile its rows)
  int up = 8;
  while (((int64_t)1 << up) < l.w.k) ++up;
  if (l.rows <= 16 && (kPieces<XT> * l.rows * 2) << up <= 65536) {
    if constexpr (!GATED) {
      if (l.w.n < 32 * (int64_t)device_cu_count()) return launch_t<FMT, XT, 1, 1, 256, 1, GATED, true>(l, up, s);
    }
    return launch_t<FMT, XT, 1, 2, 256, 1, GATED, true>(l, up, s);
  }
  if (l.rows <= 16) return launch_t<FMT, XT, 1, 2, 128, 1, GATED, false>(l, 0, s);
  if constexpr (XT != kXF32) {                 // (its three planes of 17 rows and more do not fit)
    if (l.rows <= 32) return launch_t<FMT, XT, 2, 2, 128, 1, GATED, false>(l, 0, s);
    if (l.rows <= 48) return launch_t<FMT, XT, 3, 2, 128, 1, GATED, false>(l, 0, s);
    return launch_t<FMT, XT, 4, 2, 128, 1, GATED, false>(l, 0, s);
  }
  return hipErrorInvalidValue;
}

template <int FMT, int XT>
hipError_t launch_g(const LinearLaunch& l, hipStream_t s) {
  return l.gated ? launch_m<FMT, XT, true>(l, s) : launch_m<FMT, XT, false>(l, s);
}

}  // namespace

hipError_t launch_linear_few(const LinearLaunch& l, hipStream_t s) {
  if (l.w.format == 0) {
    if (l.x_type == kXF32) return launch_g<0, kXF32>(l, s);
    return l.x_type == kXBF16 ? launch_g<0, kXBF16>(l, s) : launch_g<0, kXE4M3>(l, s);
  }
  if (l.x_type == kXF32) return launch_g<1, kXF32>(l, s);
  return l.x_type == kXBF16 ? launch_g<1, kXBF16>(l, s) : launch_g<1, kXE4M3>(l, s);
}

}  // namespace fp4q
