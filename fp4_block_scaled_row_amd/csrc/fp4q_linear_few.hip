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
  const int64_t n0 = group_number() * (16 * kSide);
  if (n0 >= half) return;                        // (whole workgroups, behind the last)
  const int64_t srow = K / (FMT == 0 ? 32 : 16);
  const int rows = (int)l.rows;
  const float gs = FMT == 1 ? tensor_scale(l.w.g) : 1.0f, power = tensor_power(gs);

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
  // Addresses, by the lane: a row's number times its bytes, in 64 bits (both factors have
  // 32).  Where the sums take most registers, the lane is hidden from the compiler, so that
  // addresses are made anew for each chunk (kept, they took up to 60 registers more than
  // there are; 40 rows of k 4096 by two factors of 10000, MXFP4: 20.8 us, so 18.3).
  constexpr bool kTight = NT * MT >= 12;
  auto this_lane = [&] {
    int ln = lane;
    if constexpr (kTight) asm volatile("" : "+v"(ln));
    return ln;
  };
  auto w_row = [&](int t, int i) {
    return min((uint32_t)n0 + 16u * (t % kSide) + (uint32_t)i, (uint32_t)half - 1u) + (t / kSide) * (uint32_t)half;
  };
  auto codes_at = [&](int ln, int t, int i) {
    return l.w.codes + (uint64_t)w_row(t, ln / kLanes + i * (64 / kLanes)) * (uint32_t)(K / 2) + 16 * (ln % kLanes);
  };
  auto scales_at = [&](int ln, int t) {
    return l.w.scales + (uint64_t)w_row(t, ln >> 2) * (uint32_t)srow + (ln & 3) * kLane;
  };
  // this lane's piece of a row of x, and the rows that it loads; rows past the last read it
  constexpr int kXLanes = CH / 8;
  const int x_piece = lane % kXLanes;
  auto x_row = [&](int ln, int i) { return (uint32_t)min(i * (64 / kXLanes) + ln / kXLanes, rows - 1); };
  // (8-bit rows are dense and 2^31 elements at most in all: offsets of 32 bits, kept, and
  // hidden where the compiler, which would keep addresses, has not the registers; 2 tiles
  // of 32 rows are 5 % faster with them)
  uint32_t x_at8[Ring::kXLoads > 0 ? Ring::kXLoads : 1];
  if constexpr (XT == kXE4M3) {
#pragma unroll
    for (int i = 0; i < Ring::kXLoads; ++i) x_at8[i] = x_row(lane, i) * (uint32_t)K + 8u * x_piece;
  }
  auto load_x = [&](int c, int ln, int i, XPiece<XT>& d) {
    if constexpr (XT == kXE4M3) {
      uint32_t at = x_at8[i];
      if constexpr (NT * MT > 4) asm volatile("" : "+v"(at));
      const u32x2_t v = load_any<u32x2_t>(static_cast<const uint8_t*>(l.x) + (int64_t)c * CH + at);
      d.w[0] = v.x;
      d.w[1] = v.y;
      d.w[2] = (l.x_scales + (int64_t)c * (CH / 32))[at >> 5];
    } else {
      load_piece<XT>(l, (int64_t)(x_row(ln, i) * (uint64_t)l.x_stride) + 8 * (ln % kXLanes) + (int64_t)c * CH, 0, d);
    }
  };

  const int whole = (int)(K / CH), chunks = (int)((K + CH - 1) / CH);
  auto load = [&](int c, Ring& d) {           // a whole chunk
    const int ln = this_lane();
#pragma unroll
    for (int i = 0; i < Ring::kXLoads; ++i) load_x(c, ln, i, d.x[i]);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) d.c[t][i] = load_codes<CH>(codes_at(ln, t, i) + (int64_t)c * (CH / 2));
      d.s[t] = load_small<kLane>(scales_at(ln, t) + (int64_t)c * kScales);
    }
  };
  auto load_end = [&](int c, Ring& d) {       // the chunk that the rows end in, zeros behind them
    const int ln = this_lane();
#pragma unroll
    for (int i = 0; i < Ring::kXLoads; ++i) {
      const int64_t k = (int64_t)c * CH + 8 * x_piece;             // (K is a multiple of 8)
      if (k < K) load_x(c, ln, i, d.x[i]);
      else no_piece<XT>(d.x[i]);
    }
    const int64_t k0 = (int64_t)c * CH, v = K - k0 - 32 * piece_at;    // v: what this lane's 32 codes have of them
    const int have = (int)(K - k0) / (FMT == 0 ? 32 : 16) - (lane & 3) * kLane;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        d.c[t][i] = u32x4_t{0u, 0u, 0u, 0u};
        const uint8_t* p = codes_at(ln, t, i) + k0 / 2;
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
        if (i < have) d.s[t] |= (uint32_t)scales_at(ln, t)[(int64_t)c * kScales + i] << (8 * i);
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
          const u32x4_t wf = weights8<FMT>(wv[t][i][j], scale_operand<FMT>(s & 0xFFu), power);
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = 0; p < P; ++p) acc[t][m] = mfma16(wf, xf[m][p], acc[t][m]);
        }
        if constexpr (NT * MT >= 12) __builtin_amdgcn_sched_barrier(0);   // (registers: one step's operands at a time)
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

  // ---- the sums of a wave's tiles, to where x was: four weight rows' of row m of x
  // a 16-byte piece, 4 of a tile (number q), m exchanged by q so that neighbouring
  // lanes' reads of 4 pieces of 4 rows meet all banks (as they lie, and read 4 bytes
  // a lane, they took 2 of 26 us of 40 rows gated)
  __syncthreads();
  f32x4_t* s_sum = reinterpret_cast<f32x4_t*>(s_x);      // [wave][tile][q][m]
  auto sum_at = [&](int w, int t, int mt, int q, int m) {
    return ((w * NT + t) * MT + mt) * 64 + q * 16 + (m ^ (4 * q));
  };
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) s_sum[sum_at(wave, t, m, g, r)] = acc[t][m];
  __syncthreads();

  const float tensor = tensor_rest(gs);
  auto sum = [&](int t, int m, int q) {
    f32x4_t v = s_sum[sum_at(0, t, m >> 4, q, m & 15)];
#pragma unroll
    for (int w = 1; w < kFewWaves; ++w) v += s_sum[sum_at(w, t, m >> 4, q, m & 15)];
    return v * tensor;
  };
  auto put = [&](void* to, int64_t at, f32x4_t v, int count, int bf16) {   // the first `count`, at most 4
    if (bf16) {
      __bf16* o = static_cast<__bf16*>(to) + at;
      if (count >= 4) store_any(o, u32x2_t{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)});
      else for (int i = 0; i < count; ++i) o[i] = (__bf16)v[i];
    } else {
      float* o = static_cast<float*>(to) + at;
      if (count >= 4) store_any(o, v);
      else for (int i = 0; i < count; ++i) o[i] = v[i];
    }
  };
  constexpr int kPieces16 = 4 * kSide;                   // of a row
  for (int e = tid; e < rows * kPieces16; e += kFewThreads) {
    const int m = e / kPieces16, q = e % kPieces16;
    const int64_t n = n0 + 4 * q;
    const int count = (int)min(half - n, (int64_t)4);
    if (count <= 0) continue;
    f32x4_t v = sum(q >> 2, m, q & 3);
    if constexpr (GATED) {
      const f32x4_t u = sum(kSide + (q >> 2), m, q & 3);
      if (l.products) {
        put(l.products, m * l.w.n + n, v, count, l.products_bf16);
        put(l.products, m * l.w.n + half + n, u, count, l.products_bf16);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
    } else if (l.bias) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < count)
          v[i] += l.out_bf16 ? (float)static_cast<const __bf16*>(l.bias)[n + i] : static_cast<const float*>(l.bias)[n + i];
    }
    put(l.out, m * half + n, v, count, l.out_bf16);
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
  const int64_t groups = (n + per - 1) / per;
  hipLaunchKernelGGL((few_kernel<FMT, XT, MT, NT, CH, D, GATED, WHOLE>), dim3(grid_x(groups), grid_y(groups)),
                     dim3(kFewThreads), lds > sums ? lds : sums, s, a);
  return hipGetLastError();
}

// 17 to 48 rows: two tiles a workgroup, or four or six, by the workgroups that CUs
// take one after another (LDS holds one at a time), each as long as its tiles and one
// and a half, for x.  Measured, MXFP4 (NVFP4) with bf16, k 4096, us, 24 rows / 40 rows
// (MXFP8 is 0 to 15 % slower, in the same order):
//   n       two tiles                  four                       six
//   4096     7.5 (7.8) /  8.8 (9.4)     9.1 (10.1) / 12.5 (13.9)  12.6 (15.5) / 15.7 (18.2)
//   16384   13.9 (15.6) / 17.7 (19.1)  10.7 (12.5) / 14.4 (16.2)  13.9 (17.3) / 17.0 (19.8)
//   20000   18.5 (21.7) / 24.5 (26.8)  18.1 (20.9) / 23.8 (28.0)  14.3 (17.2) / 17.2 (19.9)
//   28672   23.5 (28.4) / 31.7 (35.0)  18.9 (21.9) / 24.8 (28.8)  24.7 (31.4) / 30.3 (36.4)
// (Six are the ones for widths that four would give a few CUs more turns: 16400 to
// 24600 of 256 CUs.)
template <int FMT, int XT, int MT, bool GATED>
hipError_t launch_nt(const LinearLaunch& l, hipStream_t s) {
  const int64_t cus = device_cu_count();
  auto cost = [&](int nt) {
    const int64_t groups = (l.w.n + 16 * nt - 1) / (16 * nt);
    return (groups + cus - 1) / cus * (3 + 2 * nt);
  };
  if (cost(6) < cost(4) && cost(6) < cost(2)) return launch_t<FMT, XT, MT, 6, 128, 1, GATED, false>(l, 0, s);
  if (cost(4) < cost(2)) return launch_t<FMT, XT, MT, 4, 128, 1, GATED, false>(l, 0, s);
  return launch_t<FMT, XT, MT, 2, 128, 1, GATED, false>(l, 0, s);
}

// Two tiles a workgroup, which share what is read of x (24 rows of k 8192 by n
// 8192: 14.7 us; one tile 21), one where two would leave CUs without work; one chunk
// in flight (two: 15.9 us; the other waves' loads hide the rest).
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
    if (l.rows <= 32) return launch_nt<FMT, XT, 2, GATED>(l, s);
    if (l.rows <= 48) return launch_nt<FMT, XT, 3, GATED>(l, s);
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
