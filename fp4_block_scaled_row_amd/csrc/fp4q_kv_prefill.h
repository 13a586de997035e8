// fp4q_kv_prefill.h -- attention over the 4-bit cache for many query rows.
//
// A workgroup of kW waves takes a block of 32 kW query rows; it goes through the
// tokens 64 at a time, which its waves turn from codes into fp16 / bf16 in LDS
// once for all (codes of the next 64 in flight, LDS in two halves, one barrier a
// step).  Each wave works on its own 32 rows: scores by 32x32x16 products with
// the keys as the left operand, so that a lane holds one row's scores of 32
// tokens, whose weights are then its part of the second product's right
// operand, the left one being the values read transposed.
//
// Bound by matrix and vector instructions, which overlap only between a SIMD's
// two waves (42 % and 44 % of the cycles in the first of the calls below, 47 % and
// 44 % in the second): 64 tokens x 32 rows x 128 elements are 1024 cycles of the
// ones and about 1150 of the others (a third of them exponentials) a wave.
// 4 x 1000 queries of 40 heads over up to 16000 tokens, MXFP4: 810 us, 930
// TFLOP/s (a large library product reaches 1190); 4096 queries of 32 heads over
// as many tokens, NVFP4, rotated, so that queries in two pieces make the first
// product twice as long: 230 us, 600, where blocks that see half of a step and
// the ends of blocks weigh more too.  Products of the next step's scores between
// this one's exponentials in an order fixed by the source, with three steps in
// LDS, were no faster (830 us for 785).
//
// MXFP4 values are fp16 numbers, as NVFP4's are, where a block's largest lies
// between 2^-23 and 2^16.  So for bf16 outputs a workgroup takes its part of a
// unit in fp16, with one piece of weights, and if it meets a block that is not,
// leaves that and begins the part again in bf16 with two.
#pragma once

#include "fp4q_kv_attend.h"

namespace fp4q {

template <int N>
struct Const {
  static constexpr int value = N;
};

constexpr int kStepTokens = 64;
constexpr int kStepCost = 6;      // steps that beginning and ending a unit takes as long as

template <int FMT, int D, int kW, int kQ, int kP>
struct PrefillShape {
  static constexpr int kRows = 32 * kW;
  static constexpr int kThreadsWg = 64 * kW;
  static constexpr int kKStride = D + 8;                     // halves: rows 4 banks apart
  // transposed reads take 4 rows of 16 words at once: rows 16 or 48 banks apart
  static constexpr int kVStride = D == 96 ? D : D + 32;
  static constexpr int kHalf = kStepTokens * (kKStride + kVStride);
  // MXFP4 with bf16 outputs: values in fp16 where all of them fit it
  static constexpr bool kHalfValues = FMT == 0 && kP == 1;
  // two waves a SIMD where the registers allow it
  static constexpr int kWavesPerSimd = D <= 128 && kQ <= 2 && kP == 1 ? 2 : 1;
};

// The wave's query rows as right operands: lane's row l % 32, elements
// 16 c + 8 (l / 32) .. + 7 of chunk c; returns the factor from raw score to
// exponent of two.
template <int FMT, int D, int kQ>
__device__ __forceinline__ float wave_queries(const KvAttendLaunch& a, const KvUnit& u, int row, int half,
                                              u32x4_t qf[kQ][D / 16]) {
  float v[D / 16][8];
#pragma unroll
  for (int c = 0; c < D / 16; ++c) widen_q8(a, load_q8(a, u, row, 2 * c + half), v[c]);
  if constexpr (D % 128 == 0) {
    if (a.rotate) {
      // elements 1, 2, 4 apart in a lane's 8, 8 apart between the lanes' two
      // halves, 16, 32 and 64 apart between its chunks
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
#pragma unroll
        for (int h = 1; h < 8; h <<= 1)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i & h) continue;
            const float x = v[c][i], y = v[c][i + h];
            v[c][i] = x + y;
            v[c][i + h] = x - y;
          }
        const float sign = half ? -1.0f : 1.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = fmaf(v[c][i], sign, __shfl_xor(v[c][i], 32, 64));
      }
#pragma unroll
      for (int k = 0; k < D / 16; k += 8)
#pragma unroll
        for (int h = 1; h < 8; h <<= 1)
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            if (c & h) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float x = v[k + c][i], y = v[k + c + h][i];
              v[k + c][i] = x + y;
              v[k + c + h][i] = x - y;
            }
          }
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] *= a.rot_scale;
    }
  }
  float factor = fabsf(a.scale) * kLog2e * (FMT == 1 ? *a.p.kg : 1.0f), up = a.scale < 0.0f ? -1.0f : 1.0f;
  if constexpr (kv_scaled_rows<FMT>()) {
    uint32_t most = 0u;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) most = max(most, abs_max_bits8(v[c]));
    most = max(most, (uint32_t)__shfl_xor((int)most, 32, 64));
    const uint32_t e = min(max(most >> 23, 9u), 254u);
    up *= as_f((262u - e) << 23);
    factor *= as_f((e - 8u) << 23);
  }
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    uint32_t w[4][kQ];
#pragma unroll
    for (int j = 0; j < 4; ++j) pieces<FMT, kQ>(v[c][2 * j] * up, v[c][2 * j + 1] * up, w[j]);
#pragma unroll
    for (int q = 0; q < kQ; ++q) qf[q][c] = u32x4_t{w[0][q], w[1][q], w[2][q], w[3][q]};
  }
  return larger(factor, kLeast);
}

template <int FMT, int D, int kW, int kQ, int kP>
__global__ __launch_bounds__(64 * kW, (PrefillShape<FMT, D, kW, kQ, kP>::kWavesPerSimd)) void kv_prefill_kernel(
    KvAttendLaunch a, int numbers) {
  using Shape = PrefillShape<FMT, D, kW, kQ, kP>;
  using T = KvType<FMT>;
  using Lane = KvLane<FMT, D>;
  constexpr int kRows = Shape::kRows;
  constexpr int kTasks = 8 / kW;       // 16 tokens' keys or values a task: 8 in a step
  __shared__ __align__(16) uint16_t s_kv[2 * Shape::kHalf];
  __shared__ int s_scan[kW + 6];
  __shared__ NotedNans<kRows, kStepTokens> s_nans;
  __shared__ int s_misfit[2];      // kHalfValues: a step's values do not fit fp16

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4, col = lane & 31, half = lane >> 5;

  kv_clear_others<D, 64 * kW>(a);
  KvStretch st;
  KvShared* shared = kv_shared(a, blockIdx.x);
  if (tid == 0) shared->first = shared->last = 0;
  if (!kv_stretch<kRows, kStepTokens, kStepCost, 64 * kW, false>(a, numbers, st, s_scan)) return;
  const KvUnit& u = st.u;
  do {
    int group, last;      // the unit's groups [group, last) are this workgroup's
    kv_part<kStepCost>(st, group, last);
    if (group == last) continue;
    const int row0 = u.row0 + 32 * wave;
    int block_from, block_to;     // tokens that all rows of the block see
    kv_all_see<kRows>(a, u, block_from, block_to);
    const int32_t* table = a.table + u.b * a.table_stride;
    const KvHead planes = kv_head(a.p, u.head);
    const int n = u.hi;
    // task x of this wave: tokens 16 (task / 2) .. + 15 of a step, their keys
    // (even) or values (odd); see the few-row kernel for the loads
    Lane in[kTasks];
    int32_t pages[kTasks];
    bool there[kTasks];
    const int task0 = wave * kTasks;
    auto find = [&](int grp) {
#pragma unroll
      for (int x = 0; x < kTasks; ++x) {
        const int t = min(u.lo + grp * kStepTokens + 16 * ((task0 + x) >> 1) + r, n - 1);
        pages[x] = table[quotient((uint32_t)t, a.p.page)];
      }
    };
    auto fetch = [&](int grp) {
#pragma unroll
      for (int x = 0; x < kTasks; ++x) {
        const int t = u.lo + grp * kStepTokens + 16 * ((task0 + x) >> 1) + r;
        const uint32_t tt = (uint32_t)min(t, n - 1);
        const bool page = (uint32_t)pages[x] < (uint32_t)a.p.num_pages;
        const KvAt at = kv_at(a.p, page ? (uint32_t)pages[x] : 0u, tt - quotient(tt, a.p.page) * a.p.page.d);
        const bool values = (task0 + x) & 1;
        in[x].load((values ? planes.vc : planes.kc) + at.code, (values ? planes.vs : planes.ks) + at.scale, 0, 0, g);
        there[x] = page && t < n;
      }
    };
    // (fmt: the values' type, that of a format's products)
    auto put = [&](int grp, auto fmt) __attribute__((always_inline)) {
      const int t0 = u.lo + grp * kStepTokens;
      const bool edge = t0 + kStepTokens > block_to || t0 < block_from;
      uint16_t* base = s_kv + (grp & 1) * Shape::kHalf;
#pragma unroll
      for (int x = 0; x < kTasks; ++x) {
        const bool values = (task0 + x) & 1;
        in[x].keep_if(there[x]);
        if (values && edge) {
          const uint32_t dropped = in[x].drop_not_finite();
          if (__any(dropped != 0u)) s_nans.template note<FMT, D>(t0 + 16 * ((task0 + x) >> 1) + r, g, dropped);
        }
        const int t = 16 * ((task0 + x) >> 1) + r;
        uint16_t* dst = values ? base + kStepTokens * Shape::kKStride + t * Shape::kVStride : base + t * Shape::kKStride;
        if constexpr (decltype(fmt)::value != FMT) {
          if (values) {
            if (__any(!in[x].fits_half())) s_misfit[grp & 1] = 1;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) *reinterpret_cast<u32x4_t*>(dst + Lane::element(c, g)) = in[x].half_values(c);
            continue;
          }
        }
        const typename Lane::Scales sc = in[x].prepare();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) *reinterpret_cast<u32x4_t*>(dst + Lane::element(c, g)) = in[x].values(c, sc);
      }
    };
    auto begin = [&]() {
      if (n > 0) {
        find(group);
        fetch(group);
        find(group + 1);
      }
    };
    begin();      // (on their way while the queries are prepared)
    if (tid == 0) s_nans.count = s_misfit[0] = s_misfit[1] = 0;
    u32x4_t qf[kQ][D / 16];
    const float factor = wave_queries<FMT, D, kQ>(a, u, row0 + col, half, qf);
    int sees_from;
    uint32_t sees;
    kv_sees(a, u, row0 + col, sees_from, sees);
    // tokens that all of the wave's rows see; any of them: [wu.lo, wu.hi)
    int all_from, all_to;
    KvUnit wu = u;
    kv_block_at<32, kStepTokens>(a, row0, wu);
    kv_all_see<32>(a, wu, all_from, all_to);
    const bool rows = (int)quotient((uint32_t)row0, a.group_div) < u.m;

    f32x16_t o[D / 32];
    float m, l;
    // The steps of the workgroup's groups, values and weights in the type of
    // format fmt, weights in np pieces; false: some values do not fit that type.
    auto pass = [&](auto fmt, auto np) __attribute__((always_inline)) {
      constexpr int kWeights = decltype(np)::value;
      constexpr bool kMayMisfit = decltype(fmt)::value != FMT;
      using V = KvType<decltype(fmt)::value>;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) o[c] = f32x16_t{};
      m = kNoMax;
      l = 0.0f;

      __syncthreads();
      if (n > 0) {
        put(group, fmt);
        fetch(group + 1);
        find(group + 2);
      }
      __syncthreads();
      for (int grp = group; grp < last; ++grp) {
        const int t0 = u.lo + grp * kStepTokens;
        if (t0 >= n) break;                       // (a unit without tokens)
        // (a half's word is written before the barrier that ends the step before,
        // and again only after the one that ends this step: all waves read the same)
        const int misfit = kMayMisfit ? s_misfit[grp & 1] : 0;
        if (rows && t0 < wu.hi && t0 + kStepTokens > wu.lo) {
          // LDS reads set out a stage before the products that take them, and the
          // scheduler may not move them back: left alone it puts each right
          // before its product, which then waits for it.
          const uint16_t* ks = s_kv + (grp & 1) * Shape::kHalf + col * Shape::kKStride + 8 * half;
          const uint16_t* vs = s_kv + (grp & 1) * Shape::kHalf + kStepTokens * Shape::kKStride +
                               (4 * half + (r >> 2)) * Shape::kVStride + 16 * (g & 1) + 4 * (r & 3);
          constexpr int kStage = D / 16 < 8 ? D / 16 : 8, kStages = 2 * (D / 16) / kStage;   // key fragments
          u32x4_t kf[2][kStage];
          auto read_keys = [&](int stage) {
#pragma unroll
            for (int i = 0; i < kStage; ++i) {
              const int f = stage * kStage + i, x = f & 1, c = f >> 1;
              kf[stage & 1][i] = *reinterpret_cast<const u32x4_t*>(ks + 32 * x * Shape::kKStride + 16 * c);
            }
          };
          u32x4_t vf[2][D / 32];
          auto read_values = [&](int k) {
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              const u32x2_t x0 = read_transposed(vs + 16 * k * Shape::kVStride + 32 * c);
              const u32x2_t x1 = read_transposed(vs + (16 * k + 8) * Shape::kVStride + 32 * c);
              vf[k & 1][c] = u32x4_t{x0.x, x0.y, x1.x, x1.y};
            }
          };
          f32x16_t s[2] = {f32x16_t{}, f32x16_t{}};
          read_keys(0);
#pragma unroll
          for (int stage = 0; stage < kStages; ++stage) {
            __builtin_amdgcn_sched_barrier(0);
            if (stage + 1 < kStages) read_keys(stage + 1);
            else read_values(0);
#pragma unroll
            for (int i = 0; i < kStage; ++i) {
              const int f = stage * kStage + i, x = f & 1, c = f >> 1;
#pragma unroll
              for (int q = 0; q < kQ; ++q) s[x] = T::mfma32(kf[stage & 1][i], qf[q][c], s[x]);
            }
          }
          __builtin_amdgcn_sched_barrier(0);
          // token 32 x + 8 (i / 4) + 4 half + i % 4 of the step
          float y[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] = s[i >> 4][i & 15];
          if (t0 + kStepTokens > all_to || t0 < all_from) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const uint32_t j = (uint32_t)(t0 + 8 * (i >> 2) + 4 * half + (i & 3) - sees_from);
              y[i] = j < sees ? y[i] : -INFINITY;
            }
          }
          float most = y[0];
#pragma unroll
          for (int i = 1; i < 32; ++i) most = larger(most, y[i]);
          most *= factor;
          if (__any(most > m + kRaise)) {
            const float x = larger(larger(most, __shfl_xor(most, 32, 64)), m);
            const float f = __builtin_amdgcn_exp2f(m - x);
            m = x;
            l *= f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] *= f;
          }
          const float top = V::kUp - m;
          float sum = 0.0f;       // (as in the few-row kernel)
          u32x4_t w[4][kWeights];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t h[4][kWeights];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float p0 = __builtin_amdgcn_exp2f(fmaf(y[8 * k + 2 * j], factor, top));
              const float p1 = __builtin_amdgcn_exp2f(fmaf(y[8 * k + 2 * j + 1], factor, top));
              sum += p0 + p1;
              weight_pieces<decltype(fmt)::value, kWeights>(p0, p1, h[j]);
            }
#pragma unroll
            for (int q = 0; q < kWeights; ++q) w[k][q] = u32x4_t{h[0][q], h[1][q], h[2][q], h[3][q]};
          }
          l += sum;
          // weighted values: element 32 c + 8 (i / 4) + 4 half + i % 4 of the row.
          // Of a SIMD's two waves the one that is at these goes first: its
          // products fill the other's exponentials (4 x 1000 queries of 40 heads
          // over to 16000 tokens 775-779 us with this priority, 783-786 without).
          __builtin_amdgcn_s_setprio(1);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            if (k + 1 < 4) read_values(k + 1);
#pragma unroll
            for (int q = 0; q < kWeights; ++q)
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                const u32x4_t vq = values_of_piece<decltype(fmt)::value, kWeights>(q, vf[k & 1][c]);
                o[c] = V::mfma32(vq, w[k][q], o[c]);
              }
          }
          __builtin_amdgcn_sched_barrier(0);
          __builtin_amdgcn_s_setprio(0);
        }
        if (kMayMisfit && __builtin_amdgcn_readfirstlane(misfit)) return false;
        if (grp + 1 < last) {
          put(grp + 1, fmt);
          fetch(grp + 2);
          find(grp + 3);
        }
        __syncthreads();
      }
      if constexpr (V::kUp != T::kUp) {      // (weights and sums as the other passes leave them)
        constexpr float back = 1.0f / (1 << (int)(V::kUp - T::kUp));
        l *= back;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) o[c] *= back;
      }
      return true;
    };
    if constexpr (Shape::kHalfValues) {
      if (!pass(Const<1>{}, Const<1>{})) {
        if (tid == 0) s_nans.count = 0;      // (noted again; read after the passes only)
        begin();
        pass(Const<0>{}, Const<2>{});
      }
    } else {
      pass(Const<FMT>{}, Const<kP>{});
    }

    l += __shfl_xor(l, 32, 64);
    const bool whole = group == 0 && last == u.groups;
    const int rr = 32 * wave + col;
    if (s_nans.count) {
      const uint32_t nan = s_nans.seen(a, u, u.row0 + rr);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        // (elements 0 to 7 of a lane's 16 are in the lower half of the 32)
        const float f0 = (nan >> (32 * c / Lane::kBlock)) & 1u ? as_f(0x7FC00000u) : 1.0f;
        const float f1 = (nan >> ((32 * c + 16) / Lane::kBlock)) & 1u ? as_f(0x7FC00000u) : 1.0f;
        o[c] *= f32x16_t{f0, f0, f0, f0, f0, f0, f0, f0, f1, f1, f1, f1, f1, f1, f1, f1};
      }
    }
    if (whole) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
#pragma unroll
        for (int i = 0; i < 16; i += 4)
          kv_finish4<FMT, D>(a, u, u.row0 + rr, 32 * c + 2 * i + 4 * half,
                             f32x4_t{o[c][i], o[c][i + 1], o[c][i + 2], o[c][i + 3]}, m, l);
    } else {
      float* part = kv_partial<D, kRows>(a, blockIdx.x, group == 0);
      if (tid == 0) {
        if (group == 0) {
          shared->b = u.b;
          shared->head = u.head;
          shared->row0 = u.row0;
          shared->last = 1;
        } else {
          shared->first = last == u.groups ? 2 : 1;
        }
      }
      if (u.row0 + rr < u.m * a.group) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c)
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<f32x4_t*>(part + (int64_t)rr * D + 32 * c + 2 * i + 4 * half) =
                f32x4_t{o[c][i], o[c][i + 1], o[c][i + 2], o[c][i + 3]};
        if (half == 0) *reinterpret_cast<float2_t*>(part + (int64_t)kRows * D + 2 * rr) = float2_t{m, l};
      }
    }
    __syncthreads();      // (everyone has read s_nans)
  } while (kv_next<kRows, kStepTokens, kStepCost>(a, st));
}

template <int FMT, int D, int kW, int kQ, int kP>
hipError_t launch_prefill_t(const KvAttendLaunch& a, int cus, hipStream_t st) {
  using Shape = PrefillShape<FMT, D, kW, kQ, kP>;
  constexpr int kRows = Shape::kRows;
  KvAttendLaunch b = a;
  const int64_t numbers = kv_block_numbers(b, kRows);
  const int64_t most = kv_most_groups(b, numbers, kStepTokens, kStepCost);
  const int64_t resident = (int64_t)cus * (4 * Shape::kWavesPerSimd / kW);
  const int grid = (int)min(min(most, resident), (int64_t)kMostWorkgroups);
  hipLaunchKernelGGL((kv_prefill_kernel<FMT, D, kW, kQ, kP>), dim3(grid), dim3(64 * kW), 0, st, b, (int)numbers);
  const hipError_t e = hipGetLastError();
  // (a unit of one step is never shared)
  if (e != hipSuccess || a.most_tokens <= kStepTokens) return e;
  const int64_t rows = min((int64_t)kRows, (int64_t)a.max_q * a.group);
  hipLaunchKernelGGL((kv_join_kernel<FMT, D, kRows>), dim3(grid, (uint32_t)((rows * (D / 4) + kThreads - 1) / kThreads)),
                     dim3(kThreads), 0, st, a, grid);
  return hipGetLastError();
}

// Waves: 8 where two of them fit a SIMD, for blocks of 256 rows; 4 elsewhere
// and where sequences have at most 128 rows.
template <int D, int FMT>
hipError_t launch_prefill_d(const KvAttendLaunch& a, int waves, int cus, hipStream_t st) {
  if (a.dtype == kF32) return launch_prefill_t<FMT, D, 4, FMT == 1 ? 2 : 3, FMT == 1 ? 2 : 3>(a, cus, st);
  if constexpr (D <= 128) {
    if (waves == 8) {
      if (kv_bf16_pieces(a) == 2) return launch_prefill_t<FMT, D, 8, 2, 1>(a, cus, st);
      return launch_prefill_t<FMT, D, 8, 1, 1>(a, cus, st);
    }
  }
  if (kv_bf16_pieces(a) == 2) return launch_prefill_t<FMT, D, 4, 2, 1>(a, cus, st);
  return launch_prefill_t<FMT, D, 4, 1, 1>(a, cus, st);
}

}  // namespace fp4q
