// fp4q_kv_decode.h -- attention over the 4-bit cache for few query rows.
//
// One read of the cache is what such a call costs; its groups of 128 tokens
// are shared out evenly (the schedule of fp4q_kv_attend.h), lengths being read
// on the device, so that a captured launch follows them.  A unit inside one
// stretch is finished there; the others leave partial results that the last of
// their workgroups joins.
//
// In a workgroup each of the 4 waves works on 32 tokens of a group by itself:
// keys from memory into the left operand of 16x16x32 products (16 tokens x 16
// rows), values through the wave's own LDS rows.  Codes of the next two groups
// are in flight while one is worked on: a group takes a wave about 1.2 us, a
// load from HBM about as long under load.
//
// Large calls: 64 sequences of up to 8192 tokens, 8 heads of 128, NVFP4, 380 MB
// in 82 us, 4.6 TB/s (a large copy reaches 6.4), 87 to 91 with rotated queries,
// whose two pieces leave two waves a SIMD instead of three; of that call the
// vector units issue 43 % of the time and the matrix units work 16 %, so it is
// neither's issue nor the memory's rate alone but latency that more waves would
// hide.  MXFP4, 2 x 131071 tokens, 273 MB in 56 us (partly from the Infinity
// Cache) to 64; CUs are busy 73 to 84 % of it, joins and the uneven ends of the
// workgroups are the rest.  Small ones by the chain of lengths, page numbers,
// codes, products and joins: 1 x 1023 tokens 11 us.
#pragma once

#include "fp4q_kv_attend.h"

namespace fp4q {

constexpr int kGroupTokens = 128;
constexpr int kJoin = 4;          // pieces joined at a time
constexpr int kGroupCost = 2;     // groups that beginning and ending a unit takes as long as

template <int FMT, int D, int kTiles, int kQ, int kP>
struct DecodeShape {
  static constexpr int kRows = 16 * kTiles;
  static constexpr int kChunks = D / 32;
  // query pieces stay in registers up to 64 of them, in LDS beyond
  static constexpr bool kQRegs = kTiles * kQ * kChunks * 4 <= 64;
  static constexpr int kVStride = D + 16;                        // halves: rows 8 banks apart
  static constexpr int kVBytes = kWaves * 32 * kVStride * 2;
  static constexpr int kOStride = D + 4;                         // floats
  static constexpr int kOBytes = kWaves * 16 * kOStride * 4;
  static constexpr int kQBytes = kQ * kRows * (D + 8) * 2;
  static constexpr int kMax1 = kVBytes > kOBytes ? kVBytes : kOBytes;
  static constexpr int kMain = kQRegs && kQBytes > kMax1 ? kQBytes : kMax1;
  static constexpr int kShared = kMain + (kQRegs ? 0 : kQBytes);
  // as many as the registers allow: by a hair, 4 to 13 of them spilled with
  // head_dim 256 and 5 to 28 with 32 rows of 128 in two pieces
  static constexpr int kWavesPerSimd = D > 128 ? (kQ > 1 ? 1 : 2) : (kTiles == 2 || kQ > 1 ? 2 : 3);
};

template <int FMT, int D, int kTiles, int kQ, int kP, bool kWhole>
__global__ __launch_bounds__(kThreads, (DecodeShape<FMT, D, kTiles, kQ, kP>::kWavesPerSimd)) void kv_decode_kernel(
    KvAttendLaunch a, int numbers) {
  using Shape = DecodeShape<FMT, D, kTiles, kQ, kP>;
  using T = KvType<FMT>;
  using Lane = KvLane<FMT, D>;
  constexpr int kChunks = Shape::kChunks, kRows = Shape::kRows;
  __shared__ __align__(16) uint8_t s_main[Shape::kShared];
  __shared__ float s_factor[kRows];
  __shared__ uint32_t s_most[kRows];
  __shared__ float s_m[kWaves][kRows], s_l[kWaves][kRows];
  __shared__ NotedNans<kRows, 32> s_nans;
  __shared__ int s_scan[kWaves + 6];

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, g = lane >> 4;
  uint16_t* sv = reinterpret_cast<uint16_t*>(s_main) + wave * 32 * Shape::kVStride;
  float* so = reinterpret_cast<float*>(s_main);
  uint16_t* sq = reinterpret_cast<uint16_t*>(s_main + (Shape::kQRegs ? 0 : Shape::kMain));

  const float kg = FMT == 1 ? scalar(a.p.kg) : 1.0f;
  kv_clear_others<D, kThreads>(a);
  KvStretch st;
  if (!kv_stretch<kRows, kGroupTokens, kGroupCost, kThreads, Shape::kWavesPerSimd == 3>(a, numbers, st, s_scan)) return;
  const KvUnit& u = st.u;

  // Codes of 2 x 16 tokens a lane, those of two groups in flight, and the page
  // numbers of the group after them.
  //   kWhole (see kv_whole_tiles): pages are multiples of 32 tokens, so that a
  // wave's 32 tokens lie in one page: its number and their place are scalars, the
  // lanes' offsets 32-bit constants.  Tokens past the end are in the page too and are read.
  //   Other pages: every lane finds its token's page.  No branches: tokens past
  // the end are looked for at the last one's place.
  //   Pages that are none are read at page 0 and then zeroed.
  struct Tile {
    Lane k[2], v[2];
    bool there[2];
  };
  struct Pages {
    int32_t x[2];
  };
  Tile even, odd;
  Pages pages = {{0, 0}};
  QueryRows<D, kRows> rows;
  const int32_t* table = nullptr;
  KvHead planes = {};
  int group = 0, last = 0;      // the unit's groups [group, last) are this workgroup's
  int first = 0, n = 0;         // this wave's first token of group 0, the tokens' end
  const uint32_t c_lane = r * a.p.code_stride[2], s_lane = r * a.p.scale_stride[2];
  auto find = [&](int grp) {
    Pages p = {{0, 0}};
    if constexpr (kWhole) {
      const int t = min(first + grp * kGroupTokens, n - 1);
      p.x[0] = reinterpret_cast<const __attribute__((address_space(4))) int32_t*>(
          reinterpret_cast<uintptr_t>(table))[quotient((uint32_t)t, a.p.page)];
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = min(first + grp * kGroupTokens + 16 * x + r, n - 1);
        p.x[x] = table[quotient((uint32_t)t, a.p.page)];
      }
    }
    return p;
  };
  auto fetch = [&](int grp, const Pages& pages, Tile& in) {
    if constexpr (kWhole) {
      const uint32_t t = (uint32_t)min(first + grp * kGroupTokens, n - 1) & ~31u;
      const bool page = (uint32_t)pages.x[0] < (uint32_t)a.p.num_pages;
      const KvAt at = kv_at(a.p, page ? (uint32_t)pages.x[0] : 0u, t - quotient(t, a.p.page) * a.p.page.d);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const uint32_t c = c_lane + 16 * x * a.p.code_stride[2], e = s_lane + 16 * x * a.p.scale_stride[2];
        in.k[x].load(planes.kc + at.code, planes.ks + at.scale, c, e, g);
        in.v[x].load(planes.vc + at.code, planes.vs + at.scale, c, e, g);
        in.there[x] = page;
      }
    } else {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int t = first + grp * kGroupTokens + 16 * x + r;
        const uint32_t tt = (uint32_t)min(t, n - 1);
        const bool page = (uint32_t)pages.x[x] < (uint32_t)a.p.num_pages;
        const KvAt at = kv_at(a.p, page ? (uint32_t)pages.x[x] : 0u, tt - quotient(tt, a.p.page) * a.p.page.d);
        in.k[x].load(planes.kc + at.code, planes.ks + at.scale, 0, 0, g);
        in.v[x].load(planes.vc + at.code, planes.vs + at.scale, 0, 0, g);
        in.there[x] = page;
      }
    }
  };
  // Takes up the stretch's next unit with groups of its own, its first loads
  // on their way; false: there is none.
  auto take = [&](bool more) {
    for (; more; more = kv_next<kRows, kGroupTokens, kGroupCost>(a, st)) {
      kv_part<kGroupCost>(st, group, last);
      if (group == last) continue;
      table = a.table + u.b * a.table_stride;
      planes = kv_head(a.p, u.head);
      first = u.lo + 32 * wave;
      n = u.hi;
      load_queries(a, u, rows);
      if (n > 0) {
        const Pages p0 = find(group), p1 = find(group + 1);
        pages = find(group + 2);
        fetch(group, p0, even);
        fetch(group + 1, p1, odd);
      }
      return true;
    }
    return false;
  };

  // One unit a turn; it is finished in the next turn, when the next unit's loads
  // are on their way.
  KvUnit done = {};
  int begins = 0;
  bool have = false, whole = false;
  float* part = nullptr;
  f32x4_t o[kTiles][D / 16];
  float m[kTiles], l[kTiles];
  for (;;) {
    const bool more = take(have ? kv_next<kRows, kGroupTokens, kGroupCost>(a, st) : true);
    if (have) {
      // join the four waves: maxima and sums of every row, then the values
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        l[t] += __shfl_xor(l[t], 16, 64);
        l[t] += __shfl_xor(l[t], 32, 64);
        if (g == 0) {
          s_m[wave][16 * t + r] = m[t];
          s_l[wave][16 * t + r] = l[t];
        }
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        __syncthreads();
        const float top = fmaxf(fmaxf(s_m[0][16 * t + r], s_m[1][16 * t + r]), fmaxf(s_m[2][16 * t + r], s_m[3][16 * t + r]));
        const float f = __builtin_amdgcn_exp2f(m[t] - top);
        float* dst = so + (wave * 16 + r) * Shape::kOStride + 4 * g;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) *reinterpret_cast<f32x4_t*>(dst + 16 * c) = o[t][c] * f;
        __syncthreads();
        for (int item = tid; item < 16 * (D / 4); item += kThreads) {
          const int row = item / (D / 4), d = 4 * (item % (D / 4));
          const int rr = 16 * t + row;
          f32x4_t sum = *reinterpret_cast<const f32x4_t*>(so + row * Shape::kOStride + d);
#pragma unroll
          for (int w = 1; w < kWaves; ++w) sum += *reinterpret_cast<const f32x4_t*>(so + (w * 16 + row) * Shape::kOStride + d);
          if (s_nans.count && (s_nans.seen(a, done, done.row0 + rr) >> (d / Lane::kBlock)) & 1u) sum *= as_f(0x7FC00000u);
          const float mx = fmaxf(fmaxf(s_m[0][rr], s_m[1][rr]), fmaxf(s_m[2][rr], s_m[3][rr]));
          float total = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) total += s_l[w][rr] * __builtin_amdgcn_exp2f(s_m[w][rr] - mx);
          if (whole) {
            kv_finish4<FMT, D>(a, done, done.row0 + rr, d, sum, mx, total);
          } else if (done.row0 + rr < done.m * a.group) {
            put2(part + (int64_t)rr * D + d, sum.x, sum.y);
            put2(part + (int64_t)rr * D + d + 2, sum.z, sum.w);
            if (d == 0) put2(part + (int64_t)kRows * D + 2 * rr, mx, total);
          }
        }
      }
      __syncthreads();
      if (!whole) kv_join<FMT, D, kRows, kGroupCost, kThreads, kJoin>(a, done, begins, st.shares, s_most, s_m[0], s_l[0]);
      __syncthreads();
    }
    if (!more) return;
    if (tid == 0) s_nans.count = 0;
    stage_queries<FMT, D, kQ, kRows>(a, kg, rows, sq, s_factor, s_most);

    u32x4_t qf[Shape::kQRegs ? kTiles : 1][Shape::kQRegs ? kQ : 1][Shape::kQRegs ? kChunks : 1];
    float factor[kTiles];
    int sees_from[kTiles];                      // the lane's row sees `sees` tokens from here
    uint32_t sees[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      factor[t] = s_factor[16 * t + r];
      kv_sees(a, u, u.row0 + 16 * t + r, sees_from[t], sees[t]);
      if constexpr (Shape::kQRegs) {
#pragma unroll
        for (int q = 0; q < kQ; ++q)
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            qf[t][q][c] = *reinterpret_cast<const u32x4_t*>(sq + (q * kRows + 16 * t + r) * (D + 8) + Lane::element(c, g));
      }
    }
    if constexpr (Shape::kQRegs) __syncthreads();     // the values' rows overlie the queries
    int all_from, all_to;
    kv_all_see<kRows>(a, u, all_from, all_to);

#pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      m[t] = kNoMax;
      l[t] = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) o[t][c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    auto step = [&](int grp, Tile& in) {
      const int t0 = first + grp * kGroupTokens;
      const bool edge = t0 + 32 > all_to || t0 < all_from;
      if (kWhole ? !in.there[0] : true) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          in.k[x].keep_if(in.there[x]);
          in.v[x].keep_if(in.there[x]);
        }
      }
      if (edge) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int t = t0 + 16 * x + r;
          uint32_t dropped = in.v[x].drop_not_finite();
          if (t >= n) dropped = 0u;
          if (__any(dropped != 0u)) s_nans.template note<FMT, D>(t, g, dropped);
        }
      }
      // scores of 32 tokens x 16 rows, transposed: token 16 x + 4 g + i, row r
      f32x4_t s[kTiles][2];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const typename Lane::Scales sc = in.k[x].prepare();
#pragma unroll
        for (int t = 0; t < kTiles; ++t) s[t][x] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          const u32x4_t kf = in.k[x].values(c, sc);
#pragma unroll
          for (int t = 0; t < kTiles; ++t)
#pragma unroll
            for (int q = 0; q < kQ; ++q) {
              if constexpr (Shape::kQRegs) {
                s[t][x] = T::mfma16(kf, qf[t][q][c], s[t][x]);
              } else {
                const u32x4_t w = *reinterpret_cast<const u32x4_t*>(sq + (q * kRows + 16 * t + r) * (D + 8) +
                                                                    Lane::element(c, g));
                s[t][x] = T::mfma16(kf, w, s[t][x]);
              }
            }
        }
      }
      // values into the wave's LDS rows
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const typename Lane::Scales sc = in.v[x].prepare();
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
          *reinterpret_cast<u32x4_t*>(sv + (16 * x + r) * Shape::kVStride + Lane::element(c, g)) = in.v[x].values(c, sc);
      }
      // (loads come back in order: page numbers asked for before the codes can
      // be waited for without waiting for those)
      const Pages next = find(grp + 3);
      fetch(grp + 2, pages, in);
      pages = next;

      // (scalars and selects throughout: hipcc 7.2 moves the wrong elements of
      // a vector when one is replaced under a lane's condition)
      float y[kTiles][8];
      bool raise = false;
      float most[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int k = 0; k < 8; ++k) y[t][k] = s[t][k >> 2][k & 3];
        if (edge) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t j = (uint32_t)(t0 + 16 * (k >> 2) + 4 * g + (k & 3) - sees_from[t]);
            y[t][k] = j < sees[t] ? y[t][k] : -INFINITY;
          }
        }
        most[t] = y[t][0];
#pragma unroll
        for (int k = 1; k < 8; ++k) most[t] = larger(most[t], y[t][k]);
        most[t] *= factor[t];
        raise |= most[t] > m[t] + kRaise;
      }
      // raise the maxima where a score exceeds them by more than the slack
      if (__any(raise)) {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
          float x = larger(most[t], __shfl_xor(most[t], 16, 64));
          x = larger(x, __shfl_xor(x, 32, 64));
          x = larger(x, m[t]);
          const float f = __builtin_amdgcn_exp2f(m[t] - x);
          m[t] = x;
          l[t] *= f;
#pragma unroll
          for (int c = 0; c < D / 16; ++c) o[t][c] *= f;
        }
      }
      u32x4_t w[kTiles][kP];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const float top = T::kUp - m[t];
        uint32_t h[4][kP];
        // (a step's weights among themselves first: one rounding a step beside
        // what may be far larger.  Before their own: the log-sum-exp is held to fp32)
        float sum = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p0 = __builtin_amdgcn_exp2f(fmaf(y[t][2 * j], factor[t], top));
          const float p1 = __builtin_amdgcn_exp2f(fmaf(y[t][2 * j + 1], factor[t], top));
          sum += p0 + p1;
          weight_pieces<FMT, kP>(p0, p1, h[j]);
        }
        l[t] += sum;
#pragma unroll
        for (int q = 0; q < kP; ++q) w[t][q] = u32x4_t{h[0][q], h[1][q], h[2][q], h[3][q]};
      }
      // weighted values: element 16 c + 4 g + i, row r
      const uint16_t* vp = sv + (4 * g + (r >> 2)) * Shape::kVStride + 4 * (r & 3);
#pragma unroll
      for (int c = 0; c < D / 16; ++c) {
        const u32x2_t x0 = read_transposed(vp + 16 * c), x1 = read_transposed(vp + 16 * Shape::kVStride + 16 * c);
        const u32x4_t vf = {x0.x, x0.y, x1.x, x1.y};
#pragma unroll
        for (int q = 0; q < kP; ++q) {
          const u32x4_t vq = values_of_piece<FMT, kP>(q, vf);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) o[t][c] = T::mfma16(vq, w[t][q], o[t][c]);
        }
      }
    };
    // (this wave's groups: those that begin before the end)
    const int mine = min(last, first < n ? (n - first + kGroupTokens - 1) / kGroupTokens : 0);
    for (int grp = group; grp < mine; grp += 2) {
      step(grp, even);
      if (grp + 1 < mine) step(grp + 1, odd);
    }

    done = u;
    begins = st.begins;
    whole = group == 0 && last == u.groups;
    part = kv_partial<D, kRows>(a, blockIdx.x, group == 0);
    have = true;
  }
}

// Whether a wave's 32 tokens lie in one page and at 32-bit offsets from its
// start: 31 token strides and a row.
inline bool kv_whole_tiles(const KvPlanes& p) {
  return p.page.d % 32 == 0 && p.code_stride[2] <= UINT32_MAX / 32 && p.scale_stride[2] <= UINT32_MAX / 32;
}

template <int FMT, int D, int kTiles, int kQ, int kP>
hipError_t launch_decode_t(const KvAttendLaunch& a, int cus, hipStream_t st) {
  constexpr int kRows = 16 * kTiles;
  KvAttendLaunch b = a;
  const int64_t numbers = kv_block_numbers(b, kRows);
  const int64_t most = kv_most_groups(b, numbers, kGroupTokens, kGroupCost);
  const int64_t resident = (int64_t)cus * DecodeShape<FMT, D, kTiles, kQ, kP>::kWavesPerSimd;
  // Where units have no more groups than one level of the join takes pieces, a
  // workgroup a group; two groups each above, which takes less than the next
  // level (4 x 4000 tokens, 32 rows, head_dim 128: 16.2 us for 18.6; 8 heads x
  // 1000 tokens 11.9 for 11.5).
  const int64_t wanted = a.most_tokens > 2 * kJoin * kGroupTokens ? (most + 1) / 2 : most;
  const int grid = (int)min(min(wanted, resident), (int64_t)kMostWorkgroups);
  b.thirds = (uint32_t)resident;
  if (kv_whole_tiles(a.p))
    hipLaunchKernelGGL((kv_decode_kernel<FMT, D, kTiles, kQ, kP, true>), dim3(grid), dim3(kThreads), 0, st, b, (int)numbers);
  else
    hipLaunchKernelGGL((kv_decode_kernel<FMT, D, kTiles, kQ, kP, false>), dim3(grid), dim3(kThreads), 0, st, b, (int)numbers);
  return hipGetLastError();
}

// The choice of pieces (see fp4q_kv_attend.h): fp32, bf16 rotated, bf16.  More
// than 16 rows only where they fit the registers: bf16, head_dim to 128.
template <int D, int FMT>
hipError_t launch_decode_d(const KvAttendLaunch& a, int tiles, int cus, hipStream_t st) {
  if (a.dtype == kF32) return launch_decode_t<FMT, D, 1, FMT == 1 ? 2 : 3, FMT == 1 ? 2 : 3>(a, cus, st);
  constexpr int kP = FMT == 1 ? 1 : 2;
  const bool two = kv_bf16_pieces(a) == 2;
  if constexpr (D <= 128) {
    if (tiles == 2) return two ? launch_decode_t<FMT, D, 2, 2, kP>(a, cus, st) : launch_decode_t<FMT, D, 2, 1, kP>(a, cus, st);
  }
  return two ? launch_decode_t<FMT, D, 1, 2, kP>(a, cus, st) : launch_decode_t<FMT, D, 1, 1, kP>(a, cus, st);
}

}  // namespace fp4q
