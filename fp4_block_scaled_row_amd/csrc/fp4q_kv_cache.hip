// fp4q_kv_cache.hip -- writing keys and values into the paged 4-bit cache and
// reading them back.
//
// A lane holds 8 consecutive elements of one (token, head) vector, so a
// 16-block is a lane pair, a 32-block a lane quad and a 128-point transform
// 16 lanes, as in the library's other quantizers, whose bytes these match.
#include "fp4q_kv.h"
#include "fp4q_nv_common.h"

namespace fp4q {
namespace {

// ----------------------------------------------------------------------------
// NVFP4 encoding against a given tensor scale g, one block's factors computed
// where they are used: the calls that matter most write a few rows, where a
// table of every scale's factors would take longer than the rows.
//   s = RNE_E4M3(bamax / (6 g)) and codes RNE_E2M1(x / (s g)) are the roundings
// of the exact quotients.
//   - g of at most 16 significant bits (a power of two, say): 6 g, s g and
//     every decision point p times them (p to 5 bits, s 4) are fp32 numbers.
//     x is one of them or differs by a unit in the last place at least, which
//     moves the quotient by more than half of p's, so the correctly rounded
//     fp32 quotient is on the same side of p as the exact one, or on it.  It is
//     x times the rounded reciprocal, corrected by two FMAs.  (Such g make
//     exact ties common in bf16 values, in every other wave's worth: a
//     resolution of each was most of this kernel's time.)
//   - other g in [2^-100, 2^100]: fp32 products with the reciprocal off by
//     -+2^-21 bracket each quotient (product, reciprocal and bracket round by
//     2^-24 each); brackets that disagree are resolved by the sign of an exact
//     FMA residual.
//   - the rest: fp64 quotients.
__device__ __noinline__ uint32_t nv_encode_wide(const float v[8], float bamax, float g, uint32_t& scale) {
  const double mg = 6.0 * (double)g;
  scale = e4m3_encode_exact(bamax, (double)bamax / mg, mg);
  const double den = (double)e4m3_value(scale) * (double)g;
  uint32_t codes = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t mag = scale ? e2m1_rne_mag_f64(fabs((double)v[i]) / den) : 0u;
    codes |= (mag | ((as_u(v[i]) >> 31) << 3)) << (4 * i);
  }
  return codes;
}

struct NvScale {
  float g, g6, inv6;
  bool few_bits, wide;
};
__device__ __forceinline__ NvScale nv_scale(float g) {
  NvScale n;
  n.g = g;
  n.g6 = 6.0f * g;
  n.inv6 = 1.0f / n.g6;
  n.wide = !(g >= 0x1p-100f && g <= 0x1p100f);
  n.few_bits = !n.wide && (as_u(g) & 0xFFu) == 0u;
  return n;
}

__device__ __forceinline__ uint32_t pack_fp4(const float q[8]) {
  const float one = e8m0_operand(127u);
  uint32_t c = 0u;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[0], q[1], one, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[2], q[3], one, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[4], q[5], one, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[6], q[7], one, 3);
  return c;
}

// x / d correctly rounded, from inv = RN(1 / d).  (The residual negated, so that
// a zero keeps x's sign.)
__device__ __forceinline__ float quotient_rn(float x, float d, float inv) {
  const float q = x * inv;
  return fmaf(-fmaf(q, d, -x), inv, q);
}

__device__ __forceinline__ uint32_t nv_encode_block(const float v[8], float bamax, const NvScale& n, uint32_t& scale) {
  if (n.wide) return nv_encode_wide(v, bamax, n.g, scale);
  // (a block so far above the tensor scale's range that quotients may overflow
  // takes the next form)
  if (n.few_bits && bamax * n.inv6 < 0x1p20f) {
    const float t = fminf(quotient_rn(bamax, n.g6, n.inv6), 448.0f);
    const uint32_t c = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(t, t, 0, false) & 0xFFu;
    const float d = e4m3_value_hw(c) * n.g;
    const float inv = c ? 1.0f / d : 0.0f;
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = quotient_rn(v[i], d, inv);
    scale = c;
    return pack_fp4(q);
  }
  constexpr float kBelow = 1.0f - 0x1p-21f, kAbove = 1.0f + 0x1p-21f;
  const uint32_t c = nv_scale_code(bamax, n.inv6 * kBelow, n.inv6 * kAbove, 0.0, 0.0, false, 6.0f, n.g);
  const float sd = e4m3_value_hw(c);
  const float inv = c ? 1.0f / (sd * n.g) : 0.0f;
  const float lo = inv * kBelow, hi = inv * kAbove;
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * lo;
  uint32_t a = pack_fp4(q);
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i] * hi;
  const uint32_t d = (a ^ pack_fp4(q)) & 0x77777777u;
  if (d != 0u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if ((d >> (4 * i)) & 7u) {
        const uint32_t mag = e2m1_rne_mag_exact(fabsf(v[i]), (a >> (4 * i)) & 7u, sd, n.g);
        a = (a & ~(7u << (4 * i))) | (mag << (4 * i));
      }
    }
  }
  scale = c;
  return a;
}

__device__ __forceinline__ uint32_t mx_encode_block(const float v[8], uint32_t amax, uint32_t& scale) {
  const int e = (amax == 0u) ? 0 : max((int)(amax >> 23) - 129, -127);
  scale = (uint32_t)(e + 127);
  const float sc = e8m0_operand(scale);
  uint32_t codes = 0u;
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[0], v[1], sc, 0);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[2], v[3], sc, 1);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[4], v[5], sc, 2);
  codes = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, v[6], v[7], sc, 3);
  return codes;
}

// A thread takes kSlots slots, a workgroup's width apart (all loads first).
// Large calls: 6760 tokens of 8 heads x 128, bf16, keys rotated, NVFP4, 35 MB in
// 19 us, 1.9 TB/s: 178 vector instructions a slot, 8 us of issue, after loads and
// stores of 7, hardly overlapped (without the encoding 10 us).  Addresses held in
// scalars, 1, 2 or 8 slots, and workgroups that go on with the next loads in
// flight were no faster; a table of the scales' factors, whose set-up only this
// instance (four slots) would pay, has not been tried.  Small ones by latency, 3 us.
template <int FMT, int IN, int kSlots>
__global__ __launch_bounds__(kThreads) void kv_write_kernel(KvWriteLaunch w, float rot_scale, FastDiv row_slots,
                                                            FastDiv heads, uint32_t nslots) {
  const bool values = blockIdx.y != 0;
  const uint32_t s0 = blockIdx.x * (kSlots * kThreads) + threadIdx.x;
  const int64_t token_stride = values ? w.v_stride[0] : w.k_stride[0], head_stride = values ? w.v_stride[1] : w.k_stride[1];
  const void* x = values ? w.v : w.k;
  uint32_t head[kSlots], at[kSlots];
  int64_t slot[kSlots];
  SlotRaw<IN> raw[kSlots];
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    const uint32_t s = min(s0 + u * kThreads, nslots - 1);
    const uint32_t row = quotient(s, row_slots), token = quotient(row, heads);
    at[u] = s - row * row_slots.d;
    head[u] = row - token * heads.d;
    slot[u] = w.slots[token];
    const int64_t off = token * token_stride + head[u] * head_stride + 8 * at[u];
    if constexpr (IN == kF32) {
      const float* p = static_cast<const float*>(x) + off;
      const u32x4_t a = load16<true>(p), b = load16<true>(p + 4);
      raw[u].w[0] = a.x; raw[u].w[1] = a.y; raw[u].w[2] = a.z; raw[u].w[3] = a.w;
      raw[u].w[4] = b.x; raw[u].w[5] = b.y; raw[u].w[6] = b.z; raw[u].w[7] = b.w;
    } else {
      const u32x4_t a = load16<true>(static_cast<const uint16_t*>(x) + off);
      raw[u].w[0] = a.x; raw[u].w[1] = a.y; raw[u].w[2] = a.z; raw[u].w[3] = a.w;
    }
  }
  const int64_t held = (int64_t)w.p.num_pages * w.p.page.d;
  const NvScale ns = nv_scale(FMT == 0 ? 1.0f : *(values ? w.p.vg : w.p.kg));
  uint8_t* cbase = values ? w.p.vc : w.p.kc;
  uint8_t* sbase = values ? w.p.vs : w.p.ks;
#pragma unroll
  for (int u = 0; u < kSlots; ++u) {
    float v[8];
    widen_slot<IN>(raw[u], v);
    // (head_dim is a multiple of 128 here, so 16 consecutive lanes hold one chunk)
    if (w.rotate && !values) fwht128_lanes(v, threadIdx.x & 15, rot_scale);
    uint32_t amax = abs_max_bits8(v);
    amax = max(amax, dpp_u32<kQuadXor1>(amax));
    if constexpr (FMT == 0) amax = max(amax, dpp_u32<kQuadXor2>(amax));
    uint32_t scale, codes;
    if constexpr (FMT == 0) codes = mx_encode_block(v, amax, scale);
    else codes = nv_encode_block(v, as_f(amax), ns, scale);
    if (amax >= 0x7F800000u) {   // a block with an infinity or NaN: the NaN scale code
      codes = 0u;
      scale = FMT == 0 ? 0xFFu : 0x7Fu;
    }
    if (s0 + u * kThreads >= nslots || slot[u] < 0 || slot[u] >= held) continue;
    // (64-bit division only where a slot does not fit 32 bits)
    const int64_t page = slot[u] <= 0x7FFFFFFF ? (int64_t)quotient((uint32_t)slot[u], w.p.page) : slot[u] / w.p.page.d;
    const int64_t offset = slot[u] - page * w.p.page.d;
    const int64_t c = page * w.p.code_stride[0] + (int64_t)head[u] * w.p.code_stride[1] + offset * w.p.code_stride[2];
    *reinterpret_cast<uint32_t*>(cbase + c + 4 * at[u]) = codes;
    constexpr uint32_t per = FMT == 0 ? 4u : 2u;   // lanes of one block
    if ((at[u] & (per - 1)) == 0) {
      const int64_t e = page * w.p.scale_stride[0] + (int64_t)head[u] * w.p.scale_stride[1] + offset * w.p.scale_stride[2];
      sbase[e + at[u] / per] = (uint8_t)scale;
    }
  }
}

template <int FMT, int kSlots>
hipError_t launch_write_n(const KvWriteLaunch& w, uint32_t nslots, hipStream_t st) {
  const uint32_t per = (uint32_t)w.head_dim / 8;
  const dim3 grid((nslots + kSlots * kThreads - 1) / (kSlots * kThreads), 2);
  const float c = (float)(1.0 / sqrt(128.0));
  if (w.in_dtype == kF32)
    hipLaunchKernelGGL((kv_write_kernel<FMT, kF32, kSlots>), grid, dim3(kThreads), 0, st, w, c, fast_div(per),
                       fast_div((uint32_t)w.p.heads), nslots);
  else
    hipLaunchKernelGGL((kv_write_kernel<FMT, kBF16, kSlots>), grid, dim3(kThreads), 0, st, w, c, fast_div(per),
                       fast_div((uint32_t)w.p.heads), nslots);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_write_t(const KvWriteLaunch& w, int64_t first, int64_t count, hipStream_t st) {
  KvWriteLaunch part = w;
  const size_t esz = w.in_dtype == kF32 ? 4 : 2;
  part.k = static_cast<const char*>(w.k) + first * w.k_stride[0] * esz;
  part.v = static_cast<const char*>(w.v) + first * w.v_stride[0] * esz;
  part.slots = w.slots + first;
  const uint32_t nslots = (uint32_t)(count * w.p.heads * (w.head_dim / 8));
  // four slots a thread once that still leaves every CU a workgroup (865 thousand
  // slots a plane: 15 us against 18 with one)
  if (nslots >= (uint32_t)device_cu_count() * 4 * kThreads) return launch_write_n<FMT, 4>(part, nslots, st);
  return launch_write_n<FMT, 1>(part, nslots, st);
}

// ----------------------------------------------------------------------------
// Last index b < n with cu[b] <= t, of a cumulative array cu[0..n] (cu[0] = 0),
// for a t that the wave shares: 64 entries at a time, whose loads do not wait
// for each other, up to 512 of them, by bisection beyond.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int n, int64_t t) {
  const int lane = threadIdx.x & 63;
  if (n <= 512) {
    int before = 0;
    for (int i = 0; i < n; i += 64) before += __popcll(__ballot(i + lane < n && cu[min(i + lane, n)] <= t));
    return max(before - 1, 0);
  }
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Reading.  What takes time is the chain of dependent loads from an output row
// to its bytes (sequence, page number, codes), so a workgroup goes through a
// run of slots kReadSlots a thread at a time, with the codes of the next step
// and the page numbers of the one after in flight; it finds its first row's
// sequence once and goes on from there, the next kAhead sequences' bounds being
// in LDS.  Bound by the stores: 16 sequences of up to 16384 tokens, 8 heads x 128,
// 932 MB in 195 us, 4.8 TB/s (the library's copies and dequantizations of such
// sizes reach 6.1 to 6.4).
constexpr int kAhead = kThreads;

// p = RN(v g) moved by its last bit towards the exact product where it is a bf16
// midpoint and not that product itself.  The sign of the rounding error is that
// of an FMA, at a scale where nothing underflows.
__device__ __forceinline__ float off_midpoint(float v, float g, float p) {
  const float a = fabsf(v), b = fabsf(p), up = b < 1.0f ? 0x1p64f : 1.0f;
  const float e = fmaf(a * up, g, -(b * up));
  const int by = (e > 0.0f ? 1 : 0) - (e < 0.0f ? 1 : 0);
  return (as_u(p) & 0xFFFFu) == 0x8000u ? as_f(as_u(p) + (uint32_t)by) : p;
}

template <int FMT, int OUT>
__device__ __forceinline__ void read_store(float v[8], bool rotate, float g, void* out, int64_t o) {
  if constexpr (OUT == kF32) {
    if (FMT != 0 && !rotate) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= g;
    }
    u32x4_t* dst = reinterpret_cast<u32x4_t*>(static_cast<float*>(out) + o);
    __builtin_nontemporal_store(u32x4_t{as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3])}, dst);
    __builtin_nontemporal_store(u32x4_t{as_u(v[4]), as_u(v[5]), as_u(v[6]), as_u(v[7])}, dst + 1);
  } else {
    // v s g is rounded once (the rotated values are sums, rounded twice): an
    // fp32 product that sits on a bf16 midpoint is moved off it first, to the
    // side on which the exact product lies
    if (FMT != 0 && !rotate) {
      float p[8];
      bool tie = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = v[i] * g;
        tie |= (as_u(p[i]) & 0xFFFFu) == 0x8000u;
      }
      if (tie) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = off_midpoint(v[i], g, p[i]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bf16x2_t pk = {(__bf16)v[2 * i], (__bf16)v[2 * i + 1]};
      h[i] = __builtin_bit_cast(uint32_t, pk);
    }
    __builtin_nontemporal_store(u32x4_t{h[0], h[1], h[2], h[3]},
                                reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + o));
  }
}

template <int FMT, int OUT, int kReadSlots>
__global__ __launch_bounds__(kThreads) void kv_read_kernel(KvReadLaunch r, float rot_scale, FastDiv row_slots,
                                                           FastDiv heads, uint32_t nslots, int64_t first,
                                                           uint32_t steps) {
  constexpr int kReadStep = kReadSlots * kThreads;
  const bool values = r.k_out == nullptr || blockIdx.y != 0;
  const bool rotate = r.rotate && !values;
  const uint8_t* cbase = values ? r.p.vc : r.p.kc;
  const uint8_t* sbase = values ? r.p.vs : r.p.ks;
  void* out = values ? r.v_out : r.k_out;
  const float g = FMT == 0 ? 1.0f : *(values ? r.p.vg : r.p.kg);
  const int64_t holds = min((int64_t)r.table_cols * r.p.page.d, (int64_t)0x7FFFFFFF);
  const uint32_t begin = blockIdx.x * steps * kReadStep + threadIdx.x;

  // Where slots of a step are: set by look() as far as the page number, by
  // codes() from there on.
  struct Where {
    int32_t page;
    uint32_t offset, head, at;
  };
  struct Bytes {
    uint32_t codes, scale;
  };
  Where where[kReadSlots];
  Bytes bytes[kReadSlots];
  // the sequence of the slot looked at last: rows [row0, row1), which are its
  // tokens from row0 + shift on
  __shared__ int32_t s_cu[kAhead], s_start[kAhead];
  const int b0 = sequence_of(r.cu, r.seqs,
                             first + quotient(quotient(min(begin - threadIdx.x, nslots - 1), row_slots), heads));
  {
    const int i = min(b0 + (int)threadIdx.x, r.seqs);
    s_cu[threadIdx.x] = r.cu[i];
    s_start[threadIdx.x] = r.starts && i < r.seqs ? r.starts[i] : 0;
  }
  __syncthreads();
  int b = b0;
  int64_t row0 = 0, row1 = 0, shift = 0;
  auto sequence = [&](int next) {
    b = next;
    const int i = b - b0;
    if (i + 1 < kAhead) {
      row0 = s_cu[i];
      row1 = s_cu[i + 1];
      shift = s_start[i] - row0;
    } else {
      row0 = r.cu[b];
      row1 = r.cu[b + 1];
      shift = (r.starts ? r.starts[b] : 0) - row0;
    }
  };
  auto look = [&](uint32_t s0) {
#pragma unroll
    for (int u = 0; u < kReadSlots; ++u) {
      const uint32_t s = min(s0 + u * kThreads, nslots - 1);
      const uint32_t row = quotient(s, row_slots), token = quotient(row, heads);
      where[u].at = s - row * row_slots.d;
      where[u].head = row - token * heads.d;
      const int64_t t = first + token;
      while (t >= row1 && b + 1 < r.seqs) sequence(b + 1);
      const int64_t pos = t + shift;
      where[u].page = -1;
      if (t >= row0 && t < row1 && pos >= 0 && pos < holds) {
        const uint32_t col = quotient((uint32_t)pos, r.p.page);
        where[u].offset = (uint32_t)pos - col * r.p.page.d;
        where[u].page = r.table[b * r.table_stride + col];
      }
    }
  };
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < kReadSlots; ++u) {
      bytes[u] = {0u, FMT == 0 ? 127u : 0u};
      if ((uint32_t)where[u].page < (uint32_t)r.p.num_pages) {
        const uint64_t c = (uint64_t)where[u].page * r.p.code_stride[0] + (uint64_t)where[u].head * r.p.code_stride[1] +
                           (uint64_t)where[u].offset * r.p.code_stride[2];
        const uint64_t e = (uint64_t)where[u].page * r.p.scale_stride[0] + (uint64_t)where[u].head * r.p.scale_stride[1] +
                           (uint64_t)where[u].offset * r.p.scale_stride[2];
        bytes[u].codes = *reinterpret_cast<const uint32_t*>(cbase + c + 4 * where[u].at);
        bytes[u].scale = sbase[e + (FMT == 0 ? where[u].at >> 2 : where[u].at >> 1)];
      }
    }
  };
  sequence(b0);
  look(begin);
  fetch();
  if (steps > 1) look(begin + kReadStep);
  for (uint32_t i = 0; i < steps; ++i) {
    const uint32_t s0 = begin + i * kReadStep;
    if (s0 - threadIdx.x >= nslots) return;
    Bytes now[kReadSlots];
#pragma unroll
    for (int u = 0; u < kReadSlots; ++u) now[u] = bytes[u];
    if (i + 1 < steps) {
      fetch();
      look(s0 + 2 * kReadStep);
    }
#pragma unroll
    for (int u = 0; u < kReadSlots; ++u) {
      float v[8];
      const float sc = e8m0_operand(FMT == 0 ? now[u].scale : 127u);     // (E8M0 255 gives NaN)
      float2_t p;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(now[u].codes, sc, 0); v[0] = p.x; v[1] = p.y;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(now[u].codes, sc, 1); v[2] = p.x; v[3] = p.y;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(now[u].codes, sc, 2); v[4] = p.x; v[5] = p.y;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(now[u].codes, sc, 3); v[6] = p.x; v[7] = p.y;
      if constexpr (FMT != 0) {
        const uint32_t e = now[u].scale & 0x7Fu;
        const float sd = e4m3_value_hw(e);        // (0x7F gives NaN)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] *= sd;   // exact: 2 and 4 significant bits
      }
      if (rotate) {
        if constexpr (FMT != 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] *= g;
        }
        fwht128_lanes(v, threadIdx.x & 15, rot_scale);
      }
      const uint32_t s = s0 + u * kThreads;
      if (s < nslots) read_store<FMT, OUT>(v, rotate, g, out, (first * heads.d * row_slots.d + s) * 8);
    }
  }
}

template <int FMT, int kReadSlots>
hipError_t launch_read_n(const KvReadLaunch& r, int64_t first, uint32_t nslots, hipStream_t st) {
  constexpr uint32_t kReadStep = kReadSlots * kThreads;
  const uint32_t per = (uint32_t)r.head_dim / 8, planes = r.k_out && r.v_out ? 2 : 1;
  // at most 32 workgroups a CU (203 us for 0.9 GB of a batch's values, 209 with
  // 16, 226 with 8)
  const uint32_t all = (nslots + kReadStep - 1) / kReadStep, most = (uint32_t)device_cu_count() * 32 / planes;
  const uint32_t steps = (all + most - 1) / most;
  const dim3 grid((all + steps - 1) / steps, planes);
  const float c = (float)(1.0 / sqrt(128.0));
  if (r.out_dtype == kF32)
    hipLaunchKernelGGL((kv_read_kernel<FMT, kF32, kReadSlots>), grid, dim3(kThreads), 0, st, r, c, fast_div(per),
                       fast_div((uint32_t)r.p.heads), nslots, first, steps);
  else
    hipLaunchKernelGGL((kv_read_kernel<FMT, kBF16, kReadSlots>), grid, dim3(kThreads), 0, st, r, c, fast_div(per),
                       fast_div((uint32_t)r.p.heads), nslots, first, steps);
  return hipGetLastError();
}

template <int FMT>
hipError_t launch_read_t(const KvReadLaunch& r, int64_t first, int64_t count, hipStream_t st) {
  const uint32_t nslots = (uint32_t)(count * r.p.heads * (r.head_dim / 8));
  // four slots a thread once that still leaves every CU a workgroup
  if (nslots >= (uint32_t)device_cu_count() * 4 * kThreads) return launch_read_n<FMT, 4>(r, first, nslots, st);
  return launch_read_n<FMT, 1>(r, first, nslots, st);
}

// Slots of one launch fit 31 bits; longer calls run as several launches.
int64_t tokens_per_launch(int heads, int head_dim) {
  const int64_t n = ((int64_t)1 << 30) / ((int64_t)heads * (head_dim / 8));
  return n < 1 ? 1 : n;
}

}  // namespace

hipError_t launch_kv_write(const KvWriteLaunch& w, hipStream_t st) {
  const int64_t step = tokens_per_launch(w.p.heads, w.head_dim);
  for (int64_t at = 0; at < w.tokens; at += step) {
    const int64_t n = w.tokens - at < step ? w.tokens - at : step;
    const hipError_t e = w.format == 0 ? launch_write_t<0>(w, at, n, st) : launch_write_t<1>(w, at, n, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_kv_read(const KvReadLaunch& r, hipStream_t st) {
  const int64_t step = tokens_per_launch(r.p.heads, r.head_dim);
  for (int64_t at = 0; at < r.total; at += step) {
    const int64_t n = r.total - at < step ? r.total - at : step;
    const hipError_t e = r.format == 0 ? launch_read_t<0>(r, at, n, st) : launch_read_t<1>(r, at, n, st);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace fp4q
