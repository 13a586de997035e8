// fp4q_linear_few.hip -- y = x W^T and h = SiLU(x Wg^T) * (x Wu^T) for few rows
// of x: a stream over the 4-bit weight.
//
// A workgroup of 8 waves takes 16 NT rows of the weight (a gated call half of
// them from each factor) and all rows of x; its waves take every eighth chunk of
// 128 k, so that together they read 512 contiguous bytes of each row, and their
// sums meet in LDS.  Nothing crosses workgroups, so the order of sums is fixed.
//
// v_mfma_f32_16x16x32_bf16 with weights as the left operand: lane l holds row l
// mod 16 and the chunk's k = 32 (l / 16) .. + 31, 16 bytes of codes, which four
// instructions take eight at a time; x, the right operand, is read in the same
// order, 64 contiguous bytes (bf16) of row l mod 16 of x a lane.  The result has
// 4 consecutive weight rows of one x row in a lane.
#include "fp4q_ffn.h"

namespace fp4q {
namespace {

constexpr int kFewWaves = 8;
constexpr int kChunk = 128;

template <int NT>
struct FewCodes {
  u32x4_t c[NT];
  uint32_t s[NT];
};
template <int XT, int MT>
struct FewX {
  static constexpr int kWords = XT == kXF32 ? 32 : XT == kXBF16 ? 16 : 8;
  uint32_t v[MT][kWords];
  uint32_t s[MT];
};

template <int FMT, int XT, int MT, int NT, bool GATED>
__global__ __launch_bounds__(64 * kFewWaves) void few_kernel(LinearLaunch l) {
  constexpr int kHalves = GATED ? 2 : 1;
  constexpr int kSide = NT / kHalves;            // tiles of each factor
  constexpr int kElem = XT == kXF32 ? 4 : XT == kXBF16 ? 2 : 1;
  constexpr int P = kPieces<XT>;
  __shared__ float s_sum[kFewWaves][NT * MT][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t K = l.w.k, half = l.w.n / kHalves;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * kSide);
  const int64_t srow = K / (FMT == 0 ? 32 : 16);

  // rows past the ends read the last one; their results are not stored
  const uint8_t *wc[NT], *ws[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int64_t n = min(n0 + 16 * (t % kSide) + r, half - 1) + (t / kSide) * half;
    wc[t] = l.w.codes + n * (K / 2) + 16 * g;
    ws[t] = l.w.scales + n * srow + (FMT == 0 ? g : 2 * g);
  }
  const uint8_t *xp[MT], *xs[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = min((int64_t)16 * m + r, l.rows - 1);
    xp[m] = static_cast<const uint8_t*>(l.x) + (row * l.x_stride + 32 * g) * kElem;
    xs[m] = XT == kXE4M3 ? l.x_scales + row * (K / 32) + g : nullptr;
  }

  const int chunks = (int)((K + kChunk - 1) / kChunk);
  // elements of this lane's 32 that lie before the row's end: 32, 16 or none
  auto valid = [&](int c) { return K - ((int64_t)c * kChunk + 32 * g); };
  auto load_w = [&](int c, FewCodes<NT>& d) {
    const int64_t at = (int64_t)c * (kChunk / 2), sat = (int64_t)c * (FMT == 0 ? 4 : 8);
    if ((int64_t)(c + 1) * kChunk <= K) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        d.c[t] = load_any<u32x4_t>(wc[t] + at);
        d.s[t] = FMT == 0 ? ws[t][sat] : load_any<uint16_t>(ws[t] + sat);
      }
    } else {
      const int64_t v = valid(c);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        d.c[t] = u32x4_t{0u, 0u, 0u, 0u};
        d.s[t] = 0u;
        if (v >= 32) {
          d.c[t] = load_any<u32x4_t>(wc[t] + at);
          d.s[t] = FMT == 0 ? ws[t][sat] : load_any<uint16_t>(ws[t] + sat);
        } else if (v >= 16) {
          const u32x2_t w = load_any<u32x2_t>(wc[t] + at);
          d.c[t].x = w.x;
          d.c[t].y = w.y;
          d.s[t] = ws[t][sat];
        }
      }
    }
  };
  auto load_x = [&](int c, FewX<XT, MT>& d) {
    constexpr int kWords = FewX<XT, MT>::kWords;
    const int64_t at = (int64_t)c * kChunk * kElem;
    const int64_t v = valid(c);
    if ((int64_t)(c + 1) * kChunk <= K) {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          const u32x4_t w = load_any<u32x4_t>(xp[m] + at + 4 * i);
          d.v[m][i] = w.x; d.v[m][i + 1] = w.y; d.v[m][i + 2] = w.z; d.v[m][i + 3] = w.w;
        }
        if constexpr (XT == kXE4M3) d.s[m] = xs[m][4 * c];
      }
    } else {
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        d.s[m] = 0u;
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
          // (the first half of the words are the first 16 elements)
          const bool in = v >= 32 || (v >= 16 && i < kWords / 2);
          const u32x4_t w = in ? load_any<u32x4_t>(xp[m] + at + 4 * i) : u32x4_t{0u, 0u, 0u, 0u};
          d.v[m][i] = w.x; d.v[m][i + 1] = w.y; d.v[m][i + 2] = w.z; d.v[m][i + 3] = w.w;
        }
        if constexpr (XT == kXE4M3) {
          if (v >= 32) d.s[m] = xs[m][4 * c];
        }
      }
    }
  };

  f32x4_t acc[NT][MT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[t][m] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  auto multiply = [&](const FewCodes<NT>& w, const FewX<XT, MT>& x) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u32x4_t xf[MT][P];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if constexpr (XT == kXF32) split8(&x.v[m][8 * j], xf[m]);
        else if constexpr (XT == kXBF16)
          xf[m][0] = u32x4_t{x.v[m][4 * j], x.v[m][4 * j + 1], x.v[m][4 * j + 2], x.v[m][4 * j + 3]};
        else xf[m][0] = e4m3_values8(u32x2_t{x.v[m][2 * j], x.v[m][2 * j + 1]}, x.s[m]);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const uint32_t s = FMT == 0 ? w.s[t] : (w.s[t] >> (8 * (j >> 1)));
        const u32x4_t wf = weights8<FMT>(w.c[t][j], scale_operand<FMT>(s));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int p = 0; p < P; ++p) acc[t][m] = mfma16(wf, xf[m][p], acc[t][m]);
      }
    }
  };

  // two chunks of codes in flight; x comes from L2, one chunk at a time
  FewCodes<NT> w0, w1;
  if (wave < chunks) load_w(wave, w0);
  for (int c = wave; c < chunks; c += 2 * kFewWaves) {
    FewX<XT, MT> x;
    load_x(c, x);
    __builtin_amdgcn_sched_barrier(0);
    const int c1 = c + kFewWaves, c2 = c + 2 * kFewWaves;
    if (c1 < chunks) load_w(c1, w1);
    multiply(w0, x);
    if (c1 < chunks) {
      load_x(c1, x);
      __builtin_amdgcn_sched_barrier(0);
      if (c2 < chunks) load_w(c2, w0);
      multiply(w1, x);
    }
  }

#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int m = 0; m < MT; ++m)
      *reinterpret_cast<f32x4_t*>(s_sum[wave][t * MT + m][lane]) = acc[t][m];
  __syncthreads();

  // element (row of x, weight row) of the joined sums
  const float tensor = FMT == 1 ? *l.w.g : 1.0f;
  auto sum = [&](int t, int m, int n) {
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) s += s_sum[w][t * MT + (m >> 4)][(m & 15) + 16 * (n >> 2)][n & 3];
    return s * tensor;
  };
  auto put = [&](void* to, int64_t at, float v, int bf16) {
    if (bf16) static_cast<__bf16*>(to)[at] = (__bf16)v;
    else static_cast<float*>(to)[at] = v;
  };
  for (int e = threadIdx.x; e < 16 * MT * 16 * kSide; e += 64 * kFewWaves) {
    const int m = e / (16 * kSide), nn = e % (16 * kSide);
    const int64_t n = n0 + nn;
    if (m >= l.rows || n >= half) continue;
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

template <int FMT, int XT, int MT, int NT, bool GATED>
hipError_t launch_t(const LinearLaunch& l, hipStream_t s) {
  const int64_t n = GATED ? l.w.n / 2 : l.w.n;
  const int64_t per = 16 * (GATED ? NT / 2 : NT);
  hipLaunchKernelGGL((few_kernel<FMT, XT, MT, NT, GATED>), dim3((unsigned)((n + per - 1) / per)),
                     dim3(64 * kFewWaves), 0, s, l);
  return hipGetLastError();
}

template <int FMT, int XT, bool GATED>
hipError_t launch_m(const LinearLaunch& l, hipStream_t s) {
  constexpr int NT = GATED ? 2 : 1;
  if (l.rows <= 16) return launch_t<FMT, XT, 1, NT, GATED>(l, s);
  if (l.rows <= 32) return launch_t<FMT, XT, 2, 2, GATED>(l, s);
  return launch_t<FMT, XT, 4, 2, GATED>(l, s);
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
