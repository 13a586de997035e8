// fp4q_norm.hip -- root-mean-square norm with the residual's addition in front
// and MXFP8 quantization behind it, and its gradient.
//
//   s = x + residual, rounded to their type;  r = 1 / sqrt(mean(s^2) + eps);
//   y = s r w;  MXFP8: e = floor(log2(largest |y| of 32)) - 8, E4M3(y 2^-e).
//   Backward, with hat = s r and g = dy w:
//   dx = r (g - hat mean(g hat)) + ds,  dw = sum over rows of dy hat.
//
// The norm is that of the stored sum, so that the backward pass, which has the
// stored one only, is that of the same function.  A row lies in the registers of
// one wave (d to 1024), of 4 waves (to 8192) or of 16: it is read once.  Squares
// are summed in fp32, 64 at most in a thread and the rest by halves.
#include "fp4q_ffn.h"

namespace fp4q {
namespace {

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// The sum of v over a row's T threads, in every one of them; `s` one float a wave
// and row, `again` whether an earlier sum may still be read.
template <int T>
__device__ __forceinline__ float row_sum(float v, float* s, bool again) {
  v = wave_sum(v);
  if constexpr (T > 64) {
    if (again) __syncthreads();
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) v += s[i];
  }
  return v;
}

template <typename T, bool NT>
__device__ __forceinline__ T load_wide(const uint8_t* p) {
  typedef T any_t __attribute__((aligned(1)));
  if constexpr (NT) return __builtin_nontemporal_load(reinterpret_cast<const any_t*>(p));
  else return load_any<T>(p);
}

// Eight elements of a row from element c on, zeros past its end.  NT: not kept in
// the caches.
template <bool BF16, bool NT = false>
__device__ __forceinline__ void load8(const void* row, uint32_t c, uint32_t d, float (&v)[8]) {
  const uint8_t* p = static_cast<const uint8_t*>(row) + c * (BF16 ? 2u : 4u);
  if (c + 8 <= d) {
    if constexpr (BF16) {
      const u32x4_t w = load_wide<u32x4_t, NT>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf_lo(w[i]);
        v[2 * i + 1] = bf_hi(w[i]);
      }
    } else {
      const f32x4_t a = load_wide<f32x4_t, NT>(p), b = load_wide<f32x4_t, NT>(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = 0.0f;
      if (c + i < d) v[i] = BF16 ? bf_lo(load_any<uint16_t>(p + 2 * i)) : load_any<float>(p + 4 * i);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* row, uint32_t c, uint32_t d, const float (&v)[8]) {
  uint8_t* p = static_cast<uint8_t*>(row) + c * (BF16 ? 2u : 4u);
  if (c + 8 <= d) {
    if constexpr (BF16) {
      store_any(p, u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
    } else {
      store_any(p, f32x4_t{v[0], v[1], v[2], v[3]});
      store_any(p + 16, f32x4_t{v[4], v[5], v[6], v[7]});
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c + i >= d) continue;
      if constexpr (BF16) store_any(p + 2 * i, (__bf16)v[i]);
      else store_any(p + 4 * i, v[i]);
    }
  }
}

template <bool BF16>
__device__ __forceinline__ const void* at_row(const void* p, int64_t row, int64_t stride) {
  return static_cast<const uint8_t*>(p) + row * stride * (BF16 ? 2 : 4);
}

// MXFP8 of a lane's 8 values, the block being those of 4 neighbouring lanes.  A
// block with an infinity or NaN gets the NaN scale and zero codes, as the other
// quantizers give it.
__device__ __forceinline__ void mxfp8_store(const float (&y)[8], uint8_t* codes, uint8_t* scales, bool in) {
  uint32_t most = abs_max_bits8(y);
  most = max(most, dpp_u32<kQuadXor1>(most));
  most = max(most, dpp_u32<kQuadXor2>(most));
  // the exponent field less 8; below 2^-119 the scale stays at its least, 2^-127
  const bool bad = most >= 0x7F800000u;
  const int e = (int)(most >> 23) - 127 - 8;
  const uint32_t byte = bad ? 255u : most == 0u ? 127u : (uint32_t)(e < -127 ? 0 : e + 127);
  // 2^(127 - byte): byte is at most 246
  const float inv = bad ? 0.0f : as_f((254u - byte) << 23);
  uint32_t o[2] = {0u, 0u};
  if (!bad) {
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(y[i] * inv, -448.0f), 448.0f);   // (past 448: the largest code)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i], q[4 * i + 1], 0, false);
      o[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * i + 2], q[4 * i + 3], (int)o[i], true);
    }
  }
  if (in) {
    store_any(codes, u32x2_t{o[0], o[1]});
    if ((threadIdx.x & 3) == 0) *scales = (uint8_t)byte;
  }
}

// T threads a row, 8 elements a slot, NS slots a thread.  x and the residual are
// read for the last time, and not kept in the caches (8192 rows of 8192, bf16, to
// MXFP8: 98 -> 84 us, 5.6 TB/s); what is written is read next.
template <bool BF16, bool WBF16, bool QUANT, int T, int NS>
__global__ __launch_bounds__(T < 256 ? 256 : T) void norm_kernel(NormLaunch l) {
  constexpr int kRows = T < 256 ? 256 / T : 1;
  __shared__ float s_sum[T / 64];
  const int t = threadIdx.x % T;
  const int64_t row = group_number() * kRows + threadIdx.x / T;
  if (row >= l.rows) return;                  // (whole waves; several rows a workgroup have no barrier)
  float v[NS][8];
  const void* x = at_row<BF16>(l.x, row, l.x_stride);
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < NS; ++i) load8<BF16, true>(x, (int64_t)(i * T + t) * 8, l.d, v[i]);
  if (l.residual) {
    const void* res = at_row<BF16>(l.residual, row, l.residual_stride);
    uint8_t* to = static_cast<uint8_t*>(l.summed) + row * l.d * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      float u[8];
      load8<BF16, true>(res, (int64_t)(i * T + t) * 8, l.d, u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[i][j] += u[j];
        if constexpr (BF16) v[i][j] = (float)(__bf16)v[i][j];
      }
      store8<BF16>(to, (int64_t)(i * T + t) * 8, l.d, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(v[i][j], v[i][j], sum);
  sum = row_sum<T>(sum, s_sum, false);
  const float rstd = 1.0f / sqrtf(sum / (float)l.d + l.eps);
  if (l.rstd && t == 0) l.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int64_t c = (int64_t)(i * T + t) * 8;
    float w[8];
    load8<WBF16>(l.w, c, l.d, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] *= v[i][j] * rstd;
    if constexpr (QUANT) mxfp8_store(w, l.codes + row * l.d + c, l.scales + row * (l.d / 32) + c / 32, c < l.d);
    else store8<BF16>(static_cast<uint8_t*>(l.y) + row * l.d * (BF16 ? 2 : 4), c, l.d, w);
  }
}

// A workgroup takes every gridDim-th row; its threads keep their elements' sums
// of dw, which a second kernel adds in the workgroups' order.  A row is held in
// registers, or (AGAIN, d above 8192, where that would spill them) read a second
// time, from L2.  Held to the registers of two workgroups a CU (4099 rows of 5000,
// fp32: 72 us for 78).
template <bool BF16, bool WBF16, int T, int NS, bool AGAIN>
__global__ __launch_bounds__(T, T <= 512 ? 4 : 1) void norm_grad_kernel(NormGradLaunch l) {
  constexpr int kHeld = AGAIN ? 1 : NS;
  __shared__ float s_sum[T / 64];
  const int t = threadIdx.x;
  float dw[NS][8], w[kHeld][8];
  const uint32_t d = (uint32_t)l.d;
  // Hidden for each row where registers run out: else the compiler keeps all columns'
  // comparisons with the row's end, and spilled (2048 rows of 32768, bf16: 263 us, so
  // 163; 4096 of 8192, 57 and 54; shorter rows, which fit, are up to 15 % slower with it).
  constexpr bool kHide = T == 512 || NS == 4;
  int tt = t;
  auto column = [&](int i) { return (uint32_t)(i * T + tt) * 8; };
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    if constexpr (!AGAIN) load8<WBF16>(l.w, column(i), d, w[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.0f;
  }
  for (int64_t row = blockIdx.x; row < l.rows; row += gridDim.x) {
    if constexpr (kHide) asm volatile("" : "+v"(tt));
    const void* dyr = at_row<BF16>(l.dy, row, l.dy_stride);
    const void* sr = at_row<BF16>(l.s, row, l.s_stride);
    const float rstd = l.rstd[row];
    float g[kHeld][8], hat[kHeld][8], along = 0.0f;
    if constexpr (!AGAIN) {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        load8<BF16>(dyr, column(i), d, g[i]);
        load8<BF16>(sr, column(i), d, hat[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int h = AGAIN ? 0 : i;
      if constexpr (AGAIN) {
        load8<BF16>(dyr, column(i), d, g[0]);
        load8<BF16>(sr, column(i), d, hat[0]);
        load8<WBF16>(l.w, column(i), d, w[0]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hat[h][j] *= rstd;
        dw[i][j] = fmaf(g[h][j], hat[h][j], dw[i][j]);
        g[h][j] *= w[h][j];
        along = fmaf(g[h][j], hat[h][j], along);
      }
    }
    along = row_sum<T>(along, s_sum, true) / (float)l.d;
    if constexpr (kHide && AGAIN) asm volatile("" : "+v"(tt));
    uint8_t* to = static_cast<uint8_t*>(l.dx) + row * l.d * (BF16 ? 2 : 4);
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int h = AGAIN ? 0 : i;
      if constexpr (AGAIN) {
        load8<BF16>(dyr, column(i), d, g[0]);
        load8<BF16>(sr, column(i), d, hat[0]);
        load8<WBF16>(l.w, column(i), d, w[0]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          hat[0][j] *= rstd;
          g[0][j] *= w[0][j];
        }
      }
      float u[8];
      if (l.ds) {
        load8<BF16>(at_row<BF16>(l.ds, row, l.ds_stride), column(i), d, u);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = fmaf(rstd, g[h][j] - hat[h][j] * along, u[j]);
      store8<BF16>(to, column(i), d, u);
    }
  }
  float* part = l.partials + (int64_t)blockIdx.x * l.d;
#pragma unroll
  for (int i = 0; i < NS; ++i) store8<false>(part, column(i), d, dw[i]);
}

// dw = the sum of the parts: a workgroup 64 columns, its 16 waves every sixteenth
// part each, 8 of them in flight (4 waves, one at a time: 36 us for 512 parts of
// 5000).
template <bool WBF16>
__global__ __launch_bounds__(1024) void norm_grad_join_kernel(NormGradLaunch l, int parts) {
  __shared__ float s_part[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float v = 0.0f;
  if (c < l.d) {
    int i = wave;
    for (; i + 16 * 7 < parts; i += 16 * 8) {
      float p[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = l.partials[(int64_t)(i + 16 * j) * l.d + c];
#pragma unroll
      for (int j = 0; j < 8; ++j) v += p[j];
    }
    for (; i < parts; i += 16) v += l.partials[(int64_t)i * l.d + c];
  }
  s_part[wave][lane] = v;
  __syncthreads();
  if (wave == 0 && c < l.d) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += s_part[i][lane];
    if constexpr (WBF16) static_cast<__bf16*>(l.dw)[c] = (__bf16)v;
    else static_cast<float*>(l.dw)[c] = v;
  }
}

int grad_parts(int64_t rows, int64_t d) {
  const int64_t most = (int64_t)device_cu_count() * (d <= 8192 ? 2 : 1);
  return (int)(rows < most ? rows : most);
}

template <bool BF16, bool WBF16, bool QUANT>
hipError_t launch_norm_t(const NormLaunch& l, hipStream_t s) {
#define FP4Q_NORM(T, NS)                                                                                   \
  do {                                                                                                     \
    const int per = T < 256 ? 256 / T : 1;                                                                 \
    const int64_t groups = (l.rows + per - 1) / per;                                                       \
    hipLaunchKernelGGL((norm_kernel<BF16, WBF16, QUANT, T, NS>), dim3(grid_x(groups), grid_y(groups)),     \
                       dim3(T < 256 ? 256 : T), 0, s, l);                                                  \
    return hipGetLastError();                                                                              \
  } while (0)
  if (l.d <= 512) FP4Q_NORM(64, 1);
  if (l.d <= 1024) FP4Q_NORM(64, 2);
  if (l.d <= 2048) FP4Q_NORM(256, 1);
  if (l.d <= 4096) FP4Q_NORM(256, 2);
  if (l.d <= 8192) FP4Q_NORM(256, 4);
  if (l.d <= 16384) FP4Q_NORM(1024, 2);
  FP4Q_NORM(1024, 4);
#undef FP4Q_NORM
}

template <bool BF16, bool WBF16>
hipError_t launch_norm_grad_t(const NormGradLaunch& l, hipStream_t s) {
  const int parts = grad_parts(l.rows, l.d);
  if (l.rows > 0) {
#define FP4Q_GRAD(T, NS, AGAIN) \
  hipLaunchKernelGGL((norm_grad_kernel<BF16, WBF16, T, NS, AGAIN>), dim3(parts), dim3(T), 0, s, l)
    if (l.d <= 512) FP4Q_GRAD(64, 1, false);
    else if (l.d <= 2048) FP4Q_GRAD(256, 1, false);
    else if (l.d <= 4096) FP4Q_GRAD(256, 2, false);
    else if (l.d <= 8192) FP4Q_GRAD(512, 2, false);
    else if (l.d <= 16384) FP4Q_GRAD(1024, 2, true);
    else FP4Q_GRAD(1024, 4, true);
#undef FP4Q_GRAD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(norm_grad_join_kernel<WBF16>, dim3((unsigned)((l.d + 63) / 64)), dim3(1024), 0, s, l, parts);
  return hipGetLastError();
}

// MXFP8 values: a thread 8 elements.
template <int OUT>
__global__ __launch_bounds__(256) void dequant8_kernel(Dequant8Launch l, int64_t slots) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < slots; i += (int64_t)gridDim.x * 256) {
    const u32x2_t c = load_any<u32x2_t>(l.codes + 8 * i);
    const u32x4_t b = e4m3_values8(c, l.scales[i >> 2]);
    if constexpr (OUT == kBF16) {
      store_any(static_cast<uint16_t*>(l.out) + 8 * i, b);
    } else {
      // (through fp32 itself, which holds what bf16's subnormal range would round)
      const float s = e8m0_operand(l.scales[i >> 2]);
      float2_t p[4];
      p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)c.x, s, false);
      p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)c.x, s, true);
      p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)c.y, s, false);
      p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8((int)c.y, s, true);
      float* o = static_cast<float*>(l.out) + 8 * i;
      store_any(o, f32x4_t{p[0].x, p[0].y, p[1].x, p[1].y});
      store_any(o + 4, f32x4_t{p[2].x, p[2].y, p[3].x, p[3].y});
    }
  }
}

}  // namespace

hipError_t launch_rms_norm(const NormLaunch& l, hipStream_t s) {
  const bool q = l.codes != nullptr;
  if (l.bf16) {
    if (l.w_bf16) return q ? launch_norm_t<true, true, true>(l, s) : launch_norm_t<true, true, false>(l, s);
    return q ? launch_norm_t<true, false, true>(l, s) : launch_norm_t<true, false, false>(l, s);
  }
  if (l.w_bf16) return q ? launch_norm_t<false, true, true>(l, s) : launch_norm_t<false, true, false>(l, s);
  return q ? launch_norm_t<false, false, true>(l, s) : launch_norm_t<false, false, false>(l, s);
}

size_t rms_norm_grad_workspace(int64_t rows, int64_t d) { return (size_t)grad_parts(rows, d) * d * sizeof(float); }

hipError_t launch_rms_norm_grad(const NormGradLaunch& l, hipStream_t s) {
  if (l.bf16) return l.w_bf16 ? launch_norm_grad_t<true, true>(l, s) : launch_norm_grad_t<true, false>(l, s);
  return l.w_bf16 ? launch_norm_grad_t<false, true>(l, s) : launch_norm_grad_t<false, false>(l, s);
}

hipError_t launch_dequant8(const Dequant8Launch& l, hipStream_t s) {
  const int64_t slots = l.rows * l.cols / 8, want = (slots + 255) / 256;
  const int64_t cap = (int64_t)device_cu_count() * 64;
  const unsigned grid = (unsigned)(want < cap ? want : cap);
  if (l.out_dtype == kBF16) hipLaunchKernelGGL(dequant8_kernel<kBF16>, dim3(grid), dim3(256), 0, s, l, slots);
  else hipLaunchKernelGGL(dequant8_kernel<kF32>, dim3(grid), dim3(256), 0, s, l, slots);
  return hipGetLastError();
}

}  // namespace fp4q
