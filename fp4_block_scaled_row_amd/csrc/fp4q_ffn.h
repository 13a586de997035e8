// fp4q_ffn.h -- linear layers over 4-bit weights, and the norm in front of
// them: the launch interface between the C ABI (fp4q_ffn_api.hip) and the
// kernels, and what the kernels share.
//
//   y = x W^T (+ b)     dx = dy W     h = SiLU(x Wg^T) * (x Wu^T)
//
// A weight [n][k] is the quantizer's planes: codes [n][k / 2] bytes (element 2t
// in the low nibble of byte t) and scales [n][k / block], dense.
//
// Types.  An NVFP4 element without the tensor scale (E2M1 times E4M3) has at
// most 6 significant bits between 2^-10 and 2688, an MXFP4 element (E2M1 times
// a power of two) has 2: both are exact in bf16, and so is an MXFP8 one (4
// bits times a power of two).  So weights and 8-bit activations enter the
// bf16 matrix instructions as they are (an MX product outside bf16's normal range
// as in a reconstruction to bf16; a NaN scale makes its block NaN: the scaled
// conversions give NaN for scale byte 255, the E4M3 one for 0x7F).  bf16
// activations are exact too.  An fp32 one is the sum of three bf16 pieces of 8
// bits each, cut off rather than rounded, so that the sum is exact and no piece
// passes the type's range.  (From 2^-110 on: of smaller ones the last pieces fall
// under bf16's least number, 2^-133, and less than that is lost of an element.)  The tensor scale's power of two goes into the weights,
// exactly, so that sums are of the results' size; what is left of it, in [1, 2),
// multiplies the sums.  Those are fp32; bias and activation are applied in fp32, and
// outputs rounded once.
#pragma once

#include "fp4q_ffn_sizes.h"
#include "fp4q_flat.h"

namespace fp4q {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// Types of activations; kE4M3: with a plane of E8M0 scales, one for each 32.
enum XType { kXF32 = 0, kXBF16 = 1, kXE4M3 = 2 };

struct FfnWeight {
  const uint8_t* codes;
  const uint8_t* scales;
  const float* g;              // NVFP4: tensor scale (device)
  int64_t n, k;                // n: all rows, a gated weight's both halves
  int format;                  // 0 MX, 1 NV
};

struct LinearLaunch {
  FfnWeight w;
  const void* x;               // backward: the gradient of the output, [rows][n]
  const uint8_t* x_scales;     // [rows][k / 32]
  int64_t rows, x_stride;      // elements
  int x_type;
  int gated;                   // rows n / 2 of the weight on are the second factor's
  int transposed;              // dx = dy W
  const void* bias;            // [n] of the output's type, or null
  void* out;                   // [rows][n], gated [rows][n / 2], transposed [rows][k]
  void* products;              // gated: [rows][n], or null
  int out_bf16, products_bf16;
  float* partials;             // parts of sums that several workgroups share (workspace)
};

// Whether one launch takes the call's tiles.
bool linear_fits(const LinearLaunch& l);
size_t linear_workspace(const LinearLaunch& l);
hipError_t launch_linear(const LinearLaunch& l, hipStream_t s);
hipError_t launch_linear_few(const LinearLaunch& l, hipStream_t s);

// d(h) / d(products): SiLU(g) u with its derivative, elementwise.
struct GatedGradLaunch {
  const void* dh;              // [rows][f], row stride in elements
  const void* products;        // [rows][2 f], dense
  void* dproducts;             // [rows][2 f], dense
  int64_t rows, f, dh_stride;
  int bf16, products_bf16;     // dh and dproducts; products
};
hipError_t launch_gated_grad(const GatedGradLaunch& l, hipStream_t s);

struct NormLaunch {
  const void *x, *residual;    // residual may be null
  const void* w;
  void* y;                     // null when quantizing
  void* summed;                // with a residual: x + residual, rounded to the type
  float* rstd;                 // or null
  uint8_t *codes, *scales;     // MXFP8 output
  int64_t rows, d, x_stride, residual_stride;
  int bf16, w_bf16;
  float eps;
};
hipError_t launch_rms_norm(const NormLaunch& l, hipStream_t s);

struct NormGradLaunch {
  const void *dy, *s, *w, *ds; // ds: gradient that reaches the sum by other ways, or null
  const float* rstd;
  void *dx, *dw;
  int64_t rows, d, dy_stride, s_stride, ds_stride;
  int bf16, w_bf16;
  float* partials;             // workspace
};
size_t rms_norm_grad_workspace(int64_t rows, int64_t d);
hipError_t launch_rms_norm_grad(const NormGradLaunch& l, hipStream_t s);

struct Dequant8Launch {
  const uint8_t *codes, *scales;
  int64_t rows, cols;
  int out_dtype;
  void* out;
};
hipError_t launch_dequant8(const Dequant8Launch& l, hipStream_t s);

// This workgroup's number in a grid of grid_x and grid_y.
__device__ __forceinline__ int64_t group_number() { return (int64_t)blockIdx.y * kGridRow + blockIdx.x; }

// ----------------------------------------------------------------------------
// Loads of any alignment: rows need not begin on a vector's boundary.
template <typename T>
__device__ __forceinline__ T load_any(const void* p) {
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}
template <typename T>
__device__ __forceinline__ void store_any(void* p, T v) {
  __builtin_memcpy(p, &v, sizeof(T));
}

// The upper halves of two fp32 words as one word: their bf16 values where those
// are exact, else cut off.
__device__ __forceinline__ uint32_t high_halves(uint32_t lo, uint32_t hi) {
  return __builtin_amdgcn_perm(hi, lo, 0x07060302u);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2_t p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// The scale of a block as the conversions below take it: for MXFP4 the power of
// two as an exponent field, for NVFP4 the factor.
template <int FMT>
__device__ __forceinline__ float scale_operand(uint32_t byte) {
  if constexpr (FMT == 0) return e8m0_operand(byte);
  else return e4m3_value_hw(byte & 0x7Fu);
}

// The tensor scale in two factors: a power of two that the conversions below
// multiply into the elements, held to 2^-116 .. 2^115, with which the least of them
// (2^-10) is normal in bf16 and the largest (2688) finite; and the rest, which is
// exact.  (A scalar load: the rings count the vector loads that are on their way.)
__device__ __forceinline__ float tensor_scale(const float* g) {
  typedef const __attribute__((address_space(4))) float* constant_t;
  return *(constant_t)reinterpret_cast<uintptr_t>(g);
}
__device__ __forceinline__ float tensor_power(float g) {
  const uint32_t e = (as_u(g) >> 23) & 0xFFu;
  return as_f(min(max(e, 11u), 242u) << 23);
}
__device__ __forceinline__ float tensor_rest(float g) {
  return g * as_f((254u << 23) - as_u(tensor_power(g)));
}

// Eight codes of one block as bf16 pairs.  power: NVFP4, tensor_power.
template <int FMT>
__device__ __forceinline__ u32x4_t weights8(uint32_t codes, float s, float power) {
  u32x4_t o;
  if constexpr (FMT == 0) {
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
  } else {
    const float2_t a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, power, 0);
    const float2_t b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, power, 1);
    const float2_t c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, power, 2);
    const float2_t d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, power, 3);
    o.x = high_halves(as_u(a.x * s), as_u(a.y * s));
    o.y = high_halves(as_u(b.x * s), as_u(b.y * s));
    o.z = high_halves(as_u(c.x * s), as_u(c.y * s));
    o.w = high_halves(as_u(d.x * s), as_u(d.y * s));
  }
  return o;
}

// N codes (2 or 4) of one row and N of the next, each row with its own scale: pair
// j is column j's two values.
template <int FMT, int N>
__device__ __forceinline__ void weight_pairs(uint32_t ca, float sa, uint32_t cb, float sb, float power, uint32_t (&o)[N]) {
  if constexpr (FMT == 0) {
    const uint32_t a0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ca, sa, 0));
    const uint32_t b0 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cb, sb, 0));
    o[0] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
    o[1] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
    if constexpr (N == 4) {
      const uint32_t a1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(ca, sa, 1));
      const uint32_t b1 = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(cb, sb, 1));
      o[2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
      o[3] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
    }
  } else {
    const float2_t a0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ca, power, 0);
    const float2_t b0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cb, power, 0);
    o[0] = high_halves(as_u(a0.x * sa), as_u(b0.x * sb));
    o[1] = high_halves(as_u(a0.y * sa), as_u(b0.y * sb));
    if constexpr (N == 4) {
      const float2_t a1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(ca, power, 1);
      const float2_t b1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(cb, power, 1);
      o[2] = high_halves(as_u(a1.x * sa), as_u(b1.x * sb));
      o[3] = high_halves(as_u(a1.y * sa), as_u(b1.y * sb));
    }
  }
}

// Eight E4M3 codes with one E8M0 scale as bf16 pairs.
__device__ __forceinline__ u32x4_t e4m3_values8(u32x2_t codes, uint32_t scale) {
  const float s = e8m0_operand(scale);
  u32x4_t o;
  o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, s, false));
  o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.x, s, true));
  o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, s, false));
  o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes.y, s, true));
  return o;
}

// The three bf16 pieces of eight fp32 values: the upper 16 bits of what is left
// each time, which leaves nothing after three where the values' last bits are
// 2^-133 or more, bf16's least number, and less than that elsewhere.  An infinity or NaN is its own
// first piece (a NaN made quiet, so that the cut keeps it one) and leaves zeros.
__device__ __forceinline__ void split8(const uint32_t v[8], u32x4_t out[3]) {
  uint32_t h[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = as_f(v[i]);
    const bool odd = (v[i] & 0x7F800000u) == 0x7F800000u;
    h[i] = f != f ? v[i] | 0x400000u : v[i];
    const float r = odd ? 0.0f : f - as_f(h[i] & 0xFFFF0000u);
    m[i] = as_u(r);
    l[i] = as_u(r - as_f(m[i] & 0xFFFF0000u));
  }
  out[0] = u32x4_t{high_halves(h[0], h[1]), high_halves(h[2], h[3]), high_halves(h[4], h[5]), high_halves(h[6], h[7])};
  out[1] = u32x4_t{high_halves(m[0], m[1]), high_halves(m[2], m[3]), high_halves(m[4], m[5]), high_halves(m[6], m[7])};
  out[2] = u32x4_t{high_halves(l[0], l[1]), high_halves(l[2], l[3]), high_halves(l[4], l[5]), high_halves(l[6], l[7])};
}

template <int XT>
constexpr int kPieces = XT == kXF32 ? 3 : 1;

__device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0,
                                                 0, 0);
}

// SiLU(g) = g / (1 + e^-g): e^-g is infinite for g below -88, where the result
// is a zero (the limit), NaN stays NaN, and minus infinity gives -0 times ...
// NaN as the formula does.
__device__ __forceinline__ float sigmoid(float g) { return 1.0f / (1.0f + expf(-g)); }

}  // namespace fp4q
