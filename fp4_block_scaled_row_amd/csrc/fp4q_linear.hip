// fp4q_linear.hip -- which kernels a linear call takes, the joining of sums that
// several workgroups share, and the gradient of SiLU(g) u.
#include <algorithm>
#include <type_traits>

#include "fp4q_linear_many.h"

namespace fp4q {
namespace {

struct Plan {
  bool few, mx8;
  int size, splits;
};

ManyArgs many_args(const LinearLaunch& l, int size) {
  ManyArgs a;
  a.l = l;
  const ManySize t = size < 0 ? ManySize{256, 256} : many_size(l.x_type, size);
  const int64_t out = l.transposed ? l.w.k : l.gated ? l.w.n / 2 : l.w.n;
  const int64_t bn = l.gated ? t.bn / 2 : t.bn;
  const int64_t tm = (l.rows + t.bm - 1) / t.bm, tn = (out + bn - 1) / bn;
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tn;
  a.ntiles = (int)(tm * tn);
  a.stages = (int)(((l.transposed ? l.w.n : l.w.k) + kStage - 1) / kStage);
  a.splits = 1;
  a.per_split = a.stages;
  return a;
}

bool multiple(const void* p, uintptr_t of) { return reinterpret_cast<uintptr_t>(p) % of == 0; }

Plan plan(const LinearLaunch& l) {
  Plan p = {!l.transposed && l.rows <= (l.x_type == kXF32 ? 16 : 64) && (l.x_type != kXE4M3 || few_eight_fits(l.rows, l.w.k)),
            false, 1, 1};
  if (p.few) return p;
  const int cus = device_cu_count();
  // Block-scaled products for bf16 results (the instruction drops more bits than an
  // fp32 result should lose), from a quarter as many tiles as CUs on (its offsets
  // within 256 rows are 31-bit; its loads into LDS and of scales are aligned ones).
  // Measured, MXFP4, us, there / converted to bf16:
  //   k, n        rows 256       512          1024         2048
  //   8192, 8192  88 /  69    90 / 106     92 / 163    114 / 253
  //   4096, 4096  45 /  34    45 /  43     51 /  58     53 /  87
  //   8192, 1024  79 /  29    79 /  33     90 /  43     91 /  69
  p.mx8 = l.x_type == kXE4M3 && l.w.format == 0 && l.out_bf16 && (!l.products || l.products_bf16) && l.w.k > 0 &&
          l.w.k % 128 == 0 && l.w.k <= 1 << 22 && multiple(l.x, 16) && multiple(l.w.codes, 16) &&
          multiple(l.x_scales, 4) && multiple(l.w.scales, 4) && many_args(l, -1).ntiles >= cus / 4;
  if (p.mx8) return p;
  // Large tiles from one a CU on; whole stages also in parts of 32 stages or more
  // that give each CU one, forward of 128 stages or more in all.  Measured, bf16,
  // NVFP4, us, parts of large tiles / of small ones:
  //   k, n              rows 256     512         1024        2048
  //   8192, 8192        62 / 70      97 / 113
  //   4096, 16384       63 / 59
  //   4096, 4096                                 65 / 61
  //   8192, 1024                                             62 / 70
  //   gradient: 8192, 8192           107 / 133
  //   k 4096, n 16384   58 / 75      90 / 139    151 / 261
  //   4096, 4096                                 59 / 71
  const ManyArgs large = many_args(l, 1);
  const int parts = (cus + large.ntiles - 1) / large.ntiles;
  if (parts == 1) return p;
  if (ring_sizes(l) && large.stages / parts >= 32 && (l.transposed || large.stages >= 128)) {
    p.splits = parts;
    return p;
  }
  p.size = 0;
  const ManyArgs small = many_args(l, 0);
  // parts of the contraction, of 8 stages at least, until every CU has two
  const int want = (2 * cus + small.ntiles - 1) / small.ntiles;
  p.splits = std::max(1, std::min(want, small.stages / 8));
  return p;
}

// out = sum of the parts, in their order, and what follows the sum: a thread 4
// consecutive outputs of a row.
__global__ __launch_bounds__(256) void join_kernel(LinearLaunch l, int splits) {
  const int64_t half = l.w.n / 2;
  const int64_t out = l.transposed ? l.w.k : l.gated ? half : l.w.n;
  const int64_t cols = l.transposed ? l.w.k : l.w.n;
  const int64_t per = (out + 3) / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= l.rows * per) return;
  const int64_t row = at / per, col = (at - row * per) * 4;
  const int count = (int)min(out - col, (int64_t)4);
  const float tensor = l.w.format == 1 ? tensor_rest(tensor_scale(l.w.g)) : 1.0f;
  auto sum = [&](int64_t c, float (&v)[4]) {
    const float* p = l.partials + row * cols + c;
    for (int i = 0; i < 4; ++i) v[i] = 0.0f;
    for (int s = 0; s < splits; ++s, p += l.rows * cols) {
      if (count == 4) {
        const f32x4_t q = load_any<f32x4_t>(p);
        for (int i = 0; i < 4; ++i) v[i] += q[i];
      } else {
        for (int i = 0; i < count; ++i) v[i] += p[i];
      }
    }
    for (int i = 0; i < 4; ++i) v[i] *= tensor;
  };
  auto put = [&](void* to, int64_t o, const float (&v)[4], int bf16) {
    for (int i = 0; i < count; ++i) {
      if (bf16) static_cast<__bf16*>(to)[o + i] = (__bf16)v[i];
      else static_cast<float*>(to)[o + i] = v[i];
    }
  };
  float v[4];
  sum(col, v);
  if (l.gated) {
    float u[4];
    sum(half + col, u);
    if (l.products) {
      put(l.products, row * l.w.n + col, v, l.products_bf16);
      put(l.products, row * l.w.n + half + col, u, l.products_bf16);
    }
    for (int i = 0; i < 4; ++i) v[i] = v[i] * sigmoid(v[i]) * u[i];
  } else if (l.bias) {
    for (int i = 0; i < count; ++i)
      v[i] += l.out_bf16 ? (float)static_cast<const __bf16*>(l.bias)[col + i]
                         : static_cast<const float*>(l.bias)[col + i];
  }
  put(l.out, row * out + col, v, l.out_bf16);
}

// With s = 1 / (1 + e^-g):  d SiLU(g) u / dg = u s (1 + g (1 - s)),  / du = g s.
// A thread takes 8 neighbouring elements of a row: three reads and two writes, all
// memory's.
template <bool BF16, bool PBF16>
__global__ __launch_bounds__(256) void gated_grad_kernel(GatedGradLaunch l) {
  constexpr int kElem = BF16 ? 2 : 4, kPElem = PBF16 ? 2 : 4;
  const int64_t per = (l.f + 7) / 8;
  const int64_t at = group_number() * 256 + threadIdx.x;
  if (at >= l.rows * per) return;
  const int64_t row = at / per, col = (at - row * per) * 8;
  const uint8_t* dh = static_cast<const uint8_t*>(l.dh) + (row * l.dh_stride + col) * kElem;
  const uint8_t* p = static_cast<const uint8_t*>(l.products) + (row * 2 * l.f + col) * kPElem;
  uint8_t* o = static_cast<uint8_t*>(l.dproducts) + (row * 2 * l.f + col) * kElem;
  const int count = (int)min(l.f - col, (int64_t)8);
  float d[8], x[8], u[8];
  auto load = [&](const uint8_t* q, float (&v)[8], auto half) {
    constexpr bool kHalf = decltype(half)::value;
    if (count == 8) {
      if constexpr (kHalf) {
        const u32x4_t w = load_any<u32x4_t>(q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = bf_lo(w[i]);
          v[2 * i + 1] = bf_hi(w[i]);
        }
      } else {
        const f32x4_t a = load_any<f32x4_t>(q), b = load_any<f32x4_t>(q + 16);
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
        if (i < count) v[i] = kHalf ? bf_lo(load_any<uint16_t>(q + 2 * i)) : load_any<float>(q + 4 * i);
      }
    }
  };
  auto store = [&](uint8_t* q, const float (&v)[8]) {
    if (count == 8) {
      if constexpr (BF16) {
        store_any(q, u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])});
      } else {
        store_any(q, f32x4_t{v[0], v[1], v[2], v[3]});
        store_any(q + 16, f32x4_t{v[4], v[5], v[6], v[7]});
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (i >= count) continue;
        if constexpr (BF16) store_any(q + 2 * i, (__bf16)v[i]);
        else store_any(q + 4 * i, v[i]);
      }
    }
  };
  load(dh, d, std::bool_constant<BF16>());
  load(p, x, std::bool_constant<PBF16>());
  load(p + l.f * kPElem, u, std::bool_constant<PBF16>());
  float dg[8], du[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // s and 1 - s each by itself: where g is large, 1 - s of a rounded s would be rounding
    const float e = expf(-fabsf(x[i])), r = 1.0f / (1.0f + e);
    const float s = x[i] < 0.0f ? e * r : r, c = x[i] < 0.0f ? r : e * r;
    dg[i] = d[i] * u[i] * s * (1.0f + x[i] * c);
    du[i] = d[i] * x[i] * s;
  }
  store(o, dg);
  store(o + l.f * kElem, du);
}

}  // namespace

bool linear_fits(const LinearLaunch& l) {
  const Plan p = plan(l);
  return p.few || tiles_fit(many_args(l, p.mx8 ? -1 : p.size).ntiles);
}

size_t linear_workspace(const LinearLaunch& l) {
  const Plan p = plan(l);
  if (p.splits <= 1) return 0;
  return (size_t)p.splits * l.rows * (l.transposed ? l.w.k : l.w.n) * sizeof(float);
}

hipError_t launch_linear(const LinearLaunch& l, hipStream_t s) {
  const Plan p = plan(l);
  if (p.few) return launch_linear_few(l, s);
  if (p.mx8) return launch_mx8(many_args(l, -1), s);
  ManyArgs a = many_args(l, p.size);
  a.splits = p.splits;
  a.per_split = (a.stages + p.splits - 1) / p.splits;
  hipError_t e;
  if (l.transposed) e = l.w.format == 0 ? launch_many_back_mx(a, p.size, s) : launch_many_back_nv(a, p.size, s);
  else e = l.w.format == 0 ? launch_many_mx(a, p.size, s) : launch_many_nv(a, p.size, s);
  if (e != hipSuccess || p.splits <= 1) return e;
  const int64_t out = l.transposed ? l.w.k : l.gated ? l.w.n / 2 : l.w.n;
  const int64_t threads = l.rows * ((out + 3) / 4);
  hipLaunchKernelGGL(join_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, l, p.splits);
  return hipGetLastError();
}

hipError_t launch_gated_grad(const GatedGradLaunch& l, hipStream_t s) {
  const int64_t groups = (l.rows * ((l.f + 7) / 8) + 255) / 256;
  const dim3 grid(grid_x(groups), grid_y(groups));
  if (l.bf16 && l.products_bf16) hipLaunchKernelGGL((gated_grad_kernel<true, true>), grid, dim3(256), 0, s, l);
  else if (l.bf16) hipLaunchKernelGGL((gated_grad_kernel<true, false>), grid, dim3(256), 0, s, l);
  else if (l.products_bf16) hipLaunchKernelGGL((gated_grad_kernel<false, true>), grid, dim3(256), 0, s, l);
  else hipLaunchKernelGGL((gated_grad_kernel<false, false>), grid, dim3(256), 0, s, l);
  return hipGetLastError();
}

}  // namespace fp4q
