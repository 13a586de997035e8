// fp4q_linear_mx8.hip -- products of many rows of MXFP8 activations with an
// MXFP4 weight: y = x W^T and h = SiLU(x Wg^T) * (x Wu^T), on gfx950's
// block-scaled matrix instructions, which take both as they are: E4M3 codes with
// their E8M0 scales on one side, E2M1 codes with theirs on the other, at twice
// the rate of bf16 and without any conversion.  k a multiple of 128.
//
// v_mfma_scale_f32_32x32x64_f8f6f4, weights as the left operand: lane l supplies
// row l mod 32 of either side.  With h = l / 32 its 32 E2M1 codes (16 bytes), and
// its scale byte of either side, are those of k = 32 h .. + 31; its 32 E4M3 codes
// are those of 16 h .. + 15 and of 32 + 16 h .. + 15.  Result register i is weight
// row 8 (i / 4) + 4 h + i mod 4 for row l mod 32 of x: 4 consecutive outputs of a
// row.  The instruction adds eight neighbouring products at a time, lined up by the
// largest exponent among them, and drops what lies below 2^-13 of that; sums of
// eights are fp32's.  What is lost is a part of the sum of the products' magnitudes,
// 7 2^-13 of it at most.  Over a whole output it disappears under the rounding to bf16,
// the only results that these kernels write, but a single result whose products cancel
// can be off by more than its own rounding: of 2048 rows, k and n 8192, 0.2 % are, by
// 2e-6 of that sum at most (the output as a whole is 1.66e-3 from 64 bits, as with fp32
// sums).  fp32 results take the bf16 instructions, whose sums are fp32's throughout.
//
// A workgroup of 8 waves computes 256 rows of x by 256 of the weight, each wave 64
// x 128: the side with the wider elements is read twice from LDS, the other four
// times.  (128 x 128 a wave would read less and takes all 256 accumulator
// registers, which the compiler spills around.)  A stage is 128 k: 32 KiB of x and
// 16 KiB of codes, loaded straight into LDS into a ring of three buffers, asked for two
// stages ahead.  (As it is compiled, a step waits for the next stage too before its
// reads, see there: what is in flight while it multiplies is the stage that it asks for.)
// Scales come 12 bytes a row (three stages) a load, a row a lane, and are
// written beside the stage they belong to: loaded by the lanes that use them they
// would cost the load unit as long as the products take.  LDS rows are 128 and 64
// bytes, their 16-byte chunks exchanged so that reads of one chunk of 16 rows meet
// all banks.
//
// 2048 rows, k and n 8192: 105 us, 2.6 PFLOP/s, where a library's product of E4M3
// matrices of that size reaches 2.9 (converted to bf16: 253 us).
#include <type_traits>

#include "fp4q_linear_many.h"

namespace fp4q {
namespace {

constexpr int kTile8 = 256, kK8 = 128, kWaves8 = 8;
constexpr int kSubX = 2, kSubW = 4;                 // instructions of 32 rows a wave has, of either side
constexpr int kXBytes8 = kTile8 * kK8, kWBytes8 = kTile8 * kK8 / 2, kCodes8 = kXBytes8 + kWBytes8;
constexpr int kBuf8 = kCodes8 + 2 * kTile8 * 4;      // and a word of scales for each row, x's, then the weight's
constexpr int kXLoads8 = kXBytes8 / 1024 / kWaves8, kWLoads8 = kWBytes8 / 1024 / kWaves8;    // a wave's, of a stage
constexpr int kStageLoads8 = kXLoads8 + kWLoads8;
constexpr int kGroup8 = 3;                          // stages that a load of scales serves

typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef unsigned int u32x3_t __attribute__((ext_vector_type(3)));
template <bool GATED>
__global__ __launch_bounds__(64 * kWaves8) void mx8_kernel(ManyArgs a) {
  // separate objects, so that reads of one are not ordered after loads into others
  __shared__ __align__(16) uint8_t s_b0[kBuf8];
  __shared__ __align__(16) uint8_t s_b1[kBuf8];
  __shared__ __align__(16) uint8_t s_b2[kBuf8];
  const LinearLaunch& l = a.l;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);   // (the same in all lanes: descriptors go by it)
  const int wx = wave >> 1, ww = wave & 1;          // this wave's quarter of x's rows, half of the weight's

  const int w = blockIdx.x, per = (a.ntiles + 7) / 8;
  const int tile = (w % 8) * per + w / 8;
  if (tile >= a.ntiles || w / 8 >= per) return;
  const int group = tile / (4 * a.tiles_n), first = group * 4;
  const int gsize = min(a.tiles_m - first, 4), in_g = tile - group * 4 * a.tiles_n;
  const int64_t m0 = (int64_t)(first + in_g % gsize) * kTile8;
  const int64_t K = l.w.k, half = l.w.n / 2, side = GATED ? half : l.w.n;
  const int64_t o0 = (int64_t)(in_g / gsize) * (GATED ? kTile8 / 2 : kTile8);
  const int nstage = (int)(K / kK8);
  const int64_t kb = K / 2, ks = K / 32;

  // Rows past the ends read the last one, and their results are not stored.
  // Offsets from the tile's first row (of each factor) are below 2^31: K is at
  // most 2^22.  Local row i of the weight: gated, 64 of either factor a wave.
  auto w_row = [&](int i) { return GATED ? min(o0 + (i >> 7) * 64 + (i & 63), half - 1) - o0 : min(o0 + i, l.w.n - 1) - o0; };
  auto w_base = [&](int i) { return GATED && (i & 64) ? o0 + half : o0; };
  const uint8_t* x = static_cast<const uint8_t*>(l.x) + m0 * K;
  const int64_t x_bytes = (l.rows - m0) * K;
  auto issue = [&](int st, uint8_t* buf) {
#pragma unroll
    for (int i = 0; i < kXLoads8; ++i) {            // 8 rows of x, 128 bytes each
      const int region = wave * kXLoads8 + i, row = region * 8 + (lane >> 3);
      const int chunk = (lane & 7) ^ ((row >> 1) & 7);
      const int64_t r = min(m0 + row, l.rows - 1) - m0;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(x, x_bytes), (lds_void_t*)(buf + region * 1024), 16,
                                               (int)(r * K + (int64_t)st * kK8 + chunk * 16), 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < kWLoads8; ++i) {            // 16 rows of codes, 64 bytes each
      const int region = wave * kWLoads8 + i, row = region * 16 + (lane >> 2);
      const int chunk = (lane & 3) ^ ((row >> 2) & 3);
      const int64_t base = w_base(region * 16);
      __builtin_amdgcn_raw_ptr_buffer_load_lds(buffer_of(l.w.codes + base * kb, (l.w.n - base) * kb),
                                               (lds_void_t*)(buf + kXBytes8 + region * 1024), 16,
                                               (int)(w_row(row) * kb + (int64_t)st * (kK8 / 2) + chunk * 16), 0, 0, 0);
    }
  };
  // scales: this lane's row is its number, waves 0 to 3 x's, the others the weight's.
  // Bytes past a row's end, read for a last group of fewer stages, are not used
  // (past the plane's end they read as zeros).
  const int s_row = (wave & 3) * 64 + lane;
  const bool s_of_x = wave < 4;
  const int64_t s_base = s_of_x ? m0 : w_base((wave & 3) * 64);
  const __amdgpu_buffer_rsrc_t scales = buffer_of((s_of_x ? l.x_scales : l.w.scales) + s_base * ks,
                                             ((s_of_x ? l.rows : l.w.n) - s_base) * ks);
  const int s_off = (int)((s_of_x ? min(m0 + s_row, l.rows - 1) - m0 : w_row(s_row)) * ks);
  u32x3_t s_next;
  auto load_scales = [&](int gi) {
    s_next = __builtin_amdgcn_raw_buffer_load_b96(scales, s_off + 12 * min(gi, (nstage - 1) / kGroup8), 0, 0);
  };
  auto store_scales = [&](uint8_t* buf, int word) {
    // bytes 0, 2, 1, 3: those of a lane's two halves side by side
    *reinterpret_cast<uint32_t*>(buf + kCodes8 + ((s_of_x ? 0 : kTile8) + s_row) * 4) =
        __builtin_amdgcn_perm(0u, s_next[word], 0x03010200u);
  };

  f32x16_t acc[kSubW][kSubX];
#pragma unroll
  for (int i = 0; i < kSubW; ++i)
#pragma unroll
    for (int j = 0; j < kSubX; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  v8i_t xv[kSubX], wv[kSubW];
  int xe[kSubX], we[kSubW];                         // bytes 0 and 1: this lane's blocks of the stage's halves
  // (The compiler does not tell these reads from the loads into LDS that are on their way:
  // before the second one it waits for all of them, which the next stage's are.)
  auto read_scales = [&](const uint8_t* buf) {
    const int p = kCodes8 + (lane & 31) * 4 + (lane >> 5) * 2;
#pragma unroll
    for (int u = 0; u < kSubX; ++u) xe[u] = *reinterpret_cast<const uint16_t*>(buf + (p + (64 * wx + 32 * u) * 4));
#pragma unroll
    for (int u = 0; u < kSubW; ++u) we[u] = *reinterpret_cast<const uint16_t*>(buf + (p + (kTile8 + 128 * ww + 32 * u) * 4));
  };
  // The lane's offsets are hidden from the compiler: it would keep those of three
  // buffers in more registers than there are.  (Other forms of the addresses, with more
  // waits: 110 us for 106.)
  auto read = [&](const uint8_t* buf, int kk) {
    // Of the instruction's 64 a lane has 32: 4-bit ones, and the scales of both sides,
    // 32 h to 32 h + 31 (h = lane / 32); 8-bit ones 16 h to 16 h + 15 in its first four
    // registers, and those and 32 in the other four.
    const int h = lane >> 5;
    int x0 = (64 * wx + (lane & 31)) * kK8 + ((4 * kk + h) ^ ((lane >> 1) & 7)) * 16, x1 = x0 ^ 32;
    int w0 = kXBytes8 + (128 * ww + (lane & 31)) * (kK8 / 2) + ((2 * kk + h) ^ ((lane >> 2) & 3)) * 16;
    asm volatile("" : "+v"(x0), "+v"(x1), "+v"(w0));
#pragma unroll
    for (int u = 0; u < kSubX; ++u) {
      const u32x4_t v0 = *reinterpret_cast<const u32x4_t*>(buf + (x0 + 32 * u * kK8));
      const u32x4_t v1 = *reinterpret_cast<const u32x4_t*>(buf + (x1 + 32 * u * kK8));
      xv[u] = v8i_t{(int)v0.x, (int)v0.y, (int)v0.z, (int)v0.w, (int)v1.x, (int)v1.y, (int)v1.z, (int)v1.w};
    }
#pragma unroll
    for (int u = 0; u < kSubW; ++u) {
      const u32x4_t c = *reinterpret_cast<const u32x4_t*>(buf + (w0 + 32 * u * (kK8 / 2)));
      wv[u] = v8i_t{(int)c.x, (int)c.y, (int)c.z, (int)c.w, 0, 0, 0, 0};
    }
  };
  auto mma = [&](auto which) {
    constexpr int kk = decltype(which)::value;
#pragma unroll
    for (int i = 0; i < kSubW; ++i)
#pragma unroll
      for (int j = 0; j < kSubX; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(wv[i], xv[j], acc[i][j], 4, 0, kk, we[i], kk, xe[j]);
  };
  // Step st waits until only the next stage's loads are on their way, which is what it
  // needs itself.  The barrier then tells that every wave has its part of stage st in LDS
  // and is done with stage st - 1, whose buffer the refill takes.  Behind the barrier the
  // compiler waits for the next stage too (at the second read of scales), so that the
  // refill alone is on its way during the products.  Its scales are written before it, and
  // after a group's last the next group is asked for, before the refill too, so that
  // waiting for it leaves the refill on its way.  There is no branch (past the last
  // stage it is asked for again), so that counts of loads are exact.
  auto step = [&](int st, auto group_step, const uint8_t* cur, uint8_t* fill) {
    constexpr int sg = decltype(group_step)::value;
    wait_loads<kStageLoads8>();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read_scales(cur);
    read(cur, 0);
    mma(std::integral_constant<int, 0>());
    read(cur, 1);
    store_scales(fill, (sg + 2) % kGroup8);
    if (sg == 0) load_scales(st / kGroup8 + 1);
    __builtin_amdgcn_sched_barrier(0);
    issue(min(st + 2, nstage - 1), fill);
    __builtin_amdgcn_sched_barrier(0);
    mma(std::integral_constant<int, 1>());
  };
  load_scales(0);
  store_scales(s_b0, 0);
  store_scales(s_b1, 1);
  __builtin_amdgcn_sched_barrier(0);                // (the order of loads is what a count of them means)
  issue(0, s_b0);
  __builtin_amdgcn_sched_barrier(0);
  issue(min(1, nstage - 1), s_b1);
  const std::integral_constant<int, 0> g0;
  const std::integral_constant<int, 1> g1;
  const std::integral_constant<int, 2> g2;
  int st = 0;
  for (; st + 3 <= nstage; st += 3) {
    step(st, g0, s_b0, s_b2);
    step(st + 1, g1, s_b1, s_b0);
    step(st + 2, g2, s_b2, s_b1);
  }
  if (st < nstage) step(st, g0, s_b0, s_b2);
  if (st + 1 < nstage) step(st + 1, g1, s_b1, s_b0);
  wait_loads<0>();                                  // (the last stage asked for again: its LDS may be another's next)

  auto put4 = [&](void* to, int64_t at, f32x4_t v, int count) {     // (bf16: see above)
    __bf16* o = static_cast<__bf16*>(to) + at;
    if (count >= 4) {
      store_any(o, u32x2_t{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)});
    } else {
      for (int i = 0; i < count; ++i) o[i] = (__bf16)v[i];
    }
  };
#pragma unroll
  for (int j = 0; j < kSubX; ++j) {
    const int64_t row = m0 + 64 * wx + 32 * j + (lane & 31);
    if (row >= l.rows) continue;
#pragma unroll
    for (int i = 0; i < (GATED ? 2 : kSubW); ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t col = o0 + (GATED ? 64 : 128) * ww + 32 * i + 8 * q + 4 * (lane >> 5);
        const int count = (int)min(side - col, (int64_t)4);
        if (count <= 0) continue;
        f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
        if constexpr (GATED) {
          f32x4_t u = {acc[(i + 2) % kSubW][j][4 * q], acc[(i + 2) % kSubW][j][4 * q + 1],
                       acc[(i + 2) % kSubW][j][4 * q + 2], acc[(i + 2) % kSubW][j][4 * q + 3]};
          if (l.products) {
            put4(l.products, row * l.w.n + col, v, count);
            put4(l.products, row * l.w.n + half + col, u, count);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = v[e] * sigmoid(v[e]) * u[e];
        } else if (l.bias) {
          for (int e = 0; e < count; ++e) v[e] += (float)static_cast<const __bf16*>(l.bias)[col + e];
        }
        put4(l.out, row * side + col, v, count);
      }
  }
}

}  // namespace

hipError_t launch_mx8(const ManyArgs& a, hipStream_t s) {
  const dim3 grid((a.ntiles + 7) / 8 * 8);
  if (a.l.gated) hipLaunchKernelGGL(mx8_kernel<true>, grid, dim3(64 * kWaves8), 0, s, a);
  else hipLaunchKernelGGL(mx8_kernel<false>, grid, dim3(64 * kWaves8), 0, s, a);
  return hipGetLastError();
}

}  // namespace fp4q
