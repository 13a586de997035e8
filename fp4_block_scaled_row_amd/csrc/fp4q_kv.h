// fp4q_kv.h -- the paged 4-bit key/value cache: its planes as kernels see
// them, and the launch interface between the C ABI (fp4q_kv_api.hip) and the
// kernels that write, read and attend over it.
//
// A plane row is one token of one head: head_dim / 2 bytes of E2M1 codes
// (element 2k in the low nibble of byte k), or head_dim / block scale bytes
// (E4M3 for NVFP4's 16-blocks, E8M0 for MXFP4's 32-blocks).  Rows lie at
// page * stride[0] + head * stride[1] + offset * stride[2] bytes, all 64-bit,
// so any order of pages, heads and tokens is a matter of strides (each below
// 2^31; their products with page numbers are not).
#pragma once

#include "fp4q_flat.h"

namespace fp4q {

// x / d for 0 <= x < 2^31 by one high product: with 2^(s-1) < d <= 2^s and
// M = ceil(2^(31+s) / d) the error of x M / 2^(31+s) stays below 1 / d.
struct FastDiv {
  uint32_t mul;     // 0: d is 1
  uint32_t shift;
  uint32_t d;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f = {0, 0, d};
  if (d <= 1) return f;
  uint32_t s = 1;
  while (((uint64_t)1 << s) < d) ++s;
  f.mul = (uint32_t)((((uint64_t)1 << (31 + s)) + d - 1) / d);
  f.shift = s - 1;
  return f;
}
__device__ __forceinline__ uint32_t quotient(uint32_t x, const FastDiv& f) {
  return f.mul ? __umulhi(x, f.mul) >> f.shift : x;
}

struct KvPlanes {
  uint8_t *kc, *ks, *vc, *vs;    // codes and scales of keys and values
  const float *kg, *vg;          // NVFP4: tensor scales (device)
  uint32_t code_stride[3];       // bytes: page, head, token (products are 64-bit)
  uint32_t scale_stride[3];
  int32_t num_pages, heads;
  FastDiv page;                  // page size
};

struct KvWriteLaunch {
  KvPlanes p;
  int format, head_dim, in_dtype, rotate;
  int64_t tokens;
  const void *k, *v;
  int64_t k_stride[2], v_stride[2];   // elements: token, head
  const int64_t* slots;
};
hipError_t launch_kv_write(const KvWriteLaunch& w, hipStream_t s);

struct KvReadLaunch {
  KvPlanes p;
  int format, head_dim, out_dtype, rotate;
  const int32_t* table;
  int64_t table_stride;
  int32_t table_cols, seqs;
  const int32_t *cu, *starts;
  int64_t total;
  void *k_out, *v_out;
};
hipError_t launch_kv_read(const KvReadLaunch& r, hipStream_t s);

struct KvAttendLaunch {
  KvPlanes p;
  int format, head_dim, dtype, rotate;   // dtype: of q and out
  const void* q;
  int64_t q_stride[2];                   // elements: token, head
  void* out;                             // [total_q][q_heads][head_dim]
  float* lse;                            // [total_q][q_heads] or null
  int64_t total_q;
  int32_t seqs, max_q, group;            // group: query heads of one cache head
  const int32_t* cu_q;                   // null: one query a sequence
  const int32_t* lens;
  const int32_t* table;
  int64_t table_stride;
  int32_t table_cols;
  int32_t causal, window;
  float scale;
  float rot_scale;                       // fl32(1 / sqrt(128))
  uint8_t* ws;
  int64_t most_tokens;                   // what the table can hold of one sequence
  FastDiv group_div;
  FastDiv per_seq;                       // query blocks a sequence where numbered so (d 0: by bisection)
  uint32_t thirds;                       // workgroups of a launch with three on every CU
};
hipError_t launch_kv_attend(const KvAttendLaunch& a, hipStream_t s);
size_t kv_attend_workspace(const KvAttendLaunch& a);

}  // namespace fp4q
