// fp4q_kv_api.hip -- the C ABI of the paged 4-bit key/value cache (see
// include/fp4q.h): host-side checks and dispatch.  Every check runs before
// anything is enqueued.
#include <limits.h>
#include <math.h>
#include <string.h>

#include <algorithm>

#include "fp4q.h"
#include "fp4q_internal.h"
#include "fp4q_kv_attend.h"
#include "fp4q_kv_dispatch.h"

namespace fp4q {

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
fp4q_status hip_status(hipError_t e) { return e == hipSuccess ? FP4Q_OK : FP4Q_ERR_HIP; }

bool attend_dim(int d) { return d == 64 || d == 96 || d == 128 || d == 256; }

// Bytes that attention's one load of scales takes (see KvLane), 1, 2 or 4: what a
// plane's base and strides have to be multiples of.  Writing and reading take a
// byte at a time, so the head dimensions that attention does not have are free.
int scale_alignment(int format, int head_dim) {
  if (!attend_dim(head_dim) || head_dim % 128 != 0) return 1;
  return head_dim / 4 / (format == FP4Q_MXFP4 ? 32 : 16);
}

// Checks of a cache and the kernels' view of it.
fp4q_status check_cache(const fp4q_kv_cache* c, KvPlanes* p) {
  if (!c) return FP4Q_ERR_INVALID_ARG;
  if (c->format != FP4Q_MXFP4 && c->format != FP4Q_NVFP4)
    return c->format == FP4Q_IF4 ? FP4Q_ERR_UNSUPPORTED : FP4Q_ERR_INVALID_ARG;
  if (c->kv_heads <= 0 || c->head_dim <= 0 || c->page_size <= 0 || c->num_pages <= 0) return FP4Q_ERR_INVALID_ARG;
  if (c->head_dim % 32 != 0) return FP4Q_ERR_INVALID_ARG;   // incomplete blocks
  if (c->head_dim > 1024 || c->kv_heads > 4096 || c->num_pages > INT_MAX) return FP4Q_ERR_UNSUPPORTED;
  if (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales) return FP4Q_ERR_INVALID_ARG;
  if (c->format == FP4Q_NVFP4 && (!c->k_global || !c->v_global)) return FP4Q_ERR_INVALID_ARG;
  const int sa = scale_alignment(c->format, c->head_dim);
  for (int i = 0; i < 3; ++i) {
    if (c->code_stride[i] < 0 || c->scale_stride[i] < 0) return FP4Q_ERR_INVALID_ARG;
    if (c->code_stride[i] > INT_MAX || c->scale_stride[i] > INT_MAX) return FP4Q_ERR_UNSUPPORTED;
    if (c->code_stride[i] % 16 != 0 || c->scale_stride[i] % sa != 0) return FP4Q_ERR_UNSUPPORTED;
  }
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, sa) || !aligned(c->v_scales, sa))
    return FP4Q_ERR_UNSUPPORTED;
  p->kc = c->k_codes;
  p->ks = c->k_scales;
  p->vc = c->v_codes;
  p->vs = c->v_scales;
  p->kg = c->k_global;
  p->vg = c->v_global;
  for (int i = 0; i < 3; ++i) {
    p->code_stride[i] = (uint32_t)c->code_stride[i];
    p->scale_stride[i] = (uint32_t)c->scale_stride[i];
  }
  p->num_pages = (int32_t)c->num_pages;
  p->heads = c->kv_heads;
  p->page = fast_div((uint32_t)c->page_size);
  return FP4Q_OK;
}

fp4q_status check_rotation(int rotation, int head_dim) {
  if (rotation < FP4Q_ROT_NONE || rotation > FP4Q_ROT_FWHT128) return FP4Q_ERR_INVALID_ARG;
  if (rotation != FP4Q_ROT_NONE && (rotation != FP4Q_ROT_FWHT128 || head_dim % 128 != 0)) return FP4Q_ERR_UNSUPPORTED;
  return FP4Q_OK;
}

fp4q_status check_attention(const fp4q_kv_cache* cache, const fp4q_kv_attention_args* a, KvAttendLaunch* l) {
  if (!a) return FP4Q_ERR_INVALID_ARG;
  memset(l, 0, sizeof(*l));
  fp4q_status st = check_cache(cache, &l->p);
  if (st != FP4Q_OK) return st;
  if (a->dtype != FP4Q_F32 && a->dtype != FP4Q_BF16) return FP4Q_ERR_INVALID_ARG;
  if (a->total_q < 0 || a->seqs < 0 || a->q_heads <= 0 || a->q_heads % cache->kv_heads != 0)
    return FP4Q_ERR_INVALID_ARG;
  if (a->table_cols < 0 || a->table_stride < a->table_cols || a->window < 0) return FP4Q_ERR_INVALID_ARG;
  if (!(fabsf(a->scale) < INFINITY)) return FP4Q_ERR_INVALID_ARG;
  if (a->window > 0 && !a->causal) return FP4Q_ERR_UNSUPPORTED;
  st = check_rotation(a->rotation, cache->head_dim);
  if (st != FP4Q_OK) return st;
  if (!attend_dim(cache->head_dim)) return FP4Q_ERR_UNSUPPORTED;
  if (a->max_q < 0 || (!a->cu_q && (a->total_q != a->seqs || a->max_q > 1))) return FP4Q_ERR_INVALID_ARG;
  // row numbers (query, head of the group) are 31-bit
  if (a->total_q > INT_MAX / a->q_heads || a->seqs > 65535) return FP4Q_ERR_UNSUPPORTED;
  if (a->total_q > 0) {
    if (a->seqs == 0) return FP4Q_ERR_INVALID_ARG;      // (as in a read: rows without a sequence)
    if (!a->q || !a->out || !a->seq_lens || (a->table_cols > 0 && !a->page_table)) return FP4Q_ERR_INVALID_ARG;
    if (a->q_stride[0] < 0 || a->q_stride[1] < 0) return FP4Q_ERR_INVALID_ARG;
    const int64_t esz = a->dtype == FP4Q_F32 ? 4 : 2;
    if (!aligned(a->q, 16) || a->q_stride[0] * esz % 16 != 0 || a->q_stride[1] * esz % 16 != 0 || !aligned(a->out, 16))
      return FP4Q_ERR_UNSUPPORTED;
  }
  l->format = cache->format == FP4Q_MXFP4 ? 0 : 1;
  l->head_dim = cache->head_dim;
  l->dtype = a->dtype == FP4Q_F32 ? kF32 : kBF16;
  l->rotate = a->rotation == FP4Q_ROT_FWHT128;
  l->q = a->q;
  l->q_stride[0] = a->q_stride[0];
  l->q_stride[1] = a->q_stride[1];
  l->out = a->out;
  l->lse = a->lse;
  l->total_q = a->total_q;
  l->seqs = a->seqs;
  l->max_q = a->cu_q ? (a->max_q < a->total_q ? a->max_q : (int32_t)a->total_q) : 1;
  l->group = a->q_heads / cache->kv_heads;
  l->cu_q = a->cu_q;
  l->lens = a->seq_lens;
  l->table = a->page_table;
  l->table_stride = a->table_stride;
  l->table_cols = a->table_cols;
  l->causal = a->causal != 0;
  l->window = a->window;
  l->scale = a->scale;
  l->rot_scale = (float)(1.0 / sqrt(128.0));
  const int64_t most = (int64_t)a->table_cols * cache->page_size;
  l->most_tokens = most > INT_MAX - 1024 ? INT_MAX - 1024 : most;
  l->group_div = fast_div((uint32_t)l->group);
  return FP4Q_OK;
}

// Which kernels.  The few-row ones take 16 query rows of a cache head in a
// block (32 where those fit the registers: bf16, head_dim to 128) and read the
// cache once a block; the many-row ones 32 rows a wave, and turn codes into
// numbers once for 128 or 256 rows, but need many blocks and long stretches to
// earn their longer beginning, and a second kernel.  So it goes by the rows and
// by length: `shorter` with at most 2^16 tokens to pass over in all (sequences x cache heads x
// tokens of one, as far as the host knows).  Measured, bf16, head_dim 128, NVFP4,
// 16-row blocks / 32-row blocks / many-row, us:
//   sequences x heads x tokens    rows 32          rows 64          rows 128
//         1 x 1 x 2000            16 / 22 / 16     16 / 23 / 17     16 /  - / 18
//        16 x 1 x 4000            25 / 29 / 30     28 / 32 / 32     30 /  - / 37
//        16 x 8 x 1000            25 / 27 / 31     31 / 30 / 31     43 /  - / 39
//        16 x 8 x 8000            60 / 54 / 80    102 / 85 / 84    183 /  - / 99
// head_dim 64 alike.  With head_dim 256 and fp32 the many-row ones have one wave
// a SIMD: 16 x 8 x 8000 with 64 rows takes 164 / - / 204 at head_dim 256 and
// 105 / - / 182 in fp32 at 128.  With head_dim 96, whose codes are loaded 4
// bytes at a time, further reads cost more: 47 / 34 / 31 at 16 x 8 x 1000 and 64
// rows, 17 / 22 / 16 at 1 x 1 x 2000.
struct Plan {
  bool prefill;
  int tiles, waves;
};
Plan attend_plan(const KvAttendLaunch& a) {
  const int64_t rows = (int64_t)a.max_q * a.group;
  const int64_t tokens = a.window > 0 ? std::min(a.most_tokens, (int64_t)a.window + a.max_q) : a.most_tokens;
  const bool shorter = tokens * a.seqs * a.p.heads <= 1 << 16;
  const bool wide = a.dtype == kBF16 && a.head_dim <= 128;
  Plan p = {rows > (a.head_dim == 96 ? 32 : shorter ? 128 : 64), wide && rows > 16 && !shorter ? 2 : 1, 4};
  if (rows > 128 && wide) p.waves = 8;
  return p;
}

}  // namespace

// (at most 3 workgroups of the few-row kernels on a CU, 8 waves of the others)
size_t kv_attend_workspace(const KvAttendLaunch& a) {
  const Plan p = attend_plan(a);
  const int64_t cus = device_cu_count();
  if (p.prefill) return kv_workspace_bytes(cus * 8 / p.waves, 32 * p.waves, a.head_dim);
  return kv_workspace_bytes(cus * 3, 16 * p.tiles, a.head_dim);
}

// The schedule's numbers of a call (see fp4q_kv_attend.h), at most.
int64_t kv_attend_groups(const KvAttendLaunch& a) {
  const Plan p = attend_plan(a);
  KvAttendLaunch b = a;
  const int64_t numbers = kv_block_numbers(b, p.prefill ? 32 * p.waves : 16 * p.tiles);
  // (the smaller of the two kernels' steps; more than a unit costs in either)
  return kv_most_groups(b, numbers, 64, 16);
}

hipError_t launch_kv_attend(const KvAttendLaunch& a, hipStream_t s) {
  const Plan p = attend_plan(a);
  const int cus = device_cu_count();
#define FP4Q_KV_LAUNCH(D)                                                                     \
  case D:                                                                                     \
    if (p.prefill)                                                                            \
      return a.format == 1 ? launch_prefill_nv##D(a, p.waves, cus, s) : launch_prefill_mx##D(a, p.waves, cus, s); \
    return a.format == 1 ? launch_decode_nv##D(a, p.tiles, cus, s) : launch_decode_mx##D(a, p.tiles, cus, s)
  switch (a.head_dim) {
    FP4Q_KV_LAUNCH(64);
    FP4Q_KV_LAUNCH(96);
    FP4Q_KV_LAUNCH(128);
    FP4Q_KV_LAUNCH(256);
  }
#undef FP4Q_KV_LAUNCH
  return hipErrorInvalidValue;
}

}  // namespace fp4q

using namespace fp4q;

extern "C" {

fp4q_status fp4q_kv_write(const fp4q_kv_cache* cache, const fp4q_kv_write_args* args, void* hip_stream) {
  KvWriteLaunch w;
  memset(&w, 0, sizeof(w));
  fp4q_status st = check_cache(cache, &w.p);
  if (st != FP4Q_OK) return st;
  if (!args) return FP4Q_ERR_INVALID_ARG;
  if (args->tokens < 0 || (args->in_dtype != FP4Q_F32 && args->in_dtype != FP4Q_BF16)) return FP4Q_ERR_INVALID_ARG;
  st = check_rotation(args->rotation, cache->head_dim);
  if (st != FP4Q_OK) return st;
  if (args->tokens == 0) return FP4Q_OK;
  if (!args->k || !args->v || !args->slots) return FP4Q_ERR_INVALID_ARG;
  const int64_t esz = args->in_dtype == FP4Q_F32 ? 4 : 2;
  for (int i = 0; i < 2; ++i) {
    if (args->k_stride[i] < 0 || args->v_stride[i] < 0) return FP4Q_ERR_INVALID_ARG;
    if (args->k_stride[i] * esz % 16 != 0 || args->v_stride[i] * esz % 16 != 0) return FP4Q_ERR_UNSUPPORTED;
  }
  if (!aligned(args->k, 16) || !aligned(args->v, 16) || !aligned(args->slots, 8)) return FP4Q_ERR_UNSUPPORTED;
  w.format = cache->format == FP4Q_MXFP4 ? 0 : 1;
  w.head_dim = cache->head_dim;
  w.in_dtype = args->in_dtype == FP4Q_F32 ? kF32 : kBF16;
  w.rotate = args->rotation == FP4Q_ROT_FWHT128;
  w.tokens = args->tokens;
  w.k = args->k;
  w.v = args->v;
  for (int i = 0; i < 2; ++i) {
    w.k_stride[i] = args->k_stride[i];
    w.v_stride[i] = args->v_stride[i];
  }
  w.slots = args->slots;
  return hip_status(launch_kv_write(w, static_cast<hipStream_t>(hip_stream)));
}

fp4q_status fp4q_kv_read(const fp4q_kv_cache* cache, const fp4q_kv_read_args* args, void* hip_stream) {
  KvReadLaunch r;
  memset(&r, 0, sizeof(r));
  fp4q_status st = check_cache(cache, &r.p);
  if (st != FP4Q_OK) return st;
  if (!args) return FP4Q_ERR_INVALID_ARG;
  if (args->total < 0 || args->seqs < 0 || args->table_cols < 0 || args->table_stride < args->table_cols)
    return FP4Q_ERR_INVALID_ARG;
  if (args->out_dtype != FP4Q_F32 && args->out_dtype != FP4Q_BF16) return FP4Q_ERR_INVALID_ARG;
  st = check_rotation(args->rotation, cache->head_dim);
  if (st != FP4Q_OK) return st;
  if (args->total == 0 || (!args->k_out && !args->v_out)) return FP4Q_OK;
  if (args->seqs == 0 || !args->cu || (args->table_cols > 0 && !args->page_table)) return FP4Q_ERR_INVALID_ARG;
  if (!aligned(args->k_out, 16) || !aligned(args->v_out, 16)) return FP4Q_ERR_UNSUPPORTED;
  r.format = cache->format == FP4Q_MXFP4 ? 0 : 1;
  r.head_dim = cache->head_dim;
  r.out_dtype = args->out_dtype == FP4Q_F32 ? kF32 : kBF16;
  r.rotate = args->rotation == FP4Q_ROT_FWHT128;
  r.table = args->page_table;
  r.table_stride = args->table_stride;
  r.table_cols = args->table_cols;
  r.seqs = args->seqs;
  r.cu = args->cu;
  r.starts = args->starts;
  r.total = args->total;
  r.k_out = args->k_out;
  r.v_out = args->v_out;
  return hip_status(launch_kv_read(r, static_cast<hipStream_t>(hip_stream)));
}

size_t fp4q_kv_attention_workspace_bytes(const fp4q_kv_cache* cache, const fp4q_kv_attention_args* args) {
  KvAttendLaunch l;
  if (check_attention(cache, args, &l) != FP4Q_OK || l.total_q == 0 || kv_attend_groups(l) > INT_MAX) return 0;
  return kv_attend_workspace(l);
}

fp4q_status fp4q_kv_attention(const fp4q_kv_cache* cache, const fp4q_kv_attention_args* args, void* workspace,
                              size_t workspace_bytes, void* hip_stream) {
  KvAttendLaunch l;
  const fp4q_status st = check_attention(cache, args, &l);
  if (st != FP4Q_OK) return st;
  if (l.total_q == 0) return FP4Q_OK;
  if (kv_attend_groups(l) > INT_MAX) return FP4Q_ERR_UNSUPPORTED;
  const size_t need = kv_attend_workspace(l);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return FP4Q_ERR_WORKSPACE;
  l.ws = static_cast<uint8_t*>(workspace);
  return hip_status(launch_kv_attend(l, static_cast<hipStream_t>(hip_stream)));
}

}  // extern "C"
