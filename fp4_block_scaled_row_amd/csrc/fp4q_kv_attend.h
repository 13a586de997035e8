// fp4q_kv_attend.h -- attention over the paged 4-bit cache: what its kernels
// share.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j over the tokens j that query i
// of a sequence with n cached tokens and m queries sees: j < n, and causal:
// j <= n - m + i, with a window also j > n - m + i - window.
//
// Types.  NVFP4 values (E2M1 times E4M3, 6 significant bits, 2^-10 to 2688)
// and MXFP4 values (E2M1 times a power of two) are exact in fp16 and bf16, so
// the cache enters the matrix instructions without any rounding: NVFP4 in
// fp16 (one packed product per two values), MXFP4 in bf16 (the conversion
// applies the scale).  The tensor scales are applied in fp32, the keys' to
// the scores and the values' to the output.
//   The queries enter as a sum of kQ pieces in that type, each the rounding of
// what the ones before left.  A bf16 query is exact in one piece; rotated, it
// keeps 22 bits in two fp16 pieces or 16 in two bf16 ones (one fp16 piece, 11
// bits, would move a score by 2^-12 of its terms: at scores of 40 a hundredth of
// a weight; it takes 190 us where two take 229, 4096 queries of 32 heads over as
// many tokens); an fp32 one keeps 22 (fp16) or 24 (bf16).  fp16 pieces
// are scaled by a power of two per row that puts the row's largest value in
// [2^8, 2^9).  The softmax weights enter in kP pieces.  For bf16 outputs one
// in fp16 (2^-12 of the weight, an eighth of the output's own rounding: errors
// of 1.66e-3 of the output where that rounding is 1.65e-3; with two a call over
// 64 contexts took 10 % longer), two in bf16 (2^-17): one bf16 piece (2^-9) is as coarse as that rounding and left
// outputs a third further off than it.  The many-row kernel, where a second
// piece makes the call 1.33 times longer, turns MXFP4 values whose scales allow
// it into fp16 instead (see KvLane::fits_half).  For fp32 outputs two in fp16
// (see weight_pieces) and three in bf16, whose 16 bits in two left an output's
// error at 2e-6 of it, twice that of the sum in fp32.  Scores, maxima, weights' sums and outputs are
// held in fp32.
//
// Layout in the matrix instructions.  Scores are formed transposed, keys as
// the left operand and queries as the right one, so that a lane ends up with
// the weights of one query row for tokens that are also the ones it has to
// supply to the second product: weights go from one instruction to the other
// in registers.  The order of head elements inside the first contraction is
// free; it is chosen so that a lane's codes are contiguous bytes.  The values
// go through LDS, whose transposing read gives a lane 4 tokens of one element.
//
// Running maximum.  A row's maximum is raised only when a score exceeds it by
// more than 8 (in powers of two); until then weights are at most 2^8, which
// fp32 and the pieces' types hold.  So the common step has no exchange between
// lanes and no rescaling.  Sums of weights stay in their lanes to the end.
#pragma once

#include "fp4q_kv.h"

namespace fp4q {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -0x1p126f;       // a maximum before any score
// The larger one, NaN if either is: one instruction for two of them.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
constexpr float kRaise = 8.0f;            // slack of the running maximum

// The element type of a format's matrix products: fp16 for NVFP4 (FMT 1),
// bf16 for MXFP4 (FMT 0).  Weights carry a factor 2^kUp that makes use of
// fp16's range (at most 2^(kUp + kRaise) = 2^15; down to 2^-31 of the maximum).
template <int FMT>
struct KvType;
template <>
struct KvType<0> {
  static constexpr float kUp = 0.0f;
  static __device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
  static __device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const bf16x2_t p = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, p);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return bf_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf_hi(w); }
};
template <>
struct KvType<1> {
  static constexpr float kUp = 7.0f;
  static __device__ __forceinline__ f32x4_t mfma16(u32x4_t a, u32x4_t b, f32x4_t c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  }
  static __device__ __forceinline__ f32x16_t mfma32(u32x4_t a, u32x4_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const f16x2_t p = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, p);
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(f16x2_t, w)[0]; }
  static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(f16x2_t, w)[1]; }
};

// Pieces of a pair of fp32 values: out[0] their rounding, out[1] the rounding
// of the rest, and so on.
template <int FMT, int N>
__device__ __forceinline__ void pieces(float a, float b, uint32_t out[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    out[i] = KvType<FMT>::pack(a, b);
    if (i + 1 < N) {
      a -= KvType<FMT>::lo(out[i]);
      b -= KvType<FMT>::hi(out[i]);
    }
  }
}

// Pieces of a pair of softmax weights.  The second of two fp16 ones is 2^11
// times as large, so that it holds 11 bits of what the first left down to 2^-36
// (2^-43 of the largest weight at least; as it is it would end at 2^-25, and a
// hundred thousand tokens of weight 2^-17 of the largest, whose roundings all go
// one way, would be off by 3e-5), and meets values 2^-11 times as large: exact in
// fp16, NVFP4 values being multiples of 2^-10.
template <int FMT, int N>
__device__ __forceinline__ void weight_pieces(float a, float b, uint32_t out[N]) {
  if constexpr (FMT == 1 && N == 2) {
    out[0] = KvType<1>::pack(a, b);
    out[1] = KvType<1>::pack((a - KvType<1>::lo(out[0])) * 2048.0f, (b - KvType<1>::hi(out[0])) * 2048.0f);
  } else {
    pieces<FMT, N>(a, b, out);
  }
}
// The values that piece q of N meets.
template <int FMT, int N>
__device__ __forceinline__ u32x4_t values_of_piece(int q, u32x4_t v) {
  if (FMT == 1 && N == 2 && q == 1) {
    const f16x8_t by = (_Float16)(1.0f / 2048.0f);
    v = __builtin_bit_cast(u32x4_t, __builtin_bit_cast(f16x8_t, v) * by);
  }
  return v;
}

// ----------------------------------------------------------------------------
// What a lane reads of one plane row.  The lanes of group g = lane / 16 hold
// the elements e(c, g) .. + 7 of every 32-element chunk c: with head_dim 64
// or a multiple of 128 they are one run of head_dim / 4 elements (kRun), so
// that the codes are one wide load and the scales one load too; with others
// 8 elements of each chunk.
template <int FMT, int D>
struct KvLane {
  static constexpr int kChunks = D / 32;
  static constexpr bool kRun = D == 64 || D % 128 == 0;
  static constexpr int kBlock = FMT == 0 ? 32 : 16;
  // scale bytes of a lane: its run's blocks, or one byte a chunk
  static constexpr int kScales = kRun ? (D / 4 >= kBlock ? D / 4 / kBlock : 1) : kChunks;
  static __device__ __forceinline__ int element(int c, int g) { return kRun ? g * (D / 4) + 8 * c : 32 * c + 8 * g; }

  uint32_t codes[kChunks];
  uint32_t scales;                         // kScales bytes (at most 4)

  // From byte `c` of a code row and byte `e` of a scale row on (offsets apart,
  // so that the rows may be scalars).
  __device__ __forceinline__ void load(const uint8_t* row, const uint8_t* srow, uint32_t c0, uint32_t e0, int g) {
    if constexpr (kRun) {
      const uint8_t* p = row + (c0 + g * (D / 8));
      if constexpr (kChunks == 2) {
        const u32x2_t w = *reinterpret_cast<const u32x2_t*>(p);
        codes[0] = w.x;
        codes[1] = w.y;
      } else {
#pragma unroll
        for (int c = 0; c < kChunks; c += 4) {
          const u32x4_t w = *reinterpret_cast<const u32x4_t*>(p + 4 * c);
          codes[c] = w.x;
          codes[c + 1] = w.y;
          codes[c + 2] = w.z;
          codes[c + 3] = w.w;
        }
      }
      const uint8_t* q = srow + (e0 + (g * (D / 4)) / kBlock);
      if constexpr (kScales == 1) scales = *q;
      else if constexpr (kScales == 2) scales = *reinterpret_cast<const uint16_t*>(q);
      else scales = *reinterpret_cast<const uint32_t*>(q);
    } else {
      scales = 0u;
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        codes[c] = *reinterpret_cast<const uint32_t*>(row + (c0 + 16 * c + 4 * g));
        scales |= (uint32_t)srow[e0 + (FMT == 0 ? c : 2 * c + (g >> 1))] << (8 * c);
      }
    }
  }
  // Which of the scale bytes chunk c takes.
  static __device__ __forceinline__ constexpr int scale_of(int c) { return kRun ? (8 * c) / kBlock : c; }

  // Scale bytes of blocks that are no finite numbers: NVFP4's NaN code; for
  // MXFP4 253 and more, which no finite input is stored with (its largest
  // exponent less 2 is 252) and whose values pass bf16's range.
  static __device__ __forceinline__ bool not_finite(uint32_t b) { return FMT == 0 ? b >= 253u : (b & 0x7Fu) == 0x7Fu; }
  // The block that scale byte i is of.
  static __device__ __forceinline__ int block(int i, int g) {
    return kRun ? g * (D / 4) / kBlock + i : (FMT == 0 ? i : 2 * i + (g >> 1));
  }
  // Makes such blocks zero and says which there were (bit i: scale byte i).
  __device__ __forceinline__ uint32_t drop_not_finite() {
    uint32_t keep = 0xFFFFFFFFu, dropped = 0u;
#pragma unroll
    for (int i = 0; i < kScales; ++i) {
      const bool drop = not_finite((scales >> (8 * i)) & 0xFFu);
      keep &= drop ? ~(0xFFu << (8 * i)) : 0xFFFFFFFFu;
      dropped |= drop ? 1u << i : 0u;
    }
    scales &= keep;
    if constexpr (FMT == 0) {      // (scale byte 0 is 2^-127, not 0)
#pragma unroll
      for (int c = 0; c < kChunks; ++c) codes[c] = (keep >> (8 * scale_of(c))) & 1u ? codes[c] : 0u;
    }
    return dropped;
  }
  // Zeros in place of what was loaded (a token that is not there).
  __device__ __forceinline__ void keep_if(bool there) {
    scales = there ? scales : 0u;
    if constexpr (FMT == 0) {
#pragma unroll
      for (int c = 0; c < kChunks; ++c) codes[c] = there ? codes[c] : 0u;
    }
  }
  // MXFP4: whether all values are fp16 numbers, 0.5 x 2^-23 to 6 x 2^13, or zeros.
  __device__ __forceinline__ bool fits_half() const {
    static_assert(FMT == 0, "NVFP4 values always are");
    bool fits = true;
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      const uint32_t b = (scales >> (8 * scale_of(c))) & 0xFFu;
      fits &= b - 104u <= 36u || ((codes[c] & 0x77777777u) == 0u && b != 255u);
    }
    return fits;
  }
  // Chunk c of MXFP4 values that fit, in fp16.
  __device__ __forceinline__ u32x4_t half_values(int c) const {
    const float sc = e8m0_operand((scales >> (8 * scale_of(c))) & 0xFFu);
    u32x4_t o;
    o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], sc, 0));
    o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], sc, 1));
    o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], sc, 2));
    o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], sc, 3));
    return o;
  }
  // All scale bytes prepared for values(): NVFP4's as fp16 pairs.
  struct Scales {
    uint32_t h[FMT == 0 ? 1 : (kScales + 1) / 2];
  };
  __device__ __forceinline__ Scales prepare() const {
    Scales s;
    if constexpr (FMT == 0) {
      s.h[0] = scales;
    } else {
      const int b = (int)(scales & 0x7F7F7F7Fu);   // (bit 7 means nothing in an NVFP4 scale)
      s.h[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false));
      if constexpr (kScales > 2)
        s.h[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true));
    }
    return s;
  }
  // The 8 values of chunk c in the products' type, low elements first.
  __device__ __forceinline__ u32x4_t values(int c, const Scales& s) const {
    const int i = scale_of(c);
    u32x4_t o;
    if constexpr (FMT == 0) {
      const uint32_t b = (s.h[0] >> (8 * i)) & 0xFFu;
      const float sc = e8m0_operand(b);
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[c], sc, 0));
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[c], sc, 1));
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[c], sc, 2));
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes[c], sc, 3));
      // (scale byte 255 gives NaN, values past bf16's range infinity)
    } else {
      const f16x2_t pair = __builtin_bit_cast(f16x2_t, s.h[i / 2]);
      const _Float16 one = pair[i % 2];
      const f16x2_t sc = {one, one};
      o.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], 1.0f, 0) * sc);
      o.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], 1.0f, 1) * sc);
      o.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], 1.0f, 2) * sc);
      o.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes[c], 1.0f, 3) * sc);
    }
    return o;
  }
};

// Where the rows of a token are, in the planes of one cache head (the lane's
// own part of a row included): a lane's token is found by its page number and
// offset with two 64-bit multiply-adds a plane pair.
struct KvHead {
  const uint8_t *kc, *ks, *vc, *vs;
};
__device__ __forceinline__ KvHead kv_head(const KvPlanes& p, int head) {
  KvHead h;
  const uint64_t c = (uint64_t)head * p.code_stride[1], s = (uint64_t)head * p.scale_stride[1];
  h.kc = p.kc + c;
  h.vc = p.vc + c;
  h.ks = p.ks + s;
  h.vs = p.vs + s;
  return h;
}
struct KvAt {
  uint64_t code, scale;
};
__device__ __forceinline__ KvAt kv_at(const KvPlanes& p, uint32_t page, uint32_t offset) {
  KvAt a;
  a.code = (uint64_t)page * p.code_stride[0] + (uint64_t)offset * p.code_stride[2];
  a.scale = (uint64_t)page * p.scale_stride[0] + (uint64_t)offset * p.scale_stride[2];
  return a;
}

// Four tokens of one element a lane: lane l of each 16 gives the address of
// tokens' row l / 4, elements 4 (l % 4) .. + 3, and gets element l of rows 0-3.
__device__ __forceinline__ u32x2_t read_transposed(const uint16_t* p) {
  const s16x4_t r = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4_t*)(__attribute__((address_space(3))) void*)p);
  return __builtin_bit_cast(u32x2_t, r);
}

// ----------------------------------------------------------------------------
// The schedule.  A unit is one block of kRows query rows (row r of a sequence:
// query r / group, head r % group of its cache head) of one sequence and cache
// head; it has to go through the groups of kTokens tokens that any of its rows
// sees.  The groups of all units are numbered through, (sequence, block)
// first, then cache head, and workgroup w of W takes the w-th stretch of equal
// length: whatever the lengths are, all have the same to do.  A unit counts
// kCost groups more than it has, for what it takes to begin and end it (without
// that the workgroup with the shortest units of a causal prompt, 25 of them
// where others had 2, made the call 1.6 times longer).
//   Blocks go by numbers of which some are skipped, so that no list has to be
// built.  Either block k of sequence b has the number b * per_seq + k, with
// per_seq blocks the most of any sequence; or, where lengths of queries differ
// so much that most of those would be skipped, cu[b] group / kRows + b + k
// (rounded down), which skips at most one a sequence, and a thread finds a
// number's sequence by bisection.
//   All of these numbers are below 2^31 (calls that could pass it are refused).
struct KvUnit {
  int b, block, blocks;   // sequence, block of its query rows, its blocks
  int head;               // cache head
  int row0;               // first query row
  int q0, m, n;           // first row of q, queries, cached tokens
  int lo, hi;             // tokens that some row of the block sees
  int groups;             // at least 1: rows without tokens are written too
};

// A value that the whole wave reads, through the scalar cache: its wait does
// not take in the vector loads that are on their way.
template <typename T>
__device__ __forceinline__ T scalar(const T* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) T*>(reinterpret_cast<uintptr_t>(p));
}

// Row of q of sequence b's first query (never past the rows there are).
template <bool kUniform = false>
__device__ __forceinline__ int kv_first_query(const KvAttendLaunch& a, int b) {
  const int q = a.cu_q ? (kUniform ? scalar(a.cu_q + b) : a.cu_q[b]) : b;
  return min(max(q, 0), (int)a.total_q);
}

template <int kRows>
__device__ __forceinline__ int kv_block_number(const KvAttendLaunch& a, int b) {
  return (int)((uint32_t)(kv_first_query(a, b) * a.group) / kRows) + b;
}

// Blocks of a sequence of m queries; of more than max_q the blocks past those
// are left out, so that all ways of counting agree whatever cu_q holds.
template <int kRows>
__device__ __forceinline__ int kv_blocks(const KvAttendLaunch& a, int m) {
  return (int)(((uint32_t)(min(max(m, 0), a.max_q) * a.group) + kRows - 1) / kRows);
}

template <int kRows, bool kUniform = false>
__device__ __forceinline__ void kv_sequence(const KvAttendLaunch& a, int b, KvUnit& u) {
  u.b = b;
  u.q0 = kv_first_query<kUniform>(a, b);
  u.m = kv_first_query<kUniform>(a, b + 1) - u.q0;
  u.n = min(max(kUniform ? scalar(a.lens + b) : a.lens[b], 0), (int)a.most_tokens);
  u.blocks = kv_blocks<kRows>(a, u.m);
}

// Queries of the first and last of rows row0 .. row0 + kRows - 1.
template <int kRows>
__device__ __forceinline__ void kv_queries(const KvAttendLaunch& a, const KvUnit& u, int row0, int& i0, int& i1) {
  i0 = (int)quotient((uint32_t)row0, a.group_div);
  i1 = min((int)quotient((uint32_t)(row0 + kRows - 1), a.group_div), u.m - 1);
}

template <int kRows, int kTokens>
__device__ __forceinline__ void kv_block_at(const KvAttendLaunch& a, int row0, KvUnit& u) {
  u.row0 = row0;
  int i0, i1;
  kv_queries<kRows>(a, u, row0, i0, i1);
  const int past = u.n - u.m;                 // tokens before the first query's (may be negative)
  u.hi = max(0, a.causal ? past + i1 + 1 : u.n);
  const int first = a.window > 0 && past + i0 + 1 > a.window ? past + i0 + 1 - a.window : 0;
  u.lo = min(first, u.hi) & ~31;              // (whole tiles of 32: a page's, where pages allow)
  u.groups = max(1, (u.hi - u.lo + kTokens - 1) / kTokens);
}
template <int kRows, int kTokens>
__device__ __forceinline__ void kv_block(const KvAttendLaunch& a, int block, KvUnit& u) {
  u.block = block;
  kv_block_at<kRows, kTokens>(a, block * kRows, u);
}

// Block number -> sequence and block; false: a skipped number.
template <int kRows, int kTokens>
__device__ __forceinline__ bool kv_numbered(const KvAttendLaunch& a, int number, KvUnit& u) {
  int b, block;
  if (a.per_seq.d) {
    b = (int)quotient((uint32_t)number, a.per_seq);
    block = number - b * (int)a.per_seq.d;
  } else {
    b = 0;
    for (int hi = a.seqs; hi - b > 1;) {
      const int mid = (b + hi) >> 1;
      if (kv_block_number<kRows>(a, mid) <= number) b = mid;
      else hi = mid;
    }
    block = number - kv_block_number<kRows>(a, b);
  }
  kv_sequence<kRows>(a, b, u);
  if (block < 0 || block >= u.blocks) return false;
  kv_block<kRows, kTokens>(a, block, u);
  return true;
}

// The workgroups' stretches.  A CU issues its oldest waves first, so that of
// three workgroups on each CU the first ones were done in 66 us, the second in
// 72 and the third in 78 where all had the same; where a launch fills the chip
// with three a CU, they take shares of 36, 32 and 28 parts instead: 1 to 5 %
// less in seven shapes of both formats, head_dim 64 to 128, 2 to 256 sequences
// of 3000 to 131071 tokens (82.5 for 84.9 us, 69.5 for 73, 55.9 for 57.5).
constexpr uint32_t kPart0 = 36, kPart1 = 32, kPart2 = 28;
struct KvShares {
  uint32_t size0, size1, size2;      // groups of a workgroup of the first, second and last `per`
  uint32_t from1, from2;             // where the second and the last begin
  uint32_t per;
};
__device__ __forceinline__ KvShares kv_shares(uint32_t total, uint32_t workgroups, bool thirds) {
  KvShares s;
  if (thirds) {
    s.per = workgroups / 3;
    // (rounded up: sizes are for per * 96 parts of total)
    const uint32_t each = (total + s.per - 1) / s.per;
    s.size0 = (each * kPart0 + 95) / 96;
    s.size1 = (each * kPart1 + 95) / 96;
    s.size2 = (each * kPart2 + 95) / 96;
    s.from1 = s.per * s.size0;
    s.from2 = s.from1 + s.per * s.size1;
  } else {
    s.per = workgroups;
    s.size0 = s.size1 = s.size2 = (total + workgroups - 1) / workgroups;
    s.from1 = s.from2 = s.per * s.size0;
  }
  return s;
}
__device__ __forceinline__ uint32_t kv_begin(const KvShares& s, uint32_t w) {
  return w < s.per ? w * s.size0 : (w < 2 * s.per ? s.from1 + (w - s.per) * s.size1 : s.from2 + (w - 2 * s.per) * s.size2);
}
// The workgroup that has group x.
__device__ __forceinline__ uint32_t kv_owner(const KvShares& s, uint32_t x) {
  const uint32_t third = x < s.from1 ? 0u : (x < s.from2 ? 1u : 2u);
  const uint32_t from = third == 0u ? 0u : (third == 1u ? s.from1 : s.from2);
  const uint32_t size = third == 0u ? s.size0 : (third == 1u ? s.size1 : s.size2);
  return third * s.per + (x - from) / size;
}

// A workgroup's stretch: `left` counted groups from the `at`-th of unit `u` on,
// whose own first one has the number `begins`.
struct KvStretch {
  KvUnit u;
  int at, left, begins;
  KvShares shares;
};
// The groups [from, to) that a stretch has of its current unit: none where it
// ends within the unit's kCost.
template <int kCost>
__device__ __forceinline__ void kv_part(const KvStretch& st, int& from, int& to) {
  from = max(0, st.at - kCost);
  to = max(0, min(st.u.groups + kCost - st.at, st.left) + st.at - kCost);
}

// Inclusive sum over the lanes of a wave: within rows of 16 lanes, then rows 0
// and 2 into 1 and 3, then the first two into the last two.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);     // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);     // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);     // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);     // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);    // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);    // row_bcast:31
  return v;
}

// Every thread of the workgroup calls it, with all query block numbers below
// `numbers`; scratch: 6 + waves words of LDS.  False: nothing to do.  To 256
// numbers each wave goes through them all by itself, which spares the first
// step of every call its barriers.
template <int kRows, int kTokens, int kCost, int kThreadsWg, bool kThirds>
__device__ __forceinline__ bool kv_stretch(const KvAttendLaunch& a, int numbers, KvStretch& st, int* scratch) {
  constexpr int kW = kThreadsWg / 64;
  const bool alone = numbers <= 256;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int each = alone ? (numbers + 63) / 64 : (numbers + kThreadsWg - 1) / kThreadsWg;
  const int x0 = (alone ? lane : (int)threadIdx.x) * each, x1 = min(x0 + each, numbers);
  int mine = 0;
  KvUnit u = {};
  for (int x = x0; x < x1; ++x)
    if (kv_numbered<kRows, kTokens>(a, x, u)) mine += (u.groups + kCost) * a.p.heads;
  int upto = wave_scan(mine), total = 0;     // inclusive scan
  if (alone) {
    total = __builtin_amdgcn_readlane(upto, 63);
  } else {
    if (lane == 63) scratch[wave] = upto;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      if (w < wave) upto += scratch[w];
      total += scratch[w];
    }
    total = __builtin_amdgcn_readfirstlane(total);
  }
  st.shares = kv_shares((uint32_t)total, gridDim.x, kThirds && gridDim.x == a.thirds);
  const int begin = (int)min(kv_begin(st.shares, blockIdx.x), (uint32_t)total);
  const int end = (int)min(kv_begin(st.shares, blockIdx.x + 1), (uint32_t)total);
  if (begin >= end) return false;
  int before = upto - mine;
  const bool owner = begin >= before && begin < upto;
  if (owner && each > 1) {
    for (int x = x0; x < x1; ++x) {
      if (!kv_numbered<kRows, kTokens>(a, x, u)) continue;
      const int here = (u.groups + kCost) * a.p.heads;
      if (begin < before + here) break;
      before += here;
    }
  }
  int found[6] = {u.b, u.block, u.q0, u.m, u.n, begin - before};
  if (alone) {
    const int from = __ffsll((long long)__ballot(owner)) - 1;
#pragma unroll
    for (int i = 0; i < 6; ++i) found[i] = __builtin_amdgcn_readlane(found[i], from);
  } else {
    if (owner) {
#pragma unroll
      for (int i = 0; i < 6; ++i) scratch[kW + i] = found[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 6; ++i) found[i] = __builtin_amdgcn_readfirstlane(scratch[kW + i]);
  }
  st.u.b = found[0];
  st.u.q0 = found[2];
  st.u.m = found[3];
  st.u.n = found[4];
  st.u.blocks = kv_blocks<kRows>(a, st.u.m);
  kv_block<kRows, kTokens>(a, found[1], st.u);
  const int counted = st.u.groups + kCost;
  st.u.head = found[5] / counted;
  st.at = found[5] - st.u.head * counted;
  st.left = end - begin;
  st.begins = begin - st.at;
  return true;
}

// Goes on to the next unit; false: the stretch is done.
template <int kRows, int kTokens, int kCost>
__device__ __forceinline__ bool kv_next(const KvAttendLaunch& a, KvStretch& st) {
  KvUnit& u = st.u;
  st.left -= u.groups + kCost - st.at;
  if (st.left <= 0) return false;
  st.begins += u.groups + kCost;
  st.at = 0;
  if (++u.head < a.p.heads) return true;
  u.head = 0;
  int block = u.block + 1;
  while (block >= u.blocks && u.b + 1 < a.seqs) {
    kv_sequence<kRows, true>(a, u.b + 1, u);
    block = 0;
  }
  kv_block<kRows, kTokens>(a, block, u);
  return true;
}

// Numbers of all query blocks lie below this; sets the kind of numbering.
inline int64_t kv_block_numbers(KvAttendLaunch& a, int rows) {
  const int64_t most = ((int64_t)a.max_q * a.group + rows - 1) / rows;
  const int64_t all = a.seqs * (most < 1 ? 1 : most), compact = a.total_q * a.group / rows + a.seqs;
  a.per_seq = fast_div(0);
  if (all > 2 * compact || all > (1 << 30)) return compact;
  a.per_seq = fast_div((uint32_t)(most < 1 ? 1 : most));
  return all;
}
// The counted groups of a call are at most so many.
inline int64_t kv_most_groups(const KvAttendLaunch& a, int64_t numbers, int tokens, int cost) {
  const int64_t groups = (a.most_tokens + tokens - 1) / tokens;
  return numbers * a.p.heads * ((groups < 1 ? 1 : groups) + cost);
}

// The workspace: a record a workgroup, then for either end of each workgroup's
// stretch the partial result of the unit it shares with its neighbours: kRows x
// D weighted values, then each row's maximum and sum.  Units that several
// workgroups share are joined
//   - few rows: by whichever of a few neighbours finishes last, found by
//     counting arrivals in the record of the first of them, then by the last of
//     a few of those, and so on; each clears its counter again, so that all are
//     zero between calls.  Saves a launch.
//   - many rows: by a second kernel with many more workgroups, since one would
//     take too long over them (a call of 16 units of 64 rows x 256 in 16 pieces
//     each took 93 us that way, 45 with a second kernel).  The records then
//     also say which units are shared.
constexpr int kMostWorkgroups = 1024;      // of a launch
struct KvShared {
  uint32_t arrived[5];      // pieces of the unit that begins in the stretch, by level (see kv_join)
  uint32_t arrived_in[5];   // pieces of a unit that began earlier
  int32_t first;     // 1: the stretch begins with a piece of an earlier unit, 2: with its last one
  int32_t last;      // 1: it ends with the first piece of a unit, sequence b, rows row0 on of `head`
  int32_t b, head, row0;
  int32_t unused[1];      // (64 bytes: each record in a cache line of its own)
};
__device__ __forceinline__ KvShared* kv_shared(const KvAttendLaunch& a, int64_t workgroup) {
  return reinterpret_cast<KvShared*>(a.ws) + workgroup;
}
template <int D, int kRows>
__device__ __forceinline__ float* kv_partial(const KvAttendLaunch& a, int64_t workgroup, bool last) {
  return reinterpret_cast<float*>(a.ws + kMostWorkgroups * sizeof(KvShared)) +
         (2 * workgroup + (last ? 1 : 0)) * (int64_t)kRows * (D + 2);
}
inline size_t kv_workspace_bytes(int64_t workgroups, int64_t rows, int64_t head_dim) {
  return kMostWorkgroups * sizeof(KvShared) + (size_t)(workgroups * 2 * rows * (head_dim + 2)) * sizeof(float);
}

// Partial results are written and read by relaxed atomics of agent scope, which
// go past the caches that the chip's parts do not share; a workgroup counts its
// arrival after its own have completed (vmcnt 0 of every wave, then a barrier).
// The wait is an asm statement that clobbers memory: the builtin counts as
// touching none, so that the compiler would be free to move stores past it.
// Agent fences, which write back and invalidate whole L2 caches, made a call
// over a batch of 64 four times longer.
__device__ __forceinline__ void put2(float* p, float a, float b) {
  const uint64_t w = (uint64_t)as_u(a) | ((uint64_t)as_u(b) << 32);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void wait_for_own_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ float2_t get2(const float* p) {
  const uint64_t w = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return float2_t{as_f((uint32_t)w), as_f((uint32_t)(w >> 32))};
}

// Query head and row of q of row rr of a sequence; false: past its queries, or
// past max_q of them.
struct KvOutRow {
  int64_t at;     // row of out and lse, [total_q][q_heads]
};
__device__ __forceinline__ bool kv_out_row(const KvAttendLaunch& a, int q0, int m, int head, int rr, KvOutRow& o) {
  const int i = (int)quotient((uint32_t)rr, a.group_div);
  o.at = ((int64_t)q0 + i) * ((int64_t)a.p.heads * a.group) + (int64_t)head * a.group + (rr - i * a.group);
  return i < min(m, a.max_q);
}

// Zeros, and log-sum-exps of minus infinity, for queries [from, to).
template <int D, int kThreadsWg>
__device__ __forceinline__ void kv_clear(const KvAttendLaunch& a, int from, int to, int first, int workgroups) {
  const int64_t per = (int64_t)a.p.heads * a.group, r0 = from * per, r1 = to * per;   // rows of out and lse
  const int64_t at = (int64_t)first * kThreadsWg + threadIdx.x, step = (int64_t)workgroups * kThreadsWg;
  const int chunks = D * (a.dtype == kF32 ? 4 : 2) / 16;
  u32x4_t* out = static_cast<u32x4_t*>(a.out);
  for (int64_t i = r0 * chunks + at; i < r1 * chunks; i += step) out[i] = u32x4_t{0u, 0u, 0u, 0u};
  if (a.lse)
    for (int64_t i = r0 + at; i < r1; i += step) a.lse[i] = -INFINITY;
}
// Rows that no unit has, which would be left as they were: queries past the last
// sequence's (a batch padded to the size of a captured call), shared out over the
// workgroups, and queries of a sequence past max_q.
template <int D, int kThreadsWg>
__device__ __forceinline__ void kv_clear_others(const KvAttendLaunch& a) {
  if (!a.cu_q) return;      // (as many rows as sequences)
  const int end = kv_first_query<true>(a, a.seqs);
  if (end < a.total_q) kv_clear<D, kThreadsWg>(a, end, (int)a.total_q, blockIdx.x, gridDim.x);
  if (a.max_q >= a.total_q) return;
  for (int b = blockIdx.x; b < a.seqs; b += gridDim.x) {
    const int q0 = kv_first_query<true>(a, b), q1 = kv_first_query<true>(a, b + 1);
    if (q1 - q0 > a.max_q) kv_clear<D, kThreadsWg>(a, q0 + a.max_q, q1, 0, 1);
  }
}

// Pieces of bf16 queries.
inline int kv_bf16_pieces(const KvAttendLaunch& a) { return a.rotate ? 2 : 1; }

// Whether a row's pieces are scaled to fp16's range.
template <int FMT>
constexpr bool kv_scaled_rows() { return FMT == 1; }

// 8 elements of q as they are; rows past the last are zero.
struct RawQ {
  u32x4_t w[2];      // (bf16: the first alone)
};
__device__ __forceinline__ RawQ load_q8(const KvAttendLaunch& a, const KvUnit& u, int row, int at) {
  const uint32_t i = quotient((uint32_t)row, a.group_div);
  RawQ q = {{{0u, 0u, 0u, 0u}, {0u, 0u, 0u, 0u}}};
  if ((int)i < u.m) {
    const int64_t off = (u.q0 + (int64_t)i) * a.q_stride[0] +
                        ((int64_t)u.head * a.group + (row - (int)i * a.group)) * a.q_stride[1] + 8 * at;
    if (a.dtype == kF32) {
      const float* p = static_cast<const float*>(a.q) + off;
      q.w[0] = load16<false>(p);
      q.w[1] = load16<false>(p + 4);
    } else {
      q.w[0] = load16<false>(static_cast<const uint16_t*>(a.q) + off);
    }
  }
  return q;
}
__device__ __forceinline__ void widen_q8(const KvAttendLaunch& a, const RawQ& q, float v[8]) {
  if (a.dtype == kF32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = as_f(q.w[k >> 2][k & 3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = bf_lo(q.w[0][k]);
      v[2 * k + 1] = bf_hi(q.w[0][k]);
    }
  }
}

// A workgroup's ROWS query rows on their way into LDS: its threads' parts of
// them as they were loaded, and then as kQ pieces in rows of D + 8 halves,
// pieces ROWS rows apart, with each row's factor from raw score to exponent of
// two in factor[].  The factors are positive, so that masked scores stay minus
// infinity: a negative scale goes into the queries' signs, and a product of
// zero (a scale of 0; a row of zeros with a small tensor scale) becomes kLeast.
constexpr float kLeast = 0x1p-126f;
template <int D, int ROWS>
struct QueryRows {
  static constexpr int kPer = D / 8, kItems = ROWS * kPer;
  static constexpr int kEach = (kItems + kThreads - 1) / kThreads;
  RawQ raw[kEach];
};
template <int D, int ROWS>
__device__ __forceinline__ void load_queries(const KvAttendLaunch& a, const KvUnit& u, QueryRows<D, ROWS>& q) {
  using Q = QueryRows<D, ROWS>;
#pragma unroll
  for (int k = 0; k < Q::kEach; ++k) {
    const int item = threadIdx.x + k * kThreads;      // (whole waves: kItems is a multiple of 64)
    if (item < Q::kItems) q.raw[k] = load_q8(a, u, u.row0 + item / Q::kPer, item % Q::kPer);
  }
}
// Every thread of the workgroup calls it; it ends synchronised.  most[]: ROWS
// words of scratch.
template <int FMT, int D, int kQ, int ROWS>
__device__ __forceinline__ void stage_queries(const KvAttendLaunch& a, float kg, const QueryRows<D, ROWS>& in,
                                              uint16_t* sq, float* factor, uint32_t* most) {
  using Q = QueryRows<D, ROWS>;
  const int tid = threadIdx.x;
  const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
  float v[Q::kEach][8];
  if constexpr (kv_scaled_rows<FMT>()) {
    for (int i = tid; i < ROWS; i += kThreads) most[i] = 0u;
    __syncthreads();
  }
#pragma unroll
  for (int k = 0; k < Q::kEach; ++k) {
    const int item = tid + k * kThreads;
    if (item < Q::kItems) {
      widen_q8(a, in.raw[k], v[k]);
      if constexpr (D % 128 == 0) {
        if (a.rotate) fwht128_lanes(v[k], tid & 15, a.rot_scale);
      }
      if constexpr (kv_scaled_rows<FMT>()) atomicMax(most + item / Q::kPer, abs_max_bits8(v[k]));
    }
  }
  __syncthreads();
  const float base = fabsf(a.scale) * kLog2e * kg;
  for (int i = tid; i < ROWS; i += kThreads) {
    float f = base;
    if constexpr (kv_scaled_rows<FMT>()) f *= as_f((min(max(most[i] >> 23, 9u), 254u) - 8u) << 23);
    factor[i] = larger(f, kLeast);
  }
#pragma unroll
  for (int k = 0; k < Q::kEach; ++k) {
    const int item = tid + k * kThreads;
    if (item < Q::kItems) {
      const int row = item / Q::kPer, at = item % Q::kPer;
      float f = sign;
      if constexpr (kv_scaled_rows<FMT>()) f *= as_f((262u - min(max(most[row] >> 23, 9u), 254u)) << 23);
      uint32_t w[4][kQ];
#pragma unroll
      for (int j = 0; j < 4; ++j) pieces<FMT, kQ>(v[k][2 * j] * f, v[k][2 * j + 1] * f, w[j]);
#pragma unroll
      for (int q = 0; q < kQ; ++q)
        *reinterpret_cast<u32x4_t*>(sq + ((size_t)q * ROWS + row) * (D + 8) + 8 * at) =
            u32x4_t{w[0][q], w[1][q], w[2][q], w[3][q]};
    }
  }
  __syncthreads();
}

// Tokens [from, from + count) that row rr of a unit's sequence sees.
__device__ __forceinline__ void kv_sees(const KvAttendLaunch& a, const KvUnit& u, int rr, int& from, uint32_t& count) {
  const int i = (int)quotient((uint32_t)rr, a.group_div);
  const int upto = u.n - u.m + i + 1;         // the query's own token is the one before
  const int to = a.causal ? min(upto, u.n) : u.n;
  from = a.window > 0 && upto > a.window ? min(upto - a.window, u.n) : 0;
  count = i < u.m && to > from ? (uint32_t)(to - from) : 0u;
}
// Tokens [from, to) that every row of a block sees.
template <int kRows>
__device__ __forceinline__ void kv_all_see(const KvAttendLaunch& a, const KvUnit& u, int& from, int& to) {
  int i0, i1;
  kv_queries<kRows>(a, u, u.row0, i0, i1);
  const int past = u.n - u.m;
  to = max(0, a.causal ? min(u.n, past + i0 + 1) : u.n);
  from = a.window > 0 && past + i1 + 1 > a.window ? past + i1 + 1 - a.window : 0;
}

// Values that are no finite numbers, in a tile that some rows see only in part,
// enter the products as zeros: 0 times NaN must not reach the rows that do not
// see them.  Their tokens and blocks (a bit each) are noted where they are left
// out, and the rows that do see one made NaN at the end.  Such tiles are the ones
// at either end of a block's tokens: of a window's beginnings, which spread over
// kRows tokens at most, with the rest of two tiles, and of the rows' last tokens.
template <int kRows, int kTile>
struct NotedNans {
  static constexpr int kMost = 2 * kRows + 4 * kTile;
  int count;
  int token[kMost];
  uint32_t blocks[kMost];

  // The lane's part (group g of the token's row) of what was left out.
  template <int FMT, int D>
  __device__ __forceinline__ void note(int t, int g, uint32_t dropped) {
    uint32_t b = 0u;
#pragma unroll
    for (int i = 0; i < KvLane<FMT, D>::kScales; ++i) b |= ((dropped >> i) & 1u) << KvLane<FMT, D>::block(i, g);
    b |= __shfl_xor((int)b, 16, 64);
    b |= __shfl_xor((int)b, 32, 64);
    if (g != 0 || b == 0u) return;
    const int at = atomicAdd(&count, 1);
    if (at >= kMost) return;
    token[at] = t;
    blocks[at] = b;
  }
  // The noted blocks that row rr sees.
  __device__ __forceinline__ uint32_t seen(const KvAttendLaunch& a, const KvUnit& u, int rr) const {
    int from;
    uint32_t sees, b = 0u;
    kv_sees(a, u, rr, from, sees);
#pragma unroll 1
    for (int i = 0; i < min(count, kMost); ++i) b |= (uint32_t)(token[i] - from) < sees ? blocks[i] : 0u;
    return b;
  }
};

// Stores 4 consecutive elements of an output row.
__device__ __forceinline__ void store_out4(const KvAttendLaunch& a, int64_t o, f32x4_t v) {
  if (a.dtype == kF32) {
    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + o) = v;
  } else {
    *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.out) + o) =
        u32x2_t{KvType<0>::pack(v.x, v.y), KvType<0>::pack(v.z, v.w)};
  }
}

// Elements d .. d + 3 of a finished row rr: the sum of weighted values over
// the sum of weights, and with element 0 the row's log-sum-exp.
template <int FMT, int D>
__device__ __forceinline__ void kv_finish4(const KvAttendLaunch& a, const KvUnit& u, int rr, int d, f32x4_t sum,
                                           float top, float total) {
  KvOutRow out;
  if (!kv_out_row(a, u.q0, u.m, u.head, rr, out)) return;
  const float inv = total == 0.0f ? 0.0f : (FMT == 1 ? scalar(a.p.vg) : 1.0f) / total;
  store_out4(a, out.at * D + d, total == 0.0f ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : sum * inv);
  if (a.lse && d == 0)
    a.lse[out.at] = total == 0.0f ? -INFINITY : (top - KvType<FMT>::kUp + __builtin_amdgcn_logf(total)) * kLn2;
}

// After a workgroup has stored its piece of a shared unit: counts it, and where
// it is the last one joins the pieces: kBatch neighbours, their loads in flight
// together, whose sum is a piece of the next level, until at most 2 kBatch are
// left, which give the output.  A workgroup reads only about 30 GB/s here; in one
// level a unit of 16 rows x 128 took 0.27 us a piece.  With levels of 4 a call
// over 1 x 30000 tokens went from 74 us to 21, one over 2 x 131071 from 75 to 67.5
// (of 8, with more registers in use: 69 and 71).  Every thread of the workgroup
// calls it; `word`, `tops`, `totals`: LDS (a word, kRows, kRows).
template <int FMT, int D, int kRows, int kCost, int kThreadsWg, int kBatch>
__device__ __forceinline__ void kv_join(const KvAttendLaunch& a, const KvUnit& u, int begins, const KvShares& shares,
                                        unsigned int* word, float* tops, float* totals) {
  constexpr uint32_t kPiece = kRows * (D + 2) * sizeof(float);
  // its first real group and its last one say which workgroups have pieces
  const int w0 = (int)kv_owner(shares, (uint32_t)(begins + kCost));
  const int w1 = (int)kv_owner(shares, (uint32_t)(begins + kCost + u.groups - 1));
  const int rows = min(kRows, u.m * a.group - u.row0);
  // (a level's pieces lie where the first of theirs of the first level lies)
  int pieces = w1 - w0 + 1, mine = (int)blockIdx.x - w0, stride = 1;
#pragma unroll 1
  for (int level = 0;; ++level) {
    const bool final = pieces <= 2 * kBatch;
    const int base = final ? 0 : mine / kBatch * kBatch, here = final ? pieces : min(kBatch, pieces - base);
    if (here > 1) {
      wait_for_own_stores();
      __syncthreads();
      if (threadIdx.x == 0) {
        KvShared* record = kv_shared(a, w0 + base * stride);
        uint32_t* counter = base == 0 ? &record->arrived[level] : &record->arrived_in[level];
        const unsigned int arrived = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1;
        if (arrived == (unsigned int)here) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *word = arrived;
      }
      __syncthreads();
      if (*word != (unsigned int)here) return;
      // (one scalar address and 32-bit offsets, for the sake of registers)
      const uint8_t* const from = reinterpret_cast<const uint8_t*>(kv_partial<D, kRows>(a, 0, false));
      const uint32_t first = (uint32_t)(2 * (w0 + base * stride) + (base == 0)) * kPiece;
      const uint32_t second = (uint32_t)(2 * (w0 + (base + 1) * stride)) * kPiece - first;
#pragma unroll 1
      for (int item = threadIdx.x; item < rows * (D / 4); item += kThreadsWg) {
        const int rr = item / (D / 4), d = 4 * (item % (D / 4));
        const uint32_t at = 4 * (rr * D + d), at_ml = 4 * (kRows * D + 2 * rr);
        f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
        float top = kNoMax, total = 0.0f;
        uint32_t piece = first;
#pragma unroll 1
        for (int p = 0; p < here; p += kBatch) {
          float2_t x[kBatch], y[kBatch], ml[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            x[i] = get2(reinterpret_cast<const float*>(from + (piece + at)));
            y[i] = get2(reinterpret_cast<const float*>(from + (piece + at) + 8));
            ml[i] = get2(reinterpret_cast<const float*>(from + (piece + at_ml)));
            if (p + i + 1 < here) piece += p + i == 0 ? second : 2 * kPiece * stride;
          }
          float most = top;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) most = fmaxf(most, ml[i].x);
          const float f = __builtin_amdgcn_exp2f(top - most);
          top = most;
          // (small pieces among themselves before they meet a large one)
          f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
          float part_total = 0.0f;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            const float e = p + i < here ? __builtin_amdgcn_exp2f(ml[i].x - top) : 0.0f;
            part += f32x4_t{x[i].x, x[i].y, y[i].x, y[i].y} * e;
            part_total += ml[i].y * e;
          }
          sum = sum * f + part;
          total = total * f + part_total;
        }
        if (final) {
          kv_finish4<FMT, D>(a, u, u.row0 + rr, d, sum, top, total);
        } else {
          float* part = kv_partial<D, kRows>(a, w0 + base * stride, base == 0) + rr * D + d;
          put2(part, sum.x, sum.y);
          put2(part + 2, sum.z, sum.w);
          if (d == 0) {
            tops[rr] = top;
            totals[rr] = total;
          }
        }
      }
      if (final) return;
      __syncthreads();      // (the maxima and sums have been read by all)
      if ((int)threadIdx.x < rows)
        put2(kv_partial<D, kRows>(a, w0 + base * stride, base == 0) + (int64_t)kRows * D + 2 * threadIdx.x,
             tops[threadIdx.x], totals[threadIdx.x]);
    }
    mine /= kBatch;
    pieces = (pieces + kBatch - 1) / kBatch;
    stride *= kBatch;
  }
}

// The second kernel of the many-row form: a thread takes 4 elements of a row
// of the unit that begins in workgroup blockIdx.x's last piece.
template <int FMT, int D, int kRows>
__global__ __launch_bounds__(kThreads) void kv_join_kernel(KvAttendLaunch a, int workgroups) {
  constexpr int kBatch = 8;
  const int lane = threadIdx.x & 63, w0 = blockIdx.x;
  const KvShared* h = kv_shared(a, w0);
  if (!h->last) return;
  int pieces = 1;          // up to the workgroup whose first piece ends the unit
  for (int w = w0 + 1; w < workgroups; w += 64) {
    const unsigned long long found = __ballot(w + lane < workgroups && kv_shared(a, min(w + lane, workgroups - 1))->first == 2);
    pieces += found ? __ffsll((long long)found) : 64;
    if (found) break;
  }
  KvUnit u;
  u.b = h->b;
  u.head = h->head;
  u.row0 = h->row0;
  u.q0 = kv_first_query(a, u.b);
  u.m = kv_first_query(a, u.b + 1) - u.q0;
  const int item = blockIdx.y * kThreads + threadIdx.x, rr = item / (D / 4), d = 4 * (item % (D / 4));
  if (rr >= min(kRows, u.m * a.group - u.row0)) return;
  f32x4_t sum = {0.0f, 0.0f, 0.0f, 0.0f};
  float top = kNoMax, total = 0.0f;
  for (int p = 0; p < pieces; p += kBatch) {
    f32x4_t v[kBatch];
    float2_t ml[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int q = min(p + i, pieces - 1);
      const float* part = kv_partial<D, kRows>(a, w0 + q, q == 0);
      v[i] = *reinterpret_cast<const f32x4_t*>(part + (int64_t)rr * D + d);
      ml[i] = *reinterpret_cast<const float2_t*>(part + (int64_t)kRows * D + 2 * rr);
    }
    float most = top;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) most = fmaxf(most, ml[i].x);
    const float f = __builtin_amdgcn_exp2f(top - most);
    top = most;
    // (small pieces among themselves before they meet a large one)
    f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
    float part_total = 0.0f;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float e = p + i < pieces ? __builtin_amdgcn_exp2f(ml[i].x - top) : 0.0f;
      part += v[i] * e;
      part_total += ml[i].y * e;
    }
    sum = sum * f + part;
    total = total * f + part_total;
  }
  kv_finish4<FMT, D>(a, u, u.row0 + rr, d, sum, top, total);
}

}  // namespace fp4q
