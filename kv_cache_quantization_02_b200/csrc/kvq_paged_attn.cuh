// kvq_paged_attn.cuh -- what the decode and prompt attention over the paged
// 8-bit cache share: the launch parameters, codes as fp16 MMA operands, query
// rows as fp16 with a power of two each, and the softmax's formulation.
// Included at global scope, after kvq_paged.cuh.
//
// Softmax with a value scale per block.  With c^K_t, c^V_t the codes of key t,
// S_K, S_V the scales of its block, and
//     w_t = sm_scale log2(e) S_K <q, c^K_t> + log2 S_V,
// and M a running reference near max_t w_t, the output is
//     o = (sum_t P_t c^V_t) / (sum_t P_t / S_V),   P_t = 2^(w_t - M + kBoost).
// One multiply-add per score carries both scales, the codes enter both
// products as they are (exact in fp16), and P_t, an fp16 value there, is
// relative to the largest contribution to the numerator, whatever the value
// scales.  M follows the maximum lazily: it moves when some w_t exceeds it by
// more than kLazy, so P_t <= 2^(kBoost + kLazy) fits fp16 and the largest is
// at least 2^kBoost; fp16's subnormals start 2^(kBoost + 14) below that.
#pragma once

#include "kvq_paged.cuh"

namespace kvqp {

constexpr float kBoost = 6.0f, kLazy = 8.0f;

// Thread blocks of the decode kernel that an SM holds (registers and shared
// memory); a split call launches that many for each SM.  Measured on 64 ragged
// sequences of up to 4K tokens: D = 64 38 us with four, 44 with five, 41 with
// three; D = 256 69 us with three (168 registers), 75 with two.
template <int D>
constexpr int kDecodeBlocks = D == 64 ? 4 : 3;

struct AttnArgs {
  Cache c;
  const uint16_t* q;
  uint16_t* out;
  const int32_t* cu;        // [B + 1]; decode: null, one query per sequence
  const int32_t* seq_len;   // [B]
  float* part;              // split partials, or null: unsplit
  int64_t q_stride, total_q;
  int R, window;            // query heads per KV head
  int bf16, negative;       // element type; sm_scale < 0
  int blocks;               // thread blocks of a split call
  float scale;              // |sm_scale| log2(e)
};

// A code pair as fp16, exact: the bytes at bits 0-7 and 16-23 (even) or 8-15
// and 24-31 (odd) of a word.  int8: the code plus 128 in the low byte of 1024's
// significand, less 1152.  e4m3: a conversion of two neighbouring bytes; it
// makes NaN of the NaN pattern, so slots behind a sequence's last position,
// which may hold anything, have to arrive as zeros (0 x NaN is NaN).
template <int FMT>
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t& even, uint32_t& odd) {
  if constexpr (FMT == kInt8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t e = __byte_perm(u, 0x64646464u, 0x4240), o = __byte_perm(u, 0x64646464u, 0x4341);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(even) : "r"(e), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(odd) : "r"(o), "r"(0x64806480u));
  } else {
    const uint32_t p = __byte_perm(w, 0u, 0x3120);
    asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
        : "=r"(even), "=r"(odd) : "r"(p));
  }
}

// 2^x by the SFU (relative error about 2^-22, results below 2^-126 are 0).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^k for a row whose largest magnitude is `most` (bf16 rows become fp16
// without losing what matters: the largest element lands in [2^14, 2^15), and
// only elements 2^-28 of it or less round).  0, infinities and NaN: k = 0.
__device__ __forceinline__ int row_exponent(float most) {
  if (!(most > 0.0f) || isinf(most)) return 0;
  const int e = static_cast<int>(__float_as_uint(most) >> 23) - 127;     // -127 for subnormals
  return min(14 - e, 126);
}
__device__ __forceinline__ float pow2i(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

// A sequence's length, clamped to its table row.
__device__ __forceinline__ int clamped_length(const AttnArgs& a, int L, unsigned& bad) {
  const int room = a.c.max_blocks << a.c.log_block;
  if (L < 0 || L > room) {
    bad |= kFaultLength;
    L = L < 0 ? 0 : room;
  }
  return L;
}
__device__ __forceinline__ int sequence_length(const AttnArgs& a, int b, unsigned& bad) {
  return clamped_length(a, a.seq_len[b], bad);
}

}  // namespace kvqp

// The launches of each unit (arguments checked): KVQ_OK or KVQ_ERR_LAUNCH with
// the error in `err`.
__attribute__((visibility("hidden"))) int kvq_paged_decode_launch(const kvqp::AttnArgs& a, int format, int grid,
                                                                  cudaStream_t st, cudaError_t& err);
__attribute__((visibility("hidden"))) unsigned int kvq_paged_decode_fault_word(int clear);
__attribute__((visibility("hidden"))) int kvq_paged_prefill_launch(const kvqp::AttnArgs& a, int format, int64_t whole,
                                                                   int nsplit, cudaStream_t st, cudaError_t& err);
__attribute__((visibility("hidden"))) unsigned int kvq_paged_prefill_fault_word(int clear);
