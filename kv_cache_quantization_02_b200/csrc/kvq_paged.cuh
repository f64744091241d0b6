// kvq_paged.cuh -- what the units of the paged 8-bit cache share: the cache's
// parameters, 8-bit code conversions, the search for the sequence that a work
// item belongs to, and the fault word's bits.  Included at global scope.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace kvqp {

constexpr unsigned kAll = 0xffffffffu;
constexpr unsigned kFaultWait = 1u, kFaultBlock = 4u, kFaultLength = 8u;   // kvq_fault_status bits
constexpr float kScaleMin = 0x1p-40f, kScaleMax = 0x1p40f;

enum { kInt8 = 0, kE4m3 = 1 };

// The cache and its tables (include/kvq.h, "The paged 8-bit cache").
struct Cache {
  uint8_t* kc;
  uint8_t* vc;
  float* ks;
  float* vs;
  const int32_t* table;      // [B][max_blocks]
  int64_t num_blocks;
  int B, max_blocks, Hkv, D, block, log_block;
};

// The cache block of a sequence's j-th block, or -1 (and the fault bit in
// `bad`) if the table has none.
__device__ __forceinline__ int block_at(const Cache& c, int b, int64_t j, unsigned& bad) {
  int id = -1;
  if (j >= 0 && j < c.max_blocks) id = c.table[static_cast<int64_t>(b) * c.max_blocks + j];
  if (id < 0 || id >= c.num_blocks) {
    bad |= kFaultBlock;
    id = -1;
  }
  return id;
}

// Work items numbered without a prefix sum: sequence b of n_b rows has the
// items floor(cu[b] mul / per) + slack b onwards, per = 2^log_per.  It may use
// floor(n_b mul / per) + slack of them, since floor(x + n) - floor(x) >=
// floor(n); the last of them may find nothing to do.
__device__ __forceinline__ int64_t item_base(int cu, int b, int mul, int log_per, int slack) {
  return (cu > 0 ? (static_cast<int64_t>(cu) * mul) >> log_per : 0) + static_cast<int64_t>(slack) * b;
}

// The sequence of an item: its number, offsets, entry of `more` (if given) and
// the item's number in it.  A warp narrows the range 32 places at a time to
// 128, and then looks at all of them at once: one load's latency for up to 128
// sequences.  With offsets that do not ascend it ends at some sequence, whose
// ranges callers check.
struct Found {
  int b, c0, c1, more;
  int64_t item;
};
__device__ __forceinline__ Found find_sequence(const int32_t* cu, const int32_t* more, int B, int64_t item, int mul,
                                               int log_per, int slack, int lane) {
  int lo = 0, hi = B;
  while (hi - lo > 128) {
    const int step = (hi - lo + 31) >> 5;
    const int at = lo + lane * step;
    const bool le = at < hi && item_base(cu[at], at, mul, log_per, slack) <= item;
    int n = __popc(__ballot_sync(kAll, le));
    n = n < 1 ? 1 : n;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  Found f;
  if (hi - lo < 32) {                             // few sequences: one load a lane
    const int at = lo + lane;
    const int x = at <= hi ? cu[at] : 0, y = more != nullptr && at < hi ? more[at] : 0;
    int n = __popc(__ballot_sync(kAll, at < hi && item_base(x, at, mul, log_per, slack) <= item));
    n = n < 1 ? 0 : n - 1;                        // the last place that qualifies
    f.b = lo + n;
    f.c0 = __shfl_sync(kAll, x, n);
    f.c1 = __shfl_sync(kAll, x, n + 1);
    f.more = __shfl_sync(kAll, y, n);
  } else {
    int x[4], y[4], n = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = lo + 32 * k + lane;
      x[k] = at <= hi ? cu[at] : 0;
      y[k] = more != nullptr && at < hi ? more[at] : 0;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int at = lo + 32 * k + lane;
      n += __popc(__ballot_sync(kAll, at < hi && item_base(x[k], at, mul, log_per, slack) <= item));
    }
    n = n < 1 ? 0 : n - 1;
    f.b = lo + n;
    f.c0 = f.c1 = f.more = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = __shfl_sync(kAll, x[k], n & 31), v = __shfl_sync(kAll, y[k], n & 31);
      const int w = __shfl_sync(kAll, x[k], (n + 1) & 31);
      if (n >> 5 == k) { f.c0 = u; f.more = v; }
      if ((n + 1) >> 5 == k) f.c1 = w;
    }
    if (n == 127) f.c1 = cu[f.b + 1];
  }
  f.item = item - item_base(f.c0, f.b, mul, log_per, slack);
  return f;
}

// ---- codes ----------------------------------------------------------------------

// Four int8 codes as floats: the code plus 128 in the low byte of 2^23's
// significand, exact, less 2^23 + 128.
__device__ __forceinline__ void int8x4_to_float(uint32_t w, float (&f)[4]) {
  const uint32_t u = w ^ 0x80808080u;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    f[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7650 + i)) - 8388736.0f;
}
// Four e4m3 codes as floats.
__device__ __forceinline__ void e4m3x4_to_float(uint32_t w, float (&f)[4]) {
  uint32_t a, b;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.rn.f16x2.e4m3x2 %0, l;\ncvt.rn.f16x2.e4m3x2 %1, h;\n}"
      : "=r"(a), "=r"(b) : "r"(w));
  const float2 x = __half22float2(*reinterpret_cast<__half2*>(&a));
  const float2 y = __half22float2(*reinterpret_cast<__half2*>(&b));
  f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
}
template <int FMT>
__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
  if constexpr (FMT == kInt8) int8x4_to_float(w, f);
  else e4m3x4_to_float(w, f);
}

// Four values as codes, to nearest even.  int8: saturated to [-128, 127] by
// the packing conversion, then -128 raised to -127; NaN converts to 0.  e4m3:
// saturated to 448; NaN is made 0 first.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
  uint32_t w;
  if constexpr (FMT == kInt8) {
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w) : "r"(__float2int_rn(d)), "r"(__float2int_rn(c)), "r"(0u));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w) : "r"(__float2int_rn(b)), "r"(__float2int_rn(a)), "r"(w));
    return __vmaxs4(w, 0x81818181u);
  } else {
    a = a == a ? a : 0.0f; b = b == b ? b : 0.0f; c = c == c ? c : 0.0f; d = d == d ? d : 0.0f;
    asm("{\n.reg .b16 l, h;\ncvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\ncvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n"
        "mov.b32 %0, {l, h};\n}" : "=r"(w) : "f"(a), "f"(b), "f"(c), "f"(d));
    return w;
  }
}

// ---- fp16 / bf16 ------------------------------------------------------------------

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  else return __half22float2(*reinterpret_cast<__half2*>(&w));
}
template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

}  // namespace kvqp
