// kvq_paged.cu -- the paged 8-bit cache (include/kvq.h): kvq_paged_write and
// kvq_paged_read, and the C ABI of the attention over it.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "kvq.h"
#include "kvq_paged_attn.cuh"

namespace {

using namespace kvqp;

__device__ unsigned int g_paged_fault = 0;
thread_local int g_paged_cuda_error = 0;

__device__ __forceinline__ void report(unsigned bad) {
  if (bad) atomicOr(&g_paged_fault, bad);
}

struct Tokens {
  const int32_t* cu;      // [B + 1]
  const int32_t* start;   // [B]
  int64_t n_tokens;
};

// What one thread block, or one warp, works on: the tokens of one sequence that
// fall into one cache block, of one KV head, in K or V.
struct Item {
  int b;                  // sequence
  int64_t blk;            // the sequence's block, -1: nothing to do
  int head;
  bool is_v;
  int slot;               // the first token's slot
  int count;              // tokens
  int64_t row;            // the first token's row in the packed tensors
};

// Item numbers run over (sequence, block of its new tokens, head, K or V), the
// last fastest: neighbouring thread blocks read neighbouring pieces of the
// same token rows.  A sequence of n tokens touches at most floor(n / block) + 2
// blocks.  A warp finds its item; the table is read apart from that, so that
// the new tokens' loads need not wait for it.
__device__ __forceinline__ Item find_item(const Cache& c, const Tokens& t, unsigned x, int lane) {
  unsigned bad = 0;
  Item it;
  it.blk = -1;
  it.slot = it.count = 0;
  it.row = 0;
  it.is_v = x & 1;
  x >>= 1;
  it.head = static_cast<int>(x % c.Hkv);
  const Found f = find_sequence(t.cu, t.start, c.B, x / c.Hkv, 1, c.log_block, 2, lane);
  const int64_t c0 = f.c0, c1 = f.c1, p0 = f.more;
  it.b = f.b;
  if (c0 < 0 || c1 < c0 || c1 > t.n_tokens || (p0 < 0 && c1 > c0)) {
    bad |= kFaultLength;
  } else if (c1 > c0 && f.item >= 0) {
    const int64_t blk = (p0 >> c.log_block) + f.item;
    const int64_t lo = max(p0, blk << c.log_block), hi = min(p0 + (c1 - c0), (blk + 1) << c.log_block);
    if (lo < hi) {
      it.blk = blk;
      it.slot = static_cast<int>(lo & (c.block - 1));
      it.count = static_cast<int>(hi - lo);
      it.row = c0 + (lo - p0);
    }
  }
  if (lane == 0) report(bad);
  return it;
}
// A thread block's item, found by its first warp.
__device__ __forceinline__ Item find_block_item(const Cache& c, const Tokens& t) {
  __shared__ Item item;
  if (threadIdx.x < 32) {
    const Item it = find_item(c, t, blockIdx.x, threadIdx.x);
    if (threadIdx.x == 0) item = it;
  }
  __syncthreads();
  return item;
}

// Its cache block, or -1.
__device__ __forceinline__ int find_block(const Cache& c, const Item& it, int lane) {
  unsigned bad = 0;
  const int id = block_at(c, it.b, it.blk, bad);
  if (lane == 0) report(bad);
  return id;
}

// ---------------------------------------------------------------------------
// Write.  A thread block holds its tokens' channels in registers (16
// neighbouring channels a unit, at most VPT units a thread), so the cache
// block's largest magnitude is known before the codes are made and every input
// is read once.  Bound by memory: 16 resident warps an SM with eight units (256
// bytes) each in flight a thread took 34.7 us for a 32K-token prompt of 8 heads
// of 128 channels (5.8 TB/s), fewer bytes a thread 38-44 us, 20 warps with
// spilled registers 44 us.  Where an older scale has to grow, the codes of the earlier
// slots are rounded again; the arithmetic is the header's, one IEEE operation
// at a time.
// ---------------------------------------------------------------------------
template <int FMT>
__device__ __forceinline__ uint4 recode16(uint4 w, float f) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float y[4];
    decode4<FMT>(in[e], y);
    q[e] = encode4<FMT>(y[0] * f, y[1] * f, y[2] * f, y[3] * f);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}
template <int FMT, bool BF16, int T, int VPT>
__global__ void __launch_bounds__(T, 512 / T) paged_write_kernel(Cache c, Tokens t, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, int64_t k_stride,
                                                        int64_t v_stride) {
  const Item it = find_block_item(c, t);
  if (it.blk < 0) return;
  const uint16_t* x = (it.is_v ? v : k) + it.row * (it.is_v ? v_stride : k_stride) + static_cast<int64_t>(it.head) * c.D;
  const int64_t stride = it.is_v ? v_stride : k_stride;
  const int upr = c.D >> 4;                       // units of a row, a power of two
  const int lu = 31 - __clz(upr);
  const int units = it.count << lu;

  uint4 r[VPT][2];
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = threadIdx.x + i * T;
    if (u < units) {
      const uint4* p = reinterpret_cast<const uint4*>(x + (u >> lu) * stride + ((u & (upr - 1)) << 4));
      r[i][0] = __ldcs(p);
      r[i][1] = __ldcs(p + 1);
    } else {
      r[i][0] = r[i][1] = make_uint4(0, 0, 0, 0);
    }
  }
  const int id = find_block(c, it, threadIdx.x & 31);
  if (id < 0) return;                             // all of the thread block
  const int64_t bh = static_cast<int64_t>(id) * c.Hkv + it.head;
  float* scale = (it.is_v ? c.vs : c.ks) + bh;
  uint8_t* codes = (it.is_v ? c.vc : c.kc) + bh * c.block * c.D;
  const float old = it.slot > 0 ? *scale : 0.0f;  // read by all before thread 0 writes it
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {r[i][h].x, r[i][h].y, r[i][h].z, r[i][h].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack2<BF16>(w[e]);
        a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));   // a NaN is passed over
      }
    }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
  __shared__ float most[T / 32];
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = a;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < T / 32; ++w) a = fmaxf(a, most[w]);

  constexpr float inv_q = FMT == kInt8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  const float s = fminf(fmaxf(a * inv_q, kScaleMin), kScaleMax);
  const float S = fmaxf(old, s);                  // a NaN in the old scale is passed over
  const float inv = __fdiv_rn(1.0f, S);
  if (threadIdx.x == 0) *scale = S;

#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int u = threadIdx.x + i * T;
    if (u < units) {
      uint32_t q[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {r[i][h].x, r[i][h].y, r[i][h].z, r[i][h].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float2 f = unpack2<BF16>(w[2 * e]), g = unpack2<BF16>(w[2 * e + 1]);
          q[2 * h + e] = encode4<FMT>(f.x * inv, f.y * inv, g.x * inv, g.y * inv);
        }
      }
      *reinterpret_cast<uint4*>(codes + (static_cast<int64_t>(it.slot) << lu << 4) + (static_cast<int64_t>(u) << 4)) =
          make_uint4(q[0], q[1], q[2], q[3]);
    }
  }
  if (it.slot > 0 && S > old) {
    const float f = __fdiv_rn(old, S);
    uint4* p = reinterpret_cast<uint4*>(codes);
    for (int u = threadIdx.x; u < (it.slot << lu); u += T) p[u] = recode16<FMT>(p[u], f);
  }
}

// The same with a warp per item, for calls of about a token per sequence (at most
// two): four times fewer thread blocks, and no barrier.  64 tokens of 8 heads
// took 2.7 us, 7.1 us with a thread block of 128 an item.  The first 32 units stay in
// registers (two tokens at D = 256), any others are read again.  Both sides of the
// rule at its border (blocks of 64 tokens, D = 128, 8 heads): two tokens for each of 64
// sequences 3.1 us, a thread block an item 6.0; of 256 sequences 5.0 and 15.2.  Where one of
// them has all the tokens but one each: 7.0 and 6.0 us; 7.6 and 15.3.  Codes that are rounded
// again come on top: 64 tokens whose blocks' scales all grow take 6.1 us, not 2.7 (D = 128,
// blocks of 64), at D = 256 and blocks of 128 12.9 us.
template <int FMT, bool BF16>
__device__ __forceinline__ float largest(uint4 w) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
  float a = 0.0f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack2<BF16>(v[e]);
    a = fmaxf(a, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return a;
}
template <int FMT, bool BF16>
__device__ __forceinline__ uint4 encode16(uint4 lo, uint4 hi, float inv) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack2<BF16>(w[2 * e]), g = unpack2<BF16>(w[2 * e + 1]);
    q[e] = encode4<FMT>(f.x * inv, f.y * inv, g.x * inv, g.y * inv);
  }
  return make_uint4(q[0], q[1], q[2], q[3]);
}
template <int FMT, bool BF16>
__global__ void __launch_bounds__(128) paged_append_kernel(Cache c, Tokens t, int64_t items, const uint16_t* __restrict__ k,
                                                           const uint16_t* __restrict__ v, int64_t k_stride,
                                                           int64_t v_stride) {
  const int lane = threadIdx.x & 31;
  const int64_t number = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (number >= items) return;
  const Item it = find_item(c, t, static_cast<unsigned>(number), lane);
  if (it.blk < 0) return;
  const int64_t stride = it.is_v ? v_stride : k_stride;
  const uint16_t* x = (it.is_v ? v : k) + it.row * stride + static_cast<int64_t>(it.head) * c.D;
  const int upr = c.D >> 4, lu = 31 - __clz(upr), units = it.count << lu;
  auto unit_at = [&](int u) { return reinterpret_cast<const uint4*>(x + (u >> lu) * stride + ((u & (upr - 1)) << 4)); };
  uint4 r0 = make_uint4(0, 0, 0, 0), r1 = r0;
  if (lane < units) { r0 = unit_at(lane)[0]; r1 = unit_at(lane)[1]; }
  const int id = find_block(c, it, lane);
  if (id < 0) return;
  const int64_t bh = static_cast<int64_t>(id) * c.Hkv + it.head;
  float* scale = (it.is_v ? c.vs : c.ks) + bh;
  uint4* codes = reinterpret_cast<uint4*>((it.is_v ? c.vc : c.kc) + bh * c.block * c.D);
  const float old = it.slot > 0 ? *scale : 0.0f;
  float a = fmaxf(largest<FMT, BF16>(r0), largest<FMT, BF16>(r1));
  for (int u = lane + 32; u < units; u += 32)
    a = fmaxf(a, fmaxf(largest<FMT, BF16>(unit_at(u)[0]), largest<FMT, BF16>(unit_at(u)[1])));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(kAll, a, o));
  constexpr float inv_q = FMT == kInt8 ? 1.0f / 127.0f : 1.0f / 448.0f;
  const float S = fmaxf(old, fminf(fmaxf(a * inv_q, kScaleMin), kScaleMax));
  const float inv = __fdiv_rn(1.0f, S);
  __syncwarp();
  if (lane == 0) *scale = S;
  if (lane < units) codes[(it.slot << lu) + lane] = encode16<FMT, BF16>(r0, r1, inv);
  for (int u = lane + 32; u < units; u += 32)
    codes[(it.slot << lu) + u] = encode16<FMT, BF16>(unit_at(u)[0], unit_at(u)[1], inv);
  if (it.slot > 0 && S > old) {
    const float f = __fdiv_rn(old, S);
#pragma unroll 4
    for (int u = lane; u < (it.slot << lu); u += 32) codes[u] = recode16<FMT>(codes[u], f);
  }
}

// ---------------------------------------------------------------------------
// Read: the write's items, each unit of 16 codes to 32 bytes of output.  Bound
// by memory: four caches of 32K tokens, 8 heads of 128, in 129 us (6.2 TB/s).
// ---------------------------------------------------------------------------
template <int FMT, bool BF16, int T>
__global__ void __launch_bounds__(T) paged_read_kernel(Cache c, Tokens t, uint16_t* __restrict__ k,
                                                       uint16_t* __restrict__ v) {
  const Item it = find_block_item(c, t);
  if (it.blk < 0) return;
  const int id = find_block(c, it, threadIdx.x & 31);
  if (id < 0) return;
  const int64_t stride = static_cast<int64_t>(c.Hkv) * c.D;
  uint16_t* x = (it.is_v ? v : k) + it.row * stride + static_cast<int64_t>(it.head) * c.D;
  const int64_t bh = static_cast<int64_t>(id) * c.Hkv + it.head;
  const float S = (it.is_v ? c.vs : c.ks)[bh];
  const int upr = c.D >> 4, lu = 31 - __clz(upr);
  const uint4* codes = reinterpret_cast<const uint4*>((it.is_v ? c.vc : c.kc) + bh * c.block * c.D) + (it.slot << lu);
  const int units = it.count << lu;
  for (int u = threadIdx.x; u < units; u += T) {
    const uint4 w = codes[u];
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y[4];
      decode4<FMT>(in[e], y);
      o[2 * e] = pack2<BF16>(y[0] * S, y[1] * S);
      o[2 * e + 1] = pack2<BF16>(y[2] * S, y[3] * S);
    }
    uint4* p = reinterpret_cast<uint4*>(x + (u >> lu) * stride + ((u & (upr - 1)) << 4));
    __stcs(p, make_uint4(o[0], o[1], o[2], o[3]));
    __stcs(p + 1, make_uint4(o[4], o[5], o[6], o[7]));
  }
}

// ---------------------------------------------------------------------------
// Argument checks and launches.
// ---------------------------------------------------------------------------

// A table without columns and a cache without blocks are never read: they need no address (empty tensors have none).
bool missing(const void* table, int max_blocks, const void* kc, const void* vc, const void* ks, const void* vs,
             int64_t num_blocks) {
  return (!table && max_blocks > 0) || (num_blocks > 0 && (!kc || !vc || !ks || !vs));
}

bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_shape(int dtype, int format, int B, int max_blocks, int Hkv, int D, int block, int64_t num_blocks) {
  if (D != 64 && D != 128 && D != 256) return KVQ_ERR_DIM;
  if (block != 16 && block != 32 && block != 64 && block != 128) return KVQ_ERR_FORMAT;
  if ((dtype != KVQ_FP16 && dtype != KVQ_BF16) || (format != KVQ_INT8 && format != KVQ_E4M3)) return KVQ_ERR_FORMAT;
  if (B < 0 || max_blocks < 0 || Hkv < 1 || num_blocks < 0 || num_blocks > INT32_MAX) return KVQ_ERR_COUNT;
  if (static_cast<int64_t>(max_blocks) * block > INT32_MAX) return KVQ_ERR_COUNT;
  // both factors are below 2^31, so neither product overflows 64 bits
  if (num_blocks * Hkv > INT32_MAX || num_blocks * Hkv * block > INT32_MAX) return KVQ_ERR_COUNT;
  return KVQ_OK;
}

// Attention's positions are ints that are rounded up to whole key tiles, and a warp's lanes go 512 keys on from one's
// start: the last 1023 below 2^31 are kept free.
bool fits_positions(int max_blocks, int block) { return static_cast<int64_t>(max_blocks) * block <= INT32_MAX - 1023; }

int check_stride(int64_t stride, int heads, int D) {
  return stride % 8 == 0 && stride >= static_cast<int64_t>(heads) * D && stride <= (int64_t{1} << 40) ? KVQ_OK
                                                                                                   : KVQ_ERR_COUNT;
}

int sm_count() {
  static std::atomic<int> cache[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v < 1) v = 148;
    cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

// Thread blocks of a split decode call: all that the GPU holds at once, or one
// per four tiles of 32 keys if the table has room, or the window, for fewer.  0:
// up to eight tiles, two a warp, are one thread block's, which saves the second
// kernel (about 2 us, as much as six more tiles).
int decode_grid(int B, int max_blocks, int Hq, int Hkv, int D, int block, int window) {
  const int64_t items = static_cast<int64_t>(B) * Hkv * ((Hq / Hkv + 7) / 8);
  int64_t tiles = (static_cast<int64_t>(max_blocks) * block + 31) / 32 + 1;
  if (window > 0 && window / 32 + 2 < tiles) tiles = window / 32 + 2;
  if (tiles <= 8) return 0;
  const int64_t full = static_cast<int64_t>(sm_count()) *
                       (D == 64 ? kDecodeBlocks<64> : D == 128 ? kDecodeBlocks<128> : kDecodeBlocks<256>);
  if (items >= full) return static_cast<int>(full);
  const int64_t most = items * ((tiles + 3) / 4);
  return static_cast<int>(most < full ? most : full);
}
int64_t decode_bytes(int grid, int D) { return static_cast<int64_t>(grid) * (2 * 8 * (D + 4) * 4 + 16); }

// Tiles of a prompt call, and the splits of their keys.  A thread block has an
// SM to itself and a fixed cost of about six key tiles' time.
//
// Tiles see about as many keys where there is a window, or where the new tokens
// are a quarter of the table's room at most.  Up to 32 sequences are then split by
// their lengths, on the device (make_plan in kvq_paged_prefill.cu): whole = -1, and
// nsplit the thread blocks that run at once.  More sequences take full rounds of
// the GPU at half the room's keys (tables are seldom full) or the window's, and
// those rounds may be left unsplit, so that only what is left for the last one is
// split.  Without either, 5 x 256 tokens behind 4000 took 166 us; with the last round
// split 134, by the lengths 114.
//
// A prompt's tiles see anything from nothing to all, so it takes the longest
// tile's time or the average load of an SM: 4096 tokens of 8 heads took 66 us with
// two splits, not 84, and 1500 tokens 38 us without one, 48 with its last round
// split.
struct PromptGrid {
  int64_t tiles, whole;
  int nsplit;
  int64_t bytes;
};

PromptGrid prompt_grid(int B, int max_blocks, int64_t total_q, int Hq, int Hkv, int D, int block, int window) {
  const int rows = D == 256 ? 128 : 256, kt = D == 256 ? 64 : 128;
  PromptGrid g;
  g.tiles = (total_q * (Hq / Hkv) / rows + B) * Hkv;
  constexpr double kFixed = 6.0;
  const int64_t sms = sm_count(), seen = (static_cast<int64_t>(window) + rows * Hkv / Hq) / kt + 1;
  const double most = static_cast<double>(max_blocks) * block / kt;
  const double keys = window > 0 && seen < most / 2 ? static_cast<double>(seen) : most / 2;
  const bool alike = (window > 0 && seen < most / 2) || total_q * 4 <= static_cast<int64_t>(B) * max_blocks * block;
  if (alike && g.tiles <= 4 * sms && keys >= 4 && B <= 32) {  // by the lengths, on the device
    g.whole = -1;
    g.nsplit = static_cast<int>(sms);
    g.bytes = sms * rows * (D + 2) * 4;
    return g;
  }
  const int64_t rounds = alike ? g.tiles / sms : 0, rest = g.tiles % sms;
  auto cost = [&](int64_t full, int64_t split, int n) {       // `full` rounds, then `split` tiles
    if (alike) return full * (kFixed + keys) + (split * n + sms - 1) / sms * (kFixed + std::ceil(keys / n));
    return std::max(kFixed + most / n, split * (kFixed * n + keys) / sms);
  };
  g.nsplit = 1;
  g.whole = g.tiles;
  double best = cost(0, g.tiles, 1);
  for (int n = 2; n <= 16 && n <= keys / 2; ++n)
    for (const int64_t full : {int64_t{0}, rounds}) {
      const int64_t split = full > 0 ? rest : g.tiles;
      // a sixteenth more must be gained, which the partial sums cost
      const double c = cost(full, split, n) * 17 / 16;
      if (split == 0 || split >= 2 * sms || full > 3 || c >= best) continue;
      best = c;
      g.nsplit = n;
      g.whole = g.tiles - split;
    }
  g.bytes = g.nsplit > 1 ? (g.tiles - g.whole) * g.nsplit * rows * (D + 2) * 4 : 0;
  return g;
}

Cache make_cache(const void* kc, const void* vc, const float* ks, const float* vs, const int32_t* table, int B,
                 int max_blocks, int Hkv, int D, int block, int64_t num_blocks) {
  Cache c;
  c.kc = static_cast<uint8_t*>(const_cast<void*>(kc));
  c.vc = static_cast<uint8_t*>(const_cast<void*>(vc));
  c.ks = const_cast<float*>(ks);
  c.vs = const_cast<float*>(vs);
  c.table = table;
  c.num_blocks = num_blocks;
  c.B = B; c.max_blocks = max_blocks; c.Hkv = Hkv; c.D = D; c.block = block;
  c.log_block = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
  return c;
}

int finish() {
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return KVQ_OK;
  g_paged_cuda_error = static_cast<int>(e);
  return KVQ_ERR_LAUNCH;
}

// The number of items of find_item, or 0 if there are too many for one grid.
int64_t item_count(const Cache& c, int64_t n_tokens) {
  const int64_t n = (n_tokens / c.block + 2 * static_cast<int64_t>(c.B)) * c.Hkv * 2;
  return n <= INT32_MAX ? n : 0;
}

template <int FMT, bool BF16>
void launch_write(const Cache& c, const Tokens& t, unsigned grid, const void* k, const void* v, int64_t ks, int64_t vs,
                  cudaStream_t st) {
  const uint16_t *kk = static_cast<const uint16_t*>(k), *vv = static_cast<const uint16_t*>(v);
  if (t.n_tokens <= 2 * static_cast<int64_t>(c.B)) {
    paged_append_kernel<FMT, BF16><<<(grid + 3) / 4, 128, 0, st>>>(c, t, grid, kk, vv, ks, vs);
    return;
  }
  switch (c.block * c.D >> 4) {                   // units of a full cache block
    case 64: paged_write_kernel<FMT, BF16, 32, 2><<<grid, 32, 0, st>>>(c, t, kk, vv, ks, vs); break;
    case 128: paged_write_kernel<FMT, BF16, 32, 4><<<grid, 32, 0, st>>>(c, t, kk, vv, ks, vs); break;
    case 256: paged_write_kernel<FMT, BF16, 32, 8><<<grid, 32, 0, st>>>(c, t, kk, vv, ks, vs); break;
    case 512: paged_write_kernel<FMT, BF16, 64, 8><<<grid, 64, 0, st>>>(c, t, kk, vv, ks, vs); break;
    case 1024: paged_write_kernel<FMT, BF16, 128, 8><<<grid, 128, 0, st>>>(c, t, kk, vv, ks, vs); break;
    default: paged_write_kernel<FMT, BF16, 256, 8><<<grid, 256, 0, st>>>(c, t, kk, vv, ks, vs); break;
  }
}

// One of the four instances for a format and an element type.
#define KVQP_DISPATCH(FN, format, dtype, ...)                           \
  do {                                                                  \
    if ((format) == KVQ_INT8) {                                         \
      if ((dtype) == KVQ_FP16) FN<kInt8, false>(__VA_ARGS__);           \
      else FN<kInt8, true>(__VA_ARGS__);                                \
    } else {                                                            \
      if ((dtype) == KVQ_FP16) FN<kE4m3, false>(__VA_ARGS__);           \
      else FN<kE4m3, true>(__VA_ARGS__);                                \
    }                                                                   \
  } while (0)

template <int FMT, bool BF16>
void launch_read(const Cache& c, const Tokens& t, unsigned grid, void* k, void* v, cudaStream_t st) {
  paged_read_kernel<FMT, BF16, 128><<<grid, 128, 0, st>>>(c, t, static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
}

// The checks and arguments that both attentions share.  KVQ_OK with nothing to
// do leaves p.q null.
int attention_args(AttnArgs& p, const void* q, int dtype, int64_t q_stride, const int32_t* cu_q,
                   const int32_t* seq_len, const int32_t* table, int B, int max_blocks, int64_t total_q, int Hq,
                   int Hkv, int D, int block, int format, int64_t num_blocks, const void* kc, const void* vc,
                   const float* ks, const float* vs, float sm_scale, int window, void* out) {
  int rc = check_shape(dtype, format, B, max_blocks, Hkv, D, block, num_blocks);
  if (rc != KVQ_OK) return rc;
  p.q = nullptr;
  if (Hq < Hkv || Hq % Hkv != 0 || total_q < 0 || total_q > INT32_MAX || total_q * Hq > INT32_MAX || window < 0 ||
      !fits_positions(max_blocks, block) || !std::isfinite(sm_scale * 1.4426951f))      // (the scale the kernels use)
    return KVQ_ERR_COUNT;
  // a window of the whole table is none; any other reaches back from a query that may stand total_q before its sequence
  p.window = window < static_cast<int64_t>(max_blocks) * block ? window : 0;
  if (p.window + total_q > INT32_MAX) return KVQ_ERR_COUNT;
  rc = check_stride(q_stride, Hq, D);
  if (rc != KVQ_OK) return rc;
  if (B == 0 || total_q == 0) return KVQ_OK;
  if (!q || !seq_len || !out || missing(table, max_blocks, kc, vc, ks, vs, num_blocks)) return KVQ_ERR_NULL;
  if (!aligned_to(q, 16) || !aligned_to(kc, 16) || !aligned_to(vc, 16) || !aligned_to(out, 16) ||
      !aligned_to(seq_len, 4) || !aligned_to(table, 4) || !aligned_to(ks, 4) || !aligned_to(vs, 4) ||
      !aligned_to(cu_q, 4))
    return KVQ_ERR_ALIGN;
  if (num_blocks == 0) kc = vc = q;               // what copies of no bytes point to (they want an address all the same)
  p.c = make_cache(kc, vc, ks, vs, table, B, max_blocks, Hkv, D, block, num_blocks);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.cu = cu_q; p.seq_len = seq_len; p.part = nullptr;
  p.q_stride = q_stride; p.total_q = total_q;
  p.R = Hq / Hkv; p.bf16 = dtype == KVQ_BF16; p.negative = sm_scale < 0.0f;
  p.scale = static_cast<float>(std::fabs(static_cast<double>(sm_scale)) * 1.4426950408889634);
  return KVQ_OK;
}

}  // namespace

__attribute__((visibility("hidden"))) unsigned int kvq_paged_fault_word(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_paged_fault, sizeof(v)) != cudaSuccess) return 0;
  if (clear && v) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_paged_fault, &zero, sizeof(zero));
  }
  return v | kvq_paged_decode_fault_word(clear) | kvq_paged_prefill_fault_word(clear);
}
__attribute__((visibility("hidden"))) int kvq_paged_last_cuda_error() { return g_paged_cuda_error; }

extern "C" {

int kvq_paged_write(const void* k, const void* v, int dtype, int64_t k_stride, int64_t v_stride,
                    const int32_t* cu_tokens, const int32_t* start, const int32_t* block_table, int B, int max_blocks,
                    int64_t n_tokens, int Hkv, int D, int block, int format, int64_t num_blocks, void* k_codes,
                    void* v_codes, float* k_scales, float* v_scales, void* stream) {
  int rc = check_shape(dtype, format, B, max_blocks, Hkv, D, block, num_blocks);
  if (rc != KVQ_OK) return rc;
  if (n_tokens < 0 || n_tokens > INT32_MAX) return KVQ_ERR_COUNT;
  if (check_stride(k_stride, Hkv, D) != KVQ_OK || check_stride(v_stride, Hkv, D) != KVQ_OK) return KVQ_ERR_COUNT;
  if (B == 0 || n_tokens == 0) return KVQ_OK;
  if (!k || !v || !cu_tokens || !start ||
      missing(block_table, max_blocks, k_codes, v_codes, k_scales, v_scales, num_blocks))
    return KVQ_ERR_NULL;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(k_codes, 16) || !aligned_to(v_codes, 16) ||
      !aligned_to(cu_tokens, 4) || !aligned_to(start, 4) || !aligned_to(block_table, 4) || !aligned_to(k_scales, 4) ||
      !aligned_to(v_scales, 4))
    return KVQ_ERR_ALIGN;
  const Cache c = make_cache(k_codes, v_codes, k_scales, v_scales, block_table, B, max_blocks, Hkv, D, block, num_blocks);
  const Tokens t{cu_tokens, start, n_tokens};
  const int64_t items = item_count(c, n_tokens);
  if (items == 0) return KVQ_ERR_COUNT;
  (void)cudaGetLastError();
  KVQP_DISPATCH(launch_write, format, dtype, c, t, static_cast<unsigned>(items), k, v, k_stride, v_stride,
                static_cast<cudaStream_t>(stream));
  return finish();
}

int kvq_paged_read(const int32_t* cu_tokens, const int32_t* start, const int32_t* block_table, int B, int max_blocks,
                   int64_t n_tokens, int Hkv, int D, int block, int format, int64_t num_blocks, const void* k_codes,
                   const void* v_codes, const float* k_scales, const float* v_scales, int dtype, void* k_out,
                   void* v_out, void* stream) {
  int rc = check_shape(dtype, format, B, max_blocks, Hkv, D, block, num_blocks);
  if (rc != KVQ_OK) return rc;
  if (n_tokens < 0 || n_tokens > INT32_MAX) return KVQ_ERR_COUNT;
  if (B == 0 || n_tokens == 0) return KVQ_OK;
  if (!cu_tokens || !start || !k_out || !v_out ||
      missing(block_table, max_blocks, k_codes, v_codes, k_scales, v_scales, num_blocks))
    return KVQ_ERR_NULL;
  if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16) || !aligned_to(k_codes, 16) || !aligned_to(v_codes, 16) ||
      !aligned_to(cu_tokens, 4) || !aligned_to(start, 4) || !aligned_to(block_table, 4) || !aligned_to(k_scales, 4) ||
      !aligned_to(v_scales, 4))
    return KVQ_ERR_ALIGN;
  const Cache c = make_cache(k_codes, v_codes, k_scales, v_scales, block_table, B, max_blocks, Hkv, D, block, num_blocks);
  const Tokens t{cu_tokens, start, n_tokens};
  const int64_t items = item_count(c, n_tokens);
  if (items == 0) return KVQ_ERR_COUNT;
  (void)cudaGetLastError();
  KVQP_DISPATCH(launch_read, format, dtype, c, t, static_cast<unsigned>(items), k_out, v_out,
                static_cast<cudaStream_t>(stream));
  return finish();
}

static int check_workspace(int B, int max_blocks, int64_t total_q, int Hq, int Hkv, int D, int block, int window) {
  const int rc = check_shape(KVQ_FP16, KVQ_INT8, B, max_blocks, Hkv, D, block, 0);
  if (rc != KVQ_OK) return rc;
  return Hq < Hkv || Hq % Hkv != 0 || total_q < 0 || total_q > INT32_MAX || total_q * Hq > INT32_MAX || window < 0 ||
                 !fits_positions(max_blocks, block)
             ? KVQ_ERR_COUNT
             : KVQ_OK;
}

int64_t kvq_paged_decode_workspace_bytes(int B, int max_blocks, int Hq, int Hkv, int D, int block, int window) {
  if (check_workspace(B, max_blocks, B, Hq, Hkv, D, block, window) != KVQ_OK) return -1;
  return decode_bytes(decode_grid(B, max_blocks, Hq, Hkv, D, block, window), D);
}

int64_t kvq_paged_prefill_workspace_bytes(int B, int max_blocks, int64_t total_q, int Hq, int Hkv, int D, int block,
                                          int window) {
  if (check_workspace(B, max_blocks, total_q, Hq, Hkv, D, block, window) != KVQ_OK) return -1;
  return prompt_grid(B, max_blocks, total_q, Hq, Hkv, D, block, window).bytes;
}

int kvq_paged_attention_decode(const void* q, int dtype, int64_t q_stride, const int32_t* seq_len,
                               const int32_t* block_table, int B, int max_blocks, int Hq, int Hkv, int D, int block,
                               int format, int64_t num_blocks, const void* k_codes, const void* v_codes,
                               const float* k_scales, const float* v_scales, float sm_scale, int window, void* out,
                               void* workspace, int64_t workspace_bytes, void* stream) {
  AttnArgs p;
  const int rc = attention_args(p, q, dtype, q_stride, nullptr, seq_len, block_table, B, max_blocks, B, Hq, Hkv, D,
                                block, format, num_blocks, k_codes, v_codes, k_scales, v_scales, sm_scale, window, out);
  if (rc != KVQ_OK || p.q == nullptr) return rc;
  const int grid = decode_grid(B, max_blocks, Hq, Hkv, D, block, window);
  if (grid > 0 && workspace && aligned_to(workspace, 16) && workspace_bytes >= decode_bytes(grid, D))
    p.part = static_cast<float*>(workspace);
  p.blocks = grid;
  (void)cudaGetLastError();
  cudaError_t err = cudaSuccess;
  if (kvq_paged_decode_launch(p, format, grid, static_cast<cudaStream_t>(stream), err) == KVQ_OK) return KVQ_OK;
  g_paged_cuda_error = static_cast<int>(err);
  return KVQ_ERR_LAUNCH;
}

int kvq_paged_attention_prefill(const void* q, int dtype, int64_t q_stride, const int32_t* cu_q,
                                const int32_t* seq_len, const int32_t* block_table, int B, int max_blocks,
                                int64_t total_q, int Hq, int Hkv, int D, int block, int format, int64_t num_blocks,
                                const void* k_codes, const void* v_codes, const float* k_scales,
                                const float* v_scales, float sm_scale, int window, void* out, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  AttnArgs p;
  const int rc = attention_args(p, q, dtype, q_stride, cu_q, seq_len, block_table, B, max_blocks, total_q, Hq, Hkv, D,
                                block, format, num_blocks, k_codes, v_codes, k_scales, v_scales, sm_scale, window, out);
  if (rc != KVQ_OK || p.q == nullptr) return rc;
  if (!cu_q) return KVQ_ERR_NULL;
  PromptGrid g = prompt_grid(B, max_blocks, total_q, Hq, Hkv, D, block, window);
  if (g.tiles * (D == 256 ? 16 : 32) > INT32_MAX) return KVQ_ERR_COUNT;
  if (g.nsplit > 1 && workspace && aligned_to(workspace, 16) && workspace_bytes >= g.bytes)
    p.part = static_cast<float*>(workspace);
  else
    g.whole = g.tiles, g.nsplit = 1;
  (void)cudaGetLastError();
  cudaError_t err = cudaSuccess;
  if (kvq_paged_prefill_launch(p, format, g.whole, g.nsplit, static_cast<cudaStream_t>(stream), err) == KVQ_OK)
    return KVQ_OK;
  g_paged_cuda_error = static_cast<int>(err);
  return KVQ_ERR_LAUNCH;
}

}  // extern "C"
