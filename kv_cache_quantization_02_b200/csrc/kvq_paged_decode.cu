// kvq_paged_decode.cu -- attention of one token per sequence over the paged
// 8-bit cache (include/kvq.h, kvq_paged_attention_decode); the softmax's form
// is in kvq_paged_attn.cuh.
//
// Bound: the codes of K and V (2 D bytes a key and KV head), read once for every
// 8 query heads of a KV head.  With more they are streamed again: 64 ragged
// sequences of up to 4K tokens, D = 128, 4 KV heads, take 58 us with 12 or 16 query
// heads on each, where reading them once would take 24.
//
// Work.  The 32-key tiles of all (sequence, KV head, up to 8 query heads) form
// one line, and every thread block takes an equal stretch of it, so ragged
// lengths and few sequences load the GPU evenly alike.  Where a stretch ends
// inside a (sequence, head) item, both sides leave partial sums in the
// workspace, at most two per thread block whatever the lengths, and a second
// kernel, launched to overlap the first one's end, joins them.  Without a
// workspace every block takes one item whole.
//
// A warp takes every fourth tile of its block's stretch and streams the codes
// through a ring of its own in shared memory by 16-byte asynchronous copies
// (K and V alternate, NST half-tiles deep; no barrier but the warp's), across
// item boundaries, so the ring stays full.  Copies rather than tensor maps:
// a tile of 16-token blocks is two pieces, and a call needs no map.
//
// Measured at D = 128, 32 query heads on 8: 16 sequences of 32K tokens 169 us
// (6.35 TB/s) with two half-tiles a warp, 177 us with three, 184 us with four:
// 12 warps an SM ask for enough, more only queues.  64 ragged sequences of up
// to 4K 62 us (5.1 TB/s), of which about 8 us are start and join; 16 warps an
// SM (128 registers) took 70 us.
//
// Both products run as m16n8k16 MMAs on fp16 with fp32 sums, codes as A:
//   scores   M = 16 keys, K = 16 channels, N = 8 heads.  A lane's word of four
//            codes gives the fragments of one k-step by the channel order
//            (0, 2, 1, 3), which the query fragments share.
//   values   M = 16 channels, K = 16 keys: a transposing ldmatrix brings two
//            channels of two keys to a lane; byte permutes pair the keys.  The
//            weights turn from [key][head] to [head][key] by movmatrix.
// N = 8 wastes columns below 8 heads, but the tensor cores are idle otherwise.

#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kvq.h"
#include "kvq_paged_attn.cuh"

namespace {

using namespace kvqp;

__device__ unsigned int g_decode_fault = 0;

constexpr int kWarps = 4, kTile = 32, kHeads = 8;
constexpr int kMetaSlots = 8;                     // tiles whose scales are kept; more than a ring holds

template <int D>
struct Decode {
  static constexpr int HALF = kTile * D;          // bytes of one half-tile: 32 keys of K, or of V
  static constexpr int NST = D == 64 ? 4 : 2;     // half-tiles in flight a warp (see above)
  static constexpr int RING = kWarps * NST * HALF;
  static constexpr int XP = D == 256 ? 2 : 1;     // parts in which a block joins its warps' sums
  static constexpr int XCH = 2 * kHeads * D * 4 / XP;       // two warps' sums of a part
  static constexpr int META = kWarps * kMetaSlots * 32;
  static constexpr int ML = kWarps * kHeads * 8;
  static constexpr int SMEM = RING + XCH + META + ML + 128;
  static constexpr int NCH = D / 16;              // 16-channel steps
};

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
}
// With `bytes` 0 the 16 bytes become zeros and src is not read.
__device__ __forceinline__ void copy16_or_zeros(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a half-tile: the chunk index is
// mixed with the row so that eight rows of one chunk fall on all 32 banks.
template <int D>
__device__ __forceinline__ uint32_t place(int r, int c) {
  const int x = D == 64 ? (r >> 1) & 3 : r & 7;
  return static_cast<uint32_t>(r * D + ((c ^ x) << 4));
}

// Tiles of a sequence: positions lo .. L - 1 are seen, tile 0 starts at lo
// rounded down.
struct Span {
  int L, lo, first, tiles;
};
__device__ __forceinline__ Span span_of(const AttnArgs& a, int b, unsigned& bad) {
  Span s;
  s.L = sequence_length(a, b, bad);
  s.lo = a.window > 0 ? max(0, s.L - a.window) : 0;
  s.first = s.lo & ~(kTile - 1);
  s.tiles = (s.L - s.first + kTile - 1) / kTile;
  return s;
}

// One scan over the lengths, a run of sequences a thread: the tiles before this
// thread's run (b0 .. b1), and all tiles; likewise with every sequence's tiles
// rounded up to a whole number of warps' rounds.
struct Sums {
  int64_t tiles, rounded;
};
__device__ __forceinline__ int rounded(int tiles) { return (tiles + kWarps - 1) & ~(kWarps - 1); }
__device__ __forceinline__ Sums scan_tiles(const AttnArgs& a, int tid, int& b0, int& b1, Sums& total, int64_t* sums,
                                           unsigned& bad) {
  const int run = (a.c.B + kWarps * 32 - 1) / (kWarps * 32);
  b0 = min(a.c.B, tid * run);
  b1 = min(a.c.B, b0 + run);
  int64_t mine = 0, mine_r = 0;
  for (int b = b0; b < b1; ++b) {
    const int n = span_of(a, b, bad).tiles;
    mine += n;
    mine_r += rounded(n);
  }
  const int lane = tid & 31, w = tid >> 5;
  int64_t inc = mine, inc_r = mine_r;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(kAll, inc, o), y = __shfl_up_sync(kAll, inc_r, o);
    if (lane >= o) { inc += x; inc_r += y; }
  }
  if (lane == 31) { sums[w] = inc; sums[kWarps + w] = inc_r; }
  __syncthreads();
  Sums before = {inc - mine, inc_r - mine_r};
  total = {0, 0};
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    if (i < w) { before.tiles += sums[i]; before.rounded += sums[kWarps + i]; }
    total.tiles += sums[i];
    total.rounded += sums[kWarps + i];
  }
  return before;
}
// Tiles of one stretch: an equal share, but at least one for every warp.
__device__ __forceinline__ int64_t share_of(int64_t tiles, int blocks) {
  const int64_t n = (tiles + blocks - 1) / blocks;
  return n < kWarps ? kWarps : n;
}

// A piece: tiles ta .. tb - 1 of item `item` (KV head and group of query
// heads) of sequence b, the part of it inside the stretch.
struct Piece {
  Span s;
  int b, item, ta, tb;
  int64_t left;             // tiles of the stretch from ta on
};
__device__ __forceinline__ bool next_piece(const AttnArgs& a, Piece& p, int items, unsigned& bad) {
  p.left -= p.tb - p.ta;
  if (p.left <= 0) return false;
  if (p.tb == p.s.tiles) {
    p.ta = 0;
    if (++p.item == items) {
      p.item = 0;
      do {
        if (++p.b >= a.c.B) return false;
        p.s = span_of(a, p.b, bad);
      } while (p.s.tiles == 0);
    }
  } else {
    p.ta = p.tb;
  }
  p.tb = static_cast<int>(min(static_cast<int64_t>(p.s.tiles), p.ta + p.left));
  return true;
}

// The workspace: for each stretch two sets of partial sums, [head][D channels,
// reference, sum, 2 unused], and behind them all a record of the item that it
// begins and does not end: (sequence, item, which set, further stretches), the
// last 0 if there is none.
template <int D>
__device__ __forceinline__ float* part_at(const AttnArgs& a, int64_t stretch, int set) {
  return a.part + (2 * stretch + set) * kHeads * (D + 4);
}
template <int D>
__device__ __forceinline__ int4* head_at(const AttnArgs& a, int64_t stretch) {
  return reinterpret_cast<int4*>(a.part + 2 * static_cast<int64_t>(a.blocks) * kHeads * (D + 4)) + stretch;
}

// Sequences without tiles give zeros; the stretches share them out.
__device__ __forceinline__ void write_empty(const AttnArgs& a, unsigned& bad) {
  for (int b = blockIdx.x; b < a.c.B; b += gridDim.x) {
    if (span_of(a, b, bad).tiles > 0) continue;
    const int64_t n = static_cast<int64_t>(a.c.Hkv) * a.R * a.c.D / 8;
    uint4* o = reinterpret_cast<uint4*>(a.out + b * n * 8);
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) o[i] = make_uint4(0, 0, 0, 0);
  }
}

template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32, kDecodeBlocks<D>) paged_decode_kernel(AttnArgs a) {
  using C = Decode<D>;
  constexpr int NST = C::NST, NCH = C::NCH;
  extern __shared__ __align__(1024) uint8_t sm[];
  float4* xch = reinterpret_cast<float4*>(sm + C::RING);                       // [2][NCH / XP][32]
  float4* meta = reinterpret_cast<float4*>(sm + C::RING + C::XCH);             // [warp][slot]
  float2* ml = reinterpret_cast<float2*>(sm + C::RING + C::XCH + C::META);     // [warp][head]
  int64_t* sums = reinterpret_cast<int64_t*>(sm + C::RING + C::XCH + C::META + C::ML);   // [8], then the start
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, t = lane & 3;
  const int groups = (a.R + kHeads - 1) / kHeads, items = a.c.Hkv * groups;
  const int block = a.c.block;
  unsigned bad = 0;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the joining kernel may come up, and waits

  // ---- this block's stretch
  Piece p;
  int64_t share = 0;
  if (a.part != nullptr) {
    // With little to do a stretch is one round of the warps inside one item (the
    // line then counts every item as whole rounds); else an equal share.
    bool few;
    int64_t all, w0, off;
    auto lay_out = [&](const Sums& total) {
      few = total.rounded * items <= static_cast<int64_t>(gridDim.x) * kWarps;
      all = (few ? total.rounded : total.tiles) * items;
      share = few ? kWarps : share_of(all, gridDim.x);
      w0 = blockIdx.x * share;
      if (tid == 0) *head_at<D>(a, blockIdx.x) = make_int4(0, 0, 0, 0);
    };
    if (a.c.B <= 32) {                            // every warp scans for itself
      const int tiles = lane < a.c.B ? span_of(a, lane, bad).tiles : 0;
      Sums inc = {tiles, rounded(tiles)}, total;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(kAll, inc.tiles, o), y = __shfl_up_sync(kAll, inc.rounded, o);
        if (lane >= o) { inc.tiles += x; inc.rounded += y; }
      }
      total.tiles = __shfl_sync(kAll, inc.tiles, 31);
      total.rounded = __shfl_sync(kAll, inc.rounded, 31);
      lay_out(total);
      const int n = few ? rounded(tiles) : tiles;
      const int64_t end = (few ? inc.rounded : inc.tiles) * items, begin = end - static_cast<int64_t>(n) * items;
      const unsigned hit = __ballot_sync(kAll, begin <= w0 && w0 < end);
      p.b = hit ? __ffs(hit) - 1 : 0;
      off = w0 - __shfl_sync(kAll, begin, p.b);
    } else {
      int b0, b1;
      Sums total;
      const Sums before = scan_tiles(a, tid, b0, b1, total, sums, bad);
      lay_out(total);
      int64_t at = few ? before.rounded : before.tiles;
      for (int b = b0; b < b1; ++b) {
        const int tiles = span_of(a, b, bad).tiles, n = few ? rounded(tiles) : tiles;
        if (at * items <= w0 && w0 < (at + n) * items) {           // one thread finds it
          sums[2 * kWarps] = b;
          sums[2 * kWarps + 1] = w0 - at * items;
        }
        at += n;
      }
      __syncthreads();
      p.b = w0 < all ? static_cast<int>(sums[2 * kWarps]) : 0;
      off = sums[2 * kWarps + 1];
    }
    if (w0 >= all) {
      write_empty(a, bad);
      if (bad) atomicOr(&g_decode_fault, bad);
      return;
    }
    p.s = span_of(a, p.b, bad);
    const int n = few ? rounded(p.s.tiles) : p.s.tiles;
    p.item = static_cast<int>(off / n);
    p.ta = static_cast<int>(off % n);
    p.left = few ? min(kWarps, p.s.tiles - p.ta) : min(share, all - w0);
  } else {
    p.b = blockIdx.x / items;
    p.item = blockIdx.x % items;
    p.s = span_of(a, p.b, bad);
    p.ta = 0;
    p.left = p.s.tiles;
  }
  p.tb = static_cast<int>(min(static_cast<int64_t>(p.s.tiles), p.ta + p.left));

  // ---- the ring's loads
  const uint32_t ring = smem_u32(sm) + warp * NST * C::HALF;
  float4* my_meta = meta + warp * kMetaSlots * 2;
  Piece lp = p;                                   // the piece being loaded
  bool more = p.left > 0;                         // there is one
  int lt = p.ta + warp, at = 32;                  // next tile to load, its place among the 32 looked up
  int id0 = -1, id1 = -1;                         // lane i: the cache blocks of the i-th, per 16 keys
  float sk0 = 0.0f, sk1 = 0.0f, sv0 = 0.0f, sv1 = 0.0f, iv0 = 0.0f, iv1 = 0.0f;         // and S_K, log2 S_V, 1 / S_V
  bool fresh = false;                             // S_V as it was loaded
  int lslot = 0, ltiles = 0;
  bool vnext = false;
  int64_t src0 = -1, src1 = -1;                   // the tile's two 16-key parts: this lane's byte offset, or -1
  // The 16 keys of a part lie contiguous, 512 bytes of them a copy; a lane's
  // place in copy i is place<D> of row (i 512 + 16 lane) / D, whose chunk mix
  // differs from copy 0's by a constant of i.
  const uint32_t put = place<D>(lane * 16 / D, lane & (NCH - 1));
  auto mix = [](int i) -> uint32_t { return D == 64 ? 0u : D == 128 ? (i & 1) * 64u : (i & 3) * 32u; };
  int live = 0;                                   // keys from the tile's first to the sequence's end
  auto load_half = [&]() {                        // one half-tile into the ring's next place
    if (!vnext) {
      while (more && lt >= lp.tb) {
        more = next_piece(a, lp, items, bad);
        lt = lp.ta + warp;
        at = 32;
      }
      if (more) {
        const int kvh = lp.item / groups;
        if (at == 32) {                           // look up the warp's next 32 tiles of this piece
          at = 0;
          const int n = lt + kWarps * lane;
          id0 = id1 = -1;
          sk0 = sk1 = 0.0f;
          fresh = true;
          if (n < lp.tb) {
            const int key = lp.s.first + n * kTile, j = key >> a.c.log_block;
            // blocks that hold no visible position are not looked up
            if (key + 16 > lp.s.lo || block > 16) id0 = block_at(a.c, lp.b, j, bad);
            if (block > 16) id1 = id0;
            else if (key + 16 < lp.s.L) id1 = block_at(a.c, lp.b, j + 1, bad);
            if (id0 >= 0) {
              const int64_t x = static_cast<int64_t>(id0) * a.c.Hkv + kvh;
              sk0 = a.c.ks[x];
              sv0 = a.c.vs[x];
            }
            if (id1 >= 0) {
              const int64_t x = static_cast<int64_t>(id1) * a.c.Hkv + kvh;
              sk1 = a.c.ks[x];
              sv1 = a.c.vs[x];
            }
          }
        }
        const int cur0 = __shfl_sync(kAll, id0, at), cur1 = __shfl_sync(kAll, id1, at);
        live = lp.s.L - (lp.s.first + lt * kTile);
        const int slot0 = (lp.s.first + lt * kTile) & (block - 1), slot1 = (slot0 + 16) & (block - 1);
        src0 = cur0 < 0 ? -1 : static_cast<int64_t>((cur0 * a.c.Hkv + kvh) * block + slot0) * D + lane * 16;
        src1 = cur1 < 0 ? -1 : static_cast<int64_t>((cur1 * a.c.Hkv + kvh) * block + slot1) * D + lane * 16;
      } else {
        src0 = src1 = -1;
      }
    }
    const uint8_t* codes = vnext ? a.c.vc : a.c.kc;
    const uint32_t dst = ring + lslot * C::HALF;
    if (FMT == kInt8 || (more && live >= kTile && src0 >= 0 && src1 >= 0)) {
      if (src0 >= 0) {
#pragma unroll
        for (int i = 0; i < NCH / 2; ++i) copy16(dst + (put ^ mix(i)) + i * 512, codes + src0 + i * 512);
      }
      if (src1 >= 0) {
#pragma unroll
        for (int i = NCH / 2; i < NCH; ++i) copy16(dst + (put ^ mix(i)) + i * 512, codes + src1 + (i - NCH / 2) * 512);
      }
    } else if (more) {                            // e4m3: zeros where there is nothing to see
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        const int64_t src = i < NCH / 2 ? src0 + i * 512 : src1 + (i - NCH / 2) * 512;
        const bool there = (i < NCH / 2 ? src0 : src1) >= 0 && (i * 512 + lane * 16) / D < live;
        copy16_or_zeros(dst + (put ^ mix(i)) + i * 512, codes + (there ? src : 0), there ? 16 : 0);
      }
    }
    copies_commit();
    if (!vnext && more) {
      if (fresh) {                                // the scales' loads had the copies' issue to arrive in
        fresh = false;
        const float v0 = fmaxf(sv0, kScaleMin), v1 = fmaxf(sv1, kScaleMin);
        sk0 = fmaxf(sk0, kScaleMin);
        sk1 = fmaxf(sk1, kScaleMin);
        sv0 = id0 >= 0 ? log2f(v0) : -INFINITY;   // no block: weights 0
        sv1 = id1 >= 0 ? log2f(v1) : -INFINITY;
        iv0 = id0 >= 0 ? __frcp_rn(v0) : 0.0f;
        iv1 = id1 >= 0 ? __frcp_rn(v1) : 0.0f;
      }
      if (lane == at) {
        float4* m = my_meta + 2 * (ltiles & (kMetaSlots - 1));
        m[0] = make_float4(sk0, sk1, sv0, sv1);
        m[1] = make_float4(iv0, iv1, 0.0f, 0.0f);
      }
      ++ltiles;
      ++at;
      lt += kWarps;
    }
    vnext = !vnext;
    lslot = lslot + 1 == NST ? 0 : lslot + 1;
  };
#pragma unroll 1
  for (int i = 0; i < NST; ++i) load_half();

  int slot = 0, tiles_done = 0;
  const uint32_t row_at = place<D>(lane, 0);       // chunk c of this lane's row: row_at ^ (c << 4)
  bool any = p.left > 0;
  bool first_piece = true;
  while (any) {
    // ---- the query heads of this piece as B fragments: column g is head h0 + g
    const int kvh = p.item / groups, h0 = (p.item % groups) * kHeads;
    const int heads = min(kHeads, a.R - h0);
    uint32_t bq[NCH][2];
    float sc[2];                                  // heads 2t and 2t + 1: what scales their scores
    {
      const uint16_t* q = a.q + p.b * a.q_stride + static_cast<int64_t>(kvh * a.R + h0 + g) * D + 4 * t;
      uint2 raw[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) raw[c] = g < heads ? *reinterpret_cast<const uint2*>(q + 16 * c) : make_uint2(0, 0);
      float unit = a.scale;
      if (a.bf16) {
        float most = 0.0f;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const float2 x = unpack2<true>(raw[c].x), y = unpack2<true>(raw[c].y);
          most = fmaxf(most, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(y.x), fabsf(y.y))));
        }
        most = fmaxf(most, __shfl_xor_sync(kAll, most, 1));
        most = fmaxf(most, __shfl_xor_sync(kAll, most, 2));
        const int k = row_exponent(most);
        const float up = pow2i(k);
        unit *= pow2i(-k);
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const float2 x = unpack2<true>(raw[c].x), y = unpack2<true>(raw[c].y);
          raw[c].x = pack2<false>(x.x * up, x.y * up);
          raw[c].y = pack2<false>(y.x * up, y.y * up);
        }
      }
      const uint32_t sign = a.negative ? 0x80008000u : 0u;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        bq[c][0] = __byte_perm(raw[c].x, raw[c].y, 0x5410) ^ sign;    // channels 0, 2
        bq[c][1] = __byte_perm(raw[c].x, raw[c].y, 0x7632) ^ sign;    // channels 1, 3
      }
      sc[0] = __shfl_sync(kAll, unit, 8 * t);
      sc[1] = __shfl_sync(kAll, unit, 8 * t + 4);
    }
    float O[NCH][4];
#pragma unroll
    for (int i = 0; i < NCH; ++i) O[i][0] = O[i][1] = O[i][2] = O[i][3] = 0.0f;
    float M[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int n = p.ta + warp; n < p.tb; n += kWarps) {
      // ---- scores: z[mt] holds keys 16 mt + g (0, 1) and + 8 (2, 3) of heads 2t, 2t + 1
      copies_wait<NST - 1>();
      __syncwarp();
      float z[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
      const uint32_t kb = ring + slot * C::HALF + row_at;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        uint32_t w[4];
        ldsm4(w, kb ^ (c << 4));
        uint32_t e0, o0, e1, o1;
        codes_to_half2<FMT>(w[0], e0, o0);
        codes_to_half2<FMT>(w[1], e1, o1);
        mma(z[0], e0, e1, o0, o1, bq[c][0], bq[c][1]);
        codes_to_half2<FMT>(w[2], e0, o0);
        codes_to_half2<FMT>(w[3], e1, o1);
        mma(z[1], e0, e1, o0, o1, bq[c][0], bq[c][1]);
      }
      const float4 s = my_meta[2 * (tiles_done & (kMetaSlots - 1))];
      const float4 si = my_meta[2 * (tiles_done & (kMetaSlots - 1)) + 1];
      ++tiles_done;
      slot = slot + 1 == NST ? 0 : slot + 1;
      __syncwarp();
      load_half();

      // ---- weights
      const float sk[2] = {s.x, s.y}, off[2] = {s.z, s.w}, inv[2] = {si.x, si.y};
      float most[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) z[mt][e] = fmaf(z[mt][e], sc[e & 1] * sk[mt], off[mt]);
      }
      const int key = p.s.first + n * kTile + g;
      if (key - g < p.s.lo || key - g + kTile > p.s.L) {
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int k = key + 16 * mt + 8 * (e >> 1);
            if (k < p.s.lo || k >= p.s.L) z[mt][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) most[e & 1] = fmaxf(most[e & 1], z[mt][e]);
      if (__any_sync(kAll, most[0] > M[0] + kLazy || most[1] > M[1] + kLazy)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) most[j] = fmaxf(most[j], __shfl_xor_sync(kAll, most[j], o));
          const float now = fmaxf(M[j], most[j]);
          const float f = now == -INFINITY ? 1.0f : exp2_approx(M[j] - now);
          M[j] = now;
          l[j] *= f;
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            O[i][j] *= f;
            O[i][2 + j] *= f;
          }
        }
      }
      const float r0 = M[0] == -INFINITY ? 0.0f : kBoost - M[0], r1 = M[1] == -INFINITY ? 0.0f : kBoost - M[1];
      uint32_t pb[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        const float p0 = exp2_approx(z[mt][0] + r0), p1 = exp2_approx(z[mt][1] + r1);
        const float p2 = exp2_approx(z[mt][2] + r0), p3 = exp2_approx(z[mt][3] + r1);
        l[0] = fmaf(p0 + p2, inv[mt], l[0]);
        l[1] = fmaf(p1 + p3, inv[mt], l[1]);
        pb[mt][0] = transpose8(pack2<false>(p0, p1));
        pb[mt][1] = transpose8(pack2<false>(p2, p3));
      }

      // ---- values: O[i] holds channels 16 i + 2 g (0, 1) and + 1 (2, 3) of heads 2t, 2t + 1
      copies_wait<NST - 1>();
      __syncwarp();
      const uint32_t vb = ring + slot * C::HALF + row_at;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        uint32_t w[4];
        ldsm4t(w, vb ^ (i << 4));
        uint32_t e0, o0, e1, o1;
        codes_to_half2<FMT>(w[0], e0, o0);
        codes_to_half2<FMT>(w[1], e1, o1);
        mma(O[i], e0, o0, e1, o1, pb[0][0], pb[0][1]);
        codes_to_half2<FMT>(w[2], e0, o0);
        codes_to_half2<FMT>(w[3], e1, o1);
        mma(O[i], e0, o0, e1, o1, pb[1][0], pb[1][1]);
      }
      slot = slot + 1 == NST ? 0 : slot + 1;
      __syncwarp();
      load_half();
    }

    // ---- join the warps: a common reference, then pairwise sums
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[j] += __shfl_xor_sync(kAll, l[j], o);
    if (g == 0) {
      ml[warp * kHeads + 2 * t] = make_float2(M[0], l[0]);
      ml[warp * kHeads + 2 * t + 1] = make_float2(M[1], l[1]);
    }
    __syncthreads();
    float m_all[2], l_all[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      m_all[j] = -INFINITY;
      l_all[j] = 0.0f;
      float2 x[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        x[w] = ml[w * kHeads + 2 * t + j];
        m_all[j] = fmaxf(m_all[j], x[w].x);
      }
      const float ref = m_all[j] == -INFINITY ? 0.0f : m_all[j];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l_all[j] = fmaf(x[w].y, exp2_approx(x[w].x - ref), l_all[j]);
      const float f = exp2_approx(M[j] - ref);
      // sums that no key has reached are 0, and stay so
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        O[i][j] *= f;
        O[i][2 + j] *= f;
      }
    }
#pragma unroll
    for (int part = 0; part < C::XP; ++part) {
      constexpr int N = NCH / C::XP;
      if (warp >= 2) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float(&o)[4] = O[part * N + i];
          xch[((warp - 2) * N + i) * 32 + lane] = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncthreads();
      if (warp < 2) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float(&o)[4] = O[part * N + i];
          const float4 x = xch[(warp * N + i) * 32 + lane];
          o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
          if (warp == 1) xch[(N + i) * 32 + lane] = make_float4(o[0], o[1], o[2], o[3]);
        }
      }
      __syncthreads();
      if (warp == 0) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
          float(&o)[4] = O[part * N + i];
          const float4 x = xch[(N + i) * 32 + lane];
          o[0] += x.x; o[1] += x.y; o[2] += x.z; o[3] += x.w;
        }
      }
      if (part + 1 < C::XP) __syncthreads();
    }
    if (warp == 0) {
      const bool whole = p.ta == 0 && p.tb == p.s.tiles;
      // a stretch's first and last piece may be parts of an item; the one that
      // begins an item and does not end it says where its other parts are
      float* part = part_at<D>(a, blockIdx.x, first_piece ? 0 : 1);
      if (lane == 0 && p.ta == 0 && !whole)
        *head_at<D>(a, blockIdx.x) = make_int4(p.b, p.item, first_piece ? 0 : 1,
                                               static_cast<int>((p.s.tiles - p.left + share - 1) / share));
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int h = 2 * t + j;
        if (h >= heads) continue;
        if (whole) {
          // no key: 0; NaN stays
          const float inv = l_all[j] == 0.0f ? 0.0f : 1.0f / l_all[j];
          uint16_t* o = a.out + (static_cast<int64_t>(p.b) * a.c.Hkv * a.R + kvh * a.R + h0 + h) * D + 2 * g;
#pragma unroll
          for (int i = 0; i < NCH; ++i)
            *reinterpret_cast<uint32_t*>(o + 16 * i) =
                a.bf16 ? pack2<true>(O[i][j] * inv, O[i][2 + j] * inv) : pack2<false>(O[i][j] * inv, O[i][2 + j] * inv);
        } else {
          float* o = part + h * (D + 4);
#pragma unroll
          for (int i = 0; i < NCH; ++i) *reinterpret_cast<float2*>(o + 16 * i + 2 * g) = make_float2(O[i][j], O[i][2 + j]);
          if (g == 0) *reinterpret_cast<float2*>(o + D) = make_float2(m_all[j], l_all[j]);
        }
      }
    }
    __syncthreads();                              // ml and xch are free again
    first_piece = false;
    any = next_piece(a, p, items, bad);
  }
  copies_wait<0>();
  if (a.part != nullptr) write_empty(a, bad);
  if (a.part == nullptr && p.s.tiles == 0 && warp == 0) {          // an empty sequence's item
    const int kvh = p.item / groups, h0 = (p.item % groups) * kHeads, heads = min(kHeads, a.R - h0);
    uint16_t* o = a.out + (static_cast<int64_t>(p.b) * a.c.Hkv * a.R + kvh * a.R + h0) * D;
    for (int i = lane; i < heads * D / 8; i += 32) reinterpret_cast<uint4*>(o)[i] = make_uint4(0, 0, 0, 0);
  }
  if (bad) atomicOr(&g_decode_fault, bad);
}

// ---------------------------------------------------------------------------
// Join the parts of the items that several stretches covered: a block per
// stretch that begins one and per head.  The warps take every fourth part, the
// lanes the channels, and the warps' sums meet in shared memory.
// ---------------------------------------------------------------------------
template <int D, int FMT>
__global__ void __launch_bounds__(kWarps * 32) paged_decode_join_kernel(AttnArgs a) {
  constexpr int DPL = D / 32;
  __shared__ float sums[kWarps][D + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const int groups = (a.R + kHeads - 1) / kHeads;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 head = *head_at<D>(a, blockIdx.x);
  const int kvh = head.y / groups, h0 = (head.y % groups) * kHeads;
  if (head.w == 0 || h >= a.R - h0) return;
  const int parts = head.w + 1;
  float o[DPL], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < DPL; ++i) o[i] = 0.0f;
  auto at = [&](int c) -> const float* {
    return part_at<D>(a, static_cast<int64_t>(blockIdx.x) + c, c == 0 ? head.z : 0) + h * (D + 4);
  };
  for (int c = warp; c < parts; c += 8 * kWarps) {           // eight parts in flight
    float2 x[8];
    float y[8][DPL];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int part = c + k * kWarps;
      x[k] = make_float2(-INFINITY, 0.0f);
#pragma unroll
      for (int i = 0; i < DPL; ++i) y[k][i] = 0.0f;
      if (part < parts) {
        const float* p = at(part);
        x[k] = *reinterpret_cast<const float2*>(p + D);
#pragma unroll
        for (int i = 0; i < DPL; i += 2) {
          const float2 z = *reinterpret_cast<const float2*>(p + lane * DPL + i);
          y[k][i] = z.x;
          y[k][i + 1] = z.y;
        }
      }
    }
    float now = m;
#pragma unroll
    for (int k = 0; k < 8; ++k) now = fmaxf(now, x[k].x);
    const float ref = now == -INFINITY ? 0.0f : now;
    const float e = exp2_approx(m - ref);
    l *= e;
#pragma unroll
    for (int i = 0; i < DPL; ++i) o[i] *= e;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float w = exp2_approx(x[k].x - ref);
      l = fmaf(x[k].y, w, l);
#pragma unroll
      for (int i = 0; i < DPL; ++i) o[i] = fmaf(y[k][i], w, o[i]);
    }
    m = now;
  }
#pragma unroll
  for (int i = 0; i < DPL; ++i) sums[warp][lane * DPL + i] = o[i];
  if (lane == 0) {
    sums[warp][D] = m;
    sums[warp][D + 1] = l;
  }
  __syncthreads();
  float most = -INFINITY, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) most = fmaxf(most, sums[w][D]);
  const float ref = most == -INFINITY ? 0.0f : most;
  l = 0.0f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = exp2_approx(sums[w][D] - ref);
    l = fmaf(sums[w][D + 1], f[w], l);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = a.out + (static_cast<int64_t>(head.x) * a.c.Hkv * a.R + kvh * a.R + h0 + h) * D;
  for (int i = 2 * threadIdx.x; i < D; i += 2 * kWarps * 32) {
    float u = 0.0f, v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      u = fmaf(sums[w][i], f[w], u);
      v = fmaf(sums[w][i + 1], f[w], v);
    }
    *reinterpret_cast<uint32_t*>(out + i) = a.bf16 ? pack2<true>(u * inv, v * inv) : pack2<false>(u * inv, v * inv);
  }
}

template <int D, int FMT>
cudaError_t launch(const AttnArgs& a, int grid, cudaStream_t st) {
  using C = Decode<D>;
  auto k = paged_decode_kernel<D, FMT>;
  static std::atomic<int> ready[64];              // the shared-memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || ready[dev].load(std::memory_order_relaxed) == 0) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev].store(1, std::memory_order_relaxed);
  }
  const int items = a.c.Hkv * ((a.R + kHeads - 1) / kHeads);
  const int64_t all = static_cast<int64_t>(a.c.B) * items;
  if (a.part == nullptr) {
    k<<<static_cast<unsigned>(all), kWarps * 32, C::SMEM, st>>>(a);
    return cudaGetLastError();
  }
  k<<<grid, kWarps * 32, C::SMEM, st>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), static_cast<unsigned>(a.R < kHeads ? a.R : kHeads));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_decode_join_kernel<D, FMT>, a);
}

}  // namespace

__attribute__((visibility("hidden"))) int kvq_paged_decode_launch(const AttnArgs& a, int format, int grid,
                                                                  cudaStream_t st, cudaError_t& err) {
  const bool f8 = format == KVQ_E4M3;
  switch (a.c.D) {
    case 64: err = f8 ? launch<64, kE4m3>(a, grid, st) : launch<64, kInt8>(a, grid, st); break;
    case 128: err = f8 ? launch<128, kE4m3>(a, grid, st) : launch<128, kInt8>(a, grid, st); break;
    default: err = f8 ? launch<256, kE4m3>(a, grid, st) : launch<256, kInt8>(a, grid, st); break;
  }
  return err == cudaSuccess ? KVQ_OK : KVQ_ERR_LAUNCH;
}

__attribute__((visibility("hidden"))) unsigned int kvq_paged_decode_fault_word(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_decode_fault, sizeof(v)) != cudaSuccess) return 0;
  if (clear && v) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_decode_fault, &zero, sizeof(zero));
  }
  return v;
}
