// kvq_paged_prefill.cu -- causal attention of any number of new tokens per
// sequence over the paged 8-bit cache (include/kvq.h,
// kvq_paged_attention_prefill); the softmax's form is in kvq_paged_attn.cuh.
//
// Bound: tensor-core rate for long chunks (4 D flops a visible pair and query
// head), the codes' bytes for a few queries over a long cache.
//
// Work.  The query heads of a KV head share its keys, so the rows of a tile
// are (token, head) pairs of one KV head, R rows a token, packed across token
// boundaries: 2 x 128 rows a thread block (128 at D = 256).  Up to 128 rows
// share their key tiles out over both sets of warps instead.  Where the tiles do
// not fill the GPU the keys of a tile are split over several thread blocks,
// whose partial sums a second kernel joins.
//
// A thread block is 18 warps in roles, coupled by mbarriers (and two that rest):
//   0-7    softmax: a thread per row reads its scores from tensor memory,
//          makes the weights and writes them back as fp16 (warps 0-3 the first
//          128 rows, 4-7 the second; at D = 256 only 0-3);
//   8-11   K: codes from the cache to fp16 in shared memory, 128-byte swizzled;
//   12-15  V: the same;
//   16, 17 a thread each issues the MMAs of its 128 rows (tcgen05, fp16 with
//          fp32 sums in tensor memory): S = Q K^T from shared memory, O += P V
//          with P from tensor memory, 64 keys a step.  Each 128 rows have two
//          score buffers: the scores two steps on are asked for as soon as a
//          step's weights are there, while the softmax has the next step's.
// Codes are exact in fp16, so K and V are converted once per thread block and
// tile; their scales are in the softmax's exponent.  Code pairs unpack as
// channels (0, 2), (1, 3): Q's channels are laid out in that order too, and the
// outputs' are put back in the last step.
// The reference of a row's softmax moves rarely (kLazy), and only then is O
// rescaled in tensor memory, by the thread that owns the row.
//
// Measured at D = 128, 32 query heads on 8: a prompt of 8192 tokens 0.60 ms a call (911
// TFLOP/s; 586 us on the device), of 16384 (16 on 4) 1.10-1.13 ms (974-996); 8 x 32 tokens
// behind 8192 74-76 us.  8192 tokens at D = 64: 550 us (500 TFLOP/s), at D = 256 (16 on 4)
// 650 us (845).  A key tile (D = 128) takes 4,150 cycles: 2,048 of the
// exponential unit, about 2,500 of the tensor cores, the rest latencies.  With
// one score buffer of 128 keys for each 128 rows (larger MMAs, but the softmax
// waits for them) it was 0.72 ms, with sixteen softmax warps 0.64 ms.

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <type_traits>

#include "kvq.h"
#include "kvq_paged_attn.cuh"

namespace {

using namespace kvqp;

#include "kvq_async.cuh"

__device__ unsigned int g_prefill_fault = 0;

constexpr uint32_t kSpin = 1u << 22;              // bounded mbarrier waits
constexpr int kStep = 64;                         // keys of one softmax step
constexpr int kThreads = 640;                    // five warpgroups
constexpr int kFirstK = 8, kFirstV = 12, kIssuer = 16;     // warps
// Registers a thread by role.  Together they must not exceed what the block is
// launched with: 256 x 128 + 256 x 80 + 128 x 64 = 61,440 of 640 x 96.
constexpr int kSoftmaxRegs = 128, kConvertRegs = 80, kIssuerRegs = 64;
constexpr int kRegsNeeded = 256 * kSoftmaxRegs + 256 * kConvertRegs + 128 * kIssuerRegs;

template <int D>
struct Prefill {
  static constexpr int MT = D == 256 ? 1 : 2;     // 128-row tiles
  static constexpr int KT = D == 256 ? 64 : 128;  // keys of a tile in shared memory
  static constexpr int STEPS = KT / kStep;        // steps of a tile
  static constexpr int ROWS = MT * 128, LOG_ROWS = MT == 2 ? 8 : 7;
  static constexpr int CB = D / 64;               // 64-channel blocks (128-byte swizzled rows)
  static constexpr int NSUB = KT / 16;            // 16-key parts, each inside one cache block
  static constexpr int QBYTES = ROWS * D * 2;
  static constexpr int TILE = KT * D * 2;         // fp16 bytes of a K or V tile
  static constexpr int STAGES = 2;
  static constexpr int PART = ROWS * (D + 2);     // floats of a tile's partial sums, references and sums of weights
  static constexpr int META = 4 * NSUB * 16;      // scales of four tiles
  static constexpr int NBAR = 4 * STAGES + 4 + 3 * 4 + 1;
  static constexpr int SMEM = 1024 + QBYTES + 2 * STAGES * TILE + META + ROWS * 4 + 128 * 8 + NBAR * 8 + 8 + 80;
  // tensor memory columns: two score buffers (the weights over them) for each
  // 128 rows, then the outputs
  static constexpr int O0 = MT * 2 * kStep;
  static constexpr uint32_t COLS = 512;
};

// ---- tcgen05 ------------------------------------------------------------------------

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of this thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]),
         "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]),
         "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(addr)
      : "memory");
}

// And 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};"
      :: "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
         "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
      : "memory");
}

// Shared-memory matrix descriptor with the 128-byte swizzle: start address,
// leading and stride byte offsets in units of 16, descriptor version 1.
__device__ __forceinline__ uint64_t matrix_desc(uint32_t addr, uint32_t leading, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(leading >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (uint64_t{1} << 46) | (uint64_t{2} << 61);
}
// Instruction descriptor: fp16 operands, fp32 sums, M = 128.
template <int N, bool B_TRANSPOSED>
constexpr uint32_t kMmaDesc = (1u << 4) | (B_TRANSPOSED ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
                              ((128u >> 4) << 24);
// The whole warp comes here and one thread (`one`) issues: what the warp holds
// in common stays in uniform registers.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t one;
  asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(one));
  return one;
}
__device__ __forceinline__ void mma_ss(uint32_t one, uint32_t d, uint64_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               :: "r"(d), "l"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(add)), "r"(one) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t one, uint32_t d, uint32_t a, uint64_t b, uint32_t desc, bool add) {
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.b32 p, %4, 0;\nsetp.ne.b32 q, %5, 0;\n"
               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               :: "r"(d), "r"(a), "l"(b), "r"(desc), "r"(static_cast<uint32_t>(add)), "r"(one) : "memory");
}
// The barrier completes when the issuing thread's MMAs so far have.
__device__ __forceinline__ void mma_commit(uint32_t one, uint64_t* bar) {
  asm volatile("{\n.reg .pred q;\nsetp.ne.b32 q, %1, 0;\n"
               "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}"
               :: "r"(smem_addr(bar)), "r"(one) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// What a thread block works on: rows row0 .. row0 + count - 1 of the sequence's
// n R (token, head) pairs, against the key tiles first + KT i, i < tiles.
struct Job {
  int b, kvh, n, L;
  int row0, count, q0;        // q0: the sequence's first row in the packed queries
  int lo, hi;                 // keys that some row sees
  int first, tiles, steps;    // first key of the first tile; tiles and steps of this split
  int split, nsplit;
  int64_t part;               // a piece's number, for its partial sums
  bool there;                 // there is work for this thread block
};

// The keys lo .. hi - 1 that rows row0 .. row0 + count - 1 of a sequence see,
// the first key of their first tile and the number of tiles.
struct Span {
  int lo, hi, first, tiles;
};
template <int D>
__device__ __forceinline__ Span span_of(const AttnArgs& a, int L, int n, int row0, int count) {
  using C = Prefill<D>;
  const int p0 = L - n + row0 / a.R, p1 = L - n + (row0 + count - 1) / a.R;
  Span x;
  x.lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
  x.hi = max(0, p1 + 1);
  x.first = x.lo / C::KT * C::KT;
  x.tiles = x.hi > x.lo ? (x.hi - x.first + C::KT - 1) / C::KT : 0;
  return x;
}

// The splits of a call from its lengths (up to 32 sequences, one a lane).  Where
// all tiles fit the GPU at once, every tile of a sequence is split alike, into
// pieces of about as many key tiles as the shortest that still let all pieces
// start at once.  Where they do not, full rounds are left whole and what is left
// over is split to fill one more.  Tiles are numbered sequence by sequence, last
// tiles first, and pieces in the order of their tiles.
struct Plan {
  int c0, n, L;                                   // a lane's sequence: first row of q, tokens, length
  int tiles, ns;                                  // its row tiles, the pieces of each
  int pieces, before, tiles_before;               // all its pieces; those, and the tiles, of the sequences before it
  int whole, rest, rest_ns;                       // tiles before any split one (0: the lanes' ns hold), tiles after them,
};                                                // the pieces of each
__device__ __forceinline__ int sum_before(int x, int lane) {
  int y = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int z = __shfl_up_sync(kAll, y, o);
    if (lane >= o) y += z;
  }
  return y - x;
}
// The lane whose `mine` numbers from `before` on hold x, or -1.
__device__ __forceinline__ int lane_of(int x, int before, int mine) {
  return __ffs(__ballot_sync(kAll, x >= before && x - before < mine)) - 1;
}
constexpr int kPlanned = -1;                      // instead of the number of unsplit tiles; the splits are then the
                                                  // thread blocks that run at once

template <int D>
__device__ __forceinline__ Plan make_plan(const AttnArgs& a, int places, int lane, unsigned& bad) {
  using C = Prefill<D>;
  Plan p;
  const bool mine = lane < a.c.B;
  const int c0 = mine ? a.cu[lane] : 0, c1 = mine ? a.cu[lane + 1] : 0, len = mine ? a.seq_len[lane] : 0;
  const bool wrong = c0 < 0 || c1 < c0 || c1 > a.total_q;
  if (wrong) bad |= kFaultLength;
  p.c0 = c0;
  p.n = wrong ? 0 : c1 - c0;
  p.L = p.n > 0 ? clamped_length(a, len, bad) : 0;
  const int rows = p.n * a.R;                     // total_q R is an int
  p.tiles = ((rows + C::ROWS - 1) >> C::LOG_ROWS) * a.c.Hkv;
  // the key tiles of its longest row tile, at most (a window's may begin and end inside one)
  int keys = rows > 0 ? (p.L + C::KT - 1) / C::KT : 0;
  if (a.window > 0) keys = min(static_cast<int64_t>(keys), (a.window + int64_t{C::ROWS} / a.R) / C::KT + 2);
  p.tiles_before = sum_before(p.tiles, lane);
  const int most = __reduce_max_sync(kAll, keys), total = __reduce_add_sync(kAll, p.tiles);
  p.whole = p.rest = 0;
  p.rest_ns = p.ns = 1;
  p.pieces = p.tiles;
  p.before = p.tiles_before;
  if (total > places) {
    p.rest = total % places;
    p.whole = total - p.rest;
    if (p.rest > 0) p.rest_ns = max(1, min(places / p.rest, most / 2));
    return p;
  }
  const float all = static_cast<float>(total);
  float work = static_cast<float>(p.tiles) * static_cast<float>(keys);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) work += __shfl_xor_sync(kAll, work, o);
  auto pieces_of = [&](int per) { return max(1, (keys + per - 1) / per); };
  // bisection between the average load and what surely fits: pieces are at most
  // work / per + tiles
  int lo = max(2, static_cast<int>(work / static_cast<float>(places))), hi = most;
  if (all < static_cast<float>(places))
    hi = static_cast<int>(fminf(static_cast<float>(hi), work / (static_cast<float>(places) - all) + 1.0f));
  lo = min(lo, hi);
#pragma unroll 1
  while (lo < hi) {
    const int per = lo + (hi - lo) / 2;
    const int64_t mine_all = static_cast<int64_t>(p.tiles) * pieces_of(per);
    const int sum = __reduce_add_sync(kAll, static_cast<int>(min(mine_all, int64_t{1} << 20)));
    if (sum <= places) hi = per;
    else lo = per + 1;
  }
  if (most <= hi + 2) return p;                   // what joining costs
  const int ns = pieces_of(max(hi, 1));
  if (__reduce_add_sync(kAll, static_cast<int>(min(static_cast<int64_t>(p.tiles) * ns, int64_t{1} << 20))) > places)
    return p;
  p.ns = ns;
  p.pieces = p.tiles * ns;
  p.before = sum_before(p.pieces, lane);
  return p;
}

static_assert(sizeof(Job) <= 80, "its place in shared memory");

template <int D>
__device__ __forceinline__ bool find_job(const AttnArgs& a, int whole, int nsplit, Job& j, unsigned& bad) {
  using C = Prefill<D>;
  unsigned x = blockIdx.x;
  int k;
  if (whole == kPlanned) {
    const int lane = threadIdx.x & 31;
    const Plan p = make_plan<D>(a, nsplit, lane, bad);
    bad = __reduce_or_sync(kAll, bad);
    const int at = static_cast<int>(x);
    int z;                                        // the tile's number in its sequence
    if (p.whole > 0) {
      const int y = max(at - p.whole, 0), t = y / p.rest_ns;
      j.nsplit = at < p.whole ? 1 : p.rest_ns;
      j.split = y - t * p.rest_ns;
      z = min(at, p.whole) + t;
      j.part = y;
      if (t > 0 && t >= p.rest) return false;
    } else {
      z = at;
      j.part = at;
    }
    const int b = p.whole > 0 ? lane_of(z, p.tiles_before, p.tiles) : lane_of(at, p.before, p.pieces);
    if (b < 0) return false;
    if (p.whole > 0) {
      z -= __shfl_sync(kAll, p.tiles_before, b);
    } else {
      const int y = at - __shfl_sync(kAll, p.before, b);
      j.nsplit = __shfl_sync(kAll, p.ns, b);
      z = y / j.nsplit;
      j.split = y - z * j.nsplit;
    }
    j.b = b;
    j.q0 = __shfl_sync(kAll, p.c0, b);
    j.n = __shfl_sync(kAll, p.n, b);
    j.L = __shfl_sync(kAll, p.L, b);
    j.kvh = z % a.c.Hkv;
    k = __shfl_sync(kAll, p.tiles, b) / a.c.Hkv - 1 - z / a.c.Hkv;
  } else {
    j.split = 0;
    j.nsplit = 1;
    j.part = 0;
    if (x >= static_cast<unsigned>(whole)) {
      x -= static_cast<unsigned>(whole);
      j.part = x;
      j.nsplit = nsplit;
      j.split = static_cast<int>(x % static_cast<unsigned>(nsplit));
      x = x / static_cast<unsigned>(nsplit) + static_cast<unsigned>(whole);
    }
    j.kvh = static_cast<int>(x % static_cast<unsigned>(a.c.Hkv));
    // the last tiles of a sequence see most keys: they start first
    const int64_t items = (a.total_q * a.R >> C::LOG_ROWS) + a.c.B;
    const int64_t item = items - 1 - x / static_cast<unsigned>(a.c.Hkv);
    const Found f = find_sequence(a.cu, a.seq_len, a.c.B, item, a.R, C::LOG_ROWS, 1, threadIdx.x & 31);
    j.b = f.b;
    const int64_t c0 = f.c0, c1 = f.c1;
    if (c0 < 0 || c1 < c0 || c1 > a.total_q) {
      bad |= kFaultLength;
      return false;
    }
    j.n = static_cast<int>(c1 - c0);
    j.q0 = static_cast<int>(c0);
    if (f.item < 0 || f.item * C::ROWS >= (c1 - c0) * a.R) return false;
    k = static_cast<int>(f.item);
    j.L = clamped_length(a, f.more, bad);
  }
  j.row0 = k * C::ROWS;
  j.count = min(C::ROWS, j.n * a.R - j.row0);
  const Span s = span_of<D>(a, j.L, j.n, j.row0, j.count);
  j.lo = s.lo;
  j.hi = s.hi;
  const int each = s.tiles / j.nsplit, more = s.tiles - each * j.nsplit;      // the first pieces have one more
  j.first = s.first + (each * j.split + min(j.split, more)) * C::KT;
  j.tiles = each + (j.split < more ? 1 : 0);
  j.steps = j.tiles > 0 ? min(j.tiles * C::STEPS, (j.hi - j.first + kStep - 1) / kStep) : 0;
  return true;
}

// The rows in the cache of a tile's 16-key parts: lane i < NSUB gets part i's
// first row ((block id, head, slot) as one number), or -1.
template <int D>
__device__ __forceinline__ int part_row(const AttnArgs& a, const Job& j, int key0, int lane, unsigned& bad) {
  using C = Prefill<D>;
  const int key = key0 + 16 * lane;
  if (lane >= C::NSUB || key + 16 <= j.lo || key >= j.hi) return -1;
  const int id = block_at(a.c, j.b, key >> a.c.log_block, bad);
  return id < 0 ? -1 : (id * a.c.Hkv + j.kvh) * a.c.block + (key & (a.c.block - 1));
}

// One of four warps' share of a tile's codes: chunks of 512 codes (32 lanes of
// 16), chunk 4 i + which for i < N; parts that are not there become zeros.  (With
// loads of 8 codes a lane, asking for a tile took a converter's 1,100 cycles.)
template <int D>
struct Share {
  using C = Prefill<D>;
  static constexpr int N = C::KT * D / 2048;
  static constexpr int PERPART = D / 32;          // chunks of a 16-key part
  uint4 w[N];
  // (e4m3: keys from `live` on, behind the sequence's last, as zeros)
  template <int FMT>
  __device__ __forceinline__ void load(const uint8_t* codes, int rows, int live, int which, int lane) {
    const uint8_t* mine = codes + which % PERPART * 512 + lane * 16;
    const uint8_t* p = nullptr;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (4 * i % PERPART == 0) {                 // a part's first chunk for this warp
        const int row = __shfl_sync(kAll, rows, 4 * i / PERPART + which / PERPART);
        p = row < 0 ? nullptr : mine + static_cast<int64_t>(row) * D;
      }
      const bool there = p != nullptr && (FMT == kInt8 || ((4 * i + which) * 32 + lane) / (D / 16) < live);
      w[i] = there ? __ldg(reinterpret_cast<const uint4*>(p + 4 * i % PERPART * 512)) : make_uint4(0, 0, 0, 0);
    }
  }
  // To the tile at dst: row r, 8-channel unit c at unit (c mod 8) ^ (r mod 8) of
  // row r of block c / 8.  A lane has units c and c + 1, c even, and r mod 8 is the
  // same for all its chunks.  Eight lanes store at once, which have all even units of
  // one row's two blocks (D > 64): those of odd blocks begin with unit c + 1.
  template <int FMT>
  __device__ __forceinline__ void store(uint32_t dst, int which, int lane) const {
    const int x = which * 32 + lane, r = x / (D / 16), c = x % (D / 16) * 2;
    const bool odd = D > 64 && (c >> 3 & 1);
    const uint32_t at = dst + (c >> 3) * (C::KT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4) ^ (odd ? 16u : 0u);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t to = at + i * (2048 / D * 128);
      const uint32_t v[4] = {odd ? w[i].z : w[i].x, odd ? w[i].w : w[i].y, odd ? w[i].x : w[i].z, odd ? w[i].y : w[i].w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t h[4];
        codes_to_half2<FMT>(v[2 * k], h[0], h[1]);
        codes_to_half2<FMT>(v[2 * k + 1], h[2], h[3]);
        asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};"
                     :: "r"(k == 0 ? to : to ^ 16u), "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]) : "memory");
      }
    }
  }
};

template <int D, int FMT>
__global__ void __launch_bounds__(kThreads, 1) paged_prefill_kernel(AttnArgs a, int whole, int nsplit) {
  using C = Prefill<D>;
  constexpr int KT = C::KT, NSUB = C::NSUB, ST = C::STAGES;
  extern __shared__ uint8_t raw_sm[];
  uint8_t* sm = align_smem_1k(raw_sm);
  uint8_t* qs = sm;                               // [MT][CB][128 rows][128 B]
  uint8_t* kbuf = qs + C::QBYTES;                 // [stage][CB][KT rows][128 B]
  uint8_t* vbuf = kbuf + ST * C::TILE;
  float4* meta = reinterpret_cast<float4*>(vbuf + ST * C::TILE);               // [4][NSUB]: S_K, log2 S_V, 1 / S_V
  float* unit = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(meta) + C::META);
  float2* second = reinterpret_cast<float2*>(unit + C::ROWS);                  // [128]: the second set's references, sums
  uint64_t* bars = reinterpret_cast<uint64_t*>(second + 128);
  uint64_t *k_full = bars, *k_empty = bars + ST, *v_full = bars + 2 * ST, *v_empty = bars + 3 * ST;
  uint64_t *meta_full = bars + 4 * ST, *s_full = meta_full + 4, *p_full = s_full + 4, *o_full = p_full + 4;
  uint64_t* joined = o_full + 4;
  uint32_t* shared_word = reinterpret_cast<uint32_t*>(bars + C::NBAR);         // the tensor memory's address
  Job* job = reinterpret_cast<Job*>(shared_word + 2);

  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kAll, tid >> 5, 0);
  // the joining kernel's thread blocks may take their places as soon as all of
  // these have theirs; they wait for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  unsigned bad = 0;
  if (warp == 0) {                                // one warp finds the work for all
    Job found;
    const bool there = find_job<D>(a, whole, nsplit, found, bad);
    if (lane == 0) {
      found.there = there;
      *job = found;
    }
    if (!there && bad && lane == 0) atomicOr(&g_prefill_fault, bad);
  }
  __syncthreads();
  if (!job->there) return;
  const Job j = *job;

  if (warp == kIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 :: "r"(smem_addr(shared_word)), "n"(C::COLS) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  // Up to 128 rows: the second set of softmax warps takes the odd key tiles of
  // the same rows, and the two sets' sums are joined in the end.  (Place 1 of the
  // tiles in shared memory is then the second set's alone.)
  const int sets = C::MT == 2 && j.count > 128 ? 2 : 1;
  const bool dual = C::MT == 2 && sets == 1;
  // a set's steps: how many, and the tile of the i-th
  auto steps_of = [&](int mt) {
    if (!dual) return j.steps;
    return j.tiles > mt ? (j.tiles - mt + 1) / 2 * 2 - (((j.tiles - 1) & 1) == mt ? j.steps & 1 : 0) : 0;
  };
  auto tile_of = [&](int i, int mt) { return C::STEPS == 1 ? i : dual ? mt + (i & ~1) : i >> 1; };
  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&k_full[i], 4); mbar_init(&v_full[i], 4);
      mbar_init(&k_empty[i], sets); mbar_init(&v_empty[i], sets);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&meta_full[i], 1);
    // per 128 rows, steps alternate between two of each: a wait is then never two
    // phases behind, which a parity could not tell from none
    for (int i = 0; i < 4; ++i) { mbar_init(&s_full[i], 1); mbar_init(&p_full[i], 4); mbar_init(&o_full[i], 1); }
    mbar_init(joined, 4);
    mbar_fence_init();
  }

  // The converters' first tile: its loads go out before the queries'.
  const bool is_v = warp >= kFirstV;
  const uint8_t* codes = is_v ? a.c.vc : a.c.kc;
  const int which = warp & 3;
  Share<D> next;
  int rows = -1;                                  // the parts of the tile in `next`
  if (warp >= kFirstK && warp < kIssuer && j.tiles > 0) {
    rows = part_row<D>(a, j, j.first, lane, bad);
    next.template load<FMT>(codes, rows, j.L - j.first, which, lane);
  }

  // ---- the query rows, fp16 with a power of two each, channels in code order:
  // a lane has 8 channels, a row D / 8 lanes, and all loads of a warp are in
  // flight before the first is used.  (Rows of a softmax warp that has none are
  // left as they are.)
  {
    constexpr int LANES = D / 8, AT_ONCE = 32 / LANES, W = kThreads / 32 * AT_ONCE, N = (C::ROWS + W - 1) / W;
    const int c = lane % LANES, need = min(C::ROWS, (j.count + 31) & ~31);
    const int tok0 = j.row0 / a.R, head0 = j.row0 - tok0 * a.R;
    const float per = __frcp_rn(static_cast<float>(a.R));
    uint4 w[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int r = n * W + warp * AT_ONCE + lane / LANES;
      // token and head of row r: the quotient is at most one off
      int x = head0 + r, tok = static_cast<int>(static_cast<float>(x) * per);
      x -= tok * a.R;
      if (x < 0) x += a.R, --tok;
      if (x >= a.R) x -= a.R, ++tok;
      const uint16_t* q = a.q + (j.q0 + static_cast<int64_t>(tok0 + tok)) * a.q_stride +
                          static_cast<int64_t>(j.kvh * a.R + x) * D + c * 8;
      w[n] = r < j.count ? __ldg(reinterpret_cast<const uint4*>(q)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      if (n * W + warp * AT_ONCE >= need) break;
      const int r = n * W + warp * AT_ONCE + lane / LANES;
      float u = a.scale;
      uint32_t h[4] = {w[n].x, w[n].y, w[n].z, w[n].w}, sign = a.negative ? 0x80008000u : 0u;
      if (a.bf16) {
        // bf16 magnitudes are ordered as their bits are
        uint32_t most = __vmaxu2(__vmaxu2(h[0] & 0x7fff7fffu, h[1] & 0x7fff7fffu),
                                 __vmaxu2(h[2] & 0x7fff7fffu, h[3] & 0x7fff7fffu));
        if constexpr (LANES == 32) {
          most = __reduce_max_sync(kAll, max(most & 0xffffu, most >> 16));
        } else {
#pragma unroll
          for (int o = LANES / 2; o > 0; o >>= 1) most = __vmaxu2(most, __shfl_xor_sync(kAll, most, o));
          most = max(most & 0xffffu, most >> 16);
        }
        const int k = row_exponent(__uint_as_float(most << 16));
        const float up = a.negative ? -pow2i(k) : pow2i(k);
        sign = 0;
        u *= pow2i(-k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2<true>(h[i]);
          h[i] = pack2<false>(x.x * up, x.y * up);
        }
      }
      const int rr = r & 127;
      *reinterpret_cast<uint4*>(qs + ((r >> 7) * C::CB + (c >> 3)) * 16384 + rr * 128 + (((c & 7) ^ (rr & 7)) << 4)) =
          make_uint4(__byte_perm(h[0], h[1], 0x5410) ^ sign, __byte_perm(h[0], h[1], 0x7632) ^ sign,
                     __byte_perm(h[2], h[3], 0x5410) ^ sign, __byte_perm(h[2], h[3], 0x7632) ^ sign);
      if (c == 0) unit[r] = u;
    }
  }
  fence_proxy_async();
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = __shfl_sync(kAll, *shared_word, 0);
  bool ok = true;                                 // this role has met no timeout
  auto wait = [&](uint64_t* bar, uint32_t parity) {         // a whole warp, of one mind
    if (ok) ok = __all_sync(kAll, mbar_wait(bar, parity, kSpin));
    return ok;
  };

  if (warp < 8) {
    // ---- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kSoftmaxRegs));
    const int mt = warp >> 2, own = (warp & 3) * 32 + lane;
    if (mt < C::MT) {
      const int r = (dual ? 0 : mt * 128) + own, steps = steps_of(mt);
      const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
      const uint32_t o_at = lanes + C::O0 + mt * D;
      const bool live = r < j.count;
      const int row = j.row0 + r;
      // this row sees the keys low .. pos (a row that is not there: all of them, and
      // its weights are nobody's)
      const int pos = live ? j.L - j.n + row / a.R : INT32_MAX;
      const int low = a.window > 0 && live ? pos - a.window + 1 : 0;
      const bool rest = !__any_sync(kAll, live);            // no row of this warp is there
      const float u = unit[r];
      // over the warp: tiles inside [wlow, wpos] need no mask
      int wpos = pos, wlow = low;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        wpos = min(wpos, __shfl_xor_sync(kAll, wpos, o));
        wlow = max(wlow, __shfl_xor_sync(kAll, wlow, o));
      }
      float M = -INFINITY, l = 0.0f;
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        const int buf = mt * 2 + (i & 1), tile = tile_of(i, mt);
        const uint32_t s_at = lanes + buf * kStep;
        // (the scales come first)
        if (!wait(&meta_full[tile & 3], (tile >> 2) & 1) || !wait(&s_full[buf], (i >> 1) & 1)) break;
        tmem_fence_after();
        if (rest) {
          if (lane == 0) mbar_arrive(&p_full[buf]);
          continue;
        }
        const float4* sc = meta + (tile & 3) * NSUB + (C::STEPS == 2 ? (i & 1) * 4 : 0);
        const int key0 = j.first + tile * KT + (C::STEPS == 2 ? (i & 1) * kStep : 0);
        auto step = [&](auto edge) -> bool {
          uint32_t s[2][32], w[kStep / 2];
          tmem_ld32(s[0], s_at);
          tmem_ld32(s[1], s_at + 32);
          tmem_wait_ld();
          if constexpr (decltype(edge)::value) {
            const int up = pos - key0, down = low - key0;   // columns down .. up are seen
#pragma unroll
            for (int c = 0; c < kStep; ++c)
              if (c > up || c < down) s[c / 32][c % 32] = 0xff800000u;     // -inf
          }
          auto at = [&](int c) { return __uint_as_float(s[c / 32][c % 32]); };
          float most = -INFINITY, ak[kStep / 16], bk[kStep / 16], vk[kStep / 16];
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k) {
            float x = fmaxf(at(16 * k), at(16 * k + 15));
#pragma unroll
            for (int e = 1; e < 15; e += 2) x = max3(x, at(16 * k + e), at(16 * k + e + 1));
            const float4 m4 = sc[k];
            ak[k] = fmaxf(u * m4.x, 1e-30f);                // never 0, which would make NaN of -inf
            bk[k] = m4.y;
            vk[k] = m4.z;
            most = fmaxf(most, fmaf(x, ak[k], bk[k]));
          }
          if (__any_sync(kAll, most > M + kLazy)) {
            const float now = fmaxf(M, most);
            const float f = now == -INFINITY ? 1.0f : exp2_approx(M - now);
            M = now;
            l *= f;
            if (i > 0) {                                      // O so far, after its last product
              if (!wait(&o_full[mt * 2 + ((i - 1) & 1)], ((i - 1) >> 1) & 1)) return false;
              tmem_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(o, o_at + 16 * c);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st16(o_at + 16 * c, o);
              }
            }
          }
          const float ref = M == -INFINITY ? 0.0f : kBoost - M;
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k) {
            const float ck = bk[k] + ref;
            const float2 a2 = make_float2(ak[k], ak[k]), c2 = make_float2(ck, ck);
            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              float2 p = __ffma2_rn(make_float2(at(16 * k + e), at(16 * k + e + 1)), a2, c2);
              p.x = exp2_approx(p.x);
              p.y = exp2_approx(p.y);
              sum = __fadd2_rn(sum, p);
              w[8 * k + e / 2] = pack2<false>(p.x, p.y);
            }
            l = fmaf(sum.x + sum.y, vk[k], l);
          }
          tmem_st32(s_at, w);
          return true;
        };
        const bool edge = key0 + kStep - 1 > wpos || key0 < wlow;
        if (!(edge ? step(std::true_type{}) : step(std::false_type{}))) break;
        tmem_wait_st();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // ---- outputs
      if (steps > 0 && wait(&o_full[mt * 2 + ((steps - 1) & 1)], ((steps - 1) >> 1) & 1)) tmem_fence_after();
      const bool some = steps > 0 && ok;
      const bool joins = dual && mt == 0 && steps_of(1) > 0;
      float f0 = 1.0f, f1 = 0.0f;
      if (dual && mt == 1 && some) {
        second[own] = make_float2(M, l);
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(joined);
      }
      if (joins && wait(joined, 0)) {
        tmem_fence_after();
        const float2 x = second[own];
        const float now = fmaxf(M, x.x), ref = now == -INFINITY ? 0.0f : now;
        f0 = exp2_approx(M - ref);
        f1 = exp2_approx(x.x - ref);
        l = l * f0 + x.y * f1;
        M = now;
      }
      auto outputs = [&](uint32_t (&o)[32], int c) {        // 32 columns of O
        if (some) {
          tmem_ld32(o, o_at + c);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (joins) {                                        // the second set's are in the same lanes
          uint32_t o2[32];
          tmem_ld32(o2, o_at + D + c);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(__uint_as_float(o[e]) * f0 + __uint_as_float(o2[e]) * f1);
        }
      };
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (dual && mt == 1) {
        // the first set writes
      } else if (ok && j.nsplit > 1) {
        // unit by unit (four channels), all rows of a unit next to one another
        float* part = a.part + j.part * C::PART;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          outputs(o, 32 * c);
          if (live) {                                       // columns hold channels 0, 2, 1, 3 of each four
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(part + ((8 * c + e / 4) * C::ROWS + r) * 4) =
                  make_uint4(o[e], o[e + 2], o[e + 1], o[e + 3]);
          }
        }
        if (live) *reinterpret_cast<float2*>(part + D * C::ROWS + 2 * r) = make_float2(M, l);
      } else if (ok) {
        // through shared memory, where the queries are no longer needed, so that
        // rows go out whole: this warp's 32 rows, 16-byte unit c at c ^ (row mod 8)
        uint8_t* mine = qs + (mt * 128 + (warp & 3) * 32) * D * 2;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          outputs(o, 32 * c);
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float x0 = __uint_as_float(o[e + 4 * k]) * inv, x2 = __uint_as_float(o[e + 4 * k + 1]) * inv;
              const float x1 = __uint_as_float(o[e + 4 * k + 2]) * inv, x3 = __uint_as_float(o[e + 4 * k + 3]) * inv;
              h[2 * k] = a.bf16 ? pack2<true>(x0, x1) : pack2<false>(x0, x1);
              h[2 * k + 1] = a.bf16 ? pack2<true>(x2, x3) : pack2<false>(x2, x3);
            }
            const int un = 4 * c + e / 8;
            *reinterpret_cast<uint4*>(mine + lane * D * 2 + ((un ^ (lane & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        __syncwarp();
        constexpr int UNITS = D / 8, AT_ONCE = 32 / UNITS;  // units of a row, rows of one store
        const int un = lane % UNITS;
        const int64_t tok = row / a.R, head = row % a.R;    // each lane finds its row's place
        const int64_t place = live ? ((j.q0 + tok) * a.c.Hkv * a.R + j.kvh * a.R + head) * D : -1;
#pragma unroll 4
        for (int k = 0; k < 32 / AT_ONCE; ++k) {
          const int x = k * AT_ONCE + lane / UNITS;
          const int64_t to = __shfl_sync(kAll, place, x);
          const uint4 v = *reinterpret_cast<const uint4*>(mine + x * D * 2 + ((un ^ (x & 7)) << 4));
          if (to >= 0) *reinterpret_cast<uint4*>(a.out + to + un * 8) = v;
        }
      }
      tmem_fence_before();
    }
  } else if (warp >= kIssuer) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kIssuerRegs));
    {
      // ---- the MMAs
      if (warp < kIssuer + C::MT && j.tiles > 0) {
        const int mt = warp - kIssuer;
        constexpr uint32_t sdesc = kMmaDesc<kStep, false>, odesc = kMmaDesc<D, true>;
        const uint32_t one = elect_one();
        const uint64_t qd = matrix_desc(smem_addr(qs), 16, 1024), kd = matrix_desc(smem_addr(kbuf), 16, 1024);
        const uint64_t vd = matrix_desc(smem_addr(vbuf), KT * 128, 1024);
        // (start addresses count in 16 bytes.  A tile's place is handed back only
        // where a later tile takes it: no arrival is left for after the block's end.)
        const int qset = dual ? 0 : mt;
        auto scores = [&](int i) {                  // step i's, into its buffer
          const int tile = tile_of(i, mt);
          const uint64_t kt = kd + (tile % ST) * (C::TILE / 16) + (C::STEPS == 2 ? (i & 1) * (kStep * 128 / 16) : 0);
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(one, tmem + (mt * 2 + (i & 1)) * kStep, qd + (qset * C::CB + k / 4) * (16384 / 16) + (k % 4) * 2,
                   kt + (k / 4) * (KT * 128 / 16) + (k % 4) * 2, sdesc, k > 0);
          mma_commit(one, &s_full[mt * 2 + (i & 1)]);
          if ((i + 1) % C::STEPS == 0 && tile + ST < j.tiles) mma_commit(one, &k_empty[tile % ST]);
        };
        auto values = [&](int i) {
          const int tile = tile_of(i, mt);
          const uint64_t vt = vd + (tile % ST) * (C::TILE / 16) + (C::STEPS == 2 ? (i & 1) * (kStep * 128 / 16) : 0);
#pragma unroll
          for (int k = 0; k < kStep / 16; ++k)
            mma_ts(one, tmem + C::O0 + mt * D, tmem + (mt * 2 + (i & 1)) * kStep + 8 * k, vt + k * (2048 / 16), odesc,
                   i > 0 || k > 0);
          mma_commit(one, &o_full[mt * 2 + (i & 1)]);
          if ((i + 1) % C::STEPS == 0 && tile + ST < j.tiles) mma_commit(one, &v_empty[tile % ST]);
        };
        // K and V tiles are waited for at their first steps
        auto keys_in = [&](int i) {
          const int tile = tile_of(i, mt);
          if (i % C::STEPS == 0) wait(&k_full[tile % ST], (tile / ST) & 1);
          tmem_fence_after();
          return ok;
        };
        const int n = __shfl_sync(kAll, steps_of(mt), 0);
#pragma unroll 1
        for (int i = 0; i < 2 && i < n; ++i) {
          if (!keys_in(i)) break;
          scores(i);
        }
#pragma unroll 1
        for (int i = 0; i < n && ok; ++i) {
          const int tile = tile_of(i, mt);
          if (i % C::STEPS == 0 && !wait(&v_full[tile % ST], (tile / ST) & 1)) break;
          // the next keys are there before the weights are, but for a set with one
          // place for its keys
          if (!dual && i + 2 < n && !keys_in(i + 2)) break;
          if (!wait(&p_full[mt * 2 + (i & 1)], (i >> 1) & 1)) break;
          tmem_fence_after();
          values(i);
          if (dual && i + 2 < n && !keys_in(i + 2)) break;
          // the buffer is free once that product has read it, which is before
          // the next one of this thread writes it
          if (i + 2 < n) scores(i + 2);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kConvertRegs));
    {
      // ---- codes to fp16, the next tile's loads in flight over this one's
      // conversion and wait
      uint64_t *full = is_v ? v_full : k_full, *empty = is_v ? v_empty : k_empty;
      const uint32_t base = smem_addr(is_v ? vbuf : kbuf);
      int rows2 = -1;                             // the parts of the tile after the one in `next`
      if (j.tiles > 1) rows2 = part_row<D>(a, j, j.first + KT, lane, bad);
#pragma unroll 1
      for (int i = 0; i < j.tiles; ++i) {
        const int st = i % ST;
        float4 m4 = make_float4(0.0f, -INFINITY, 0.0f, 0.0f);        // no block: weights 0
        if (warp == kFirstK && rows >= 0) {
          const int x = rows >> a.c.log_block;
          const float v = fmaxf(a.c.vs[x], kScaleMin);
          m4 = make_float4(fmaxf(a.c.ks[x], kScaleMin), log2f(v), __frcp_rn(v), 0.0f);
        }
        if (i >= ST && !wait(&empty[st], (i / ST - 1) & 1)) break;
        if (warp == kFirstK) {
          if (lane < NSUB) meta[(i & 3) * NSUB + lane] = m4;
          __syncwarp();
          if (lane == 0) mbar_arrive(&meta_full[i & 3]);
        }
        next.template store<FMT>(base + st * C::TILE, which, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&full[st]);
        rows = rows2;
        if (i + 1 < j.tiles) next.template load<FMT>(codes, rows, j.L - j.first - (i + 1) * KT, which, lane);
        if (i + 2 < j.tiles) rows2 = part_row<D>(a, j, j.first + (i + 2) * KT, lane, bad);
      }
    }
  }
  if (!ok) atomicOr(&g_prefill_fault, kFaultWait);
  if (bad) atomicOr(&g_prefill_fault, bad);
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  if (warp == kIssuer)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "n"(C::COLS) : "memory");
}

// ---------------------------------------------------------------------------
// Join the splits of a tile's rows: a warp has 8 rows' 32 channels, so that the
// rows of a unit are read and the units of a row written next to one another.
// ---------------------------------------------------------------------------
template <int D>
constexpr int kJoinRows = 2048 / D;                // rows of a thread block of 8 warps

template <int D, int FMT>
__global__ void __launch_bounds__(256) paged_prefill_join_kernel(AttnArgs a, int whole, int nsplit) {
  using C = Prefill<D>;
  constexpr int PERTILE = C::ROWS / kJoinRows<D>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = static_cast<int>(blockIdx.x % PERTILE) * kJoinRows<D> + warp / (D / 32) * 8 + (lane & 7);
  const int unit = warp % (D / 32) * 8 + (lane >> 3);         // and unit + 4
  int64_t tile = blockIdx.x / PERTILE, piece = 0, c0 = 0, n = 0, k = 0;          // n = 0: nothing to join
  int kvh = 0;
  if (whole == kPlanned) {
    unsigned bad = 0;
    const Plan p = make_plan<D>(a, nsplit, lane, bad);
    const int at = static_cast<int>(tile);
    int b, z;
    if (p.whole > 0) {
      b = p.rest_ns == 1 || at >= p.rest ? -1 : lane_of(p.whole + at, p.tiles_before, p.tiles);
      z = p.whole + at - __shfl_sync(kAll, p.tiles_before, b & 31);
      nsplit = p.rest_ns;
      piece = static_cast<int64_t>(at) * nsplit;
    } else {
      const int mine = p.ns > 1 ? p.tiles : 0, before = sum_before(mine, lane);
      b = lane_of(at, before, mine);
      z = at - __shfl_sync(kAll, before, b & 31);
      nsplit = __shfl_sync(kAll, p.ns, b & 31);
      piece = __shfl_sync(kAll, p.before, b & 31) + z * nsplit;
    }
    c0 = __shfl_sync(kAll, p.c0, b & 31);
    n = b < 0 ? 0 : __shfl_sync(kAll, p.n, b & 31);
    kvh = z % a.c.Hkv;
    k = __shfl_sync(kAll, p.tiles, b & 31) / a.c.Hkv - 1 - z / a.c.Hkv;
  } else {
    piece = tile * nsplit;
    tile += whole;
    const int64_t items = (a.total_q * a.R >> C::LOG_ROWS) + a.c.B, item = items - 1 - tile / a.c.Hkv;
    kvh = static_cast<int>(tile % a.c.Hkv);
    const Found at = find_sequence(a.cu, nullptr, a.c.B, item, a.R, C::LOG_ROWS, 1, lane);
    c0 = at.c0;
    n = c0 < 0 || at.c1 > a.total_q || at.item < 0 ? 0 : at.c1 - c0;
    k = at.item;
  }
  const int64_t row = k * C::ROWS + r;
  const bool none = n == 0 || row < 0 || row >= n * a.R;
  // This grid's end stands for the first one's, so one thread block waits for that
  // even if it has nothing to do.
  if (none && blockIdx.x > 0) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (none) return;
  float o[8], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.0f;
  const float* p = a.part + piece * C::PART;
#pragma unroll 4
  for (int s = 0; s < nsplit; ++s, p += C::PART) {
    const float2 x = *reinterpret_cast<const float2*>(p + D * C::ROWS + 2 * r);
    const float4 y0 = *reinterpret_cast<const float4*>(p + (unit * C::ROWS + r) * 4);
    const float4 y1 = *reinterpret_cast<const float4*>(p + ((unit + 4) * C::ROWS + r) * 4);
    const float now = fmaxf(m, x.x), ref = now == -INFINITY ? 0.0f : now;
    const float e0 = exp2_approx(m - ref), e1 = exp2_approx(x.x - ref);
    l = l * e0 + x.y * e1;
    const float y[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = o[i] * e0 + y[i] * e1;
    m = now;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* out = a.out + ((c0 + row / a.R) * a.c.Hkv * a.R + kvh * a.R + row % a.R) * D + unit * 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float x0 = o[4 * i] * inv, x1 = o[4 * i + 1] * inv, x2 = o[4 * i + 2] * inv, x3 = o[4 * i + 3] * inv;
    *reinterpret_cast<uint2*>(out + 16 * i) = a.bf16 ? make_uint2(pack2<true>(x0, x1), pack2<true>(x2, x3))
                                                     : make_uint2(pack2<false>(x0, x1), pack2<false>(x2, x3));
  }
}

template <int D, int FMT>
cudaError_t launch(const AttnArgs& a, int64_t whole, int nsplit, cudaStream_t st) {
  using C = Prefill<D>;
  auto k = paged_prefill_kernel<D, FMT>;
  static std::atomic<int> ready[64];              // the shared-memory opt-in, once per device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || ready[dev].load(std::memory_order_relaxed) == 0) {
    e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, k);
    if (e != cudaSuccess) return e;
    if (fa.numRegs * kThreads < kRegsNeeded) return cudaErrorInvalidKernelImage;
    if (dev < 64) ready[dev].store(1, std::memory_order_relaxed);
  }
  const int64_t tiles = ((a.total_q * a.R >> C::LOG_ROWS) + a.c.B) * a.c.Hkv;
  // (a planned call's nsplit: the places, all thread blocks that run at once)
  const int64_t split = whole == kPlanned ? std::min<int64_t>(tiles, nsplit / 2) : tiles - whole;
  const unsigned grid = static_cast<unsigned>(whole != kPlanned ? whole + split * nsplit
                                              : tiles <= nsplit ? nsplit : (tiles / nsplit + 1) * nsplit);
  k<<<grid, kThreads, C::SMEM, st>>>(a, static_cast<int>(whole), nsplit);
  e = cudaGetLastError();
  if (e != cudaSuccess || nsplit == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(split * (C::ROWS / kJoinRows<D>)));
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_prefill_join_kernel<D, FMT>, a, static_cast<int>(whole), nsplit);
}

}  // namespace

__attribute__((visibility("hidden"))) int kvq_paged_prefill_launch(const AttnArgs& a, int format, int64_t whole,
                                                                   int nsplit, cudaStream_t st, cudaError_t& err) {
  const bool f8 = format == KVQ_E4M3;
  switch (a.c.D) {
    case 64: err = f8 ? launch<64, kE4m3>(a, whole, nsplit, st) : launch<64, kInt8>(a, whole, nsplit, st); break;
    case 128: err = f8 ? launch<128, kE4m3>(a, whole, nsplit, st) : launch<128, kInt8>(a, whole, nsplit, st); break;
    default: err = f8 ? launch<256, kE4m3>(a, whole, nsplit, st) : launch<256, kInt8>(a, whole, nsplit, st); break;
  }
  return err == cudaSuccess ? KVQ_OK : KVQ_ERR_LAUNCH;
}

__attribute__((visibility("hidden"))) unsigned int kvq_paged_prefill_fault_word(int clear) {
  unsigned int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_prefill_fault, sizeof(v)) != cudaSuccess) return 0;
  if (clear && v) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_prefill_fault, &zero, sizeof(zero));
  }
  return v;
}
