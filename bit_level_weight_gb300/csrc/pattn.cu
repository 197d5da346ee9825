// pattn.cu - attention of new tokens over a paged bf16 cache.
//
// o = softmax(q K^T / sqrt(128)) V over the positions up to the row's own, in
// one pass over the keys with the running maximum and sum of the softmax.
//
// Work. The query heads of one kv head are rows of one product: flat row f of
// a sequence is token f / G, head f % G of the group. A unit is 256 flat rows
// of one (sequence, kv head); its keys are taken in tiles of 128. The tiles of
// all units form one line that is cut into equal pieces, one a CTA (one CTA
// an SM), so single tokens over uneven contexts, a few drafted rows and long
// prompt chunks balance alike. A CTA whose piece starts or ends inside a unit
// writes the partial result (maximum, sum, unnormalised output) to the
// workspace and attn_join_kernel merges the pieces. Lengths are read on the
// device: every CTA finds its place on the line from row_start and kv_len.
//
// A CTA holds two slots of 128 rows with a softmax warpgroup each. Units of
// more than 128 rows put their two halves in the slots and share each key
// tile; smaller units (decoding, drafted tokens) take even key tiles in slot 0
// and odd ones in slot 1 and merge the two at the end, so that one slot's
// softmax runs while the tensor cores work for the other in both cases.
//
//   warps 4-7, 8-11 softmax of slot 0, 1: S from tensor memory (a row a
//                   thread), P back as bf16, O rescaled there when a row's
//                   maximum grows by more than 2^8 (probabilities relative to
//                   an older maximum are as exact), epilogue
//   warp 1, 2       TMA: K and V tiles from their pages, five 32 KB buffers
//   warp 0          issues tcgen05.mma: S = Q K^T (both from shared memory),
//                   O += P V (P from tensor memory, V with the head dimension
//                   contiguous)
//   warp 3          finds the CTA's units and hands them to the others one
//                   ahead, with their Q rows
//
// What bounds it (measured on GB300, 8 kv heads, 32 query heads):
//   one token a sequence: the K and V stream. 61 sequences of up to 8K: 172-177
//     us for 1.0 GB = 5.7-5.8 TB/s, 83-86 % of the measured copy rate; one sequence of 32K:
//     41 us for 134 MB, of which about 8 us are the way to the first tile (place
//     on the line, page table, first TMA) and 4 us the join.
//   long chunks: 2048 rows over 32K in 686-706 us = 1.51-1.55 PFLOP/s by themselves,
//     78-80 % of cuBLAS's burst rate on this GPU; 750 us = 1.42 PFLOP/s in long runs,
//     where the power cap holds the SMs at 1790 MHz, 73 % of the burst rate and 81 %
//     of cuBLAS's sustained one. A key tile takes 1.6 us where its four products
//     need 1.05: a slot's chain S -> softmax (0.7 us) -> P V, S is longer than what
//     the other slot hides, and tensor memory holds no third slot (2 x (128 S +
//     128 O) columns are all 512). Tried and slower: P V in two halves behind two
//     barriers (790 us), two threads a row in sixteen softmax warps (880 us), the
//     exponentials ahead of the maximum (790 us): each puts more waits or
//     instructions next to the issuing warp, whose products then lag.
//   short ragged chunks: a change of units costs a slot about 3 us (last
//     product, output, first scores), which kUnitCells weighs in.
//
// The 4-bit cache (cas_paged4_attn, more than 32 rows of a kv head a sequence): the same
// with a fourth warpgroup that writes the tiles which TMA writes here: 2048 rows over 32K
// in 759 us = 1.40 PFLOP/s. (By the two loading warps: 2711 us.) Its softmax spills 76 bytes
// a thread.
//
// Every wait is bounded: one that gives up marks the CTA, whose warps then
// leave their loops, and sets a status that cas_device_status reads. Units that
// such a CTA holds a piece of are not joined.
//
// Rounding: scores, statistics and sums are fp32; P is rounded to bf16 for the
// product with V, the sum takes it unrounded. In calls of at most 128 rows of a
// kv head a sequence on average (LOW: decoding, drafted tokens) units of at most
// 128 rows multiply V by what that rounding left as well, a second product with
// P good to 2^-17 as in the compressed cache's attention; the output's distance
// from 64 bits is then that of its own rounding (0.168 % instead of 0.24 %). That
// costs one token over 32K 41 instead of 38 us, 61 ragged ones 173 instead of
// 167; for units of 256 rows it would be 983 instead of 702 us (2048 rows over
// 32K), and the unused code alone 105 instead of 93 us for five ragged prompts
// (first fetch of the instructions), so prompts have a kernel without it.
//
// The tensor cores cut the sums of their accumulators instead of rounding them
// (as measured: the output of a unit that one CTA takes whole came out 0.05 %
// small at 128K tokens, 0.33 % at 1M, 1.5 % at 4M), so a slot folds its O into
// fp32 memory every kFold tiles: 0.011 % at every length from 128K to 4M, for 6 us
// a fold (units of 1024 tiles each in a CTA: 1516 -> 1539 us).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "mma.cuh"
#include "paged.cuh"
#include "pline.cuh"
#include "q4.cuh"
#include "tc05.cuh"

namespace cas {
namespace {

constexpr int kTile = 128;                 // keys a tile, rows a slot
constexpr int kUnit = 2 * kTile;           // flat rows a unit
constexpr int kRing = 5;                   // K / V buffers: with two Q tiles all of the shared memory
constexpr uint32_t kBuf = kTile * 256;     // bytes of a K or V tile
constexpr uint32_t kHalf = kBuf / 2;       // 64 of the 128 dimensions
constexpr int kLowPart = kTile / 2;        // columns of S behind P
constexpr int kThreads = 384;               // three warpgroups of 168 registers a thread at launch
constexpr int kThreads4 = 512;              // four of 128
// Registers of the softmax, which keeps a row of S, and of the others: 2 * 216 + 72 = 3 * 168. With the
// 4-bit cache's decoders, a fourth warpgroup: 2 * 184 + 72 + 72 = 4 * 128 (with 2 * 176 + 88 the softmax spills more: 836 instead of 740 us).
template <bool Q4>
struct Regs {
  static constexpr int kSoftmax = Q4 ? 184 : 216, kOther = 72, kDecode = 72;
};
constexpr int kUnitCells = 2;              // cells of the line for a change of units: about two tiles' time
                                           // (1, 2, 3 of them: 104, 98, 98 us on five ragged prompts)
constexpr int kMinCells = kUnitCells + 2;  // cells a CTA takes at least
constexpr uint32_t kSpins = 1u << 20;        // polls of a wait
constexpr int kFold = 256;                   // tiles that a slot's O adds up before it is folded away: a power of two

__device__ int g_attn_status = 0;
// Polls of a wait before it gives up; 0 (tests) also hands out no units, so that
// the waits for one run out. 1 (tests): so in every second CTA.
__constant__ uint32_t c_attn_spins = kSpins;
__device__ __forceinline__ uint32_t spins() {
  return c_attn_spins == 1 ? (blockIdx.x & 1 ? 0 : kSpins) : c_attn_spins;
}

struct AttnArgs : JoinArgs {
  const uint16_t* q;
  float* ws1;        // [grid] pieces of min(piece_rows, 128) rows: what slot 1 folds of units of few rows
  bool wide;         // o is 32-byte aligned
  bool q_box;        // G divides 128: Q by TMA
};
using Units = UnitLine<kUnit, kTile, kUnitCells>;

// A unit, or the part of it that a CTA takes.
struct Unit {
  int b, start, hk, f0, rows;  // sequence and its first row, kv head, flat rows
  int pos0, kv_end;            // position of the sequence's first row, end of what it holds
  int first_pos;               // position of the unit's first row
  int t0, n;                   // key tiles
  int flags;                   // below
};
enum { kWhole = 1, kFirst = 2, kLast = 4, kNone = 8, kTileB = 16 };  // kTileB: Q in the second tile

// ---------------------------------------------------------------- shared memory
struct Aux {
  uint64_t kv_full[kRing], kv_empty[kRing];
  uint64_t u_full[2], u_empty[2], q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], merge, merged, spoilt, drain;
  uint64_t seen[2];  // slot 1 is through with the marks below: of even, of odd units
  uint32_t tmem;
  int abort;
  Unit unit[2];
  Cut cut;
  // values that are not finite and that not every row of the unit sees, for an
  // even and an odd unit: whether there are any, and the first position for each
  // dimension, counted from the unit's first row's. Slot 0 may be two units ahead
  // of slot 1 (with one key tile, a unit's O of slot 0 is out before slot 1's P is
  // waited for), but then waits for slot 1 in seen[u & 1] before it marks. Slot 1 is
  // one ahead at most: its O of unit u, or the merge of the two, needs slot 0's P
  // of u, which follows all that slot 0 does for u - 1.
  int any_bad[2];
  uint16_t bad[2][CAS_BLK];
  float m[2][kTile], l[2][kTile];
};

__device__ __forceinline__ bool wait_long(uint64_t* bar, uint32_t phase, volatile int* abort, uint64_t tiles) {
  const uint64_t limit = spins() * tiles;
  for (uint64_t i = 0; i < limit; ++i) {
    if (mbar_try_wait(bar, phase)) return true;
    if ((i & 63) == 63 && *abort) return false;
  }
  *abort = 1;
  atomicExch(&g_attn_status, CAS_ERR_TIMEOUT);
  return false;
}
// Warp-wide; false when any lane gave up. tiles: what the wait may have to
// outlast, a few for all but the scheduler's, which lie behind whole units.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t phase, Aux* x, uint64_t tiles = 1) {
  bool ok = mbar_try_wait(bar, phase);
  if (!__all_sync(CAS_FULL, ok)) ok = ok || wait_long(bar, phase, &x->abort, tiles);
  return __all_sync(CAS_FULL, ok);
}
__device__ __forceinline__ void arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
// Unit number `u` of the CTA, read by a warp that then frees its place.
__device__ __forceinline__ bool take_unit(uint32_t u, Aux* x, Unit& w) {
  if (!wait(&x->u_full[u & 1], (u >> 1) & 1, x)) return false;
  w = x->unit[u & 1];
  arrive_warp(&x->u_empty[u & 1]);
  return true;
}

// K and V tiles take the buffers in turn: K0 V0 K1 V1 ... A turn is a buffer and
// the parity of its use; each of the two streams takes every second one.
struct Turn {
  uint32_t slot, phase;
  __device__ __forceinline__ void next() {
    slot += 2;
    if (slot >= kRing) {
      slot -= kRing;
      phase ^= 1;
    }
  }
};

// ---------------------------------------------------------------- units and Q
__device__ void scheduler(const AttnArgs& a, const CUtensorMap* qm, uint8_t* q_sm, Aux* x) {
  const int lane = threadIdx.x & 31;
  Units::Line line;
  Place p;
  Unit w{};
  if (spins() == 0) return;
  Seq s;
  const bool any = Units::find_place(a, blockIdx.x, gridDim.x, kMinCells, line, p, s);
  if (!any) {
    if (lane == 0) {
      w.flags = kNone | kLast;
      x->unit[0] = w;
    }
    arrive_warp(&x->u_full[0]);
    return;
  }
  int64_t left = min(line.per, line.total - (int64_t)blockIdx.x * line.per);
  int cell = p.cell;
  uint32_t uses[2] = {0, 0};  // of the Q tiles
  uint64_t handed = 1;        // tiles of the units so far: the limit of the waits grows with them
  uint32_t loads = 0;         // units whose Q was fetched by TMA
  for (uint32_t u = 0;; ++u) {
    const int all = Units::unit_tiles(s, a, p.qt);
    const int end = (int)min((int64_t)all + kUnitCells, cell + left);
    w.b = p.b, w.start = s.start, w.hk = p.hk, w.f0 = p.qt * kUnit;
    w.rows = min(kUnit, s.R - w.f0);
    w.pos0 = s.len - s.T;
    w.kv_end = min(s.cap, s.len);
    w.first_pos = w.pos0 + div_g(a, w.f0);
    w.t0 = max(0, cell - kUnitCells);
    w.n = max(0, end - kUnitCells) - w.t0;
    left -= end - cell;
    const bool two = w.rows > kTile, tile_b = !two && (u & 1);
    w.flags = (w.n == all ? kWhole : 0) | (u == 0 ? kFirst : 0) | (tile_b ? kTileB : 0);
    const bool last = left <= kUnitCells;  // (a next unit's first cells hold no tile)
    if (last) w.flags |= kLast;
    if (!wait(&x->u_empty[u & 1], ((u >> 1) & 1) ^ 1, x, handed)) break;
    if (lane == 0) x->unit[u & 1] = w;
    arrive_warp(&x->u_full[u & 1]);
    if (w.t0 == 0 && w.n > 0 && w.n < all && lane == 0) {  // the unit's first piece: its cut
      Cut& cut = x->cut;
      cut.pieces = 1 + (int)div64(all - w.n + line.per - 1, line.per);
      cut.start = w.start, cut.hk = w.hk, cut.f0 = w.f0, cut.rows = w.rows;
      cut.first = u == 0 ? 0 : 1;
    }
    // Q: rows of 256 bytes in swizzled halves. Rows that the unit does not have
    // hold another sequence's or what was there: nothing of them is used.
    const int first = tile_b ? 1 : 0, count = two ? 2 : 1;
    bool ok = true;
    for (int t = first; t < first + count; ++t) ok = ok && wait(&x->q_empty[t], (uses[t]++ & 1) ^ 1, x, handed);
    if (!ok) break;
    handed += w.n;
    if (a.q_box) {  // boxes of the group's heads x 128 / G tokens
      if (lane == 0) {
        mbar_arrive_tx(&x->q_full[u & 1], count * kBuf);
        for (int t = 0; t < count; ++t) {
          uint8_t* dst = q_sm + (first + t) * kBuf;
          const int tok = w.start + div_g(a, w.f0 + t * kTile);
          tma_load_3d(dst, qm, 0, w.hk * a.G, tok, &x->q_full[u & 1]);
          tma_load_3d(dst + kHalf, qm, 64, w.hk * a.G, tok, &x->q_full[u & 1]);
        }
      }
      __syncwarp();
      loads = u + 1;
    } else {  // other group sizes: 16 bytes a lane
      const int c = lane & 15, f = w.f0 + (lane >> 4);
      int t = div_g(a, f), h = f - t * a.G;
      const uint16_t* src = a.q + ((int64_t)(w.start + t) * a.Hq + w.hk * a.G + h) * CAS_BLK + 8 * c;
      const int64_t next_token = (int64_t)(a.Hq - a.G) * CAS_BLK;
      const uint32_t dst = smem_u32(q_sm) + first * kBuf + (c >> 3) * kHalf;
#pragma unroll 4
      for (int row = lane >> 4; row < w.rows; row += 2) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst + (row >> 7) * kBuf + (row & 127) * 128 +
                                                                     (((c & 7) ^ (row & 7)) << 4)),
                     "l"(src)
                     : "memory");
        src += 2 * CAS_BLK;  // the group's next head but one, or that of a later token
        for (h += 2; h >= a.G; h -= a.G) src += next_token;
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      fence_async_smem();
      arrive_warp(&x->q_full[u & 1]);
    }
    if (last) break;
    cell = 0;
    if (++p.qt >= Units::unit_count(s)) {
      p.qt = 0;
      if (++p.hk >= a.d.H) {
        p.hk = 0;
        do s = ++p.b < a.d.batch ? seq_of(a, p.b) : Seq{};
        while (s.R == 0 && p.b < a.d.batch);
      }
    }
  }
  if (*(volatile int*)&x->abort)  // after a wait that gave up, copies in flight land before the block ends
    for (uint32_t u = loads > 2 ? loads - 2 : 0; u < loads; ++u)
      mbar_wait_bounded(&x->q_full[u & 1], (u >> 1) & 1, kSpins);
}

// ---------------------------------------------------------------- K and V
// One warp loads K, another V: pages of 16 tokens take 16 boxes a tile, whose
// issue would bound one warp.
template <bool IS_V>
__device__ void producer(const AttnArgs& a, const CUtensorMap* map, uint8_t* ring, Aux* x) {
  const int lane = threadIdx.x & 31;
  const int shift = min(a.d.shift, 7);  // log2 of tokens a box
  const int boxes = kTile >> shift;     // boxes a tile
  Turn turn{IS_V ? 1u : 0u, 0};
  uint32_t used = 0, phase = 0;  // buffers this warp has filled, and the phase of its newest copy
  bool ok = true;
  for (uint32_t u = 0; ok; ++u) {
    Unit w;
    if (!take_unit(u, x, w) || (w.flags & kNone)) break;
    // page of this lane's box of tile j; pages past the last token and bad ids load zeros
    auto page_at = [&](int j) -> int {
      const int64_t tok = (int64_t)(w.t0 + j) * kTile + ((int64_t)lane << shift);
      if (lane >= boxes || j >= w.n || tok >= w.kv_end) return (int)a.d.n_pages;
      const int64_t id = page_of(a.d, w.b, tok);
      return id < 0 ? (int)a.d.n_pages : (int)id;
    };
    int cur = page_at(0), nxt = page_at(1);
    for (int j = 0; j < w.n; ++j) {
      const uint32_t slot = turn.slot;
      ok = wait(&x->kv_empty[slot], turn.phase ^ 1, x);
      if (!ok) break;
      used |= 1u << slot;
      phase = (phase & ~(1u << slot)) | turn.phase << slot;
      turn.next();
      if (lane == 0) mbar_arrive_tx(&x->kv_full[slot], kBuf);
      __syncwarp();
      if (lane < boxes) {
        const int in_page = (int)(((int64_t)(w.t0 + j) * kTile + (lane << shift)) & ((1 << a.d.shift) - 1));
        uint8_t* dst = ring + slot * kBuf + ((uint32_t)lane << shift) * 128;
        tma_load_4d(dst, map, 0, in_page, w.hk, cur, &x->kv_full[slot]);
        tma_load_4d(dst + kHalf, map, 64, in_page, w.hk, cur, &x->kv_full[slot]);
      }
      cur = nxt;
      nxt = page_at(j + 2);
    }
    if (w.flags & kLast) break;
  }
  // after a wait that gave up, copies in flight land before the block ends
  if (*(volatile int*)&x->abort)
    for (int i = 0; i < kRing; ++i)
      if (used >> i & 1) mbar_wait_bounded(&x->kv_full[i], phase >> i & 1, kSpins);
}

// ---------------------------------------------------------------- K and V of the 4-bit cache
// The same tiles from records (q4.cuh), made by a warpgroup of its own: warp d of it takes
// tokens 32d..32d+31 of every K and V tile in turn. Four lanes read a token's 64 bytes of
// codes, 32 dimensions each, and write them as bf16 chunks of 16 bytes where TMA with a
// 128-byte swizzle would put them; lanes of the upper dimensions take their chunks in
// another order, so that the eight lanes that write together, two rows of four, take
// different banks. Codes are loaded a tile ahead. What is not there reads as zeros, and
// nothing in a tile is infinite.
struct Codes {
  uint4 w;
  uint32_t s;
};
__device__ void decoder(const AttnArgs& a, uint8_t* ring, Aux* x) {
  constexpr int kBatches = 4;  // of 8 tokens
  const int lane = threadIdx.x & 31, q = lane & 3, tr = lane >> 2, first = (threadIdx.x >> 5 & 3) * 32;
  const int shift = min(a.d.shift, 7), boxes = kTile >> shift;
  const bool upper = q & 2;
  const Q4Bf16 q4;
  uint32_t place[4];  // of the lane's chunks in a row of its half
#pragma unroll
  for (int i = 0; i < 4; ++i)
    place[i] = (uint32_t)(((4 * (q & 1) + (i ^ (upper ? 2 : 0))) ^ tr) << 4) + (q >> 1) * kHalf + (first + tr) * 128;
  const uint8_t* rec0 = a.d.rec + tr * a.d.token_stride;
  uint32_t slot = 0, phase = 1;
  bool ok = true;
  for (uint32_t u = 0; ok; ++u) {
    Unit w;
    if (!take_unit(u, x, w) || (w.flags & kNone)) break;
    // page of this lane's box of tile j
    auto page_at = [&](int j) -> int {
      const int64_t tok = (int64_t)(w.t0 + j) * kTile + ((int64_t)lane << shift);
      if (lane >= boxes || j >= w.n || tok >= w.kv_end) return -1;
      return (int)page_of(a.d, w.b, tok);
    };
    const uint8_t* head = rec0 + w.hk * a.d.head_stride;
    auto load = [&](Codes* to, int j, int pages, bool v) {
#pragma unroll
      for (int k = 0; k < kBatches; ++k) {
        const int t = first + 8 * k;  // (a box has 8 tokens or more)
        const int page = __shfl_sync(CAS_FULL, pages, t >> shift);
        const int in_page = (int)(((uint32_t)(w.t0 + j) * kTile + t) & ((1u << a.d.shift) - 1));
        to[k].w = make_uint4(0, 0, 0, 0);
        to[k].s = 0;
        if (page >= 0) {
          const uint8_t* rec = head + page * a.d.page_stride + in_page * a.d.token_stride;
          to[k].w = *reinterpret_cast<const uint4*>(rec + (v ? kRecV : 0) + 16 * q);
          to[k].s = *reinterpret_cast<const uint16_t*>(rec + (v ? kRecVs : kRecKs) + 2 * q);
        }
      }
    };
    auto put = [&](const Codes* from) {
      ok = ok && wait(&x->kv_empty[slot], phase, x);
      if (!ok) return;
      uint8_t* tile = ring + slot * kBuf;
#pragma unroll
      for (int k = 0; k < kBatches; ++k) {
        const Codes& t = from[k];
        const uint32_t word[4] = {upper ? t.w.z : t.w.x, upper ? t.w.w : t.w.y, upper ? t.w.x : t.w.z, upper ? t.w.y : t.w.w};
        const uint32_t s = upper ? __byte_perm(t.s, 0, 0x4401) : t.s;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t s2 = q4_scale2(half ? s >> 8 : s & 255), n2 = q4_offset(s2);
#pragma unroll
          for (int i = 2 * half; i < 2 * half + 2; ++i)
            *reinterpret_cast<uint4*>(tile + place[i] + 8 * k * 128) = q4.word(word[i], s2, n2);
        }
      }
      fence_async_smem();
      arrive_warp(&x->kv_full[slot]);
      if (++slot == kRing) slot = 0, phase ^= 1;
    };
    int pages = page_at(0);
    Codes ck[kBatches], cv[kBatches];
    load(ck, 0, pages, false);
    load(cv, 0, pages, true);
    pages = page_at(1);
    for (int j = 0; ok && j < w.n; ++j) {
      put(ck);
      load(ck, j + 1, pages, false);
      put(cv);
      load(cv, j + 1, pages, true);
      pages = page_at(j + 2);
    }
    if (w.flags & kLast) break;
  }
}

// ---------------------------------------------------------------- products
// A step of a slot is P V of one tile and the scores of the next: one elected
// lane issues both and their signals without a wait in between, since the K and
// V tiles that it needs are waited for before P is (they are there long since).
template <bool LOW>
__device__ void issuer(uint32_t q_sm, uint32_t ring_sm, Aux* x) {
  const uint32_t tm = __reduce_max_sync(CAS_FULL, x->tmem);
  constexpr uint32_t id_s = tc_idesc_bf16(kTile, kTile, false), id_o = tc_idesc_bf16(kTile, CAS_BLK, true);
  uint32_t np[2] = {0, 0};
  Turn kt{0, 0}, vt{1, 0};  // buffers of the next K and V tile
  bool ok = true;
  auto arrived = [&](const Turn& t) { ok = ok && wait(&x->kv_full[t.slot], t.phase, x); };
  auto wait_p = [&](int slot) {
    ok = ok && wait(&x->p_full[slot], np[slot]++ & 1, x);
    tc_fence_after();
  };
  auto scores = [&](int slot, uint32_t tile, const Turn& k) {
    tc_product_ss(tm + slot * kTile, tc_desc_lo(q_sm + tile * kBuf, 16), tc_desc_lo(ring_sm + k.slot * kBuf, 16), id_s);
    tc_commit(&x->s_full[slot]);
  };
  auto values = [&](int slot, const Turn& v, bool add, bool low) {
    const uint32_t o = tm + 2 * kTile + slot * CAS_BLK, p = tm + slot * kTile, b = tc_desc_lo(ring_sm + v.slot * kBuf, kHalf);
    tc_product_ts(o, p, b, id_o, add);
    if (low) tc_product_ts(o, p + kLowPart, b, id_o, 1);
  };
  auto release = [&](const Turn& t) { tc_commit(&x->kv_empty[t.slot]); };
  for (uint32_t u = 0; ok; ++u) {
    Unit w;
    if (!take_unit(u, x, w) || (w.flags & kNone)) break;
    ok = wait(&x->q_full[u & 1], (u >> 1) & 1, x);
    const int n = w.n;
    if (w.rows > kTile) {
      arrived(kt);
      tc_fence_after();
      if (ok && elect_one()) {
        scores(0, 0, kt);
        scores(1, 1, kt);
        release(kt);
        if (n == 1) tc_commit(&x->q_empty[0]), tc_commit(&x->q_empty[1]);
      }
      __syncwarp();
      kt.next();
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n, last = j + 2 == n;
        arrived(vt);
        if (more) arrived(kt);
        wait_p(0);
        if (ok && elect_one()) {
          values(0, vt, j & (kFold - 1), false);
          if (more) {
            scores(0, 0, kt);
            if (last) tc_commit(&x->q_empty[0]);
          } else {
            tc_commit(&x->o_full[0]);
          }
        }
        __syncwarp();
        wait_p(1);
        if (ok && elect_one()) {
          values(1, vt, j & (kFold - 1), false);
          release(vt);
          if (more) {
            scores(1, 1, kt);
            release(kt);
            if (last) tc_commit(&x->q_empty[1]);
          } else {
            tc_commit(&x->o_full[1]);
          }
        }
        __syncwarp();
        vt.next();
        if (more) kt.next();
      }
    } else {
      const int t = (w.flags & kTileB) ? 1 : 0;
      for (int j = 0; j < min(n, 2); ++j) {
        arrived(kt);
        tc_fence_after();
        if (ok && elect_one()) {
          scores(j, t, kt);
          release(kt);
          if (j + 1 == n) tc_commit(&x->q_empty[t]);
        }
        __syncwarp();
        kt.next();
      }
      for (int j = 0; j < n && ok; ++j) {
        const int i = j & 1;
        const bool more = j + 2 < n;
        // few rows wait for memory: nothing waits for a K tile that it does not need
        arrived(vt);
        wait_p(i);
        if (ok && elect_one()) {
          values(i, vt, (j >> 1) & (kFold - 1), LOW);
          release(vt);
          if (!more) tc_commit(&x->o_full[i]);
        }
        __syncwarp();
        if (more) {
          arrived(kt);
          if (ok && elect_one()) {
            scores(i, t, kt);
            release(kt);
            if (j + 3 == n) tc_commit(&x->q_empty[t]);
          }
          __syncwarp();
        }
        vt.next();
        if (more) kt.next();
      }
    }
    if (w.flags & kLast) break;
  }
  if (elect_one()) tc_commit(&x->drain);  // products in flight end before the block does
  __syncwarp();
  mbar_wait_bounded(&x->drain, 0, kSpins);
}

// ---------------------------------------------------------------- softmax
// Scale of the scores in powers of two: log2(e) / sqrt(128).
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;

__device__ __forceinline__ void store32(void* p, const uint32_t* v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// A probability of zero does not hide what is not finite: 0 * NaN would reach
// rows that do not see the token. Tiles at the end of what a unit's rows see are
// looked over by a thread a V row: rows behind the last token, which may hold
// anything, become zeros; values of tokens that only some rows see become zeros
// where they are not finite, and the epilogue makes the outputs of that
// dimension NaN for the rows that see the first of them.
__device__ __forceinline__ bool guards(const Unit& w, int key0) {
  return min(key0 + kTile, w.kv_end) - 1 > w.first_pos;  // a token that the unit's first row does not see
}
__device__ bool guard_values(const Unit& w, uint32_t u, int slot, int key0, uint32_t item, uint8_t* ring, Aux* x) {
  const int r = threadIdx.x & 127, turn = u & 1;
  if (slot == 0 && !wait(&x->seen[turn], ((u >> 1) & 1) ^ 1, x)) return false;  // of unit u - 2
  if (!wait(&x->kv_full[item % kRing], (item / kRing) & 1, x)) return false;
  uint8_t* row = ring + (item % kRing) * kBuf + r * 128;
  bool wrote = false;
  if (key0 + r >= w.kv_end) {
    wrote = true;
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint4*>(row + c * 16) = *reinterpret_cast<uint4*>(row + kHalf + c * 16) = make_uint4(0, 0, 0, 0);
  } else if (key0 + r > w.first_pos) {
    uint32_t top = 0;  // the largest magnitudes of two lanes
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int c = 0; c < 8; ++c) {  // rotated, so that a warp's threads read different banks
        const uint4 v = *reinterpret_cast<const uint4*>(row + h * kHalf + (((c + r) & 7) << 4));
        top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                     __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
      }
    }
    if ((top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u) {
      wrote = true;
      for (int d = 0; d < CAS_BLK; ++d) {
        uint16_t* p = reinterpret_cast<uint16_t*>(row + (d >> 6) * kHalf + ((((d >> 3) & 7) ^ (r & 7)) << 4)) + (d & 7);
        if ((*p & 0x7F80u) == 0x7F80u) {
          *p = 0;
          const uint16_t at = (uint16_t)(key0 + r - w.first_pos);
          for (uint16_t old = x->bad[turn][d]; at < old;) {
            const uint16_t was = atomicCAS(&x->bad[turn][d], old, at);
            if (was == old) break;
            old = was;
          }
          x->any_bad[turn] = 1;
        }
      }
    }
  }
  if (wrote) fence_async_smem();
  return true;
}

// A maximum is rounded once, by up to 2^-24 of itself, and the scores that it is taken from are not: up to
// here that makes all of a row's P alike wrong by 2^(2^-4), beyond it too large or zero.
constexpr float kFar = 0x1p20f;

// P = 2^(s kScaleLog2 - ref) of a row's 128 scores as bf16 into its columns at
// tm_s, with LOW what the rounding left of it behind; returns the sum of P. FAR: a
// ref beyond kFar is taken from scores that are rounded as it was.
template <bool LOW, bool FAR = false>
__device__ __forceinline__ float weigh_keys(const uint32_t s[kTile], float ref, uint32_t tm_s) {
  const uint64_t sc2 = pack2(kScaleLog2, kScaleLog2), ref2 = pack2(-ref, -ref);
  uint64_t ls[2] = {0, 0};
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t p[32], q[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) {
      float e0, e1;
      unpack2(fma2(pack2(__uint_as_float(s[64 * c + 2 * k]), __uint_as_float(s[64 * c + 2 * k + 1])), sc2, ref2), e0, e1);
      if (FAR && fabsf(ref) > kFar) {
        e0 = __fadd_rn(__fmul_rn(__uint_as_float(s[64 * c + 2 * k]), kScaleLog2), -ref);
        e1 = __fadd_rn(__fmul_rn(__uint_as_float(s[64 * c + 2 * k + 1]), kScaleLog2), -ref);
      }
      e0 = ex2(e0);
      e1 = ex2(e1);
      ls[k & 1] = add2(ls[k & 1], pack2(e0, e1));
      p[k] = pack_bf16x2(e0, e1);
      if (LOW) q[k] = pack_bf16x2(e0 - __uint_as_float(p[k] << 16), e1 - __uint_as_float(p[k] & 0xFFFF0000u));
    }
    tm_st32(tm_s + 32 * c, p);
    if (LOW) tm_st32(tm_s + kLowPart + 32 * c, q);
  }
  float l0, l1;
  unpack2(add2(ls[0], ls[1]), l0, l1);
  return l0 + l1;
}

// The same of a warp that has a row with its maximum beyond kFar: rare, and apart, as the loop over the tiles has
// no registers left. The scores are read again; the last that the row sees is number `last`. (The look for such
// rows takes 2048 rows over 32K of the 4-bit cache from 746 to 759 us, of the bf16 cache nothing.)
template <bool LOW>
__device__ __noinline__ float weigh_far_keys(float ref, uint32_t tm_s, int last) {
  uint32_t s[kTile];
#pragma unroll
  for (int c = 0; c < kTile; c += 32) tm_ld32(s + c, tm_s + c);
#pragma unroll
  for (int c = 0; c < kTile; c += 32) tm_wait_ld(s + c);
#pragma unroll
  for (int c = 0; c < kTile; ++c)
    if (c > last) s[c] = 0xFF800000u;
  return weigh_keys<LOW, true>(s, ref, tm_s);
}

// The tensor cores cut their sums, so a slot's O takes kFold tiles at most: then
// it is added, relative to the maximum m of now, to what the row's place in the
// workspace holds (`more`), and starts anew; at the unit's end (`back`) the sum
// of both goes to tensor memory. Warp-wide; a thread reads what it wrote itself.
__device__ __noinline__ void fold(const AttnArgs& a, bool own, bool first, int fr, bool mine, uint32_t tm_o, float m,
                                  bool more, bool back) {
  const int rows = own ? a.piece_rows : min(a.piece_rows, kTile);
  float* place = own ? a.ws + (int64_t)(2 * blockIdx.x + (first ? 0 : 1)) * rows * kPieceFloats
                     : a.ws1 + (int64_t)blockIdx.x * rows * kPieceFloats;
  float* top = place + (int64_t)CAS_BLK * rows + fr;
  const float fac = more && mine && m != -INFINITY ? ex2(*top - m) : 0.f;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t v[32];
    tm_ld32(v, tm_o + 32 * c);
    tm_wait_ld(v);
    float4* at = reinterpret_cast<float4*>(place) + (int64_t)8 * c * rows + fr;
    if (more && mine) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float4 t = at[(int64_t)k * rows];
        const float old[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * k + i] = __float_as_uint(fmaf(old[i], fac, __uint_as_float(v[4 * k + i])));
      }
    }
    if (back) {
      tm_st32(tm_o + 32 * c, v);
    } else if (mine) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        at[(int64_t)k * rows] = make_float4(__uint_as_float(v[4 * k]), __uint_as_float(v[4 * k + 1]),
                                            __uint_as_float(v[4 * k + 2]), __uint_as_float(v[4 * k + 3]));
    }
  }
  if (back)
    tm_wait_st();
  else if (mine)
    *top = m;
}

template <bool LOW, bool Q4>
__device__ void softmax(const AttnArgs& a, uint8_t* ring, Aux* x) {
  const int slot = (threadIdx.x >> 7) - 1, r = threadIdx.x & 127, warp = r >> 5;
  const uint32_t tm = x->tmem + ((uint32_t)warp << 21);
  const uint32_t tm_s = tm + slot * kTile, tm_o = tm + 2 * kTile + slot * CAS_BLK;
  uint32_t base = 0, ns = 0, no = 0, nm = 0, nb = 0;  // base: tiles of the units before
  bool pending = false;  // the other slot may still read this slot's O
  Unit w;
  if (!take_unit(0, x, w) || (w.flags & kNone)) return;
  for (uint32_t u = 0;; ++u) {
    const bool two = w.rows > kTile;  // both slots share the key tiles
    // this thread's row: the last position it sees (-1: none)
    const int fr = two ? slot * kTile + r : r;
    const bool mine = fr < w.rows;
    const int f = w.f0 + (mine ? fr : w.rows - 1), tok = div_g(a, f);
    const int lim = max(0, min(w.kv_end, w.pos0 + tok + 1)) - 1;
    const bool busy = __any_sync(CAS_FULL, mine);
    float m = -INFINITY, l = 0.f, l_fold = 0.f;
    int done = 0;
    auto folds = [&](bool more, bool back) {
      fold(a, two || slot == 0, w.flags & kFirst, fr, mine, tm_o, m, more, back);
      l_fold += l;
      l = 0.f;
    };
    const int step = two ? 1 : 2;
    for (int j = two ? 0 : slot; j < w.n;) {
      if (__builtin_expect(done > 0, 0)) {  // (the product before a tile's S is complete when S is)
        if (!wait(&x->s_full[slot], ns & 1, x)) return;
        tc_fence_after();
        if (busy) folds(done > kFold, false);
      }
      for (const int end = min(w.n, j + kFold * step); j < end; j += step) {
        const int key0 = (w.t0 + j) * kTile;
        if (!Q4 && (slot == 0 || !two) && (key0 + kTile > w.kv_end || guards(w, key0))) {
          if (!guard_values(w, u, slot, key0, 2 * (base + j) + 1, ring, x)) return;
        }
        if (!wait(&x->s_full[slot], ns++ & 1, x)) return;
        tc_fence_after();
        if (busy) {
          uint32_t s[kTile];
          tm_ld32(s, tm_s);
          tm_ld32(s + 32, tm_s + 32);
          tm_wait_ld(s);
          tm_wait_ld(s + 32);
          tm_ld32(s + 64, tm_s + 64);
          tm_ld32(s + 96, tm_s + 96);
          const bool edge = __any_sync(CAS_FULL, key0 + kTile - 1 > lim);
          const int last = lim - key0;
          if (edge) {
#pragma unroll
            for (int c = 0; c < 64; ++c)
              if (c > last) s[c] = 0xFF800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 64; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
          tm_wait_ld(s + 64);
          tm_wait_ld(s + 96);
          if (edge) {
#pragma unroll
            for (int c = 64; c < kTile; ++c)
              if (c > last) s[c] = 0xFF800000u;
          }
#pragma unroll
          for (int c = 64; c < kTile; c += 8)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx[k] = max3(mx[k], __uint_as_float(s[c + 2 * k]), __uint_as_float(s[c + 2 * k + 1]));
          const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]) * kScaleLog2;
          const bool grow = mine && top > m + 8.f;
          if (done == 0) {
            m = top;
          } else if (__any_sync(CAS_FULL, grow)) {
            // rescale O
            const float fac = grow ? ex2(m - top) : 1.f;
            if (grow) m = top;
            l *= fac;
            l_fold *= fac;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t v[32];
              tm_ld32(v, tm_o + 32 * c);
              tm_wait_ld(v);
#pragma unroll
              for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * fac);
              tm_st32(tm_o + 32 * c, v);
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          // (what is expected lies in the loop: one token over 32K 40.8 us, 41.8 the other way round)
          if (__builtin_expect(__any_sync(CAS_FULL, fabsf(ref) > kFar), 0))
            l += LOW && !two ? weigh_far_keys<LOW>(ref, tm_s, last) : weigh_far_keys<false>(ref, tm_s, last);
          else if (LOW && __builtin_expect(!two, 1))
            l += weigh_keys<true>(s, ref, tm_s);
          else
            l += weigh_keys<false>(s, ref, tm_s);
          tm_wait_st();
        }
        ++done;
        tc_fence_before();
        if (pending) {
          if (!wait(&x->merged, (nm - 1) & 1, x)) return;
          pending = false;
        }
        arrive_warp(&x->p_full[slot]);
      }
    }
    base += w.n;
    // ---- epilogue
    if (pending) {  // (no tile was this slot's)
      if (!wait(&x->merged, (nm - 1) & 1, x)) return;
      pending = false;
    }
    if (done > 0) {
      if (!wait(&x->o_full[slot], no++ & 1, x)) return;
      tc_fence_after();
      if (__builtin_expect(busy && done > kFold, 0)) {
        folds(true, true);
        l = l_fold;
      }
    }
    float w0 = 1.f, w1 = 0.f;  // weights of the two slots' outputs
    int c0 = 0, c1 = 4;        // 32-column chunks that this thread writes
    if (!two) {
      x->m[slot][r] = m;
      x->l[slot][r] = l;
      tc_fence_before();
      arrive_warp(&x->merge);
      if (!wait(&x->merge, nm & 1, x)) return;
      tc_fence_after();
      const bool other = w.n > 1;  // slot 1 had tiles
      const float mb = other ? x->m[1][r] : -INFINITY;
      const float top = fmaxf(x->m[0][r], mb), ref = top == -INFINITY ? 0.f : top;
      w0 = ex2(x->m[0][r] - ref);
      w1 = ex2(mb - ref);
      l = x->l[0][r] * w0 + (other ? x->l[1][r] * w1 : 0.f);
      m = top;
      c0 = 2 * slot;
      c1 = c0 + 2;
    }
    const bool spoilt = *(volatile int*)&x->any_bad[u & 1];  // (the tiles' products follow the look at their values)
    if (busy) {
      const bool whole = w.flags & kWhole;
      const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      float* part = a.ws + (int64_t)(2 * blockIdx.x + (w.flags & kFirst ? 0 : 1)) * a.piece_rows * kPieceFloats;
      uint16_t* out = a.o + ((int64_t)(w.start + tok) * a.Hq + w.hk * a.G + (f - tok * a.G)) * CAS_BLK;
      const uint32_t o0 = two ? tm_o : tm + 2 * kTile;
#pragma unroll 1
      for (int c = c0; c < c1; ++c) {
        uint32_t v[32];
        tm_ld32(v, o0 + 32 * c);
        tm_wait_ld(v);
        if (!two && w.n > 1) {
          uint32_t t[32];
          tm_ld32(t, o0 + CAS_BLK + 32 * c);
          tm_wait_ld(t);
#pragma unroll
          for (int k = 0; k < 32; ++k)
            v[k] = __float_as_uint(__uint_as_float(v[k]) * w0 + __uint_as_float(t[k]) * w1);
        }
        if (!mine) continue;
        if (whole) {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            v[k] = pack_bf16x2(__uint_as_float(v[2 * k]) * inv, __uint_as_float(v[2 * k + 1]) * inv);
          store32(out + 32 * c, v, a.wide);
          store32(out + 32 * c + 16, v + 8, a.wide);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(part + ((int64_t)(8 * c + k) * a.piece_rows + fr) * 4) =
                make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          if (c == 0) {
            part[(int64_t)CAS_BLK * a.piece_rows + fr] = m;
            part[(int64_t)(CAS_BLK + 1) * a.piece_rows + fr] = l;
          }
        }
      }
      if (spoilt && mine) {
#pragma unroll 1
        for (int d = 32 * c0; d < 32 * c1; ++d)
          if (lim >= 0 && lim - w.first_pos >= (int)x->bad[u & 1][d]) {
            if (whole)
              out[d] = 0x7FC0;
            else
              part[((int64_t)(d >> 2) * a.piece_rows + fr) * 4 + (d & 3)] = __uint_as_float(0x7FC00000u);
          }
      }
    }
    tc_fence_before();
    if (spoilt) {  // clean for the next unit, when all have read it
      arrive_warp(&x->spoilt);
      if (!wait(&x->spoilt, nb++ & 1, x)) return;
      if (slot == 0) x->bad[u & 1][r] = 0xFFFF;
      x->any_bad[u & 1] = 0;
      arrive_warp(&x->spoilt);
      if (!wait(&x->spoilt, nb++ & 1, x)) return;
    }
    if (slot == 1) arrive_warp(&x->seen[u & 1]);
    if (!two) {  // both slots' O, m and l are read before either is written again
      arrive_warp(&x->merged);
      ++nm;
      pending = true;
    }
    if (w.flags & kLast) return;
    if (!take_unit(u + 1, x, w)) return;
  }
}

template <bool LOW, bool Q4>
__global__ void __launch_bounds__(Q4 ? kThreads4 : kThreads, 1)
    paged_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap km,
                      const __grid_constant__ CUtensorMap vm, const __grid_constant__ CUtensorMap qm) {
  extern __shared__ __align__(1024) uint8_t q_sm[];
  uint8_t* ring = q_sm + 2 * kBuf;
  Aux* x = reinterpret_cast<Aux*>(ring + kRing * kBuf);
  const int warp = threadIdx.x >> 5;
  if (smem_u32(q_sm) & 1023) {  // swizzled tiles need it; dynamic shared memory starts there
    if (threadIdx.x == 0) {
      atomicExch(&g_attn_status, CAS_ERR_CUDA);
      a.cuts[blockIdx.x] = Cut{};
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&x->kv_full[i], Q4 ? 4 : 1);
      mbar_init(&x->kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x->u_full[i], 1);
      mbar_init(&x->u_empty[i], Q4 ? 13 : 11);  // eight softmax warps, two producers or four decoders, the issuer
      mbar_init(&x->q_full[i], 1);
      mbar_init(&x->q_empty[i], 1);
      mbar_init(&x->s_full[i], 1);
      mbar_init(&x->p_full[i], 4);
      mbar_init(&x->o_full[i], 1);
      mbar_init(&x->seen[i], 4);
    }
    mbar_init(&x->merge, 8);
    mbar_init(&x->merged, 8);
    mbar_init(&x->spoilt, 8);
    mbar_init(&x->drain, 1);
    x->abort = x->any_bad[0] = x->any_bad[1] = 0;
    x->cut = Cut{};
    fence_mbar_init();
    fence_async_smem();
  }
  if (!Q4 && warp == 1) tma_prefetch_map(&km);
  if (!Q4 && warp == 2) tma_prefetch_map(&vm);
  if (warp == 3 && a.q_box) tma_prefetch_map(&qm);
  if (threadIdx.x >= 128 && threadIdx.x < 128 + 2 * CAS_BLK) x->bad[0][threadIdx.x - 128] = 0xFFFF;
  if (warp == 0) tm_alloc(&x->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  pdl_trigger();
  if (Q4 && warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<Q4>::kDecode));
    decoder(a, ring, x);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<Q4>::kSoftmax));
    softmax<LOW, Q4>(a, ring, x);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<Q4>::kOther));
    if (Q4 && (warp == 1 || warp == 2))
      ;
    else if (warp == 1)
      producer<false>(a, &km, ring, x);
    else if (warp == 2)
      producer<true>(a, &vm, ring, x);
    else if (warp == 0)
      issuer<LOW>(smem_u32(q_sm), smem_u32(ring), x);
    else
      scheduler(a, &qm, q_sm, x);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tm_free(x->tmem, 512);
  if (threadIdx.x == 0) {
    x->cut.ok = !x->abort;
    a.cuts[blockIdx.x] = x->cut;
  }
}
constexpr size_t kSmem = (2 + kRing) * (size_t)kBuf + sizeof(Aux);
static_assert(kSmem <= 232448, "shared memory of a CTA");

// ---------------------------------------------------------------- host
// (d, slot, head, page) of a pool, boxes of 64 dimensions x min(page, 128) slots, 128-byte swizzle.
bool make_map(CUtensorMap* m, const cas_paged_kv* kv, uint16_t* pool) {
  const cuuint64_t dims[4] = {CAS_BLK, (cuuint64_t)kv->page_size, (cuuint64_t)kv->n_kv_heads, (cuuint64_t)kv->n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)kv->token_stride * 2, (cuuint64_t)kv->head_stride * 2,
                                 (cuuint64_t)kv->page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(kv->page_size, kTile), 1, 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// (d, head, token) of q, boxes of 64 dimensions x G heads x 128 / G tokens: 128 flat rows.
bool make_q_map(CUtensorMap* m, const uint16_t* q, int rows, int Hq, int G) {
  const cuuint64_t dims[3] = {CAS_BLK, (cuuint64_t)Hq, (cuuint64_t)rows};
  const cuuint64_t strides[2] = {CAS_BLK * 2, (cuuint64_t)Hq * CAS_BLK * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)(kTile / G)};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t*>(q), dims, strides, box,
                      CU_TENSOR_MAP_SWIZZLE_128B);
}

int piece_rows(int rows, int Hq, int Hkv) {
  const int64_t flat = (int64_t)std::max(rows, 1) * (Hq / std::max(Hkv, 1));
  return (int)std::min<int64_t>(kUnit, (flat + 31) / 32 * 32);
}

// The rest of the arguments, the launch and that of the join.
template <class K>
int launch_attn(K kernel, int threads, AttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, const uint16_t* q, int Hq, int Hkv,
                uint16_t* o, void* workspace, cudaStream_t st) {
  const int grid = sm_count();
  a.q = q;
  a.o = o;
  a.cuts = (Cut*)workspace;
  a.ctas = grid;
  a.ws = (float*)((uint8_t*)workspace + cuts_bytes(grid));
  set_group(a, Hq, Hkv);
  a.wide = ((uintptr_t)o & 31) == 0;
  a.piece_rows = piece_rows(a.d.rows, Hq, Hkv);
  a.ws1 = a.ws + (int64_t)2 * grid * a.piece_rows * kPieceFloats;
  a.q_box = kTile % a.G == 0;
  CUtensorMap qm{};
  if (a.q_box && !make_q_map(&qm, q, a.d.rows, Hq, a.G)) return CAS_ERR_CUDA;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem) != cudaSuccess)
    return CAS_ERR_CUDA;
  if (const int e = launch_k(kernel, grid, threads, kSmem, st, a, km, vm, qm)) return e;
  if (grid < 2) return CAS_OK;
  // directly behind our own kernel: its launch may overlap that kernel's tail
  // (pieces of 256 rows: two items a thread; of few rows: all in flight together)
  return launch_with(true, attn_join_kernel<256, 5>, dim3(grid - 1, a.piece_rows > 128 ? 16 : 8), 256, 0, st, (JoinArgs)a);
}

}  // namespace

int attn_wait_status(bool clear) {
  int s = 0;
  if (cudaMemcpyFromSymbol(&s, g_attn_status, sizeof(s)) != cudaSuccess) return CAS_ERR_CUDA;
  if (s && clear) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_attn_status, &z, sizeof(z)) != cudaSuccess) return CAS_ERR_CUDA;
  }
  return s;
}

int set_attn_spins(uint32_t n) {
  return cudaMemcpyToSymbol(c_attn_spins, &n, sizeof(n)) == cudaSuccess ? CAS_OK : CAS_ERR_CUDA;
}

}  // namespace cas

using namespace cas;

extern "C" uint64_t cas_paged_attn_workspace_bytes(int rows, int n_q_heads, int n_kv_heads) {
  if (rows < 1 || n_q_heads < 1 || n_kv_heads < 1) return 16;
  const int64_t g = sm_count(), r = piece_rows(rows, n_q_heads, n_kv_heads);
  return cuts_bytes((int)g) + g * (2 * r + std::min<int64_t>(r, kTile)) * kPieceFloats * 4;
}

extern "C" int cas_paged_attn(const cas_paged_kv* kv, const cas_paged_batch* b, const uint16_t* q, int n_q_heads,
                              uint16_t* o, void* workspace, uint64_t workspace_bytes, void* stream) {
  const int s = check_paged(kv, b);
  if (s) return s;
  if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % kv->n_kv_heads) return CAS_ERR_INVALID;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o)) return CAS_ERR_INVALID;
  if ((int64_t)b->rows * n_q_heads > 0x7FFFFFFF - kUnit) return CAS_ERR_INVALID;
  // o may be q: a row is written when all CTAs that need its q are through with it, by the CTA that takes
  // its unit whole or by the join, and what a Q tile holds of other units' rows is not used
  const uint64_t n = (uint64_t)b->rows * n_q_heads * CAS_BLK * sizeof(uint16_t);
  const uint64_t qa = (uint64_t)(uintptr_t)q, oa = (uint64_t)(uintptr_t)o;
  if (qa != oa && qa < oa + n && oa < qa + n) return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < cas_paged_attn_workspace_bytes(b->rows, n_q_heads, kv->n_kv_heads))
    return CAS_ERR_BUFFER;
  AttnArgs a{};
  a.d = make_paged_dev(kv, b);
  CUtensorMap km, vm;
  if (!make_map(&km, kv, kv->k) || !make_map(&vm, kv, kv->v)) return CAS_ERR_CUDA;
  // few rows a sequence on average: bound by the traffic
  const bool low = (int64_t)b->rows * (n_q_heads / kv->n_kv_heads) <= (int64_t)kTile * b->batch;
  return launch_attn(low ? paged_attn_kernel<true, false> : paged_attn_kernel<false, false>, kThreads, a, km, vm, q,
                     n_q_heads, kv->n_kv_heads, o, workspace, (cudaStream_t)stream);
}

namespace cas {
// Attention of cas_paged4_attn over long chunks, whose checks that call has made.
int paged4_attn_long(const cas_paged4_kv* kv, const cas_paged_batch* b, const uint16_t* q, int n_q_heads, uint16_t* o,
                     void* workspace, cudaStream_t st) {
  AttnArgs a{};
  a.d = make_paged_dev(kv, b);
  const CUtensorMap none{};
  return launch_attn(paged_attn_kernel<false, true>, kThreads4, a, none, none, q, n_q_heads, kv->n_kv_heads, o, workspace, st);
}
}  // namespace cas
