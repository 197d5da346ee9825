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
//   warps 0-3, 4-7  softmax of slot 0, 1: S from tensor memory (a row a
//                   thread), P back as bf16, O rescaled there when a row's
//                   maximum grows by more than 2^8 (probabilities relative to
//                   an older maximum are as exact), epilogue
//   warp 8          TMA: K and V tiles from their pages, five 32 KB buffers
//   warp 9          one thread issues tcgen05.mma: S = Q K^T (both from shared memory), O += P V
//                   (P from tensor memory, V with the head dimension contiguous);
//                   warps 10-11 complete its warpgroup and only give up registers
//
// Rounding: scores, statistics and sums are fp32; P is rounded to bf16 for the
// product with V (2^-8 relative each, the size of the output's own rounding),
// the sum takes it unrounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "mma.cuh"
#include "paged.cuh"
#include "tc05.cuh"

namespace cas {
namespace {

constexpr int kTile = 128;                 // keys a tile, rows a slot
constexpr int kUnit = 2 * kTile;           // flat rows a unit
constexpr int kRing = 5;                   // K / V buffers
constexpr uint32_t kBuf = kTile * 256;     // bytes of a K or V tile
constexpr uint32_t kHalf = kBuf / 2;       // 64 of the 128 dimensions
constexpr int kThreads = 384;               // three warpgroups of 168 registers a thread at launch
constexpr int kRegsSoftmax = 216, kRegsOther = 72;  // 2 * 216 + 72 = 3 * 168: the softmax keeps a row of S
constexpr int kMinTiles = 4;               // tiles a CTA takes at least
constexpr uint32_t kSpins = 1u << 20;
constexpr int64_t kPieceFloats = kTile + 2;  // a row of a partial result: output, maximum, sum

__device__ int g_attn_status = 0;

struct AttnArgs {
  PagedDev d;
  const uint16_t* q;
  uint16_t* o;
  float* ws;  // [2 * grid][piece_rows] rows of 128 + 2 floats
  int Hq, G, piece_rows;
};

// ---------------------------------------------------------------- the line of tiles
struct Seq {
  int start, T, len, R;  // first row, rows, tokens in the cache, flat rows
  int cap;               // positions that the block table holds
};
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
  const SeqSpan s = seq_span(a.d, b);
  Seq q;
  q.start = s.start;
  q.T = s.end - s.start;
  q.len = s.len;
  q.R = q.T * a.G;
  q.cap = (int)min((int64_t)0x7FFFFF00, (int64_t)a.d.max_pages << a.d.shift);
  return q;
}
__device__ __forceinline__ int unit_count(const Seq& s) { return (s.R + kUnit - 1) / kUnit; }
// key tiles of unit qt: up to the position of its last row; one (masked) tile at least
__device__ __forceinline__ int unit_tiles(const Seq& s, int G, int qt) {
  const int tok = (min(s.R, (qt + 1) * kUnit) - 1) / G;
  const int64_t seen = min((int64_t)s.cap, (int64_t)s.len - s.T + tok + 1);
  return seen <= 0 ? 1 : (int)((seen + kTile - 1) / kTile);
}
// Tiles of one kv head of sequences b0 + lane (warp-wide call).
__device__ int64_t head_tiles(const AttnArgs& a, int b, int lane) {
  Seq s{};
  int nq = 0;
  if (b < a.d.batch) {
    s = seq_of(a, b);
    nq = unit_count(s);
  }
  int64_t sum = 0;
  if (nq <= 4)
    for (int i = 0; i < nq; ++i) sum += unit_tiles(s, a.G, i);
  unsigned big = __ballot_sync(CAS_FULL, nq > 4);
  while (big) {  // long chunks: the warp counts one together
    const int src = __ffs(big) - 1;
    big &= big - 1;
    const int bb = __shfl_sync(CAS_FULL, b, src);
    const Seq t = seq_of(a, bb);
    const int n = unit_count(t);
    int part = 0;
    for (int i = lane; i < n; i += 32) part += unit_tiles(t, a.G, i);
    part = warp_sum(part);
    if (lane == src) sum = part;
  }
  return sum;
}

struct Place {
  int b, hk, qt, tile;  // unit and its key tile
  int64_t unit0;        // the unit's first tile on the line
};
struct Line {
  int64_t total, per;  // tiles of all units, tiles a CTA takes
};

// Warp-wide: the line's length, and the place of tile `c * per` on it (false
// when the line is shorter).
__device__ bool find_place(const AttnArgs& a, int64_t c, int grid, Line& line, Place& p) {
  const int lane = threadIdx.x & 31;
  int64_t total = 0, first = 0;
  for (int b0 = 0; b0 < a.d.batch; b0 += 32) {
    int64_t t = head_tiles(a, b0 + lane, lane) * a.d.H;
    if (b0 == 0) first = t;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) t += __shfl_xor_sync(CAS_FULL, t, d);
    total += t;
  }
  line.total = total;
  line.per = max((int64_t)kMinTiles, (total + grid - 1) / grid);
  const int64_t want = c * line.per;
  if (want >= total) return false;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.d.batch; b0 += 32) {
    const int64_t t = b0 == 0 ? first : head_tiles(a, b0 + lane, lane) * a.d.H;
    int64_t incl = t;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t u = __shfl_up_sync(CAS_FULL, incl, d);
      if (lane >= d) incl += u;
    }
    const unsigned hit = __ballot_sync(CAS_FULL, base + incl > want);
    if (hit) {
      const int src = __ffs(hit) - 1;
      const int64_t before = base + __shfl_sync(CAS_FULL, incl - t, src);
      const int64_t per_head = __shfl_sync(CAS_FULL, t, src) / a.d.H;
      p.b = b0 + src;
      const int64_t rem = want - before;
      p.hk = (int)(rem / per_head);
      int64_t left = rem - p.hk * per_head;
      p.unit0 = before + p.hk * per_head;
      const Seq s = seq_of(a, p.b);
      const int nq = unit_count(s);
      for (int q0 = 0; q0 < nq; q0 += 32) {
        const int n = q0 + lane < nq ? unit_tiles(s, a.G, q0 + lane) : 0;
        const int up = warp_incl_add(n, lane);
        const unsigned in = __ballot_sync(CAS_FULL, up > left);
        if (in) {
          const int w = __ffs(in) - 1;
          const int below = __shfl_sync(CAS_FULL, up - n, w);
          p.qt = q0 + w;
          p.tile = (int)(left - below);
          p.unit0 += below;
          return true;
        }
        const int all = __shfl_sync(CAS_FULL, up, 31);
        left -= all;
        p.unit0 += all;
      }
      return false;  // not reached: the unit lies in the sequence
    }
    base += __shfl_sync(CAS_FULL, incl, 31);
  }
  return false;
}

// The units of a CTA's piece of the line, walked by every warp in step.
struct Walk {
  int b, hk, qt;
  int t0, n, all;  // first tile, tiles taken here, tiles of the unit
  int64_t left;    // tiles of the piece from this unit on
  Seq s;
  bool first;
  __device__ __forceinline__ void set(const AttnArgs& a) {
    all = unit_tiles(s, a.G, qt);
    n = (int)min((int64_t)(all - t0), left);
  }
  __device__ __forceinline__ void begin(const AttnArgs& a, const Place& p, int64_t tiles) {
    b = p.b, hk = p.hk, qt = p.qt, t0 = p.tile, left = tiles, first = true;
    s = seq_of(a, b);
    set(a);
  }
  __device__ __forceinline__ bool next(const AttnArgs& a) {
    left -= n;
    if (left <= 0) return false;
    first = false;
    t0 = 0;
    if (++qt >= unit_count(s)) {
      qt = 0;
      if (++hk >= a.d.H) {
        hk = 0;
        do {
          if (++b >= a.d.batch) return false;
          s = seq_of(a, b);
        } while (s.R == 0);
      }
    }
    set(a);
    return true;
  }
  __device__ __forceinline__ int rows() const { return min(kUnit, s.R - qt * kUnit); }
  __device__ __forceinline__ bool shared() const { return rows() > kTile; }  // both slots share the key tiles
};

// ---------------------------------------------------------------- shared memory
struct Aux {
  uint64_t kv_full[kRing], kv_empty[kRing], q_full, s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int abort, any;
  Place place;
  int64_t tiles;
};

__device__ __forceinline__ bool wait_slow(uint64_t* bar, uint32_t phase, volatile int* abort) {
  for (uint32_t i = 0; i < kSpins; ++i) {
    if (mbar_try_wait(bar, phase)) return true;
    if ((i & 63) == 63 && *abort) return false;
  }
  *abort = 1;
  atomicExch(&g_attn_status, CAS_ERR_TIMEOUT);
  return false;
}
// A wait that gave up marks the CTA; its threads then run through their loops
// without waiting, computing or writing, so that all reach the end.
__device__ __forceinline__ void wait_or_die(uint64_t* bar, uint32_t phase, Aux* x, bool& dead) {
  if (!dead && !mbar_try_wait(bar, phase)) dead = !wait_slow(bar, phase, &x->abort);
}

// Ring position of K and V tile j of n: K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ uint32_t k_item(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ uint32_t v_item(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

// ---------------------------------------------------------------- the roles
__device__ void producer(const AttnArgs& a, const CUtensorMap* km, const CUtensorMap* vm, uint8_t* ring, Aux* x,
                         const Place& place, int64_t tiles) {
  const int lane = threadIdx.x & 31;
  const int shift = min(a.d.shift, 7);  // log2 of tokens a box
  const int boxes = kTile >> shift;     // boxes a tile
  uint32_t base = 0, issued = 0;
  bool dead = false;
  Walk w;
  w.begin(a, place, tiles);
  do {
    // page and slot of this lane's box of tile j; pages past the last token and bad ids load zeros
    const int seen = (int)min((int64_t)w.s.cap, (int64_t)w.s.len);
    auto page_at = [&](int j) -> int {
      const int64_t tok = (int64_t)(w.t0 + j) * kTile + ((int64_t)lane << shift);
      if (lane >= boxes || j >= w.n || tok >= seen) return -1;
      return (int)page_of(a.d, w.b, tok);
    };
    auto load = [&](const CUtensorMap* map, uint32_t item, int j, int page) {
      const uint32_t it = base + item, slot = it % kRing;
      wait_or_die(&x->kv_empty[slot], ((it / kRing) & 1) ^ 1, x, dead);
      dead = __any_sync(CAS_FULL, dead);
      if (dead) return;
      issued = it + 1;
      if (lane == 0) mbar_arrive_tx(&x->kv_full[slot], kBuf);
      __syncwarp();
      if (lane < boxes) {
        const int in_page = (int)(((int64_t)(w.t0 + j) * kTile + (lane << shift)) & ((1 << a.d.shift) - 1));
        uint8_t* dst = ring + slot * kBuf + ((uint32_t)lane << shift) * 128;
        const int pg = page >= 0 ? page : (int)a.d.n_pages;
        tma_load_4d(dst, map, 0, in_page, w.hk, pg, &x->kv_full[slot]);
        tma_load_4d(dst + kHalf, map, 64, in_page, w.hk, pg, &x->kv_full[slot]);
      }
    };
    int prev = -1, cur = page_at(0), nxt = page_at(1);
    for (int j = 0; j < w.n; ++j) {
      load(km, k_item(j), j, cur);
      if (j > 0) load(vm, v_item(j - 1, w.n), j - 1, prev);
      prev = cur;
      cur = nxt;
      nxt = page_at(j + 2);
    }
    load(vm, v_item(w.n - 1, w.n), w.n - 1, prev);
    base += 2 * w.n;
  } while (w.next(a));
  if (dead)  // copies in flight land before the block ends
    for (uint32_t it = issued > kRing ? issued - kRing : 0; it < issued; ++it)
      mbar_wait_bounded(&x->kv_full[it % kRing], (it / kRing) & 1, kSpins);
}

__device__ void issuer(const AttnArgs& a, uint32_t q_sm, uint32_t ring_sm, Aux* x, const Place& place, int64_t tiles) {
  const uint32_t tm = x->tmem;
  constexpr uint32_t id_s = tc_idesc_bf16(kTile, kTile, false), id_o = tc_idesc_bf16(kTile, CAS_BLK, true);
  uint32_t base = 0, np[2] = {0, 0}, unit = 0;
  bool dead = false;
  auto wait_kv = [&](uint32_t item) {
    const uint32_t it = base + item;
    wait_or_die(&x->kv_full[it % kRing], (it / kRing) & 1, x, dead);
  };
  auto free_kv = [&](uint32_t item) {
    if (!dead) tc_commit(&x->kv_empty[(base + item) % kRing]);
  };
  auto mma_s = [&](int slot, uint32_t q_tile, uint32_t item) {
    if (dead) return;
    const uint32_t kb = ring_sm + ((base + item) % kRing) * kBuf, qb = q_sm + q_tile * kBuf;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t off = (k >> 2) * kHalf + (k & 3) * 32;
      tc_mma_ss(tm + slot * kTile, tc_desc(qb + off, 16, 1024), tc_desc(kb + off, 16, 1024), id_s, k > 0);
    }
    tc_commit(&x->s_full[slot]);
  };
  auto mma_o = [&](int slot, uint32_t item, bool add) {
    if (dead) return;
    const uint32_t vb = ring_sm + ((base + item) % kRing) * kBuf;
    tc_fence_after();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      tc_mma_ts(tm + 2 * kTile + slot * CAS_BLK, tm + slot * kTile + 8 * k, tc_desc(vb + k * 2048, kHalf, 1024), id_o,
                add || k > 0);
  };
  auto wait_p = [&](int slot) { wait_or_die(&x->p_full[slot], np[slot]++ & 1, x, dead); };
  Walk w;
  w.begin(a, place, tiles);
  do {
    wait_or_die(&x->q_full, unit++ & 1, x, dead);
    const int n = w.n;
    if (w.shared()) {
      wait_kv(k_item(0));
      mma_s(0, 0, k_item(0));
      mma_s(1, 1, k_item(0));
      free_kv(k_item(0));
      for (int j = 0; j < n; ++j) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          wait_p(i);
          if (i == 0) wait_kv(v_item(j, n));
          mma_o(i, v_item(j, n), j > 0);
          if (i == 1) free_kv(v_item(j, n));
          if (j + 1 < n) {
            if (i == 0) wait_kv(k_item(j + 1));
            mma_s(i, i, k_item(j + 1));
            if (i == 1) free_kv(k_item(j + 1));
          } else if (!dead) {
            tc_commit(&x->o_full[i]);
          }
        }
      }
    } else {
      for (int j = 0; j < min(n, 2); ++j) {
        wait_kv(k_item(j));
        mma_s(j, 0, k_item(j));
        free_kv(k_item(j));
      }
      for (int j = 0; j < n; ++j) {
        const int i = j & 1;
        wait_p(i);
        wait_kv(v_item(j, n));
        mma_o(i, v_item(j, n), j >= 2);
        free_kv(v_item(j, n));
        if (j + 2 < n) {
          wait_kv(k_item(j + 2));
          mma_s(i, 0, k_item(j + 2));
          free_kv(k_item(j + 2));
        } else if (!dead) {
          tc_commit(&x->o_full[i]);
        }
      }
    }
    base += 2 * n;
  } while (w.next(a));
  tc_commit(&x->drain);  // products in flight end before the block does
  mbar_wait_bounded(&x->drain, 0, kSpins);
}

// Scale of the scores in powers of two: log2(e) / sqrt(128).
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;

__device__ void softmax(const AttnArgs& a, uint8_t* q_sm, uint8_t* ring, Aux* x, const Place& place, int64_t tiles) {
  const int slot = threadIdx.x >> 7, r = threadIdx.x & 127, warp = r >> 5;
  const uint32_t tm = x->tmem + ((uint32_t)warp << 21);
  const uint32_t tm_s = tm + slot * kTile, tm_o = tm + 2 * kTile + slot * CAS_BLK;
  uint32_t base = 0, ns = 0, no = 0;
  bool dead = false;
  Walk w;
  w.begin(a, place, tiles);
  do {
    const bool two = w.shared();
    const int rows = w.rows();
    const int f0 = w.qt * kUnit;
    // Q: rows of 256 bytes into swizzled halves; both warpgroups load the unit's rows
    {
      const int nrow = two ? kUnit : kTile;
      for (int i = threadIdx.x; i < nrow * 16; i += 256) {
        const int row = i >> 4, c = i & 15;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (row < rows) {
          const int f = f0 + row, t = f / a.G, h = w.hk * a.G + (f - t * a.G);
          v = __ldg(reinterpret_cast<const uint4*>(a.q + ((int64_t)(w.s.start + t) * a.Hq + h) * CAS_BLK) + c);
        }
        *reinterpret_cast<uint4*>(q_sm + (row >> 7) * kBuf + (c >> 3) * kHalf + (row & 127) * 128 +
                                  (((c & 7) ^ (row & 7)) << 4)) = v;
      }
      fence_async_smem();
      mbar_arrive(&x->q_full);
    }
    // this thread's row: the last position it sees
    const int fr = two ? slot * kTile + r : r;  // row in the unit
    const bool mine = fr < rows;
    const int f = f0 + fr;
    const int64_t seen = min((int64_t)w.s.cap, (int64_t)w.s.len - w.s.T + (mine ? f / a.G : w.s.T - 1) + 1);
    const int lim = (int)max((int64_t)0, seen) - 1;  // -1: sees nothing
    const bool busy = __any_sync(CAS_FULL, mine);
    const int kv_end = (int)min((int64_t)w.s.cap, (int64_t)w.s.len);
    float m = -INFINITY, l = 0.f;
    int done = 0;
    const int j0 = two ? 0 : slot, step = two ? 1 : 2;
    for (int j = j0; j < w.n; j += step) {
      const int key0 = (w.t0 + j) * kTile;
      wait_or_die(&x->s_full[slot], ns++ & 1, x, dead);
      tc_fence_after();
      if (busy && !dead) {
        uint32_t s[kTile];
#pragma unroll
        for (int c = 0; c < 4; ++c) tm_ld32(s + 32 * c, tm_s + 32 * c);
        tm_wait_ld();
        if (__any_sync(CAS_FULL, key0 + kTile - 1 > lim)) {
          const int last = lim - key0;
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            if (c > last) s[c] = 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < kTile; c += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmaxf(fmaxf(mx[k], __uint_as_float(s[c + k])), __uint_as_float(s[c + 4 + k]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kScaleLog2;
        const bool grow = top > m + 8.f;
        if (done == 0) {
          m = top;
        } else if (__any_sync(CAS_FULL, grow)) {
          // rescale O: the product before this tile's S is complete when S is
          const float fac = grow ? ex2(m - top) : 1.f;
          if (grow) m = top;
          l *= fac;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t v[32];
            tm_ld32(v, tm_o + 32 * c);
            tm_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * fac);
            tm_st32(tm_o + 32 * c, v);
          }
        }
        const float ref = m == -INFINITY ? 0.f : m;
        float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t p[32];
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const float e0 = ex2(fmaf(__uint_as_float(s[64 * c + 2 * k]), kScaleLog2, -ref));
            const float e1 = ex2(fmaf(__uint_as_float(s[64 * c + 2 * k + 1]), kScaleLog2, -ref));
            ls[k & 1] += e0;
            ls[2 + (k & 1)] += e1;
            p[k] = pack_bf16x2(e0, e1);
          }
          tm_st32(tm_s + 32 * c, p);
        }
        l += (ls[0] + ls[1]) + (ls[2] + ls[3]);
        tm_wait_st();
      }
      ++done;
      if (key0 + kTile > kv_end && (slot == 0 || !two)) {
        // slots behind the last token may hold anything: their V rows become zeros
        const uint32_t it = base + v_item(j, w.n);
        wait_or_die(&x->kv_full[it % kRing], (it / kRing) & 1, x, dead);
        if (key0 + r >= kv_end && !dead) {
          uint4* row = reinterpret_cast<uint4*>(ring + (it % kRing) * kBuf + r * 128);
#pragma unroll
          for (int c = 0; c < 8; ++c) row[c] = row[kHalf / 16 + c] = make_uint4(0, 0, 0, 0);
        }
        fence_async_smem();
      }
      tc_fence_before();
      mbar_arrive(&x->p_full[slot]);
    }
    base += 2 * w.n;
    // ---- epilogue
    if (done > 0) {
      wait_or_die(&x->o_full[slot], no++ & 1, x, dead);
      tc_fence_after();
    }
    float w0 = 1.f, w1 = 0.f;  // weights of the two slots' outputs
    int c0 = 0, c1 = 4;        // 32-column chunks that this thread writes
    if (!two) {
      float* ml = reinterpret_cast<float*>(q_sm + kBuf);  // the second Q tile is not used here
      ml[slot * kTile + r] = m;
      ml[(2 + slot) * kTile + r] = l;
      tc_fence_before();
      named_sync(1, 256);
      tc_fence_after();
      const float ma = ml[r], mb = ml[kTile + r];
      const float top = fmaxf(ma, mb), ref = top == -INFINITY ? 0.f : top;
      w0 = ex2(ma - ref);
      w1 = w.n > 1 ? ex2(mb - ref) : 0.f;
      l = ml[2 * kTile + r] * w0 + (w.n > 1 ? ml[3 * kTile + r] * w1 : 0.f);
      m = top;
      c0 = 2 * slot;
      c1 = c0 + 2;
    }
    if (busy && !dead) {
      const bool whole = w.n == w.all;
      const float inv = whole ? (l > 0.f || l != l ? 1.f / l : 0.f) : 1.f;
      const int t = f / a.G, h = w.hk * a.G + (f - t * a.G);
      uint16_t* out = a.o + ((int64_t)(w.s.start + t) * a.Hq + h) * CAS_BLK;
      float* part = a.ws + ((int64_t)(2 * blockIdx.x + (w.first ? 0 : 1)) * a.piece_rows + fr) * kPieceFloats;
      const uint32_t o0 = two ? tm_o : tm + 2 * kTile;
      for (int c = c0; c < c1; ++c) {
        uint32_t v[32];
        tm_ld32(v, o0 + 32 * c);
        tm_wait_ld();
        if (!two) {
          if (w.n > 1) {
            uint32_t u[32];
            tm_ld32(u, o0 + CAS_BLK + 32 * c);
            tm_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; ++k)
              v[k] = __float_as_uint(__uint_as_float(v[k]) * w0 + __uint_as_float(u[k]) * w1);
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * w0);
          }
        }
        if (!mine) continue;
        if (whole) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 q;
            q.x = pack_bf16x2(__uint_as_float(v[8 * k]) * inv, __uint_as_float(v[8 * k + 1]) * inv);
            q.y = pack_bf16x2(__uint_as_float(v[8 * k + 2]) * inv, __uint_as_float(v[8 * k + 3]) * inv);
            q.z = pack_bf16x2(__uint_as_float(v[8 * k + 4]) * inv, __uint_as_float(v[8 * k + 5]) * inv);
            q.w = pack_bf16x2(__uint_as_float(v[8 * k + 6]) * inv, __uint_as_float(v[8 * k + 7]) * inv);
            *reinterpret_cast<uint4*>(out + 32 * c + 8 * k) = q;
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k)
            *reinterpret_cast<float2*>(part + 32 * c + 2 * k) =
                make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
          if (c == 0) *reinterpret_cast<float2*>(part + CAS_BLK) = make_float2(m, l);
        }
      }
    }
    tc_fence_before();
    // O of both slots, and the rows' m and l, are read before the next unit writes them;
    // Q is free too: both slots' scores are complete
    named_sync(2, 256);
    tc_fence_after();
  } while (w.next(a));
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_attn_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap km,
                      const __grid_constant__ CUtensorMap vm) {
  extern __shared__ uint8_t raw[];
  uint8_t* base = raw + (1024 - (smem_u32(raw) & 1023)) % 1024;
  uint8_t* q_sm = base;
  uint8_t* ring = base + 2 * kBuf;
  Aux* x = reinterpret_cast<Aux*>(ring + kRing * kBuf);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&x->kv_full[i], 1);
      mbar_init(&x->kv_empty[i], 1);
    }
    mbar_init(&x->q_full, 256);
    mbar_init(&x->drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&x->s_full[i], 1);
      mbar_init(&x->p_full[i], kTile);
      mbar_init(&x->o_full[i], 1);
    }
    x->abort = 0;
    fence_mbar_init();
    fence_async_smem();
  }
  if (warp == 9) tm_alloc(&x->tmem, 512);
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    Line line;
    Place p;
    const bool any = find_place(a, blockIdx.x, gridDim.x, line, p);
    if (threadIdx.x == 0) {
      x->any = any;
      x->place = p;
      x->tiles = any ? min(line.per, line.total - (int64_t)blockIdx.x * line.per) : 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (x->any) {
    const Place p = x->place;
    const int64_t tiles = x->tiles;
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      softmax(a, q_sm, ring, x, p, tiles);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
      if (warp == 8)
        producer(a, &km, &vm, ring, x, p, tiles);
      else if (threadIdx.x == 9 * 32)
        issuer(a, smem_u32(q_sm), smem_u32(ring), x, p, tiles);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tm_free(x->tmem, 512);
}
constexpr size_t kSmem = 1024 + (2 + kRing) * (size_t)kBuf + sizeof(Aux);
static_assert(kSmem <= 232448, "shared memory of a CTA");

// ---------------------------------------------------------------- joining the pieces
// Block (c, y) looks at the cut between CTA c and c + 1: if it is the first cut
// inside a unit, it merges the unit's pieces for rows 32 y to 32 y + 31.
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs a, int grid) {
  __shared__ Place sp;
  __shared__ Line sl;
  __shared__ int any;
  // row_start and kv_len are older than the attention kernel, whose start this kernel's start follows
  if (threadIdx.x < 32) {
    Line line;
    Place p;
    const bool ok = find_place(a, blockIdx.x + 1, grid, line, p);
    if (threadIdx.x == 0) sp = p, sl = line, any = ok;
  }
  pdl_wait();
  pdl_trigger();
  __syncthreads();
  if (!any) return;
  const Place p = sp;
  const int64_t per = sl.per;
  if (p.tile == 0 || (int64_t)blockIdx.x * per > p.unit0) return;  // no cut, or not the unit's first
  const Seq s = seq_of(a, p.b);
  const int64_t end = p.unit0 + unit_tiles(s, a.G, p.qt);
  const int c0 = blockIdx.x, c1 = (int)((end - 1) / per);
  const int rows = min(kUnit, s.R - p.qt * kUnit), lane = threadIdx.x & 31;
  for (int i = 0; i < 4; ++i) {
    const int fr = blockIdx.y * 32 + (threadIdx.x >> 5) * 4 + i;
    if (fr >= rows) return;
    // CTA c0 met the unit as its first one only if its piece starts with it
    auto piece = [&](int c) {
      const int which = (int64_t)c * per >= p.unit0 ? 0 : 1;
      return a.ws + ((int64_t)(2 * c + which) * a.piece_rows + fr) * kPieceFloats;
    };
    float m = -INFINITY, l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = c0; c <= c1; ++c) {
      const float* w = piece(c);
      const float pm = w[CAS_BLK], pl = w[CAS_BLK + 1];
      const float2 v0 = *reinterpret_cast<const float2*>(w + 4 * lane);
      const float2 v1 = *reinterpret_cast<const float2*>(w + 4 * lane + 2);
      const float top = fmaxf(m, pm), ref = top == -INFINITY ? 0.f : top;
      const float f = ex2(m - ref), g = ex2(pm - ref);
      l = l * f + pl * g;
      acc[0] = acc[0] * f + v0.x * g;
      acc[1] = acc[1] * f + v0.y * g;
      acc[2] = acc[2] * f + v1.x * g;
      acc[3] = acc[3] * f + v1.y * g;
      m = top;
    }
    const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
    const int f = p.qt * kUnit + fr, t = f / a.G, h = p.hk * a.G + (f - t * a.G);
    uint2 out;
    out.x = pack_bf16x2(acc[0] * inv, acc[1] * inv);
    out.y = pack_bf16x2(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(a.o + ((int64_t)(s.start + t) * a.Hq + h) * CAS_BLK + 4 * lane) = out;
  }
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  return fn;
}

// (d, slot, head, page) of a pool, boxes of 64 dimensions x min(page, 128) slots, 128-byte swizzle.
bool make_map(CUtensorMap* m, const cas_paged_kv* kv, uint16_t* pool) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {CAS_BLK, (cuuint64_t)kv->page_size, (cuuint64_t)kv->n_kv_heads, (cuuint64_t)kv->n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)kv->token_stride * 2, (cuuint64_t)kv->head_stride * 2,
                                 (cuuint64_t)kv->page_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)std::min(kv->page_size, kTile), 1, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, pool, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int piece_rows(int rows, int Hq, int Hkv) {
  const int64_t flat = (int64_t)std::max(rows, 1) * (Hq / std::max(Hkv, 1));
  return (int)std::min<int64_t>(kUnit, (flat + 31) / 32 * 32);
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

}  // namespace cas

using namespace cas;

extern "C" uint64_t cas_paged_attn_workspace_bytes(int rows, int n_q_heads, int n_kv_heads) {
  return (uint64_t)2 * sm_count() * piece_rows(rows, n_q_heads, n_kv_heads) * kPieceFloats * 4;
}

extern "C" int cas_paged_attn(const cas_paged_kv* kv, const cas_paged_batch* b, const uint16_t* q, int n_q_heads,
                              uint16_t* o, void* workspace, uint64_t workspace_bytes, void* stream) {
  const int s = check_paged(kv, b);
  if (s) return s;
  if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % kv->n_kv_heads) return CAS_ERR_INVALID;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o)) return CAS_ERR_INVALID;
  if ((int64_t)b->rows * n_q_heads > 0x7FFFFFFF - kUnit) return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < cas_paged_attn_workspace_bytes(b->rows, n_q_heads, kv->n_kv_heads))
    return CAS_ERR_BUFFER;
  AttnArgs a{};
  a.d = make_paged_dev(kv, b);
  a.q = q;
  a.o = o;
  a.ws = (float*)workspace;
  a.Hq = n_q_heads;
  a.G = n_q_heads / kv->n_kv_heads;
  a.piece_rows = piece_rows(b->rows, n_q_heads, kv->n_kv_heads);
  CUtensorMap km, vm;
  if (!make_map(&km, kv, kv->k) || !make_map(&vm, kv, kv->v)) return CAS_ERR_CUDA;
  if (occupancy((const void*)paged_attn_kernel, kThreads, kSmem) < 1) return CAS_ERR_CUDA;
  const int grid = sm_count();
  const cudaStream_t st = (cudaStream_t)stream;
  if (const int e = launch_k(paged_attn_kernel, grid, kThreads, kSmem, st, a, km, vm)) return e;
  if (grid < 2) return CAS_OK;
  // directly behind our own kernel: its launch may overlap that kernel's tail
  return launch_with(true, attn_join_kernel, dim3(grid - 1, (a.piece_rows + 31) / 32), 256, 0, st, a, grid);
}
