// p4attn.cu - the 4-bit paged cache read back, and attention of few new tokens
// a sequence over it.
//
// o = softmax(q K^T / sqrt(128)) V with K and V the values of the records
// (q4.cuh), in one pass with the running maximum and sum of the softmax. The
// work is cut as pline.cuh says: units of 8 NT flat rows, tiles of 128 keys.
//
// The products are transposed, so that keys are the long side of a tensor core
// product and few rows its short one: S^T = K Q^T and O^T = V^T P^T with
// mma.m16n8k16, 8 rows a product. The codes become fp16 in the registers that the
// product reads, and pass through shared memory once, as codes. That pipe makes 1024
// multiply-adds a clock and SM: a tile of 128 keys takes 256 of its clocks for 8 rows,
// 512 for 16 and 1024 for 32, where the tile's 18 KB take 865 of the memory. So up to 16
// rows the memory may bound it; 32 rows would have to go through tcgen05, with the keys
// on its side of 128, and through a copy of K and V as 16-bit values. That is not done.
//
// A warp takes 32 keys of a tile. In a product's A operand lane (g, t) holds rows
// g and g + 8 and the columns 2t, 2t + 1, 2t + 8, 2t + 9; which keys and dimensions
// these are is free where the other operand follows:
//   K  rows are keys; lane t's columns of all eight steps are dimensions 32t..32t+31,
//      16 bytes of codes and two scales, and Q is loaded in that order
//   V  rows are dimensions: lane g has 16g..16g+15, 8 bytes of codes and one scale of
//      each of its four keys, and two keys' halves are put side by side in a register
//   keys: row g is key g (even g) or 8 + (g + 3) % 8 (odd), row g + 8 the one after
//      it: keys of lanes that a load serves together then lie on different banks, both
//      as rows of K (16 bytes a lane) and as columns of V (8 bytes)
// movmatrix turns the probabilities from rows of S^T into columns of P^T.
//
// Warps hold the maximum, sum and output of their keys by themselves and are
// joined at a unit's end. A row's maximum is renewed when it grows by more than
// 2^8, which a vote finds.
//
// A CTA's four warps share the tiles, 32 keys each, and a few stages of them. They are
// loaded by bulk copies where a page's records of a head lie next to one another, else
// by tiled TMA, which takes rows of 144 bytes one by one.
//
// What bounds it (measured on GB300, 8 kv heads, 32 query heads):
//   one token a sequence: 61 ragged sequences of up to 8K in 66 us for 282 MB, 4.3 TB/s. Twice
//     the lengths take 114 us and four times 212: what comes on top runs at 5.7-5.9 TB/s,
//     86-88 % of the measured copy rate, at 57 % of the issue slots (310 instructions of a warp
//     for 16 keys), and 17 us are the start, the ends of units and the join. With tiled TMA 86
//     us, without the loading warp (and a CTA more an SM) 88, with bf16 operands and P in two
//     terms 86, with one CTA of 16 warps an SM 139.
//   one token over 32K: 20 us for 38 MB, 10 to the first tile and 5 for the join.
//   4 rows of 4 heads (units of 16): 32 sequences of 8K in 102 us for 302 MB, 3.0 TB/s; of 16K
//     in 179. The products' pipe is 32 % busy, the issue slots 47 %.
//   7 rows of 4 heads: units of 32 rows hold 242 registers a thread, so that two warps a
//     scheduler have to hide their products' and logic's latencies: 32 sequences of 8K in 150
//     us, 2.0 TB/s, the products' pipe 42 % busy (2 x 7 rows over 16K: 33 us). The kernel of long
//     chunks takes 10 % more for 32 x 7 rows over 16K.
//
// Every wait is bounded as in pattn.cu; a CTA whose wait gave up writes no output
// and its units' pieces are not joined.
//
// Rounding: scores, statistics and sums are fp32. The products take fp16: K and V are
// exact in it, Q times a power of two of its row as good as exact, and P has 2^-11 of
// itself, which leaves the output's distance from 64 bits at that of its own rounding (two
// bf16 terms of P, good to 2^-17, cost half a product more and the same distance). The
// tensor cores cut their sums, so a warp's O is put away every kFold tiles, into fp32
// memory where it is added with rounding.
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
int paged4_attn_long(const cas_paged4_kv* kv, const cas_paged_batch* b, const uint16_t* q, int n_q_heads, uint16_t* o,
                     void* workspace, cudaStream_t st);
namespace {

// ---------------------------------------------------------------- reading back
struct ReadArgs {
  PagedDev d;
  uint16_t *k, *v;
};
// A warp takes four heads of a row, eight lanes a head, 16 dimensions of K and V a lane. Bound by
// the chain row bounds -> page -> record (2048 rows of 8 heads 4.9 us for 10.7 MB, 14 rows 2.8).
constexpr int kReadThreads = 128;
__device__ __forceinline__ void put16(uint16_t* to, uint2 codes, uint32_t scale) {
  const Q4Bf16 q4;
  const uint32_t s2 = q4_scale2(scale), n2 = q4_offset(s2);
  reinterpret_cast<uint4*>(to)[0] = q4.word(codes.x, s2, n2);
  reinterpret_cast<uint4*>(to)[1] = q4.word(codes.y, s2, n2);
}
__global__ void __launch_bounds__(kReadThreads) paged4_read_kernel(const __grid_constant__ ReadArgs a) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, j = lane & 7, per_row = (a.d.H + 3) / 4;
  const int64_t unit = ((int64_t)blockIdx.x * kReadThreads + threadIdx.x) >> 5, row = unit / per_row;
  if (row >= a.d.rows) return;
  const int h = (int)(unit - row * per_row) * 4 + (lane >> 3);
  const int seq = seq_of_row(a.d, row, lane);
  const SeqSpan s = seq_span(a.d, seq);
  if (row < s.start || row >= s.end || h >= a.d.H) return;
  const int64_t p = (int64_t)s.len - (s.end - row), page = page_of(a.d, seq, p);
  uint2 ck = make_uint2(0, 0), cv = ck;
  uint32_t sk = 0, sv = 0;
  if (page >= 0) {
    const uint8_t* rec = a.d.rec + page * a.d.page_stride + (p & ((1 << a.d.shift) - 1)) * a.d.token_stride +
                         h * a.d.head_stride;
    ck = *reinterpret_cast<const uint2*>(rec + 8 * j);
    cv = *reinterpret_cast<const uint2*>(rec + kRecV + 8 * j);
    sk = rec[kRecKs + j];
    sv = rec[kRecVs + j];
  }
  const int64_t to = (row * a.d.H + h) * CAS_BLK + 16 * j;
  put16(a.k + to, ck, sk);
  put16(a.v + to, cv, sv);
}

// ---------------------------------------------------------------- attention of few rows
constexpr int kTile = 128;
constexpr uint32_t kStage = kTile * kRec;  // bytes of a tile's records
constexpr int kWarps = 4;                  // of a CTA that compute
constexpr int kCells = 2;                  // cells of the line for a change of units
constexpr uint32_t kSpins = 1u << 20;      // polls of a wait
constexpr int kFold = 128;                 // tiles that a warp's O adds up before it is put away

__device__ int g_p4_status = 0;
__constant__ uint32_t c_p4_spins = kSpins;  // 0 (tests): waits give up at once; 1: in every second CTA
__device__ __forceinline__ uint32_t spins() {
  return c_p4_spins == 1 ? (blockIdx.x & 1 ? 0 : kSpins) : c_p4_spins;
}

// NT: products of 8 rows side by side. A CTA has four computing warps, an SM as many
// CTAs as their registers leave room for: one changes units while the others compute. The
// smallest units leave room for a fifth warp that loads ahead, over the ends of units, too;
// with more rows the last warp that is through with a stage fills it. (2 x 7 rows over 16K
// with eight warps a CTA and a loading one: 59 us instead of 34.)
template <int NT>
struct Shape {
  static constexpr int kUnit = 8 * NT;
  static constexpr bool kLoads = NT == 1;            // a warp that loads
  static constexpr int kThreads = 32 * kWarps + (kLoads ? 32 : 0);
  // CTAs an SM, of 128, 168, 255 registers a thread. Units of 8 rows spill 48 bytes a thread, of 16 rows 40: a
  // variant with 0 and 20 took 64.4 instead of 65.3 us (61 ragged tokens) and 97.6 instead of 101.8 (32 x 4 rows
  // over 8K), but units of 32 rows, which spill nothing either way, 153 instead of 150 (32 x 7 rows).
  static constexpr int kCtas = NT == 4 ? 2 : 3;
  static constexpr int kStages = NT == 4 ? 4 : 3;
  static constexpr int kHalves = NT <= 2 ? 2 : 1;    // of 16 keys that a warp takes in a step
  static constexpr bool kQShared = NT > 2;           // Q's operands in shared memory instead of registers
  static constexpr int kFoldFloat4 = (NT * 9) * 32;  // a warp's: O, maxima
  struct Smem {
    uint8_t ring[kStages][kStage];
    float o[kWarps][8][CAS_BLK];
    uint2 q[kQShared ? NT : 1][8][32];
    int q_exp[kUnit];
    float m[kWarps][kUnit], l[kWarps][kUnit];
    uint64_t full[kStages], empty[kStages];
    uint32_t done[kStages], loads[kStages];  // warps through with a stage's tiles, tiles loaded
    uint64_t walk[12], next[4];
    int abort;
  };
  static_assert(kCtas * (sizeof(Smem) + 1024) <= 233472, "shared memory of an SM");
};
struct P4Args : JoinArgs {
  const uint16_t* q;
  float4* fold;      // [grid][warps] of kFoldFloat4
  bool whole_boxes;  // a page's records of a head lie next to one another
};

__device__ __noinline__ bool wait_long(uint64_t* bar, uint32_t phase, volatile int* abort) {
  const uint32_t limit = spins();
  for (uint32_t i = 0; i < limit && !*abort; ++i)
    if (mbar_try_wait(bar, phase)) return true;
  if (!*abort) {
    *abort = 1;
    atomicExch(&g_p4_status, CAS_ERR_TIMEOUT);
  }
  return false;
}
// Warp-wide; false when any lane gave up.
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t phase, int* abort) {
  bool ok = spins() != 0 && mbar_try_wait(bar, phase);
  if (!__all_sync(CAS_FULL, ok)) ok = ok || wait_long(bar, phase, abort);
  return __all_sync(CAS_FULL, ok);
}

// The units of a CTA, or its parts of them. One warp finds the first; then every warp
// walks them by itself, but one thread looks at the lengths of the sequences that follow
// for all computing warps: these meet at barriers whose number hangs on the units, so every
// one of them has to see the same lengths, also where a caller changes them under the
// kernel (the output then means nothing). N: what counts cells.
struct Unit {
  int b, start, hk, f0, rows;  // sequence and its first row, kv head, flat rows
  int pos0, kv_end;            // position of the sequence's first row, end of what it holds
  int t0, n, all;              // key tiles of this CTA, of the unit
  bool first, last;            // of this CTA's
};
// A sequence that has rows; b = batch: there is none.
struct NextSeq {
  int b;
  Seq s;
};
template <int NT, class N>
struct Walk {
  using L = UnitLine<Shape<NT>::kUnit, kTile, kCells, N>;
  N per, left;
  Place p;
  Seq s;
  int cell;
  bool any, first;
  __device__ __forceinline__ void begin(const LineArgs& a) {
    typename L::Line line;
    first = true;
    any = L::find_place(a, (N)blockIdx.x, gridDim.x, kCells + 1, line, p, s);
    per = line.per;
    left = min(per, line.total - (N)blockIdx.x * per);
    cell = p.cell;
  }
  __device__ __forceinline__ Unit take(const LineArgs& a) {
    Unit w;
    w.all = L::unit_tiles(s, a, p.qt);
    const int end = (int)min((N)w.all + kCells, cell + left);
    w.b = p.b, w.start = s.start, w.hk = p.hk, w.f0 = p.qt * Shape<NT>::kUnit;
    w.rows = min(Shape<NT>::kUnit, s.R - w.f0);
    w.pos0 = s.len - s.T;
    w.kv_end = min(s.cap, s.len);
    w.t0 = max(0, cell - kCells);
    w.n = max(0, end - kCells) - w.t0;
    left -= end - cell;
    w.first = first;
    w.last = left <= kCells;  // (a next unit's first cells hold no tile)
    first = false;
    cell = 0;
    return w;
  }
  // Whether the next unit lies in another sequence, and that sequence.
  __device__ __forceinline__ bool leaves(const LineArgs& a) const {
    return p.qt + 1 >= L::unit_count(s) && p.hk + 1 >= a.d.H;
  }
  __device__ __forceinline__ NextSeq look(const LineArgs& a) const {
    NextSeq n{p.b, Seq{}};
    do n.s = ++n.b < a.d.batch ? seq_of(a, n.b) : Seq{};
    while (n.s.R == 0 && n.b < a.d.batch);
    return n;
  }
  __device__ __forceinline__ void next(const LineArgs& a, const NextSeq& n) {
    if (++p.qt < L::unit_count(s)) return;
    p.qt = 0;
    if (++p.hk < a.d.H) return;
    p.hk = 0;
    p.b = n.b, s = n.s;
    any = p.b < a.d.batch;
  }
};

// A warp that loads tile j of a unit into a stage that nobody reads any more.
template <int NT>
struct Loader {
  const P4Args& a;
  const CUtensorMap* map;
  typename Shape<NT>::Smem* x;
  int lane, shift, boxes;  // log2 of tokens a box, boxes a tile
  __device__ __forceinline__ Loader(const P4Args& a_, const CUtensorMap* map_, typename Shape<NT>::Smem* x_)
      : a(a_), map(map_), x(x_), lane(threadIdx.x & 31), shift(min(a_.d.shift, 7)), boxes(kTile >> shift) {}
  // Page of this lane's box of tile j; n_pages where there is nothing to load.
  __device__ __forceinline__ int page_at(const Unit& w, int j) const {
    const uint32_t tok = (uint32_t)(w.t0 + j) * kTile + ((uint32_t)lane << shift);
    if (lane >= boxes || j >= w.n || tok >= (uint32_t)w.kv_end) return (int)a.d.n_pages;
    const int id = a.d.pages[(int64_t)w.b * a.d.max_pages + (tok >> a.d.shift)];
    return (uint32_t)id < (uint32_t)a.d.n_pages ? id : (int)a.d.n_pages;
  }
  __device__ __forceinline__ void load(const Unit& w, int j, int page, uint32_t slot) const {
    const uint32_t tok = (uint32_t)(w.t0 + j) * kTile + ((uint32_t)lane << shift);
    const int in_page = (int)(tok & ((1u << a.d.shift) - 1));
    uint8_t* dst = x->ring[slot] + ((uint32_t)lane << shift) * kRec;
    const uint32_t bytes = (uint32_t)kRec << shift;
    const bool good = lane < boxes && page < a.d.n_pages;
    if (lane == 0) ++x->loads[slot];
    if (a.whole_boxes) {  // a box is one piece of memory: plain copies of those that are there
      const unsigned some = __ballot_sync(CAS_FULL, good);
      // pages that do not exist read as zeros; what lies behind the last token is not looked at
      for (unsigned zero = __ballot_sync(CAS_FULL, lane < boxes && !good && tok < (uint32_t)w.kv_end); zero; zero &= zero - 1) {
        uint8_t* z = x->ring[slot] + ((uint32_t)(__ffs(zero) - 1) << shift) * kRec;
        for (uint32_t i = 16 * lane; i < bytes; i += 512) *reinterpret_cast<uint4*>(z + i) = make_uint4(0, 0, 0, 0);
        fence_async_smem();
      }
      __syncwarp();
      if (lane == 0) {
        if (some)
          mbar_arrive_tx(&x->full[slot], bytes * __popc(some));
        else
          mbar_arrive(&x->full[slot]);
      }
      __syncwarp();
      if (good)
        bulk_g2s(dst, a.d.rec + w.hk * a.d.head_stride + page * a.d.page_stride + in_page * kRec, bytes, &x->full[slot]);
    } else {
      if (lane == 0) mbar_arrive_tx(&x->full[slot], kStage);
      __syncwarp();
      if (lane < boxes) tma_load_4d(dst, map, 0, in_page, w.hk, page, &x->full[slot]);
    }
  }
};

template <class T>
__device__ __forceinline__ T at(const uint8_t* p, uint32_t offset) {
  return *reinterpret_cast<const T*>(p + offset);
}
// Transpose of an 8x8 matrix of 16-bit values, lane (g, t) holding row g, columns 2t and 2t + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// Place of four values of a row of O in shared memory: the eight lanes that write
// together, four rows and two chunks, take different banks.
__device__ __forceinline__ int swizzle(int row, int chunk) { return chunk ^ ((row >> 1) & 3); }
// Counts a warp that is through with a stage; how many were before it.
__device__ __forceinline__ uint32_t count_done(uint32_t* at) {
  uint32_t n;
  asm volatile("atom.acq_rel.cta.shared.add.u32 %0, [%1], 1;" : "=r"(n) : "r"(smem_u32(at)) : "memory");
  return n;
}

// Scale of the scores in powers of two: log2(e) / sqrt(128).
constexpr float kScaleLog2 = 0.08838834764831845f * 1.4426950408889634f;

// A probability relative to the maximum of then is at most 2^8; 2^7 times as much
// keeps what fp16 holds exactly down to 2^-31 of the maximum.
constexpr float kUp = 7.f;
constexpr float kNone = 3.4028234663852886e38f;

// The computing warps of a CTA, among themselves.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kWarps) : "memory"); }

__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23); }

template <int NT, class N>
__device__ void compute(const P4Args& a, const CUtensorMap* map, typename Shape<NT>::Smem* x, Walk<NT, N> walk) {
  using Sh = Shape<NT>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  const int key = (g & 1) ? 8 + ((g + 3) & 7) : g;  // of row g; row g + 8: the next
  // this lane's K codes and V codes in its warp's part of a stage
  const uint32_t at_k = (warp * 32 + key) * kRec;
  const uint32_t at_va = (warp * 32 + 2 * t) * kRec, at_vb = (warp * 32 + 8 + ((2 * t + 4) & 7)) * kRec;
  const Q4Const q4;
  uint32_t tile0 = 0;  // tiles of the units before
  const Loader<NT> loader(a, map, x);
  Cut cut{};
  bool ok = true;
  auto first_tiles = [&](const Unit& w) {
    if constexpr (!Sh::kLoads) {
      int page[Sh::kStages];
#pragma unroll
      for (int k = 0; k < Sh::kStages; ++k) page[k] = loader.page_at(w, k);
#pragma unroll
      for (int k = 0; k < Sh::kStages; ++k)
        if (k < w.n) loader.load(w, k, page[k], (tile0 + k) % Sh::kStages);
    }
  };
  while (walk.any) {
    const Unit w = walk.take(a);
    if (w.t0 == 0 && w.n > 0 && w.n < w.all) {  // the unit's first piece: its cut
      cut.pieces = 1 + (int)div64((N)(w.all - w.n) + walk.per - 1, walk.per);
      cut.start = w.start, cut.hk = w.hk, cut.f0 = w.f0, cut.rows = w.rows;
      cut.first = w.first ? 0 : 1;
    }
    if (warp == 0 && ok) first_tiles(w);  // (all warps are through with the unit before)
    // ---- Q: lane (g, t) has dimensions 32t..32t+31 of row g of each product, as fp16 and times a power of
    // two that takes the row's largest magnitude to 2^14..2^15 (what fp16 then cuts is below 2^-38 of it)
    uint32_t q[Sh::kQShared ? 1 : NT][16];
    float to_log2[NT][2];  // of rows 2t and 2t + 1
    auto load_q = [&](int nt, uint32_t* to) {
      const int f = w.f0 + 8 * nt + g, tok = div_g(a, min(f, w.f0 + w.rows - 1));
      const uint4* from = reinterpret_cast<const uint4*>(
          a.q + ((int64_t)(w.start + tok) * a.Hq + w.hk * a.G + (f - tok * a.G)) * CAS_BLK + 32 * t);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 v = 8 * nt + g < w.rows ? from[i] : make_uint4(0, 0, 0, 0);
        to[4 * i] = v.x, to[4 * i + 1] = v.y, to[4 * i + 2] = v.z, to[4 * i + 3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) top = __vmaxu2(top, to[i] & 0x7FFF7FFFu);
      int e = (int)max(top >> 23, (top >> 7) & 0xFFu);  // biased exponent of the largest
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) e = max(e, __shfl_xor_sync(CAS_FULL, e, d));
      e = max(e, 14);
      const float up = __uint_as_float((uint32_t)(127 + 14 + 127 - e) << 23);  // 2^(14 - (e - 127))
#pragma unroll
      for (int i = 0; i < 16; ++i)
        to[i] = pack_f16x2(__uint_as_float(to[i] << 16) * up, __uint_as_float(to[i] & 0xFFFF0000u) * up);
      return e - 127 - 14 + 3;  // (the keys are taken as eighths)
    };
    if (Sh::kQShared) {
      for (int nt = warp; nt < NT; nt += kWarps) {
        uint32_t v[16];
        const int e = load_q(nt, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x->q[nt][i][lane] = make_uint2(v[2 * i], v[2 * i + 1]);
        if (t == 0) x->q_exp[8 * nt + g] = e;
      }
      meet();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int e = Sh::kQShared ? 0 : load_q(nt, q[Sh::kQShared ? 0 : nt]);
#pragma unroll
      for (int c = 0; c < 2; ++c)
        to_log2[nt][c] = kScaleLog2 * exp2_int(Sh::kQShared ? x->q_exp[8 * nt + 2 * t + c]
                                                            : __shfl_sync(CAS_FULL, e, 4 * (2 * t + c)));
    }
    const int least = max(0, min(w.kv_end, w.pos0 + div_g(a, w.f0) + 1)) - 1;  // of the unit's first row
    // r: what takes a score, in powers of two, to the exponent of its probability: kUp - the maximum (without one
    // yet so large that the first score asks for it)
    float o[NT][8][4], l[NT][2], r[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < 8; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;
      r[nt][0] = r[nt][1] = kNone;
      l[nt][0] = l[nt][1] = 0.f;
    }
    float4* away = a.fold + ((int64_t)blockIdx.x * kWarps + warp) * Sh::kFoldFloat4 + lane;
    int steps = 0;
    // Adds what lies in memory, relative to the r of then, to O; `put`: and puts the sum there.
    auto fold = [&](bool more, bool put) {
#pragma unroll 1
      for (int nt = 0; nt < NT; ++nt) {
        float f0 = 0.f, f1 = 0.f, r0 = 0.f, r1 = 0.f;
#pragma unroll
        for (int k = 0; k < NT; ++k)
          if (k == nt) r0 = r[k][0], r1 = r[k][1];
        if (more) {
          const float4 was = away[(NT * 8 + nt) * 32];
          f0 = ex2(r0 - was.x);
          f1 = ex2(r1 - was.y);
        }
#pragma unroll
        for (int k = 0; k < NT; ++k)
          if (k == nt) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float* v = o[k][i];
              if (more) {
                const float4 was = away[(k * 8 + i) * 32];
                v[0] = fmaf(was.x, f0, v[0]), v[1] = fmaf(was.y, f1, v[1]);
                v[2] = fmaf(was.z, f0, v[2]), v[3] = fmaf(was.w, f1, v[3]);
              }
              if (put) {
                away[(k * 8 + i) * 32] = make_float4(v[0], v[1], v[2], v[3]);
                v[0] = v[1] = v[2] = v[3] = 0.f;
              }
            }
          }
        if (put) away[(NT * 8 + nt) * 32] = make_float4(r0, r1, 0.f, 0.f);
      }
    };
    // ---- 16 * kHalves keys of a tile: scores, softmax, values
    constexpr int kHalves = Sh::kHalves;
    auto step = [&](const uint8_t* base, int pos, bool edge) {
      float s[kHalves][NT][4];
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint8_t* kp = base + h * 16 * kRec + at_k;
        const uint4 ca = at<uint4>(kp, 16 * t), cb = at<uint4>(kp, kRec + 16 * t);
        const uint32_t sa = at<uint16_t>(kp, kRecKs + 2 * t), sb = at<uint16_t>(kp, kRec + kRecKs + 2 * t);
        const uint32_t wa[4] = {ca.x, ca.y, ca.z, ca.w}, wb[4] = {cb.x, cb.y, cb.z, cb.w};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) s[h][nt][0] = s[h][nt][1] = s[h][nt][2] = s[h][nt][3] = 0.f;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          Q4Half d(q4);  // of the lane's two keys
          d.set(__byte_perm(sa, sb, half ? 0x2521 : 0x2420));  // (byte 2 is zero)
#pragma unroll
          for (int e = 2 * half; e < 2 * half + 2; ++e)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t u = i ? wa[e] >> 8 : wa[e], v = i ? wb[e] >> 8 : wb[e];
              const uint32_t f[4] = {d.low_by<0>(u), d.low_by<1>(v), d.high_by<0>(u), d.high_by<1>(v)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                if (Sh::kQShared) {
                  const uint2 b = x->q[nt][2 * e + i][lane];
                  mma_f16(s[h][nt], f, b.x, b.y);
                } else {
                  mma_f16(s[h][nt], f, q[Sh::kQShared ? 0 : nt][4 * e + 2 * i], q[Sh::kQShared ? 0 : nt][4 * e + 2 * i + 1]);
                }
              }
            }
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // the last position that the row sees (rows that the unit does not have: any)
            const int fr = 8 * nt + 2 * t + c;
            const int lim = fr < w.rows ? max(0, min(w.kv_end, w.pos0 + div_g(a, w.f0 + fr) + 1)) - 1 : 0x7FFFFFFF;
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
              if (pos + 16 * h > lim) s[h][nt][c] = -INFINITY;
              if (pos + 16 * h + 1 > lim) s[h][nt][c + 2] = -INFINITY;
            }
          }
      }
      bool grow = false;
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          top[nt][c] = -INFINITY;
#pragma unroll
          for (int h = 0; h < kHalves; ++h) {
            // (rounded here once, so that the largest is 0 below its maximum however large it is)
            s[h][nt][c] = __fmul_rn(s[h][nt][c], to_log2[nt][c]);
            s[h][nt][c + 2] = __fmul_rn(s[h][nt][c + 2], to_log2[nt][c]);
            top[nt][c] = max3(top[nt][c], s[h][nt][c], s[h][nt][c + 2]);
          }
          grow = grow || top[nt][c] + r[nt][c] > kUp + 8.f;
        }
      if (__any_sync(CAS_FULL, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float v = top[nt][c];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) v = fmaxf(v, __shfl_xor_sync(CAS_FULL, v, d));
            if (v + r[nt][c] > kUp + 8.f) {  // (no row's renewal hangs on another's)
              const float fac = ex2(kUp - v - r[nt][c]);
              r[nt][c] = kUp - v;
              l[nt][c] *= fac;
#pragma unroll
              for (int i = 0; i < 8; ++i) o[nt][i][c] *= fac, o[nt][i][c + 2] *= fac;
            }
          }
      }
      uint32_t p[kHalves][NT][2];
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float p0 = ex2(__fadd_rn(s[h][nt][0], r[nt][0])), p1 = ex2(__fadd_rn(s[h][nt][1], r[nt][1]));
          const float p2 = ex2(__fadd_rn(s[h][nt][2], r[nt][0])), p3 = ex2(__fadd_rn(s[h][nt][3], r[nt][1]));
          l[nt][0] += p0 + p2;
          l[nt][1] += p1 + p3;
          p[h][nt][0] = transpose8(pack_f16x2(p0, p1));
          p[h][nt][1] = transpose8(pack_f16x2(p2, p3));
        }
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint8_t *pa = base + h * 16 * kRec + at_va, *pb = base + h * 16 * kRec + at_vb;
        const uint2 a0 = at<uint2>(pa, kRecV + 8 * g), b0 = at<uint2>(pb, kRecV + 8 * g);
        const uint2 a1 = at<uint2>(pa, kRec + kRecV + 8 * g), b1 = at<uint2>(pb, kRec + kRecV + 8 * g);
        const uint32_t va = at<uint8_t>(pa, kRecVs + g), vb = at<uint8_t>(pb, kRecVs + g);
        const uint32_t va1 = at<uint8_t>(pa, kRec + kRecVs + g), vb1 = at<uint8_t>(pb, kRec + kRecVs + g);
        // (what no row sees may hold any byte, but has to stay finite beside a probability of zero)
        Q4Half d0(q4), d1(q4);
        d0.set(__vminu2(va | vb << 16, kScaleMost * 0x10001u));
        d1.set(__vminu2(va1 | vb1 << 16, kScaleMost * 0x10001u));
#pragma unroll
        for (int e = 0; e < 2; ++e) {  // 8 of the lane's 16 dimensions
          const uint32_t u = e ? a0.y : a0.x, v = e ? b0.y : b0.x, y = e ? a1.y : a1.x, z = e ? b1.y : b1.x;
          uint32_t e0 = __byte_perm(u, v, 0x5410), o0 = __byte_perm(u, v, 0x7632);
          uint32_t e1 = __byte_perm(y, z, 0x5410), o1 = __byte_perm(y, z, 0x7632);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t f[4] = {i & 1 ? d0.high(e0) : d0.low(e0), i & 1 ? d0.high(o0) : d0.low(o0),
                                   i & 1 ? d1.high(e1) : d1.low(e1), i & 1 ? d1.high(o1) : d1.low(o1)};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][4 * e + i], f, p[h][nt][0], p[h][nt][1]);
            if (i == 1) e0 >>= 8, o0 >>= 8, e1 >>= 8, o1 >>= 8;
          }
        }
      }
    };
    for (int j = 0; ok && j < w.n; ++j) {
      const uint32_t turn = (tile0 + j) / Sh::kStages, slot = (tile0 + j) - turn * Sh::kStages;
      ok = wait(&x->full[slot], turn & 1, &x->abort);
      if (!ok) break;
      const int key0 = (w.t0 + j) * kTile + warp * 32;
      if (steps && steps % kFold == 0) fold(steps > kFold, true);
      ++steps;
#pragma unroll 1
      for (int h = 0; h < 2; h += kHalves)
        step(x->ring[slot] + h * 16 * kRec, key0 + 16 * h + key, key0 + 16 * (h + kHalves) - 1 > least);
      if (Sh::kLoads) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&x->empty[slot]);
      } else if (j + Sh::kStages < w.n) {  // the last warp that is through with a stage fills it
        uint32_t before = 0;
        __syncwarp();
        if (lane == 0) before = count_done(&x->done[slot]);
        if ((__shfl_sync(CAS_FULL, before, 0) & (kWarps - 1)) == kWarps - 1) loader.load(w, j + Sh::kStages, loader.page_at(w, j + Sh::kStages), slot);
      }
    }
    tile0 += w.n;
    if (steps > kFold) fold(true, false);
    // ---- join the warps
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float v = l[nt][c];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(CAS_FULL, v, d);
        if (g == 0) {
          x->m[warp][8 * nt + 2 * t + c] = r[nt][c] == kNone ? -INFINITY : -r[nt][c];
          x->l[warp][8 * nt + 2 * t + c] = v;
        }
      }
    const bool whole = w.n == w.all;
    float* part = a.ws + (int64_t)(2 * blockIdx.x + (w.first ? 0 : 1)) * a.piece_rows * kPieceFloats;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (8 * nt >= w.rows) break;  // (the same for all warps)
      if (nt > 0) meet();
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 8; i += 2)
          *reinterpret_cast<float4*>(&x->o[warp][2 * t + c][4 * swizzle(2 * t + c, 4 * g + i / 2)]) =
              make_float4(o[nt][i][c], o[nt][i][c + 2], o[nt][i + 1][c], o[nt][i + 1][c + 2]);
      meet();
      // a warp takes every kWarps-th row, a lane four of its values
#pragma unroll
      for (int row = warp; row < 8; row += kWarps) {
        const int fr = 8 * nt + row;
        if (fr >= w.rows || !ok || *(volatile int*)&x->abort) break;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) top = fmaxf(top, x->m[k][fr]);
        const float ref = top == -INFINITY ? 0.f : top;
        float sum = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float fac = ex2(x->m[k][fr] - ref);
          const float4 u = *reinterpret_cast<const float4*>(&x->o[k][row][4 * swizzle(row, lane)]);
          sum = fmaf(x->l[k][fr], fac, sum);
          v.x = fmaf(u.x, fac, v.x), v.y = fmaf(u.y, fac, v.y), v.z = fmaf(u.z, fac, v.z), v.w = fmaf(u.w, fac, v.w);
        }
        sum *= 0.125f;  // (the values are taken as eighths)
        if (whole) {
          const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
          const int f = w.f0 + fr, tok = div_g(a, f);
          uint16_t* out = a.o + ((int64_t)(w.start + tok) * a.Hq + w.hk * a.G + (f - tok * a.G)) * CAS_BLK + 4 * lane;
          *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
        } else {
          *reinterpret_cast<float4*>(part + ((int64_t)lane * a.piece_rows + fr) * 4) = v;
          if (lane == 0) {
            part[(int64_t)CAS_BLK * a.piece_rows + fr] = top;
            part[(int64_t)(CAS_BLK + 1) * a.piece_rows + fr] = sum;
          }
        }
      }
    }
    // (read behind this meeting, written behind the one of the unit's first rows)
    NextSeq& following = *reinterpret_cast<NextSeq*>(x->next);
    if (threadIdx.x == 0 && !w.last && walk.leaves(a)) following = walk.look(a);
    __syncwarp();
    meet();  // what is shared is read before the next unit's is written
    if (w.last) break;
    walk.next(a, following);
  }
  if (threadIdx.x == 0) {
    cut.ok = 1;  // (taken back where a wait gave up)
    a.cuts[blockIdx.x] = cut;
  }
}

template <int NT, class N>
__device__ void produce(const P4Args& a, const CUtensorMap* map, typename Shape<NT>::Smem* x, Walk<NT, N> walk) {
  constexpr int kStages = Shape<NT>::kStages;
  const Loader<NT> loader(a, map, x);
  uint32_t slot = 0, phase = 1;
  while (walk.any) {
    const Unit w = walk.take(a);
    int ahead[4] = {loader.page_at(w, 0), loader.page_at(w, 1), loader.page_at(w, 2), loader.page_at(w, 3)};
    for (int j = 0; j < w.n; ++j) {
      if (!wait(&x->empty[slot], phase, &x->abort)) return;
      loader.load(w, j, ahead[0], slot);
      ahead[0] = ahead[1], ahead[1] = ahead[2], ahead[2] = ahead[3];
      ahead[3] = loader.page_at(w, j + 4);
      if (++slot == kStages) slot = 0, phase ^= 1;
    }
    if (w.last) return;
    walk.next(a, walk.leaves(a) ? walk.look(a) : NextSeq{});
  }
}

template <int NT, class N>
__global__ void __launch_bounds__(Shape<NT>::kThreads, Shape<NT>::kCtas)
    paged4_attn_kernel(const __grid_constant__ P4Args a, const __grid_constant__ CUtensorMap map) {
  using Sh = Shape<NT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  auto* x = reinterpret_cast<typename Sh::Smem*>(smem);
  Walk<NT, N>& walk = *reinterpret_cast<Walk<NT, N>*>(x->walk);
  static_assert(sizeof(walk) <= sizeof(x->walk) && sizeof(NextSeq) <= sizeof(x->next), "room for the walk");
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < Sh::kStages; ++i) {
      mbar_init(&x->full[i], 1);
      mbar_init(&x->empty[i], kWarps);
      x->done[i] = x->loads[i] = 0;
    }
    x->abort = 0;
    if (!a.whole_boxes) tma_prefetch_map(&map);
    fence_mbar_init();
    fence_async_smem();
  }
  pdl_wait();
  pdl_trigger();
  if (warp == 0) {
    Walk<NT, N> mine;
    mine.begin(a);
    if ((threadIdx.x & 31) == 0) walk = mine;
  }
  __syncthreads();
  if (warp < kWarps)
    compute<NT, N>(a, &map, x, walk);
  else
    produce<NT, N>(a, &map, x, walk);
  // after a wait that gave up, copies in flight land before the block ends
  __syncthreads();
  if (*(volatile int*)&x->abort && threadIdx.x == 0) {
    for (int k = 0; k < Sh::kStages; ++k)
      if (x->loads[k]) mbar_wait_bounded(&x->full[k], (x->loads[k] - 1) & 1, kSpins);
    a.cuts[blockIdx.x].ok = 0;
  }
}

// ---------------------------------------------------------------- host
// (byte, slot, head, page) of the records, boxes of a record x min(page, 128) slots.
bool make_map(CUtensorMap* m, const cas_paged4_kv* kv) {
  const cuuint64_t dims[4] = {kRec, (cuuint64_t)kv->page_size, (cuuint64_t)kv->n_kv_heads, (cuuint64_t)kv->n_pages};
  const cuuint64_t strides[3] = {(cuuint64_t)kv->token_stride, (cuuint64_t)kv->head_stride, (cuuint64_t)kv->page_stride};
  const cuuint32_t box[4] = {kRec, (cuuint32_t)std::min(kv->page_size, kTile), 1, 1};
  return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, kv->records, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_NONE);
}

// Units of 8, 16 or 32 rows: the least that hold a sequence's flat rows on average; 0:
// more than 32, for pattn.cu's units of 256. The host knows no more than rows and
// sequences. (At the border, of 4 heads over 8K: 32 x 8 rows take 151 us here, 32 x 9 in
// units of 256 179.) What the average hides costs time, not results: a sequence far above it
// has its keys read again by every small unit, and sequences without rows lower it. 2048 rows
// over 32K take 760 us alone or beside 63 empty sequences, 3900 us beside 255 and 6300
// beside 1023; 63 single tokens over 8K with a chunk of 448 rows over 32K 1170 us, with one of 451
// (the long chunks' kernel for all) 600. A caller whose table has many empty places had better pass
// the sequences that have rows.
int units_of(int64_t flat, int64_t batch) {
  return flat <= 8 * batch ? 1 : flat <= 16 * batch ? 2 : flat <= 32 * batch ? 4 : 0;
}

template <int NT>
uint64_t workspace_of(int sms) {
  const int grid = sms * Shape<NT>::kCtas;
  return cuts_bytes(grid) + (uint64_t)grid * 2 * 8 * NT * kPieceFloats * 4 +
         (uint64_t)grid * kWarps * Shape<NT>::kFoldFloat4 * 16;
}
template <int NT>
int launch(P4Args& a, const cas_paged4_kv* kv, void* workspace, cudaStream_t st) {
  using Sh = Shape<NT>;
  static_assert(sizeof(typename Sh::Smem) <= 232448, "shared memory of a CTA");
  const int grid = sm_count() * Sh::kCtas;
  a.cuts = (Cut*)workspace;
  a.ctas = grid;
  a.ws = (float*)((uint8_t*)workspace + cuts_bytes(grid));
  a.piece_rows = 8 * NT;
  a.fold = (float4*)(a.ws + (int64_t)grid * 2 * a.piece_rows * kPieceFloats);
  a.whole_boxes = kv->token_stride == kRec;
  CUtensorMap map{};
  if (!a.whole_boxes && !make_map(&map, kv)) return CAS_ERR_CUDA;
  // cells of the line at most: units of all sequences and heads, and the tiles that the block table has room for
  const double units = (double)a.d.H * ((double)a.d.rows * a.G / Sh::kUnit + a.d.batch);
  const double tiles = (double)a.d.max_pages * (1 << a.d.shift) / kTile + 1 + kCells;
  const auto kernel = units * tiles < 2e9 ? paged4_attn_kernel<NT, int> : paged4_attn_kernel<NT, int64_t>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(typename Sh::Smem)) !=
      cudaSuccess)
    return CAS_ERR_CUDA;
  if (const int e = launch_k(kernel, grid, Sh::kThreads, sizeof(typename Sh::Smem), st, a, map)) return e;
  if (grid < 2) return CAS_OK;
  // directly behind our own kernel: its launch may overlap that kernel's tail
  // (Few units have many pieces: their values are shared out. One token over 32K in 20.0 us with four CTAs of 128
  // threads a unit, 21.1 with eight; 2 x 7 rows over 16K in 32.7 with eight of 256, 33.6 with eight of 128.)
  constexpr int kJoin = NT == 4 ? 256 : 128;
  const int shares = units < grid / 8 ? (NT == 4 ? 8 : 4) : units < 2 * grid ? 2 : 1;
  return launch_with(true, attn_join_kernel<kJoin, 1024 / kJoin>, dim3(grid - 1, shares), kJoin, 0, st, (JoinArgs)a);
}

}  // namespace

int p4_wait_status(bool clear) {
  int s = 0;
  if (cudaMemcpyFromSymbol(&s, g_p4_status, sizeof(s)) != cudaSuccess) return CAS_ERR_CUDA;
  if (s && clear) {
    const int z = 0;
    if (cudaMemcpyToSymbol(g_p4_status, &z, sizeof(z)) != cudaSuccess) return CAS_ERR_CUDA;
  }
  return s;
}

int set_p4_spins(uint32_t n) {
  return cudaMemcpyToSymbol(c_p4_spins, &n, sizeof(n)) == cudaSuccess ? CAS_OK : CAS_ERR_CUDA;
}

}  // namespace cas

using namespace cas;

extern "C" int cas_paged4_read(const cas_paged4_kv* kv, const cas_paged_batch* b, uint16_t* k, uint16_t* v,
                               void* stream) {
  if (const int s = check_paged(kv, b)) return s;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!k || !v || !aligned16(k) || !aligned16(v)) return CAS_ERR_INVALID;
  ReadArgs a{make_paged_dev(kv, b), k, v};
  const int64_t blocks = ((int64_t)b->rows * ((kv->n_kv_heads + 3) / 4) * 32 + kReadThreads - 1) / kReadThreads;
  if (blocks > 0x7FFFFFFF) return CAS_ERR_INVALID;
  return launch_k(paged4_read_kernel, (unsigned)blocks, kReadThreads, 0, (cudaStream_t)stream, a);
}

extern "C" uint64_t cas_paged4_attn_workspace_bytes(int rows, int n_q_heads, int n_kv_heads) {
  if (rows < 1 || n_q_heads < 1 || n_kv_heads < 1) return 16;
  const int g = sm_count();
  const int64_t flat = (int64_t)rows * (n_q_heads / n_kv_heads);
  // the largest of what a batch of any size may choose
  uint64_t n = workspace_of<1>(g);
  if (flat > 8) n = std::max(n, workspace_of<2>(g));
  if (flat > 16) n = std::max(n, workspace_of<4>(g));
  if (flat > 32) n = std::max(n, cas_paged_attn_workspace_bytes(rows, n_q_heads, n_kv_heads));
  return n;
}

extern "C" int cas_paged4_attn(const cas_paged4_kv* kv, const cas_paged_batch* b, const uint16_t* q, int n_q_heads,
                               uint16_t* o, void* workspace, uint64_t workspace_bytes, void* stream) {
  if (const int s = check_paged(kv, b)) return s;
  if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % kv->n_kv_heads) return CAS_ERR_INVALID;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o)) return CAS_ERR_INVALID;
  if ((int64_t)b->rows * n_q_heads > 0x7FFFFFFF - 256) return CAS_ERR_INVALID;
  // o may be q: a unit's rows are written when all warps and CTAs that need its q are through with it
  const uint64_t n = (uint64_t)b->rows * n_q_heads * CAS_BLK * sizeof(uint16_t);
  const uint64_t qa = (uint64_t)(uintptr_t)q, oa = (uint64_t)(uintptr_t)o;
  if (qa != oa && qa < oa + n && oa < qa + n) return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < cas_paged4_attn_workspace_bytes(b->rows, n_q_heads, kv->n_kv_heads))
    return CAS_ERR_BUFFER;
  P4Args a{};
  a.d = make_paged_dev(kv, b);
  a.q = q;
  a.o = o;
  set_group(a, n_q_heads, kv->n_kv_heads);
  const cudaStream_t st = (cudaStream_t)stream;
  switch (units_of((int64_t)b->rows * a.G, b->batch)) {
    case 1: return launch<1>(a, kv, workspace, st);
    case 2: return launch<2>(a, kv, workspace, st);
    case 4: return launch<4>(a, kv, workspace, st);
    default: return paged4_attn_long(kv, b, q, n_q_heads, o, workspace, st);
  }
}
