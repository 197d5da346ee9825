// pline.cuh - what the paged attention kernels share: the line of key tiles
// that is cut evenly over the CTAs, and the kernel that joins the pieces of a
// unit that several CTAs have taken.
//
// The query heads of one kv head are rows of one product: flat row f of a
// sequence is token f / G, head f % G of the group. A unit is some flat rows of
// one (sequence, kv head); its keys are taken in tiles. The tiles of all units
// form one line, each unit's behind a few cells for the change of units.
#pragma once
#include "mma.cuh"
#include "paged.cuh"
#include "tc05.cuh"

namespace cas {
namespace {

constexpr int64_t kPieceFloats = CAS_BLK + 2;  // floats a row of a partial result: output, maximum, sum

struct LineArgs {
  PagedDev d;
  int Hq, G;
  uint32_t gmul;     // f / G = (umulhi(f, gmul) + f) >> gshift for 0 <= f < 2^31
  int gshift;
};
struct Cut {
  int pieces;        // of the unit, CTAs c .. c + pieces - 1; 0: none
  int ok;            // CTA c has written all its pieces
  int start, hk, f0, rows, first;  // first row of the sequence, kv head, flat rows; the first piece's place
};
struct JoinArgs : LineArgs {
  uint16_t* o;
  Cut* cuts;         // [grid]: the unit that the cut behind CTA c is the first one in
  float* ws;         // [2 * grid] pieces of piece_rows rows: output [32][rows][4], maximum [rows], sum [rows]
  int piece_rows, ctas;  // ctas: of the kernel that wrote the pieces
};
// Heads, group and its division; the rest of the arguments is the caller's.
inline void set_group(LineArgs& a, int Hq, int Hkv) {
  a.Hq = Hq;
  a.G = Hq / Hkv;
  a.gshift = 0;
  while ((1 << a.gshift) < a.G) ++a.gshift;
  a.gmul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << a.gshift) - a.G)) / a.G + 1);
}
__device__ __forceinline__ int div_g(const LineArgs& a, int f) {
  return (int)((__umulhi((uint32_t)f, a.gmul) + (uint32_t)f) >> a.gshift);
}
__device__ __forceinline__ int div64(int x, int y) { return (int)((uint32_t)x / (uint32_t)y); }
// a / b where both mostly fit 32 bits
__device__ __forceinline__ int64_t div64(int64_t x, int64_t y) {
  return ((x | y) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)y) : x / y;
}

// ---------------------------------------------------------------- the line of tiles
struct Seq {
  int start, T, len, R;  // first row, rows, tokens in the cache, flat rows
  int cap;               // positions that the block table holds
};
__device__ __forceinline__ Seq seq_of(const LineArgs& a, int b) {
  const SeqSpan s = seq_span(a.d, b);
  Seq q;
  q.start = s.start;
  q.T = s.end - s.start;
  q.len = s.len;
  q.R = q.T * a.G;
  q.cap = (int)min((int64_t)0x7FFFFF00, (int64_t)a.d.max_pages << a.d.shift);
  return q;
}
template <class N>
__device__ __forceinline__ N warp_incl(N v, int lane) {
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const N u = __shfl_up_sync(CAS_FULL, v, d);
    if (lane >= d) v += u;
  }
  return v;
}

struct Place {
  int b, hk, qt, cell;  // unit and the cell inside it
};
// Units of UNIT flat rows over tiles of TILE keys, CELLS cells for the change of units,
// counted in N: 64 bits, or 32 where the caller knows that the line fits (one warp finds its
// place on it before anything else begins).
template <int UNIT, int TILE, int CELLS, class N = int64_t>
struct UnitLine {
  struct Line {
    N total, per;  // cells of all units, cells a CTA takes
  };
  static __device__ __forceinline__ int unit_count(const Seq& s) { return (s.R + UNIT - 1) / UNIT; }
  // key tiles of unit qt: up to the position of its last row; one (masked) tile at least
  static __device__ __forceinline__ int unit_tiles(const Seq& s, const LineArgs& a, int qt) {
    const int tok = div_g(a, min(s.R, (qt + 1) * UNIT) - 1);
    const int64_t seen = min((int64_t)s.cap, (int64_t)s.len - s.T + tok + 1);
    return seen <= 0 ? 1 : (int)((seen + TILE - 1) / TILE);
  }
  // Cells of one kv head of sequence b (a lane each, warp-wide call; b beyond the
  // batch: none): a unit's tiles behind CELLS for the change of units.
  static __device__ __forceinline__ N head_cells(const LineArgs& a, int b, int lane) {
    Seq s{};
    int nq = 0;
    if (b < a.d.batch) {
      s = seq_of(a, b);
      nq = unit_count(s);
    }
    N sum = 0;
    if (nq <= 4)
      for (int i = 0; i < nq; ++i) sum += unit_tiles(s, a, i) + CELLS;
    unsigned big = __ballot_sync(CAS_FULL, nq > 4);
    while (big) {  // long chunks: the warp counts one together
      const int src = __ffs(big) - 1;
      big &= big - 1;
      const int bb = __shfl_sync(CAS_FULL, b, src);
      const Seq t = seq_of(a, bb);
      const int n = unit_count(t);
      N part = 0;
      for (int i = lane; i < n; i += 32) part += unit_tiles(t, a, i) + CELLS;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) part += __shfl_xor_sync(CAS_FULL, part, d);
      if (lane == src) sum = part;
    }
    return sum;
  }
  // Warp-wide: the line's length, and the place of cell `c * per` on it (false
  // when the line is shorter). A lane adds up `each` neighbouring sequences; the
  // lane that holds the place has its sequences looked at again by the warp.
  static __device__ bool find_place(const LineArgs& a, N c, int grid, int min_cells, Line& line, Place& p, Seq& s) {
    const int lane = threadIdx.x & 31;
    const int each = (a.d.batch + 31) / 32;
    N own = 0;
#pragma unroll 1
    for (int k = 0; k < each; ++k) own += head_cells(a, lane * each + k, lane);
    N incl = warp_incl(own, lane);
    line.total = __shfl_sync(CAS_FULL, incl, 31) * a.d.H;
    line.per = max((N)min_cells, div64(line.total + grid - 1, (N)grid));
    const N want = c * line.per;
    if (want >= line.total) return false;
    // the sequence whose cells, of all its heads, hold the wanted one
    unsigned hit = __ballot_sync(CAS_FULL, incl * a.d.H > want);
    if (!hit) return false;  // (neither this nor the two below: bounds of a count that overflowed)
    int src = __ffs(hit) - 1;
    N before = __shfl_sync(CAS_FULL, incl - own, src), per_head = __shfl_sync(CAS_FULL, own, src);
    p.b = src * each;
#pragma unroll 1
    for (int k0 = 0; each > 1 && k0 < each; k0 += 32) {
      const int b = src * each + k0 + lane;
      const N h = head_cells(a, k0 + lane < each ? b : a.d.batch, lane);
      incl = warp_incl(h, lane);
      hit = __ballot_sync(CAS_FULL, (before + incl) * a.d.H > want);
      if (hit) {
        const int w = __ffs(hit) - 1;
        p.b += k0 + w;
        per_head = __shfl_sync(CAS_FULL, h, w);
        before += __shfl_sync(CAS_FULL, incl - h, w);
        break;
      }
      before += __shfl_sync(CAS_FULL, incl, 31);
    }
    N left = want - before * a.d.H;
    if (!hit || per_head <= 0) return false;  // not reached: the sequence lies in the lane's
    p.hk = (int)div64(left, per_head);
    if (p.hk < 0 || p.hk >= a.d.H || p.b >= a.d.batch) return false;
    left -= p.hk * per_head;
    s = seq_of(a, p.b);
    const int nq = unit_count(s);
    for (int q0 = 0; q0 < nq; q0 += 32) {
      const int n = q0 + lane < nq ? unit_tiles(s, a, q0 + lane) + CELLS : 0;
      const int up = warp_incl_add(n, lane);
      const unsigned in = __ballot_sync(CAS_FULL, up > left);
      if (in) {
        const int w = __ffs(in) - 1;
        p.qt = q0 + w;
        p.cell = (int)(left - __shfl_sync(CAS_FULL, up - n, w));
        return true;
      }
      left -= __shfl_sync(CAS_FULL, up, 31);
    }
    return false;  // not reached: the unit lies in the sequence
  }
};

// ---------------------------------------------------------------- joining the pieces
// Block (c, y) merges a part of the pieces of the unit whose first cut lies
// behind CTA c: 128 / gridDim.y of the values of its rows. An item is 4 values of a row,
// neighbouring threads take neighbouring rows; where there are fewer items than
// threads, several threads share an item's pieces, so that all loads are in
// flight together.
struct Part {
  float m, l;
  float4 o;
  __device__ __forceinline__ void add(float pm, float pl, float4 v) {
    const float top = fmaxf(m, pm), ref = top == -INFINITY ? 0.f : top;
    const float f = ex2(m - ref), g = ex2(pm - ref);
    m = top;
    l = l * f + pl * g;
    o.x = o.x * f + v.x * g;
    o.y = o.y * f + v.y * g;
    o.z = o.z * f + v.z * g;
    o.w = o.w * f + v.w * g;
  }
};
template <int kJoinThreads, int CTAS>
__global__ void __launch_bounds__(kJoinThreads, CTAS) attn_join_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ Part sp[kJoinThreads];
  pdl_wait();
  pdl_trigger();
  const int at = blockIdx.x;
  Cut cut = a.cuts[at];
  const int ctas = a.ctas - at;  // from the cut's on
  cut.pieces = min(cut.pieces, ctas);  // (more only where lengths changed while the pieces were made)
  bool ok = threadIdx.x >= ctas || a.cuts[at + threadIdx.x].ok || threadIdx.x >= cut.pieces;
  if (cut.pieces < 2) return;
  for (int k = threadIdx.x + kJoinThreads; k < cut.pieces; k += kJoinThreads) ok = ok && a.cuts[at + k].ok;
  if (!__syncthreads_and(ok)) return;  // a CTA gave up: what lies at its pieces' places is not this call's
  const int chunks = 32 / gridDim.y, items = cut.rows * chunks;
  int width = 4;  // threads side by side on items: a power of two
  while (width < items && width < kJoinThreads) width *= 2;
  const int share = min(kJoinThreads / width, cut.pieces), mine = threadIdx.x & (width - 1), sub = threadIdx.x / width;
  const int64_t size = (int64_t)a.piece_rows * kPieceFloats, half = (int64_t)CAS_BLK * a.piece_rows;
  const float* base = a.ws + (int64_t)2 * at * size;
  for (int i0 = 0; i0 < items; i0 += width) {
    const int i = i0 + mine, q = i / cut.rows, fr = i - q * cut.rows, c = blockIdx.y * chunks + q;
    Part p{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    if (i < items && sub < share) {
#pragma unroll 4
      for (int k = sub; k < cut.pieces; k += share) {
        // the unit is the first of every CTA but, perhaps, the first one
        const float* w = base + (k == 0 ? cut.first : 2 * k) * size;
        p.add(w[half + fr], w[half + a.piece_rows + fr],
              *reinterpret_cast<const float4*>(w + ((int64_t)c * a.piece_rows + fr) * 4));
      }
    }
    if (share > 1) {
      sp[threadIdx.x] = p;
      __syncthreads();
      if (sub == 0)
        for (int k = 1; k < share; ++k) {
          const Part& t = sp[k * width + mine];
          p.add(t.m, t.l, t.o);
        }
    }
    if (sub == 0 && i < items) {
      const float inv = p.l > 0.f || p.l != p.l ? 1.f / p.l : 0.f;
      const int f = cut.f0 + fr, t = div_g(a, f), h = cut.hk * a.G + (f - t * a.G);
      uint2 out;
      out.x = pack_bf16x2(p.o.x * inv, p.o.y * inv);
      out.y = pack_bf16x2(p.o.z * inv, p.o.w * inv);
      *reinterpret_cast<uint2*>(a.o + ((int64_t)(cut.start + t) * a.Hq + h) * CAS_BLK + 4 * c) = out;
    }
  }
}

// ---------------------------------------------------------------- host
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// A tensor map without interleaving whose elements lie next to one another and that reads zeros outside.
inline bool encode_tiled(CUtensorMap* m, CUtensorMapDataType type, int rank, void* base, const cuuint64_t* dims,
                         const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return (EncodeFn)p;
  }();
  const cuuint32_t elem[5] = {1, 1, 1, 1, 1};
  return fn && fn(m, type, (cuuint32_t)rank, base, dims, strides, box, elem, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [grid] cuts, then pieces: the caller's workspace.
inline uint64_t cuts_bytes(int grid) { return ((uint64_t)grid * sizeof(Cut) + 255) / 256 * 256; }

}  // namespace
}  // namespace cas
