// spec.cu - acceptance of drafted tokens by given random numbers.
//
// Three kernels, each over the whole GPU whatever the batch:
//   stats_kernel  reads every logit that can matter once and leaves (maximum,
//                 sum of exponentials) of slices of rows: HBM bound;
//   sums_kernel   joins the slices, takes the ratios and the number of accepted
//                 tokens, and adds up the one or two rows that the draw uses;
//   rest_kernel   adds up the remainder max(p - q, 0) after a rejection; the last
//                 CTA of a sequence draws the next token.
//
// Ratios need fp32 accuracy. The drawn index does not forgive it: with 150000
// tokens the cumulative sum passes a border every 2^-17, so an error of 2^-24
// in the sums would move one draw in a hundred to a neighbour, and results would
// depend on the order of additions. So the rows that the draw uses are taken in
// more than fp32:
//   - exponentials to about 2^-37: y = logit * log2(e) / T as two floats, split
//     into n + j / 32 + g with |g| <= 1 / 64 (table-driven, after P. Tang, 1989); 2^(j/32) from a table of two
//     floats, 2^g - 1 = g ln 2 (two floats) + a short polynomial (fp32, below
//     2^-14 of the value); two logits at a time in packed arithmetic. fp64 has
//     2 lanes a SM and clock: 30 operations of it cost a row more than reading it;
//   - 64-bit fixed point P, Q, so that sums are exact and the same in any order;
//     the remainder is P sum(Q) - Q sum(P) by its upper halves, without division.
//
// What bounds it: one sequence of 4 drafts over 128256 tokens, three launches and
// their dependent loads (18.5 us for 4.6 MB); 29 sequences of up to 6 drafts over
// 151936 tokens take 76 us: the stats at 4.8 TB/s (24 us for 114 MB), then the
// arithmetic of the sums and the rest, about 50 instructions a weight, with the
// logits loaded ahead of it. Tried: fp64 (320 us), one cluster of 16 CTAs a sequence
// (185 us), weights kept as pairs of floats to the end (84 us), a table of 1024
// steps and a shorter polynomial (81 us, but 22.5 us for the single sequence).
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "mma.cuh"
#include "tc05.cuh"

namespace cas {
namespace {

constexpr int kStatThreads = 256;
constexpr int kThreads = 256;  // of the sums and the rest
constexpr int kMaxGamma = 64;
constexpr int kAhead = 4;  // tokens of a row that a thread loads before it weighs the ones in hand: 29 sequences
                           // of up to 6 drafts over 151936 tokens took 83 us without, 77.5 with 2, 76 with 4

struct SpecArgs {
  const float *target, *draft, *u;
  const int32_t *x, *n_draft;
  int64_t ts, ds, V;
  int batch, gamma, slices;
  int64_t vecs;  // 16-byte groups a slice
  double temp;
  float c, c_lo;  // log2(e) / T as two floats
  int32_t *n_accepted, *tokens;
  float* ratio;
  float span;    // 80 / c: logits further below the maximum weigh nothing
  float2* part;  // [batch][2 gamma + 1][slices]: maximum and sum, or maximum and its index
  struct Seq* seq;     // [batch]
  ulonglong2* sum;     // [batch][parts]: sums of P and Q over a part of the vocabulary
  uint64_t* rest;      // [batch][parts]: and of the remainder
  int parts;
  int64_t per;         // tokens a part
};

// NaN counts as -inf (fmaxf returns its other argument)
__device__ __forceinline__ float clean(float l) { return fmaxf(l, -INFINITY); }
__device__ __forceinline__ int drafted(const SpecArgs& a, int b) {
  return a.n_draft ? max(0, min(a.gamma, a.n_draft[b])) : a.gamma;
}

// Running maximum and sum; m starts at the lowest finite value, so -inf
// weighs nothing; equal infinities weigh one each.
struct Stat {
  float m, s;
  __device__ __forceinline__ void add(const float* v, float c) {  // 16 values, any
    float t = m;
#pragma unroll
    for (int i = 0; i < 16; ++i) t = fmaxf(t, v[i]);
    if (t > m) {
      s *= ex2((m - t) * c);
      m = t;
    }
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const float l = clean(v[i]);
      s += ex2(l == m ? 0.f : (l - m) * c);
    }
  }
  // 16 values; the sum becomes NaN where one is NaN or +inf
  __device__ __forceinline__ void add_fast(const float* v, float c) {
    float t = m;
#pragma unroll
    for (int i = 0; i < 16; i += 2) t = max3(t, v[i], v[i + 1]);
    if (t > m) {
      s *= ex2((m - t) * c);
      m = t;
    }
    const uint64_t nm = pack2(-m, -m), c2 = pack2(c, c);
    uint64_t s2 = 0;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      float a, b;
      unpack2(mul2(add2(pack2(v[i], v[i + 1]), nm), c2), a, b);
      s2 = add2(s2, pack2(ex2(a), ex2(b)));
    }
    float a, b;
    unpack2(s2, a, b);
    s += a + b;
  }
  __device__ __forceinline__ void join(float om, float os, float c) {
    const float t = fmaxf(m, om);
    s = s * ex2(m == t ? 0.f : (m - t) * c) + os * ex2(om == t ? 0.f : (om - t) * c);
    m = t;
  }
};

// One CTA: a slice of one row. GREEDY: the maximum and its lowest index, target rows only.
template <bool GREEDY>
__global__ void __launch_bounds__(kStatThreads) stats_kernel(SpecArgs a) {
  pdl_wait();
  pdl_trigger();
  const int per = GREEDY ? a.gamma + 1 : 2 * a.gamma + 1;
  const int64_t r = blockIdx.x;
  const int b = (int)(r / per), k = (int)(r - (int64_t)b * per), nd = drafted(a, b);
  if (k <= a.gamma ? k > nd : k - a.gamma - 1 >= nd) return;  // decides nothing
  const float* row = k <= a.gamma ? a.target + ((int64_t)b * (a.gamma + 1) + k) * a.ts
                                  : a.draft + ((int64_t)b * a.gamma + k - a.gamma - 1) * a.ds;
  // 16-byte groups from the aligned address at or below the row's start
  const int mis = (int)(((uintptr_t)row >> 2) & 3);
  const float4* base = reinterpret_cast<const float4*>(row - mis);
  const int64_t nvec = (a.V + mis + 3) / 4;
  const int64_t v0 = blockIdx.y * a.vecs, v1 = min(nvec, v0 + a.vecs);
  if (blockIdx.y == 0 && k == 0 && threadIdx.x == 0 && !GREEDY) a.seq[b].done = 0;
  auto load = [&](int64_t v, float x[16]) {
    const int64_t first = v - threadIdx.x;  // of the block's 4 * kStatThreads groups
    if (first > 0 && first + 4 * kStatThreads <= v1 && 4 * (first + 4 * kStatThreads) - mis <= a.V) {  // all whole
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 t = __ldg(base + v + i * kStatThreads);
        x[4 * i] = t.x, x[4 * i + 1] = t.y, x[4 * i + 2] = t.z, x[4 * i + 3] = t.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t g = v + i * kStatThreads;
      const int64_t e = 4 * g - mis;  // first element of the group
      if (g < v1 && e >= 0 && e + 4 <= a.V) {
        const float4 t = __ldg(base + g);
        x[4 * i] = t.x, x[4 * i + 1] = t.y, x[4 * i + 2] = t.z, x[4 * i + 3] = t.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[4 * i + j] = g < v1 && e + j >= 0 && e + j < a.V ? row[e + j] : -INFINITY;
      }
    }
  };
  Stat st{-FLT_MAX, 0.f};
  float best = -INFINITY;
  int64_t idx = a.V;
  float x[16];
  for (int64_t v = v0 + threadIdx.x; v < v1; v += 4 * kStatThreads) {
    load(v, x);
    if (GREEDY) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (x[i] > best) {  // indices grow within a thread: the first of a tie stays; NaN never wins
          best = x[i];
          idx = 4 * (v + (i >> 2) * kStatThreads) - mis + (i & 3);
        }
    } else {
      st.add_fast(x, a.c);
    }
  }
  if (!GREEDY && st.s != st.s) {  // a NaN or +inf among them
    st = Stat{-FLT_MAX, 0.f};
    for (int64_t v = v0 + threadIdx.x; v < v1; v += 4 * kStatThreads) {
      load(v, x);
      st.add(x, a.c);
    }
  }
  __shared__ float sm[kStatThreads / 32], ss[kStatThreads / 32];
  __shared__ int64_t si[kStatThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (GREEDY) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float ob = __shfl_xor_sync(CAS_FULL, best, d);
      const int64_t oi = __shfl_xor_sync(CAS_FULL, idx, d);
      if (ob > best || (ob == best && oi < idx)) best = ob, idx = oi;
    }
    if (lane == 0) sm[warp] = best, si[warp] = idx;
  } else {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float om = __shfl_xor_sync(CAS_FULL, st.m, d), os = __shfl_xor_sync(CAS_FULL, st.s, d);
      // the lower lane's pair first, so that both lanes form the same bits
      Stat lo = (lane & d) ? Stat{om, os} : st;
      const Stat hi = (lane & d) ? st : Stat{om, os};
      lo.join(hi.m, hi.s, a.c);
      st = lo;
    }
    if (lane == 0) sm[warp] = st.m, ss[warp] = st.s;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 out;
    if (GREEDY) {
      for (int w = 1; w < kStatThreads / 32; ++w)
        if (sm[w] > best || (sm[w] == best && si[w] < idx)) best = sm[w], idx = si[w];
      out = make_float2(best, __int_as_float((int)idx));
    } else {
      for (int w = 1; w < kStatThreads / 32; ++w) st.join(sm[w], ss[w], a.c);
      out = make_float2(st.m, st.s);
    }
    a.part[r * a.slices + blockIdx.y] = out;
  }
}

// Greedy acceptance: a warp a sequence.
__global__ void __launch_bounds__(32) greedy_kernel(SpecArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, G = a.gamma, nd = drafted(a, b), lane = threadIdx.x;
  int n = nd;
  int32_t next = -1;
  for (int j = 0; j <= G; ++j) {
    bool hit = false;
    if (j <= nd) {
      const float2* p = a.part + ((int64_t)b * (G + 1) + j) * a.slices;
      float best = -INFINITY;
      int idx = 0x7FFFFFFF;
      for (int s = lane; s < a.slices; s += 32) {
        const float2 t = p[s];
        if (t.x > best) best = t.x, idx = __float_as_int(t.y);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const float ob = __shfl_xor_sync(CAS_FULL, best, d);
        const int oi = __shfl_xor_sync(CAS_FULL, idx, d);
        if (ob > best || (ob == best && oi < idx)) best = ob, idx = oi;
      }
      const int32_t top = best > -INFINITY ? idx : -1;
      hit = j < nd && top >= 0 && a.x[(int64_t)b * G + j] == top;
      if (j < nd && !hit) n = min(n, j);
      if (j == n) next = top;
    }
    if (a.ratio && j < G && lane == 0) a.ratio[(int64_t)b * G + j] = hit ? 1.f : 0.f;
  }
  if (lane == 0) a.n_accepted[b] = n;
  for (int j = lane; j <= G; j += 32)
    a.tokens[(int64_t)b * (G + 1) + j] = j < n ? a.x[(int64_t)b * G + j] : j == n ? next : -1;
}

// ---------------------------------------------------------------- exact weights
// How a row's logits become fixed-point weights, the largest near 2^59 / sum.
struct Weigh {
  float m, low;          // the row's maximum; below `low` a weight is nothing
  int off;               // shift of a weight of exponent 0
  bool diff, inf, none;  // y of (logit - m): for large |m * c|; infinite maximum; no mass
};
// What sums_kernel tells rest_kernel about a sequence.
struct Seq {
  int n;          // accepted tokens
  int sub;        // the draw is from a remainder
  Weigh p, q;
  uint32_t done;  // CTAs of rest_kernel that have finished
};
constexpr float kMagic = 393216.f;  // 1.5 * 2^18: adding it rounds to multiples of 1 / 32
constexpr float kLn2Hi = 0x1.62e43p-1f, kLn2Lo = -0x1.05c61p-29f;
constexpr int kFrac = 42;           // fraction bits of a table product
constexpr int kMaxParts = 4096;

// 2^(j / 32) as two floats
__constant__ float2 kPow2[32] = {
    {0x1.0000000000000p+0f, 0x0.0p+0f}, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f},
    {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f},
    {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f},
    {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f},
    {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f},
    {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f},
    {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f},
    {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f},
    {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f},
    {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f},
    {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f},
    {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f},
    {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f},
    {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f},
    {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f},
    {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}};

// Weights of two logits.
__device__ __forceinline__ void weigh2(float l0, float l1, const Weigh& w, const SpecArgs& a, const float2* table,
                                       uint64_t out[2]) {
  if (w.inf) {
    out[0] = l0 == INFINITY ? 1ull << 30 : 0ull;
    out[1] = l1 == INFINITY ? 1ull << 30 : 0ull;
    return;
  }
  auto both = [](float v) { return pack2(v, v); };
  const uint64_t one = both(-1.f);  // negates in the multiply-add that follows
  const uint64_t ch = both(a.c);
  uint64_t x = pack2(l0, l1), e = 0;
  if (w.diff) {  // l - m as two floats
    const uint64_t l = x, m = both(w.m);
    x = fma2(m, one, l);
    const uint64_t bb = fma2(l, one, x);                                       // x - l
    e = mul2(fma2(add2(m, bb), one, fma2(fma2(bb, one, x), one, l)), ch);      // (l - (x - bb)) - (m + bb)
  }
  const uint64_t yh = mul2(x, ch), yn = mul2(yh, one);
  const uint64_t yl = add2(fma2(x, both(a.c_lo), fma2(x, ch, yn)), e);
  const uint64_t t = add2(yh, both(kMagic));                                   // 32 n + j in its low bits
  const uint64_t g0 = fma2(add2(t, both(-kMagic)), one, yh);
  const uint64_t g = add2(g0, yl), gl = fma2(fma2(g0, one, g), one, yl);
  // 2^g - 1 as h + r
  const uint64_t h = mul2(g, both(kLn2Hi)), hn = mul2(g, both(-kLn2Hi));
  uint64_t r = fma2(g, both(kLn2Hi), hn);
  r = fma2(g, both(kLn2Lo), r);
  r = fma2(gl, both(kLn2Hi), r);
  uint64_t p = fma2(g, both(1.33335581e-3f), both(9.61812911e-3f));  // ln^5 2 / 120, ln^4 2 / 24
  p = fma2(g, p, both(5.55041087e-2f));                               // ln^3 2 / 6
  p = fma2(g, p, both(2.40226507e-1f));                               // ln^2 2 / 2
  r = fma2(mul2(g, g), p, r);
  float t0, t1;
  unpack2(t, t0, t1);
  const int k0 = __float_as_int(t0) - __float_as_int(kMagic), k1 = __float_as_int(t1) - __float_as_int(kMagic);
  const float2 b0 = table[k0 & 31], b1 = table[k1 & 31];
  const uint64_t th = pack2(b0.x, b1.x), tl = pack2(b0.y, b1.y);
  const uint64_t ph = mul2(th, h), s = add2(th, ph);
  r = fma2(th, r, fma2(th, h, mul2(th, hn)));
  r = add2(r, add2(fma2(tl, h, tl), fma2(fma2(th, one, s), one, ph)));
  // s: 24 bits down to 2^-24 of at most 2.1; |r| below 2^-12
  float s0, s1, r0, r1;
  unpack2(mul2(s, both(268435456.f)), s0, s1);        // 2^28
  unpack2(mul2(r, both(4398046511104.f)), r0, r1);    // 2^42
  auto fix = [&](float hi, float lo, int k, float l) -> uint64_t {
    const uint64_t full = (uint64_t)((int64_t)__float2int_rn(hi) * (1 << (kFrac - 28)) + __float2int_rn(lo));
    const int sh = l >= w.low ? 20 - ((k >> 5) + w.off) : 64;  // of the weight 20 bits up: never to the left
    return sh < 64 ? (full << 20) >> sh : 0ull;
  };
  out[0] = fix(s0, r0, k0, l0);
  out[1] = fix(s1, r1, k1, l1);
}

__device__ __forceinline__ Weigh row_weigh(const SpecArgs& a, float M, float Z) {
  Weigh w;
  const float top = M * a.c;
  w.m = M;
  w.none = !(Z > 0.f);
  w.inf = M == INFINITY;
  w.low = fmaxf(M - a.span, -FLT_MAX);
  w.diff = fabsf(top) > 16384.f;
  const int N = w.none || w.inf || w.diff ? 0 : (int)floorf(top);
  // a weight is below 2.1, Z >= 1 - 2^-20 up to its rounding: sums stay below 2^62
  const int up = w.none || w.inf ? 0 : max(0, ilogbf(Z)) + 1;
  w.off = 60 - up - kFrac - N;
  return w;
}

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(CAS_FULL, v, d);
  return v;
}
__device__ __forceinline__ uint64_t block_sum64(uint64_t v, uint64_t* sm) {  // every thread gets it
  v = warp_sum64(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int k = 0; k < kThreads / 32; ++k) v += sm[k];
  return v;
}
__device__ __forceinline__ void load_table(float2* table) {
  if (threadIdx.x < 32) table[threadIdx.x] = kPow2[threadIdx.x];
}

// One CTA: a part of the vocabulary of one sequence.
__global__ void __launch_bounds__(kThreads) sums_kernel(SpecArgs a) {
  __shared__ float sM[2 * kMaxGamma + 1], sZ[2 * kMaxGamma + 1], sr[kMaxGamma];
  __shared__ float2 table[32];
  __shared__ uint64_t red[kThreads / 32];
  __shared__ int sn;
  load_table(table);
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, G = a.gamma, nd = drafted(a, b), rows = 2 * G + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // rows: join the slices
  for (int k = warp; k < rows; k += kThreads / 32) {
    Stat st{-FLT_MAX, 0.f};
    if (k <= G ? k <= nd : k - G - 1 < nd) {
      const float2* p = a.part + ((int64_t)b * rows + k) * a.slices;
      for (int i = lane; i < a.slices; i += 32) {
        const float2 v = p[i];
        st.join(v.x, v.y, a.c);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const float om = __shfl_xor_sync(CAS_FULL, st.m, d), os = __shfl_xor_sync(CAS_FULL, st.s, d);
        Stat lo = (lane & d) ? Stat{om, os} : st;
        const Stat hi = (lane & d) ? st : Stat{om, os};
        lo.join(hi.m, hi.s, a.c);
        st = lo;
      }
    }
    if (lane == 0) sM[k] = st.m, sZ[k] = st.s;
  }
  __syncthreads();
  // ratios and the number of accepted tokens
  if (threadIdx.x < G) {
    const int j = threadIdx.x, kq = G + 1 + j;
    const int64_t x = a.x[(int64_t)b * G + j];
    float ratio = 0.f;
    if (j < nd && x >= 0 && x < a.V && sZ[j] > 0.f) {
      const float tl = clean(a.target[((int64_t)b * (G + 1) + j) * a.ts + x]);
      const float dl = clean(a.draft[((int64_t)b * G + j) * a.ds + x]);
      const float zp = tl == sM[j] ? 0.f : (tl - sM[j]) * a.c, zq = dl == sM[kq] ? 0.f : (dl - sM[kq]) * a.c;
      // a probability below the smallest double is zero
      const bool p0 = tl == -INFINITY || zp < -1075.f;
      const bool q0 = !(sZ[kq] > 0.f) || dl == -INFINITY || zq < -1075.f;
      if (!p0) ratio = q0 ? 1.f : fminf(1.f, ex2(zp - zq) * (sZ[kq] / sZ[j]));
    }
    sr[j] = ratio;
    if (blockIdx.y == 0 && a.ratio) a.ratio[(int64_t)b * G + j] = ratio;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    while (n < nd && a.u[(int64_t)b * (G + 1) + n] < sr[n]) ++n;
    sn = n;
  }
  __syncthreads();
  const int n = sn;
  const Weigh wp = row_weigh(a, sM[n], sZ[n]);
  const Weigh wq = n < nd ? row_weigh(a, sM[G + 1 + n], sZ[G + 1 + n]) : Weigh{};
  const bool sub = n < nd && !wp.none && !wq.none;
  if (blockIdx.y == 0) {
    if (threadIdx.x == 0) {
      Seq& s = a.seq[b];
      s.n = n;
      s.sub = sub;
      s.p = wp;
      s.q = wq;
      a.n_accepted[b] = n;
    }
    for (int j = threadIdx.x; j <= G; j += kThreads)  // rest_kernel writes place n
      a.tokens[(int64_t)b * (G + 1) + j] = j < n ? a.x[(int64_t)b * G + j] : -1;
  }
  // the sums over this part
  const float* pr = a.target + ((int64_t)b * (G + 1) + n) * a.ts;
  const float* qr = sub ? a.draft + ((int64_t)b * G + n) * a.ds : nullptr;
  const int64_t i0 = blockIdx.y * a.per, i1 = min(a.V, i0 + a.per);
  uint64_t tp = 0, tq = 0;
  if (!wp.none) {
    auto load = [&](const float* row, int64_t i, float v[kAhead]) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v[k] = i + k * kThreads < i1 ? __ldg(row + i + k * kThreads) : -INFINITY;
    };
    float p[kAhead], q[kAhead];
    load(pr, i0 + threadIdx.x, p);
    if (sub) load(qr, i0 + threadIdx.x, q);
#pragma unroll 1
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kAhead * kThreads) {
      float pn[kAhead], qn[kAhead];
      load(pr, i + kAhead * kThreads, pn);
      if (sub) load(qr, i + kAhead * kThreads, qn);
      uint64_t w[2];
#pragma unroll
      for (int k = 0; k < kAhead; k += 2) {
        weigh2(p[k], p[k + 1], wp, a, table, w);
        tp += w[0] + w[1];
        if (sub) {
          weigh2(q[k], q[k + 1], wq, a, table, w);
          tq += w[0] + w[1];
        }
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) p[k] = pn[k], q[k] = qn[k];
    }
  }
  tp = block_sum64(tp, red);
  if (sub) tq = block_sum64(tq, red);
  if (threadIdx.x == 0) a.sum[(int64_t)b * a.parts + blockIdx.y] = make_ulonglong2(tp, tq);
}

// The weight r of two tokens that the draw is from.
struct Draw {
  const float *pr, *qr;
  Weigh p, q;
  uint64_t zp, zq;  // sums, shifted up to their upper bits
  int lp, lq;       // by these
  bool sub;
  __device__ __forceinline__ void get2(float p0, float p1, float q0, float q1, const SpecArgs& a, const float2* table,
                                       uint64_t r[2]) const {
    weigh2(p0, p1, p, a, table, r);
    if (!sub) return;
    uint64_t w[2];
    weigh2(q0, q1, q, a, table, w);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint64_t x = __umul64hi(r[k] << lp, zq), y = __umul64hi(w[k] << lq, zp);
      r[k] = x > y ? x - y : 0ull;
    }
  }
};

// One CTA: a part of the vocabulary of one sequence. The last CTA of a
// sequence to finish draws the token.
__global__ void __launch_bounds__(kThreads) rest_kernel(SpecArgs a) {
  __shared__ float2 table[32];
  __shared__ uint64_t red[kThreads / 32], scan[kThreads / 32];
  __shared__ uint64_t goal_s;
  __shared__ int part_s, last_s;
  load_table(table);
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, G = a.gamma, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const Seq& s = a.seq[b];
  const int n = s.n;
  Draw d;
  d.sub = s.sub;
  if (!d.sub && blockIdx.y > 0) return;  // the sums say all
  d.p = s.p;
  d.q = s.q;
  d.pr = a.target + ((int64_t)b * (G + 1) + n) * a.ts;
  d.qr = d.sub ? a.draft + ((int64_t)b * G + n) * a.ds : d.pr;
  const ulonglong2* sums = a.sum + (int64_t)b * a.parts;
  uint64_t R, zq = 0;
  {
    uint64_t x = 0, y = 0;
    for (int k = threadIdx.x; k < a.parts; k += kThreads) {
      const ulonglong2 v = sums[k];
      x += v.x;
      y += v.y;
    }
    R = block_sum64(x, red);
    if (d.sub) zq = block_sum64(y, red);
  }
  const uint64_t Zp = R;
  if (d.sub) {
    d.lp = __clzll(R);
    d.lq = __clzll(zq);
    d.zp = R << d.lp;
    d.zq = zq << d.lq;
    const int64_t i0 = blockIdx.y * a.per, i1 = min(a.V, i0 + a.per);
    uint64_t t = 0;
    auto load = [&](const float* row, int64_t i, float v[kAhead]) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) v[k] = i + k * kThreads < i1 ? __ldg(row + i + k * kThreads) : -INFINITY;
    };
    float p[kAhead], q[kAhead];
    load(d.pr, i0 + threadIdx.x, p);
    load(d.qr, i0 + threadIdx.x, q);
#pragma unroll 1
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kAhead * kThreads) {
      float pn[kAhead], qn[kAhead];
      load(d.pr, i + kAhead * kThreads, pn);
      load(d.qr, i + kAhead * kThreads, qn);
#pragma unroll
      for (int k = 0; k < kAhead; k += 2) {
        uint64_t r[2];
        d.get2(p[k], p[k + 1], q[k], q[k + 1], a, table, r);
        t += r[0] + r[1];
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) p[k] = pn[k], q[k] = qn[k];
    }
    t = block_sum64(t, red);
    if (threadIdx.x == 0) {
      a.rest[(int64_t)b * a.parts + blockIdx.y] = t;
      __threadfence();
      last_s = atomicAdd(&a.seq[b].done, 1u) == (uint32_t)a.parts - 1;
    }
    __syncthreads();
    if (!last_s) return;
    __threadfence();
    uint64_t x = 0;
    for (int k = threadIdx.x; k < a.parts; k += kThreads) x += __ldcg(a.rest + (int64_t)b * a.parts + k);
    R = block_sum64(x, red);
    if (R == 0) d.sub = false, R = Zp;  // nothing remains: draw from p itself
  }
  if (R == 0) return;  // no mass: the token stays -1
  // lowest index whose cumulative sum passes u R, in whole units: floor(u R) = mantissa R >> -exponent
  if (threadIdx.x == 0) {
    const float u = a.u[(int64_t)b * (G + 1) + G];
    uint64_t goal = 0;
    if (u >= 1.f) {
      goal = R - 1;
    } else if (u > 0.f) {
      const uint32_t bits = __float_as_uint(u), ex = bits >> 23;
      const uint64_t mant = ex ? (bits & 0x7FFFFFu) | 0x800000u : bits & 0x7FFFFFu;
      const int sh = 126 - (int)(ex ? ex : 1u);
      goal = sh < 64 ? __umul64hi(mant << 40, R) >> sh : 0ull;
    }
    goal_s = goal;
    part_s = 0;
  }
  __syncthreads();
  uint64_t goal = goal_s;
  // inclusive prefix of `own` over the block, and the block's total
  auto prefix = [&](uint64_t own, uint64_t& total) {
    uint64_t incl = own;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const uint64_t t = __shfl_up_sync(CAS_FULL, incl, k);
      if (lane >= k) incl += t;
    }
    __syncthreads();
    if (lane == 31) scan[warp] = incl;
    __syncthreads();
    total = 0;
    uint64_t ahead = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k == warp) ahead = total;
      total += scan[k];
    }
    return ahead + incl;
  };
  // the part that holds the goal
  for (int k0 = 0; k0 < a.parts; k0 += kThreads) {
    const int k = k0 + threadIdx.x;
    uint64_t own = 0, total;
    if (k < a.parts) own = d.sub ? __ldcg(a.rest + (int64_t)b * a.parts + k) : sums[k].x;
    const uint64_t to = prefix(own, total), from = to - own;
    if (own && goal >= from && goal < to) {
      goal_s = goal - from;
      part_s = k;
    }
    const bool here = goal < total;
    __syncthreads();
    if (here) break;
    goal -= total;
  }
  goal = goal_s;
  const int64_t i0 = part_s * a.per, i1 = min(a.V, i0 + a.per);
  for (int64_t base = i0; base < i1; base += 4 * kThreads) {
    const int64_t i = base + 4 * threadIdx.x;
    uint64_t r[4], own = 0, total;
#pragma unroll
    for (int k = 0; k < 4; k += 2) {
      float p0 = -INFINITY, p1 = -INFINITY, q0 = -INFINITY, q1 = -INFINITY;
      if (i + k < i1) p0 = d.pr[i + k], q0 = d.qr[i + k];
      if (i + k + 1 < i1) p1 = d.pr[i + k + 1], q1 = d.qr[i + k + 1];
      d.get2(p0, p1, q0, q1, a, table, r + k);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) own += r[k];
    const uint64_t to = prefix(own, total), from = to - own;
    if (own && goal >= from && goal < to) {
      uint64_t left = goal - from;
      int k = 0;
#pragma unroll
      for (int t = 0; t < 3; ++t)
        if (k == t && left >= r[t]) left -= r[t], k = t + 1;
      a.tokens[(int64_t)b * (G + 1) + n] = (int32_t)(i + k);
    }
    if (goal < total) return;
    goal -= total;
  }
}

// Slices of a row: enough CTAs for every SM, long enough to amortise their reduction.
void slice(int rows, int64_t vocab, int* slices, int64_t* vecs) {
  const int64_t nvec = (vocab + 6) / 4;  // with up to 3 elements before an unaligned row
  const int64_t unit = 4 * kStatThreads;
  const int64_t want = std::max<int64_t>(1, (int64_t)sm_count() * 8 / std::max(rows, 1));
  const int64_t units = std::max<int64_t>(1, (nvec + unit - 1) / unit);
  const int64_t each = std::max<int64_t>(1, units / std::min(units, want));
  *vecs = each * unit;
  *slices = (int)((nvec + *vecs - 1) / *vecs);
}

}  // namespace
}  // namespace cas

using namespace cas;

namespace {
// Workspace: sequences, sums, remainders, slices.
struct Plan {
  int slices, parts;
  int64_t vecs, per;
  uint64_t sum, rest, part, bytes;
};
Plan plan_of(int batch, int gamma, int64_t vocab, bool greedy) {
  Plan p{};
  const int rows = batch * (greedy ? gamma + 1 : 2 * gamma + 1);
  slice(rows, vocab, &p.slices, &p.vecs);
  // parts of the vocabulary: four tokens a thread at least, eight CTAs an SM wanted, since sequences differ in
  // the rows that they sum (29 sequences: 108, 92, 78, 76, 83 us for 3, 4, 6, 8, 12; a single one the same)
  const int64_t want = std::max<int64_t>(1, (int64_t)sm_count() * 8 / batch);
  p.per = std::max<int64_t>(4 * kThreads, (vocab + want - 1) / want);
  p.per = std::max<int64_t>((p.per + 2 * kThreads - 1) / (2 * kThreads) * (2 * kThreads), (vocab + kMaxParts - 1) / kMaxParts);
  p.parts = (int)((vocab + p.per - 1) / p.per);
  auto up = [](uint64_t x) { return (x + 15) & ~15ull; };
  p.sum = up(sizeof(Seq) * (uint64_t)batch);
  p.rest = up(p.sum + sizeof(ulonglong2) * (uint64_t)batch * p.parts);
  p.part = up(p.rest + 8ull * batch * p.parts);
  p.bytes = up(p.part + sizeof(float2) * (uint64_t)rows * p.slices);
  return p;
}
}  // namespace

extern "C" uint64_t cas_spec_verify_workspace_bytes(int batch, int gamma, int64_t vocab) {
  if (batch < 1 || batch > 65535 || gamma < 0 || gamma > kMaxGamma || vocab < 1 || vocab > 0x7FFFFFFF) return 16;
  return std::max(plan_of(batch, gamma, vocab, false).bytes, plan_of(batch, gamma, vocab, true).bytes);
}

extern "C" int cas_spec_verify(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                               const int32_t* x, const float* u, const int32_t* n_draft, int batch, int gamma,
                               int64_t vocab, double temperature, int32_t* n_accepted, int32_t* tokens, float* ratio,
                               void* workspace, uint64_t workspace_bytes, void* stream) {
  if (batch < 0 || batch > 65535 || gamma < 0 || gamma > kMaxGamma || vocab < 1 || vocab > 0x7FFFFFFF ||
      target_stride < vocab ||
      !(temperature == 0.0 || (temperature >= 1e-6 && temperature <= 1e6)))
    return CAS_ERR_INVALID;
  const bool greedy = temperature == 0.0;
  if (!greedy && gamma > 0 && draft_stride < vocab) return CAS_ERR_INVALID;
  if (batch == 0) return CAS_OK;
  if (!target || !n_accepted || !tokens || (gamma > 0 && !x) || (!greedy && (!u || (gamma > 0 && !draft))))
    return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) || workspace_bytes < cas_spec_verify_workspace_bytes(batch, gamma, vocab))
    return CAS_ERR_BUFFER;
  SpecArgs a{};
  a.target = target, a.draft = draft, a.u = u, a.x = x, a.n_draft = n_draft, a.ts = target_stride;
  a.ds = draft_stride, a.V = vocab, a.batch = batch, a.gamma = gamma, a.temp = temperature;
  if (!greedy) {
    const double c = 1.4426950408889634074 / temperature;
    a.c = (float)c;
    a.c_lo = (float)(c - (double)a.c);
    a.span = (float)(80.0 / c);
  }
  a.n_accepted = n_accepted, a.tokens = tokens, a.ratio = ratio;
  const Plan p = plan_of(batch, gamma, vocab, greedy);
  uint8_t* ws = (uint8_t*)workspace;
  a.seq = (Seq*)ws, a.sum = (ulonglong2*)(ws + p.sum), a.rest = (uint64_t*)(ws + p.rest);
  a.part = (float2*)(ws + p.part);
  a.slices = p.slices, a.vecs = p.vecs, a.parts = p.parts, a.per = p.per;
  const int rows = batch * (greedy ? gamma + 1 : 2 * gamma + 1);
  const cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)rows, (unsigned)a.slices), grid2((unsigned)batch, (unsigned)a.parts);
  // the later kernels follow our own: their launch may overlap the tail of the one before
  if (greedy) {
    if (const int e = launch_k(stats_kernel<true>, grid, kStatThreads, 0, st, a)) return e;
    return launch_with(true, greedy_kernel, batch, 32, 0, st, a);
  }
  if (const int e = launch_k(stats_kernel<false>, grid, kStatThreads, 0, st, a)) return e;
  if (const int e = launch_with(true, sums_kernel, grid2, kThreads, 0, st, a)) return e;
  return launch_with(true, rest_kernel, grid2, kThreads, 0, st, a);
}
