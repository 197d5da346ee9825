// spec.cu - acceptance of drafted tokens by given random numbers.
//
// Two kernels. stats_kernel reads every logit that can matter once and leaves
// (maximum, sum of exponentials) of slices of rows: HBM bound. accept_kernel
// (a cluster of 16 CTAs a sequence) joins the slices, takes the ratios and the
// number of accepted tokens, and draws the next token.
//
// Ratios need fp32 accuracy. The drawn index does not forgive it: with 150000
// tokens the cumulative sum passes a border every 2^-17, so an error of 2^-24
// in the sums would move one draw in a hundred to a neighbour, and results would
// depend on the order of additions. So the one or two rows that the draw uses
// are taken again in more than fp32:
//   - exponentials to about 2^-37: y = logit * log2(e) / T as two floats, split
//     into n + j / 32 + g with |g| <= 1 / 64; 2^(j/32) from a table of two
//     floats, 2^g - 1 = g ln 2 (two floats) + a short polynomial (fp32, below
//     2^-14 of the value);
//   - 64-bit fixed point, so that sums are exact and the same in any order.
// A sequence whose tokens were all accepted needs one row's sums (one pass);
// after a rejection the two rows' sums come first and then the remainder's,
// whose weights take 1 / sum from the table.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace cas {
namespace {

constexpr int kStatThreads = 256;
constexpr int kCluster = 16;
constexpr int kThreads = 1024;
constexpr int kMaxGamma = 64;

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
  float2* part;  // [batch][2 gamma + 1][slices]: maximum and sum, or maximum and its index
};

__device__ __forceinline__ float ex2f(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// NaN counts as -inf (fmaxf returns its other argument)
__device__ __forceinline__ float clean(float l) { return fmaxf(l, -INFINITY); }
__device__ __forceinline__ int drafted(const SpecArgs& a, int b) {
  return a.n_draft ? max(0, min(a.gamma, a.n_draft[b])) : a.gamma;
}

// Running maximum and sum; m starts at the lowest finite value, so -inf
// weighs nothing; equal infinities weigh one each.
struct Stat {
  float m, s;
  __device__ __forceinline__ void add(const float* v, int n, float c) {
    float t = m;
    for (int i = 0; i < n; ++i) t = fmaxf(t, v[i]);
    if (t > m) {
      s *= ex2f((m - t) * c);
      m = t;
    }
    for (int i = 0; i < n; ++i) s += ex2f(v[i] == m ? 0.f : (v[i] - m) * c);
  }
  __device__ __forceinline__ void join(float om, float os, float c) {
    const float t = fmaxf(m, om);
    s = s * ex2f(m == t ? 0.f : (m - t) * c) + os * ex2f(om == t ? 0.f : (om - t) * c);
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
  Stat st{-FLT_MAX, 0.f};
  float best = -INFINITY;
  int64_t idx = a.V;
  for (int64_t v = v0 + threadIdx.x; v < v1; v += 4 * kStatThreads) {
    float x[16];
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
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = clean(x[i]);
    if (GREEDY) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (x[i] > best) {  // indices grow within a thread: the first of a tie stays
          best = x[i];
          idx = 4 * (v + (i >> 2) * kStatThreads) - mis + (i & 3);
        }
    } else {
      st.add(x, 16, a.c);
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
struct Scale {      // log2(e) / T as two floats
  float hi, lo;
};
// How a row's logits become fixed-point weights 2^(y - N) * factor.
struct Weigh {
  const float2* table;  // 2^(j/32) * factor as two floats, j = 0..31
  float m, low;         // the row's maximum; below `low` a weight is nothing
  int off;              // shift of the result
  bool diff, inf, none; // y of (logit - m): for large |m * c|; infinite maximum; no mass
};
constexpr float kMagic = 393216.f;  // 1.5 * 2^18: adding it rounds to multiples of 1 / 32
constexpr float kLn2Hi = 0.693147182464599609375f, kLn2Lo = -1.904654299957768e-09f;
constexpr int kFrac = 42;           // fraction bits of a table product

__device__ __forceinline__ uint64_t weight(float l, const Weigh& w, Scale c) {
  l = clean(l);
  if (w.inf) return l == INFINITY ? 1ull << 30 : 0ull;
  if (!(l >= w.low)) return 0ull;
  float x = l, e = 0.f;
  if (w.diff) {  // l - m as two floats
    x = l - w.m;
    const float bb = x - l;
    e = ((l - (x - bb)) - (w.m + bb)) * c.hi;
  }
  const float yh = x * c.hi;
  const float yl = fmaf(x, c.lo, fmaf(x, c.hi, -yh)) + e;
  const float t = yh + kMagic;
  const int k = __float_as_int(t) - __float_as_int(kMagic);  // 32 n + j
  const float g0 = yh - (t - kMagic);
  const float g = g0 + yl, gl = yl - (g - g0);
  // 2^g - 1 as h + r
  const float h = g * kLn2Hi;
  float r = fmaf(g, kLn2Hi, -h);
  r = fmaf(g, kLn2Lo, r);
  r = fmaf(gl, kLn2Hi, r);
  float p = fmaf(g, 1.33335581e-3f, 9.61812911e-3f);  // ln^5 2 / 120, ln^4 2 / 24
  p = fmaf(g, p, 5.55041087e-2f);                      // ln^3 2 / 6
  p = fmaf(g, p, 2.40226507e-1f);                      // ln^2 2 / 2
  r = fmaf(g * g, p, r);
  const float2 tb = w.table[k & 31];
  const float ph = tb.x * h, s = tb.x + ph;
  r = fmaf(tb.x, r, fmaf(tb.x, h, -ph));
  r += fmaf(tb.y, h, tb.y) + (ph - (s - tb.x));
  // s has at most 24 bits down to 2^-23 (factor 1..2, table 1..2); r below 2^-11
  const int64_t full = ((int64_t)__float2int_rn(s * 268435456.f) << (kFrac - 28)) +
                       (int64_t)__float2int_rn(r * 4398046511104.f);
  const int sh = (k >> 5) + w.off;
  return sh >= 0 ? (uint64_t)full << sh : sh > -64 ? (uint64_t)full >> -sh : 0ull;
}

// 2^(j / 32)
__constant__ double kPow2[32] = {
    1.0, 1.0218971486541166, 1.0442737824274138, 1.0671404006768237,
    1.0905077326652577, 1.1143867425958924, 1.1387886347566916, 1.1637248587775775,
    1.189207115002721, 1.215247359980469, 1.241857812073484, 1.2690509571917332,
    1.2968395546510096, 1.3252366431597413, 1.3542555469368927, 1.383909881963832,
    1.4142135623730951, 1.4451808069770467, 1.4768261459394993, 1.5091644275934228,
    1.5422108254079407, 1.5759808451078865, 1.6104903319492543, 1.645755478153965,
    1.681792830507429, 1.718619298122478, 1.7562521603732995, 1.7947090750031072,
    1.8340080864093424, 1.8741676341103, 1.9152065613971474, 1.9571441241754002};

struct Shared {
  float M[2 * kMaxGamma + 1], Z[2 * kMaxGamma + 1];
  float ratio[kMaxGamma];
  float2 table[3][32];  // plain, target / sum, draft / sum
  Weigh w[4];           // target, draft; the same over their sums
  double factor[2];
  uint64_t goal;
  uint64_t warp[2][kThreads / 32];
  uint64_t sum[2];      // this CTA's share of the target's and the draft's weights
  uint64_t rest;        // and of the remainder's
  int n;
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(CAS_FULL, v, d);
  return v;
}

// Table entry j of factor f in [1, 2).
__device__ __forceinline__ float2 table_entry(int j, double f) {
  const double v = kPow2[j] * f;
  const float hi = (float)v;
  return make_float2(hi, (float)(v - (double)hi));
}

__device__ Weigh plain_weigh(const SpecArgs& a, const Shared& s, float M, float Z) {
  Weigh w;
  const double c = 1.4426950408889634074 / a.temp, top = (double)M * c;
  w.table = s.table[0];
  w.m = M;
  w.none = !(Z > 0.f);
  w.inf = M == INFINITY;
  w.low = w.none || w.inf ? 0.f : fmaxf((float)((double)M - 80.0 / c), -FLT_MAX);
  w.diff = fabs(top) > 16384.0;
  const int N = w.diff || w.inf ? 0 : (int)floor(top);
  // sums stay below 2^62: weights below 2, their sum below 2 Z (1 + 2^-20)
  const int up = w.none || w.inf ? 0 : (int)ceil(log2((double)Z));
  w.off = 59 - up - kFrac - N;
  return w;
}
// The same weights divided by their sum, in units of 2^-61.
__device__ Weigh normal_weigh(Weigh w, const float2* table, uint64_t sum, double* factor) {
  int ex;
  *factor = frexp(1.0 / (double)sum, &ex) * 2.0;  // 1 / sum = factor * 2^(ex - 1)
  w.table = table;
  w.off += ex - 1 + 61;
  return w;
}

__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads) accept_kernel(SpecArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ Shared s;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank();
  const int b = blockIdx.x / kCluster, G = a.gamma, nd = drafted(a, b), rows = 2 * G + 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // ---- rows: join the slices
  for (int k = warp; k < rows; k += kThreads / 32) {
    Stat st{-FLT_MAX, 0.f};
    if (k <= G ? k <= nd : k - G - 1 < nd) {
      const float2* p = a.part + ((int64_t)b * rows + k) * a.slices;
      for (int i = lane; i < a.slices; i += 32) st.join(p[i].x, p[i].y, a.c);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) {
        const float om = __shfl_xor_sync(CAS_FULL, st.m, d), os = __shfl_xor_sync(CAS_FULL, st.s, d);
        Stat lo = (lane & d) ? Stat{om, os} : st;
        const Stat hi = (lane & d) ? st : Stat{om, os};
        lo.join(hi.m, hi.s, a.c);
        st = lo;
      }
    }
    if (lane == 0) s.M[k] = st.m, s.Z[k] = st.s;
  }
  if (threadIdx.x < 32) s.table[0][threadIdx.x] = table_entry(threadIdx.x, 1.0);
  __syncthreads();
  // ---- ratios and the number of accepted tokens
  if (threadIdx.x < G) {
    const int j = threadIdx.x;
    const int64_t x = a.x[(int64_t)b * G + j];
    float ratio = 0.f;
    if (j < nd && x >= 0 && x < a.V && s.Z[j] > 0.f) {
      // exponents in 64 bits, the exponential in 32; below -745 a probability is zero in 64 bits too
      const int kq = G + 1 + j;
      const float tl = clean(a.target[((int64_t)b * (G + 1) + j) * a.ts + x]);
      const float dl = clean(a.draft[((int64_t)b * G + j) * a.ds + x]);
      const double zp = tl == s.M[j] ? 0.0 : ((double)tl - (double)s.M[j]) / a.temp;
      const double zq = dl == s.M[kq] ? 0.0 : ((double)dl - (double)s.M[kq]) / a.temp;
      const bool p0 = tl == -INFINITY || zp < -745.0;
      const bool q0 = !(s.Z[kq] > 0.f) || dl == -INFINITY || zq < -745.0;
      if (!p0) ratio = q0 ? 1.f : fminf(1.f, expf((float)(zp - zq)) * (s.Z[kq] / s.Z[j]));
    }
    s.ratio[j] = ratio;
    if (rank == 0 && a.ratio) a.ratio[(int64_t)b * G + j] = ratio;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int n = 0;
    while (n < nd && a.u[(int64_t)b * (G + 1) + n] < s.ratio[n]) ++n;
    s.n = n;
    // a GPU has few fp64 lanes: the rows' scalars are formed once, not by every thread
    s.w[0] = plain_weigh(a, s, s.M[n], s.Z[n]);
    if (n < nd) s.w[1] = plain_weigh(a, s, s.M[G + 1 + n], s.Z[G + 1 + n]);
  }
  __syncthreads();
  const int n = s.n;
  const bool both = n < nd;
  const Scale c{a.c, a.c_lo};
  const float* pr = a.target + ((int64_t)b * (G + 1) + n) * a.ts;
  const float* qr = both ? a.draft + ((int64_t)b * G + n) * a.ds : nullptr;
  const Weigh wp = s.w[0], wq = both ? s.w[1] : Weigh{};
  const bool use_q = both && !wq.none;
  // ---- this CTA's part of the vocabulary, and the sums over it
  const int64_t per = (a.V + kCluster - 1) / kCluster, i0 = min(a.V, rank * per), i1 = min(a.V, i0 + per);
  auto block_total = [&](uint64_t v, int which) {  // every thread gets it
    v = warp_sum64(v);
    __syncthreads();
    if (lane == 0) s.warp[which][warp] = v;
    __syncthreads();
    return warp_sum64(s.warp[which][lane]);
  };
  {
    uint64_t tp = 0, tq = 0;
    if (!wp.none)
      for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
        tp += weight(__ldg(pr + i), wp, c);
        if (use_q) tq += weight(__ldg(qr + i), wq, c);
      }
    tp = block_total(tp, 0);
    tq = block_total(tq, 1);
    if (threadIdx.x == 0) s.sum[0] = tp, s.sum[1] = tq, s.rest = 0;
  }
  cl.sync();
  uint64_t Zp = 0, Zq = 0;
  for (int k = 0; k < kCluster; ++k) {
    const uint64_t* o = cl.map_shared_rank(s.sum, k);
    Zp += o[0];
    Zq += o[1];
  }
  // ---- after a rejection: the remainder max(p - q, 0)
  bool sub = use_q && Zp > 0;
  if (sub) {
    if (threadIdx.x == 0) {
      s.w[2] = normal_weigh(wp, s.table[1], Zp, &s.factor[0]);
      s.w[3] = normal_weigh(wq, s.table[2], Zq, &s.factor[1]);
    }
    __syncthreads();
    if (threadIdx.x < 64) s.table[1 + warp][lane] = table_entry(lane, s.factor[warp]);
    __syncthreads();
  }
  const Weigh np = sub ? s.w[2] : wp, nq = sub ? s.w[3] : wq;
  // infinite maxima: equal shares of 2^61
  const uint64_t ip = wp.inf && Zp ? (1ull << 61) / (Zp >> 30) : 0, iq = wq.inf && Zq ? (1ull << 61) / (Zq >> 30) : 0;
  auto rest = [&](int64_t i) -> uint64_t {
    const float lp = __ldg(pr + i);
    if (!sub) return weight(lp, wp, c);
    const uint64_t p = np.inf ? (lp == INFINITY ? ip : 0ull) : weight(lp, np, c);
    if (p == 0) return 0ull;
    const float lq = __ldg(qr + i);
    const uint64_t q = nq.inf ? (lq == INFINITY ? iq : 0ull) : weight(lq, nq, c);
    return p > q ? p - q : 0ull;
  };
  uint64_t share = s.sum[0], R = Zp, before = 0;
  if (sub) {
    uint64_t t = 0;
    for (int64_t i = i0 + threadIdx.x; i < i1; i += kThreads) t += rest(i);
    t = block_total(t, 0);
    if (threadIdx.x == 0) s.rest = t;
  }
  cl.sync();
  if (sub) {
    R = 0;
    for (int k = 0; k < kCluster; ++k) R += *cl.map_shared_rank(&s.rest, k);
    if (R == 0) sub = false, R = Zp;  // nothing remains: draw from p itself
  }
  for (int k = 0; k < rank; ++k) before += sub ? *cl.map_shared_rank(&s.rest, k) : cl.map_shared_rank(s.sum, k)[0];
  share = sub ? s.rest : s.sum[0];
  cl.sync();  // no CTA's shared memory is read from here on
  if (rank == 0) {
    if (threadIdx.x == 0) a.n_accepted[b] = n;
    for (int j = threadIdx.x; j <= G; j += kThreads)
      if (j != n || R == 0) a.tokens[(int64_t)b * (G + 1) + j] = j < n ? a.x[(int64_t)b * G + j] : -1;
  }
  if (R == 0) return;
  // lowest index whose cumulative sum passes u R, in whole units
  if (threadIdx.x == 0) {
    const float u = a.u[(int64_t)b * (G + 1) + G];
    s.goal = u >= 1.f ? R - 1 : u > 0.f ? min(R - 1, (uint64_t)((double)u * (double)R)) : 0ull;
  }
  __syncthreads();
  uint64_t goal = s.goal;
  if (goal < before || goal - before >= share) return;  // another CTA's
  goal -= before;
  for (int64_t base = i0; base < i1; base += 4 * kThreads) {
    uint64_t w[4], own = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t i = base + 4 * threadIdx.x + k;
      w[k] = i < i1 ? rest(i) : 0ull;
      own += w[k];
    }
    uint64_t incl = own;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint64_t t = __shfl_up_sync(CAS_FULL, incl, d);
      if (lane >= d) incl += t;
    }
    __syncthreads();
    if (lane == 31) s.warp[0][warp] = incl;
    __syncthreads();
    uint64_t ahead = 0, all = 0;
    for (int k = 0; k < kThreads / 32; ++k) {
      if (k < warp) ahead += s.warp[0][k];
      all += s.warp[0][k];
    }
    const uint64_t from = ahead + incl - own;
    if (goal >= from && goal - from < own) {
      uint64_t left = goal - from;
      int k = 0;
      while (left >= w[k]) left -= w[k++];
      a.tokens[(int64_t)b * (G + 1) + n] = (int32_t)(base + 4 * threadIdx.x + k);
    }
    if (goal < all) return;
    goal -= all;
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

extern "C" uint64_t cas_spec_verify_workspace_bytes(int batch, int gamma, int64_t vocab) {
  if (batch < 1 || gamma < 0 || vocab < 1) return 16;
  const int rows = batch * (2 * gamma + 1);
  int n, ng;
  int64_t v;
  slice(rows, vocab, &n, &v);
  slice(batch * (gamma + 1), vocab, &ng, &v);
  const uint64_t a = (uint64_t)rows * n, b = (uint64_t)batch * (gamma + 1) * ng;
  return (std::max(a, b) * sizeof(float2) + 15) / 16 * 16;
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
  }
  a.n_accepted = n_accepted, a.tokens = tokens, a.ratio = ratio, a.part = (float2*)workspace;
  const int rows = batch * (greedy ? gamma + 1 : 2 * gamma + 1);
  slice(rows, vocab, &a.slices, &a.vecs);
  const cudaStream_t st = (cudaStream_t)stream;
  const dim3 grid((unsigned)rows, (unsigned)a.slices);
  if (greedy) {
    if (const int e = launch_k(stats_kernel<true>, grid, kStatThreads, 0, st, a)) return e;
    return launch_with(true, greedy_kernel, batch, 32, 0, st, a);
  }
  if (const int e = launch_k(stats_kernel<false>, grid, kStatThreads, 0, st, a)) return e;
  if (cudaFuncSetAttribute(accept_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
    return CAS_ERR_CUDA;
  // directly behind our own kernel: its launch may overlap that kernel's tail
  return launch_with(true, accept_kernel, batch * kCluster, kThreads, 0, st, a);
}
