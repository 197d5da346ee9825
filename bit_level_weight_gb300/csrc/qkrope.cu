// qkrope.cu - the split of a fused QKV product with per-head RMSNorm of q and
// k and the rotary embedding in one pass (the evaluated Qwen3-8B normalises
// its heads; Cassandra paper, evaluation), writing either dense rows
// (cas_qk_norm_rope), the slots of a paged cache (cas_paged_append) or the records
// of a 4-bit paged cache (cas_paged4_append; the codes are in q4.cuh).
//
// Per head x of 128 values: y = x * rsqrt(mean(x^2) + eps) * gamma, then the
// pairs (i, i + 64) turn by p * theta^(-i/64). Each value is read once and
// written once.
//
// What bounds it: many rows, the traffic (fp32 rows of 13 ragged sequences into
// pages: 35 us for 204 MB = 5.8 TB/s, 86 % of the measured copy rate; 4096 bf16
// rows: 22.6 us for 101 MB = 4.5 TB/s, where half of the issue slots are taken);
// a few rows, the launch (5-6 us). Into records, neither: a true division a value and the
// packing of codes by 20 to 24 warps an SM (96 and 80 registers a thread), whose latencies
// they do not hide: 2048 bf16 rows 21 us for 44 MB (2.1 TB/s, 53 % of the issue slots), 2224
// fp32 rows 21 us for 75 MB (3.6 TB/s, 39 %).
//
// Angle: theta^(-i/64) / 2 pi is a fraction of a turn per position, held as a
// 64-bit fixed-point number f_i in units of 2^-64 turns, the product of two
// constants. p * f_i modulo 2^64 is the angle reduced to a turn. f_i is off by less
// than 2^-55 turns (the constants' rounding: 2^-63 turns in A, a few 2^-53 of itself
// in both), the angle by |p| times that: 2^-24 turns at |p| = 2^31. Its top 32 bits
// go to sincospif: no double precision sine per row, whose 64 evaluations would
// cost more than the row's traffic on a GPU with 2 fp64 lanes a SM and clock.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "mma.cuh"
#include "paged.cuh"
#include "q4.cuh"
#include "tc05.cuh"

namespace cas {

namespace {
template <class KV>
PagedDev paged_dev(const KV* kv, const cas_paged_batch* b) {
  PagedDev d{};
  d.n_pages = kv->n_pages;
  d.page_stride = kv->page_stride;
  d.token_stride = kv->token_stride;
  d.head_stride = kv->head_stride;
  d.row_start = b->row_start;
  d.kv_len = b->kv_len;
  d.pages = b->pages;
  d.H = kv->n_kv_heads;
  for (d.shift = 0; (1 << d.shift) < kv->page_size;) ++d.shift;
  d.batch = b->batch;
  d.rows = b->rows;
  d.max_pages = b->max_pages;
  return d;
}
template <class KV>
bool good_paged(const KV* kv, const cas_paged_batch* b, int64_t least_stride, int64_t stride_unit) {
  if (!kv || !b || b->batch < 0 || b->batch > CAS_MAX_BATCH || b->rows < 0 || b->max_pages < 1) return false;
  const int S = kv->page_size;
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 4096 || S < 8 || S > 1024 || (S & (S - 1)) || kv->n_pages < 1 ||
      kv->n_pages > 0x7FFFFFFF)
    return false;
  const int64_t strides[3] = {kv->page_stride, kv->token_stride, kv->head_stride};
  for (int i = 0; i < 3; ++i)
    if (strides[i] < least_stride || strides[i] % stride_unit || strides[i] >= (1ll << 38)) return false;
  return !(b->batch > 0 && b->rows > 0 && (!b->row_start || !b->kv_len || !b->pages));
}
}  // namespace

PagedDev make_paged_dev(const cas_paged_kv* kv, const cas_paged_batch* b) {
  PagedDev d = paged_dev(kv, b);
  d.k = kv->k;
  d.v = kv->v;
  return d;
}
PagedDev make_paged_dev(const cas_paged4_kv* kv, const cas_paged_batch* b) {
  PagedDev d = paged_dev(kv, b);
  d.rec = kv->records;
  return d;
}

int check_paged(const cas_paged_kv* kv, const cas_paged_batch* b) {
  if (!good_paged(kv, b, CAS_BLK, 8)) return CAS_ERR_INVALID;
  return kv->k && kv->v && aligned16(kv->k) && aligned16(kv->v) ? CAS_OK : CAS_ERR_INVALID;
}
int check_paged(const cas_paged4_kv* kv, const cas_paged_batch* b) {
  if (!good_paged(kv, b, kRec, 16)) return CAS_ERR_INVALID;
  return kv->records && aligned16(kv->records) ? CAS_OK : CAS_ERR_INVALID;
}

namespace {

constexpr int kHeadsMax = 4096;
constexpr int kThreads = 128;
constexpr int kAhead = 2;         // groups of four heads whose loads a warp has in flight
constexpr int kHeadsPer = 16;     // heads a warp takes at most: a multiple of 4
constexpr int kWarpsWanted = 48;  // a SM, before a warp takes more than four heads

enum { kDense, kPaged, kPaged4 };  // where keys and values go

struct QkArgs {
  const void* qkv;
  const uint16_t *gq, *gk;
  const int32_t* pos;
  int64_t pos0;
  int rows, Hq, Hkv, rps, hpw, per_row;  // hpw: heads per warp, per_row: warps per row
  float eps;
  uint16_t *q, *k, *v;
  int64_t ks, vs;
  PagedDev pg;
  uint64_t A[8], B[8];  // theta^(-i/8) / (2 pi) in units of 2^-66, theta^(-i/64) in units of 2^-63
};

// Eight consecutive values of a head as they are loaded, and as pairs.
template <class T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void get(uint64_t x[4]) const {
    x[0] = pack2(a.x, a.y), x[1] = pack2(a.z, a.w), x[2] = pack2(b.x, b.y), x[3] = pack2(b.z, b.w);
  }
};
__device__ __forceinline__ uint64_t widen2(uint32_t t) {
  return pack2(__uint_as_float(t << 16), __uint_as_float(t & 0xFFFF0000u));
}
template <>
struct Raw<uint16_t> {
  uint4 t;
  __device__ __forceinline__ void load(const uint16_t* p) { t = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(uint64_t x[4]) const {
    x[0] = widen2(t.x), x[1] = widen2(t.y), x[2] = widen2(t.z), x[3] = widen2(t.w);
  }
};
__device__ __forceinline__ uint32_t round2(uint64_t v) {
  float a, b;
  unpack2(v, a, b);
  return pack_bf16x2(a, b);
}
__device__ __forceinline__ void store8(uint16_t* p, const uint64_t x[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(round2(x[0]), round2(x[1]), round2(x[2]), round2(x[3]));
}

// (4096 bf16 rows with half-warps on a head and 8-byte lanes: 61 us with one
// head each, 31 us with twelve; quarter-warps with packed arithmetic: 25 us;
// with 16 instead of 64 frequency constants: 22.6 us.)
// A warp takes hpw consecutive heads of one row, four at a time: eight lanes a
// head, lane l of them the values 8l..8l+7 and 64+8l..64+8l+7, so that a pair
// stays in one lane, loads and stores are 16 bytes and the arithmetic is on
// packed pairs. The row's 64 sines and cosines: each lane forms two of the
// eight that it needs, the quarters of the warp exchange them.
template <class T, int TO>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 4 ? 5 : 6) qk_norm_rope_kernel(const __grid_constant__ QkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int H = a.Hq + 2 * a.Hkv, lane = threadIdx.x & 31, l = lane & 7, quarter = lane >> 3;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t row = unit / a.per_row;
  if (row >= a.rows) return;
  const int h0 = (int)(unit - row * a.per_row) * a.hpw, h1 = min(H, h0 + a.hpw);
  const T* src = (const T*)a.qkv + (row * H + h0 + quarter) * CAS_BLK + 8 * l;
  Raw<T> rx[kAhead], ry[kAhead];  // groups of four heads in flight
  auto load = [&](int hb) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (hb + 4 * i + quarter < h1) {
        const T* from = src + (int64_t)(hb + 4 * i - h0) * CAS_BLK;
        rx[i].load(from);
        ry[i].load(from + 64);
      }
  };
  load(h0);
  int64_t p, slot = -1;
  if (TO != kDense) {
    const int seq = seq_of_row(a.pg, row, lane);
    const SeqSpan s = seq_span(a.pg, seq);
    if (row < s.start || row >= s.end) return;  // padding: left as it was
    p = (int64_t)s.len - (s.end - row);
    const int64_t page = page_of(a.pg, seq, p);
    if (page >= 0) slot = page * a.pg.page_stride + (p & ((1 << a.pg.shift) - 1)) * a.pg.token_stride;
  } else {
    p = a.pos ? (int64_t)a.pos[row] : a.pos0 + row % a.rps;
  }
  uint64_t cs[4], sn[4];
  {
    float c[8], s[8], mc[2], ms[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {  // pairs 8 l + 2 quarter + j: turns a position in units of 2^-64
      const uint64_t f = __umul64hi(a.A[l], a.B[2 * quarter + j]) >> 1;
      const int32_t turn = (int32_t)(((uint64_t)p * f) >> 32);
      if (TO == kPaged4) {
        // (codes have borders: the nearest quarter turn apart, the rest keeps two bits more in fp32)
        const uint32_t quarters = ((uint32_t)turn + 0x20000000u) >> 30;
        const int32_t rest = (int32_t)((uint32_t)turn - (quarters << 30));
        float s0, c0;
        sincospif((float)rest * 4.656612873077392578125e-10f, &s0, &c0);
        const float sw = quarters & 1 ? c0 : s0, cw = quarters & 1 ? s0 : c0;
        ms[j] = quarters & 2 ? -sw : sw;
        mc[j] = quarters == 1 || quarters == 2 ? -cw : cw;
      } else {
        sincospif((float)turn * 4.656612873077392578125e-10f /* 2^-31 */, &ms[j], &mc[j]);
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      c[k] = __shfl_sync(CAS_FULL, mc[k & 1], (k >> 1) * 8 + l);
      s[k] = __shfl_sync(CAS_FULL, ms[k & 1], (k >> 1) * 8 + l);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) cs[k] = pack2(c[2 * k], c[2 * k + 1]), sn[k] = pack2(s[2 * k], s[2 * k + 1]);
  }
  for (int hb = h0;;) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = hb + 4 * i + quarter;
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      const uint16_t* g = is_q ? a.gq : is_v ? nullptr : a.gk;
      uint64_t x[4], y[4];
      if (h < h1) {
        rx[i].get(x);
        ry[i].get(y);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = y[k] = 0;
      }
      if (a.gq || a.gk) {  // warp-uniform: every lane takes part in the sums
        uint64_t s2 = mul2(x[0], x[0]);
#pragma unroll
        for (int k = 1; k < 4; ++k) s2 = fma2(x[k], x[k], s2);
#pragma unroll
        for (int k = 0; k < 4; ++k) s2 = fma2(y[k], y[k], s2);
        float s0, s1;
        unpack2(s2, s0, s1);
        float ss = s0 + s1;
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) ss += __shfl_xor_sync(CAS_FULL, ss, d);
        if (g) {
          const float mean = ss * (1.f / CAS_BLK) + a.eps, inv = TO == kPaged4 ? __frsqrt_rn(mean) : rsqrtf(mean);
          const uint64_t i2 = pack2(inv, inv);
          Raw<uint16_t> gr;
          uint64_t gx[4];
          gr.load(g + 8 * l);
          gr.get(gx);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = mul2(mul2(x[k], i2), gx[k]);
          gr.load(g + 64 + 8 * l);
          gr.get(gx);
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] = mul2(mul2(y[k], i2), gx[k]);
        }
      }
      if (!is_v) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint64_t u = x[k], w = y[k];
          float d0, d1;
          unpack2(mul2(w, sn[k]), d0, d1);
          x[k] = fma2(u, cs[k], pack2(-d0, -d1));
          y[k] = fma2(w, cs[k], mul2(u, sn[k]));
        }
      }
      if (TO == kPaged4 && hb + 4 * i + 3 >= a.Hq) {  // warp-uniform: a key or value head among the four
        float u[8], w[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) unpack2(x[k], u[2 * k], u[2 * k + 1]), unpack2(y[k], w[2 * k], w[2 * k + 1]);
        float tu = 0.f, tw = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) tu = fmaxf(tu, fabsf(u[k])), tw = fmaxf(tw, fabsf(w[k]));
        // two lanes hold the 16 values of a scale
        tu = fmaxf(tu, __shfl_xor_sync(CAS_FULL, tu, 1));
        tw = fmaxf(tw, __shfl_xor_sync(CAS_FULL, tw, 1));
        if (h < h1 && !is_q && slot >= 0) {
          const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
          uint8_t* rec = a.pg.rec + slot + hk * a.pg.head_stride;
          const uint32_t bu = q4_scale_byte(tu), bw = q4_scale_byte(tw);
          uint32_t* codes = reinterpret_cast<uint32_t*>(rec + (is_v ? kRecV : 0));
          codes[l] = q4_word(u, q4_scale_value(bu));
          codes[8 + l] = q4_word(w, q4_scale_value(bw));
          if (!(l & 1)) {
            uint8_t* s = rec + (is_v ? kRecVs : kRecKs) + (l >> 1);
            s[0] = (uint8_t)bu;
            s[4] = (uint8_t)bw;
          }
        }
      }
      uint16_t* dst;
      bool put = h < h1 && (TO != kPaged4 || is_q);
      if (is_q) {
        dst = a.q + (row * a.Hq + h) * CAS_BLK;
      } else {
        const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        if (TO == kPaged4) {
          dst = nullptr;
        } else if (TO == kPaged) {
          put = put && slot >= 0;
          dst = (is_v ? a.pg.v : a.pg.k) + slot + hk * a.pg.head_stride;
        } else {
          dst = is_v ? a.v + row * a.vs + (int64_t)hk * CAS_BLK : a.k + row * a.ks + (int64_t)hk * CAS_BLK;
        }
      }
      if (put) {
        store8(dst + 8 * l, x);
        store8(dst + 64 + 8 * l, y);
      }
    }
    hb += 4 * kAhead;
    if (hb >= h1) break;
    load(hb);
  }
}

int check_common(const void* qkv, int type, int rows, int Hq, int Hkv, const uint16_t* gq, const uint16_t* gk,
                 float eps, double theta) {
  if (rows < 0 || Hq < 1 || Hkv < 1 || Hq > kHeadsMax || Hkv > kHeadsMax || (type != CAS_T_F32 && type != CAS_T_BF16) ||
      !(theta > 1.0) || std::isinf(theta) || !(eps >= 0.f))
    return CAS_ERR_INVALID;
  if (rows > 0 && (!qkv || !aligned16(qkv) || !aligned16(gq) || !aligned16(gk))) return CAS_ERR_INVALID;
  return CAS_OK;
}

template <int TO>
int launch_qk(QkArgs& a, int type, double theta, cudaStream_t st) {
  const double lt = std::log(theta);
  for (int i = 0; i < 8; ++i) {  // (16 constants: 64 read by 64 lanes cost a constant-cache pass each)
    a.A[i] = (uint64_t)std::llround(std::ldexp(std::exp(-lt * i / 8.0) / 6.283185307179586476925286766559, 62)) << 4;
    a.B[i] = (uint64_t)std::ldexp(std::exp(-lt * i / 64.0), 63);
  }
  const int H = a.Hq + 2 * a.Hkv;
  // A warp forms its row's sines once, whatever number of heads it takes; few
  // rows are spread over more warps.
  const int64_t warps = (int64_t)sm_count() * kWarpsWanted;
  const int groups = (H + 3) / 4;
  int each = (int)std::min<int64_t>(kHeadsPer / 4, std::max<int64_t>(1, (int64_t)a.rows * groups / warps));
  a.per_row = (groups + each - 1) / each;
  a.hpw = 4 * ((groups + a.per_row - 1) / a.per_row);
  const int64_t units = (int64_t)a.rows * a.per_row;
  const int64_t blocks = (units * 32 + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFF) return CAS_ERR_INVALID;
  return type == CAS_T_F32 ? launch_k(qk_norm_rope_kernel<float, TO>, (unsigned)blocks, kThreads, 0, st, a)
                           : launch_k(qk_norm_rope_kernel<uint16_t, TO>, (unsigned)blocks, kThreads, 0, st, a);
}

}  // namespace
}  // namespace cas

using namespace cas;

extern "C" int cas_qk_norm_rope(const void* qkv, int qkv_type, int rows, int n_q_heads, int n_kv_heads,
                                const uint16_t* gamma_q, const uint16_t* gamma_k, float eps, const int32_t* pos,
                                int64_t pos0, int rows_per_seq, double theta, uint16_t* q, uint16_t* k,
                                int64_t k_row_stride, uint16_t* v, int64_t v_row_stride, void* stream) {
  const int s = check_common(qkv, qkv_type, rows, n_q_heads, n_kv_heads, gamma_q, gamma_k, eps, theta);
  if (s) return s;
  if (!pos && (pos0 < 0 || rows_per_seq < 1)) return CAS_ERR_INVALID;
  if (rows == 0) return CAS_OK;
  const int64_t w = (int64_t)n_kv_heads * CAS_BLK;
  if (!q || !k || !v || !aligned16(q) || !aligned16(k) || !aligned16(v) || k_row_stride < w || v_row_stride < w ||
      (k_row_stride & 7) || (v_row_stride & 7))
    return CAS_ERR_INVALID;
  QkArgs a{};
  a.qkv = qkv, a.gq = gamma_q, a.gk = gamma_k, a.pos = pos, a.pos0 = pos0, a.rows = rows, a.Hq = n_q_heads;
  a.Hkv = n_kv_heads, a.rps = rows_per_seq, a.eps = eps, a.q = q, a.k = k, a.v = v;
  a.ks = k_row_stride, a.vs = v_row_stride;
  return launch_qk<kDense>(a, qkv_type, theta, (cudaStream_t)stream);
}

template <int TO, class KV>
static int append(const KV* kv, const cas_paged_batch* b, const void* qkv, int qkv_type, int n_q_heads,
                  const uint16_t* gamma_q, const uint16_t* gamma_k, float eps, double theta, uint16_t* q, void* stream) {
  int s = check_paged(kv, b);
  if (s) return s;
  s = check_common(qkv, qkv_type, b->batch ? b->rows : 0, n_q_heads, kv->n_kv_heads, gamma_q, gamma_k, eps, theta);
  if (s) return s;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!q || !aligned16(q)) return CAS_ERR_INVALID;
  QkArgs a{};
  a.qkv = qkv, a.gq = gamma_q, a.gk = gamma_k, a.rows = b->rows, a.Hq = n_q_heads, a.Hkv = kv->n_kv_heads;
  a.eps = eps, a.q = q, a.pg = make_paged_dev(kv, b);
  return launch_qk<TO>(a, qkv_type, theta, (cudaStream_t)stream);
}

extern "C" int cas_paged_append(const cas_paged_kv* kv, const cas_paged_batch* b, const void* qkv, int qkv_type,
                                int n_q_heads, const uint16_t* gamma_q, const uint16_t* gamma_k, float eps,
                                double theta, uint16_t* q, void* stream) {
  return append<kPaged>(kv, b, qkv, qkv_type, n_q_heads, gamma_q, gamma_k, eps, theta, q, stream);
}

extern "C" int cas_paged4_append(const cas_paged4_kv* kv, const cas_paged_batch* b, const void* qkv, int qkv_type,
                                 int n_q_heads, const uint16_t* gamma_q, const uint16_t* gamma_k, float eps,
                                 double theta, uint16_t* q, void* stream) {
  return append<kPaged4>(kv, b, qkv, qkv_type, n_q_heads, gamma_q, gamma_k, eps, theta, q, stream);
}
