// qkrope.cu - the split of a fused QKV product with per-head RMSNorm of q and
// k and the rotary embedding in one pass (the evaluated Qwen3-8B normalises
// its heads; Cassandra paper, evaluation), writing either dense rows
// (cas_qk_norm_rope) or the slots of a paged cache (cas_paged_append).
//
// Per head x of 128 values: y = x * rsqrt(mean(x^2) + eps) * gamma, then the
// pairs (i, i + 64) turn by p * theta^(-i/64). Each value is read once and
// written once.
//
// Angle: theta^(-i/64) / 2 pi is a fraction of a turn per position, held as
// a 64-bit fixed-point number F_i (units of 2^-64 turns). p * F_i modulo 2^64
// is the angle reduced to a turn exactly, with an error of p * 2^-65 turns from
// F_i's rounding, and the top 32 bits of it go to sincospif: no double
// precision sine per row, whose 64 evaluations would cost more than the row's
// traffic on a GPU with 2 fp64 lanes per SM and clock.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "paged.cuh"

namespace cas {

PagedDev make_paged_dev(const cas_paged_kv* kv, const cas_paged_batch* b) {
  PagedDev d{};
  d.k = kv->k;
  d.v = kv->v;
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

int check_paged(const cas_paged_kv* kv, const cas_paged_batch* b) {
  if (!kv || !b || b->batch < 0 || b->rows < 0 || b->max_pages < 1) return CAS_ERR_INVALID;
  const int S = kv->page_size;
  if (kv->n_kv_heads < 1 || kv->n_kv_heads > 4096 || S < 8 || S > 1024 || (S & (S - 1)) || kv->n_pages < 1 ||
      kv->n_pages > 0x7FFFFFFF)
    return CAS_ERR_INVALID;
  if (!kv->k || !kv->v || !aligned16(kv->k) || !aligned16(kv->v)) return CAS_ERR_INVALID;
  for (const int64_t s : {kv->page_stride, kv->token_stride, kv->head_stride})
    if (s < CAS_BLK || (s & 7) || s >= (1ll << 38)) return CAS_ERR_INVALID;
  if (b->batch > 0 && b->rows > 0 && (!b->row_start || !b->kv_len || !b->pages)) return CAS_ERR_INVALID;
  return CAS_OK;
}

namespace {

constexpr int kHeadsMax = 4096;
constexpr int kHalfWarps = 64;  // wanted a SM before a half-warp takes more than one head
constexpr int kHeadsPer = 12;   // heads a half-warp takes at most
constexpr int kThreads = 256;
constexpr int kAhead = 4;  // heads whose loads a half-warp has in flight

struct QkArgs {
  const void* qkv;
  const uint16_t *gq, *gk;
  const int32_t* pos;
  int64_t pos0;
  int rows, Hq, Hkv, rps, hpu;  // hpu: heads per half-warp
  float eps;
  uint16_t *q, *k, *v;
  int64_t ks, vs;
  PagedDev pg;
  uint64_t F[64];  // theta^(-i/64) / (2 pi) in units of 2^-64
};

__device__ __forceinline__ void unpack4(uint2 t, float x[4]) {
  x[0] = __uint_as_float(t.x << 16), x[1] = __uint_as_float(t.x & 0xFFFF0000u);
  x[2] = __uint_as_float(t.y << 16), x[3] = __uint_as_float(t.y & 0xFFFF0000u);
}
template <class T>
struct Raw;  // four values as they were loaded
template <>
struct Raw<float> {
  float4 t;
  __device__ __forceinline__ void load(const float* p) { t = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float x[4]) const { x[0] = t.x, x[1] = t.y, x[2] = t.z, x[3] = t.w; }
};
template <>
struct Raw<uint16_t> {
  uint2 t;
  __device__ __forceinline__ void load(const uint16_t* p) { t = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float x[4]) const { unpack4(t, x); }
};
__device__ __forceinline__ void store4(uint16_t* p, const float x[4]) {
  uint2 t;
  t.x = f2bf(x[0]) | (uint32_t)f2bf(x[1]) << 16;
  t.y = f2bf(x[2]) | (uint32_t)f2bf(x[3]) << 16;
  *reinterpret_cast<uint2*>(p) = t;
}

// A half-warp takes hpu consecutive heads of one row; its lane l holds the
// values 4l..4l+3 and 64+4l..64+4l+3 of a head, so a pair stays in one lane
// and a head's loads and stores are contiguous halves of 256 (128) bytes.
template <class T, bool PAGED>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const __grid_constant__ QkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int H = a.Hq + 2 * a.Hkv;
  const int per_row = (H + a.hpu - 1) / a.hpu;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 4;
  const int64_t row = unit / per_row;
  if (row >= a.rows) return;  // both halves of a warp may differ: no warp-wide operation below but within a half
  const int h0 = (int)(unit - row * per_row) * a.hpu, h1 = min(H, h0 + a.hpu);
  const int l = threadIdx.x & 15;
  const uint32_t half = (threadIdx.x & 16) ? 0xFFFF0000u : 0x0000FFFFu;
  int64_t p, page = -1, slot = 0;
  int seq = 0;
  if (PAGED) {
    // the last sequence that starts at or before the row
    int lo = 0, hi = a.pg.batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.pg.row_start[mid] <= row) lo = mid; else hi = mid;
    }
    seq = lo;
    const SeqSpan s = seq_span(a.pg, seq);
    if (row < s.start || row >= s.end) return;  // padding: left as it was
    p = (int64_t)s.len - (s.end - row);
    page = page_of(a.pg, seq, p);
    slot = page * a.pg.page_stride + (p & ((1 << a.pg.shift) - 1)) * a.pg.token_stride;
  } else {
    p = a.pos ? (int64_t)a.pos[row] : a.pos0 + row % a.rps;
  }
  float cs[4], sn[4];
  if (h0 < a.Hq + a.Hkv) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t turn = (int32_t)(((uint64_t)p * a.F[4 * l + j]) >> 32);
      sincospif((float)turn * 4.656612873077392578125e-10f /* 2^-31 */, &sn[j], &cs[j]);
    }
  }
  const uint2 none = make_uint2(0, 0);
  const uint2 gq0 = a.gq ? *reinterpret_cast<const uint2*>(a.gq + 4 * l) : none;
  const uint2 gq1 = a.gq ? *reinterpret_cast<const uint2*>(a.gq + 64 + 4 * l) : none;
  const uint2 gk0 = a.gk ? *reinterpret_cast<const uint2*>(a.gk + 4 * l) : none;
  const uint2 gk1 = a.gk ? *reinterpret_cast<const uint2*>(a.gk + 64 + 4 * l) : none;
  const T* src = (const T*)a.qkv + row * H * CAS_BLK + 4 * l;
  for (int hb = h0; hb < h1; hb += kAhead) {
    Raw<T> rx[kAhead], ry[kAhead];  // loads of kAhead heads in flight
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (hb + i < h1) {
        rx[i].load(src + (int64_t)(hb + i) * CAS_BLK);
        ry[i].load(src + (int64_t)(hb + i) * CAS_BLK + 64);
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int h = hb + i;
      if (h >= h1) break;
      float x[4], y[4];
      rx[i].get(x);
      ry[i].get(y);
      const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
      if (is_q ? a.gq != nullptr : !is_v && a.gk != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) ss = fmaf(x[j], x[j], fmaf(y[j], y[j], ss));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) ss += __shfl_xor_sync(half, ss, d);
        const float inv = rsqrtf(ss * (1.f / CAS_BLK) + a.eps);
        float gx[4], gy[4];
        unpack4(is_q ? gq0 : gk0, gx);
        unpack4(is_q ? gq1 : gk1, gy);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] *= inv * gx[j];
          y[j] *= inv * gy[j];
        }
      }
      if (!is_v) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float c = x[j], d = y[j];
          x[j] = fmaf(c, cs[j], -d * sn[j]);
          y[j] = fmaf(d, cs[j], c * sn[j]);
        }
      }
      uint16_t* dst;
      if (is_q) {
        dst = a.q + (row * a.Hq + h) * CAS_BLK;
      } else {
        const int hk = is_v ? h - a.Hq - a.Hkv : h - a.Hq;
        if (PAGED) {
          if (page < 0) continue;
          dst = (is_v ? a.pg.v : a.pg.k) + slot + hk * a.pg.head_stride;
        } else {
          dst = is_v ? a.v + row * a.vs + (int64_t)hk * CAS_BLK : a.k + row * a.ks + (int64_t)hk * CAS_BLK;
        }
      }
      store4(dst + 4 * l, x);
      store4(dst + 64 + 4 * l, y);
    }
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

template <bool PAGED>
int launch_qk(QkArgs& a, int type, double theta, cudaStream_t st) {
  const double lt = std::log(theta);
  for (int i = 0; i < 64; ++i)  // below 2^64 / 6: the product is a whole number of 2^-64 turns
    a.F[i] = (uint64_t)std::llround(std::ldexp(std::exp(-lt * i / 64.0) / 6.283185307179586476925286766559, 62)) << 2;
  const int H = a.Hq + 2 * a.Hkv;
  // A half-warp pays for its row's sines once, whatever number of heads it
  // takes; few rows are spread over as many half-warps as there are heads.
  const int64_t half_warps = (int64_t)sm_count() * kHalfWarps;
  a.hpu = (int)std::min<int64_t>(kHeadsPer, std::max<int64_t>(1, (int64_t)a.rows * H / half_warps));
  const int64_t units = (int64_t)a.rows * ((H + a.hpu - 1) / a.hpu);
  const int64_t blocks = (units * 16 + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFF) return CAS_ERR_INVALID;
  return type == CAS_T_F32 ? launch_k(qk_norm_rope_kernel<float, PAGED>, (unsigned)blocks, kThreads, 0, st, a)
                           : launch_k(qk_norm_rope_kernel<uint16_t, PAGED>, (unsigned)blocks, kThreads, 0, st, a);
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
  return launch_qk<false>(a, qkv_type, theta, (cudaStream_t)stream);
}

extern "C" int cas_paged_append(const cas_paged_kv* kv, const cas_paged_batch* b, const void* qkv, int qkv_type,
                                int n_q_heads, const uint16_t* gamma_q, const uint16_t* gamma_k, float eps,
                                double theta, uint16_t* q, void* stream) {
  int s = check_paged(kv, b);
  if (s) return s;
  s = check_common(qkv, qkv_type, b->batch ? b->rows : 0, n_q_heads, kv->n_kv_heads, gamma_q, gamma_k, eps, theta);
  if (s) return s;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!q || !aligned16(q)) return CAS_ERR_INVALID;
  QkArgs a{};
  a.qkv = qkv, a.gq = gamma_q, a.gk = gamma_k, a.rows = b->rows, a.Hq = n_q_heads, a.Hkv = kv->n_kv_heads;
  a.eps = eps, a.q = q, a.pg = make_paged_dev(kv, b);
  return launch_qk<true>(a, qkv_type, theta, (cudaStream_t)stream);
}
