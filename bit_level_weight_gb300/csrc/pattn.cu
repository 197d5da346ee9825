// pattn.cu - attention of new tokens over a paged bf16 cache.
//
// o = softmax(q K^T / sqrt(128)) V over the positions up to the row's own, in
// one pass over the keys with the running maximum and sum: a warp per (row,
// query head), 4 of the 128 values a lane.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "paged.cuh"

namespace cas {
namespace {

__global__ void __launch_bounds__(128) paged_attn_kernel(PagedDev d, const uint16_t* __restrict__ q, int Hq,
                                                         uint16_t* __restrict__ o) {
  pdl_wait();
  pdl_trigger();
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  const int64_t row = w / Hq;
  if (row >= d.rows) return;
  const int h = (int)(w - row * Hq), hk = h / (Hq / d.H);
  int lo = 0, hi = d.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (d.row_start[mid] <= row) lo = mid; else hi = mid;
  }
  const SeqSpan s = seq_span(d, lo);
  if (row < s.start || row >= s.end) return;
  const int64_t p = min((int64_t)s.len - (s.end - row), ((int64_t)d.max_pages << d.shift) - 1);
  float qf[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int j = 0; j < 4; ++j) qf[j] = bf2f(q[(row * Hq + h) * CAS_BLK + 4 * lane + j]);
  for (int64_t t = 0; t <= p; ++t) {
    const int64_t page = page_of(d, lo, t);
    float kf[4] = {0.f, 0.f, 0.f, 0.f}, vf[4] = {0.f, 0.f, 0.f, 0.f};
    if (page >= 0) {
      const int64_t at = page * d.page_stride + (t & ((1 << d.shift) - 1)) * d.token_stride + hk * d.head_stride +
                         4 * lane;
      for (int j = 0; j < 4; ++j) {
        kf[j] = bf2f(d.k[at + j]);
        vf[j] = bf2f(d.v[at + j]);
      }
    }
    float x = 0.f;
    for (int j = 0; j < 4; ++j) x = fmaf(qf[j], kf[j], x);
    x = warp_sumf(x) * 0.08838834764831845f;
    const float m2 = fmaxf(m, x);
    const float f = expf(m - m2), e = expf(x - m2);
    l = l * f + e;
    for (int j = 0; j < 4; ++j) acc[j] = fmaf(acc[j], f, e * vf[j]);
    m = m2;
  }
  for (int j = 0; j < 4; ++j) o[(row * Hq + h) * CAS_BLK + 4 * lane + j] = f2bf(l > 0.f ? acc[j] / l : 0.f);
}

}  // namespace
}  // namespace cas

using namespace cas;

extern "C" uint64_t cas_paged_attn_workspace_bytes(int rows, int n_q_heads, int n_kv_heads) {
  (void)rows, (void)n_q_heads, (void)n_kv_heads;
  return 256;
}

extern "C" int cas_paged_attn(const cas_paged_kv* kv, const cas_paged_batch* b, const uint16_t* q, int n_q_heads,
                              uint16_t* o, void* workspace, uint64_t workspace_bytes, void* stream) {
  const int s = check_paged(kv, b);
  if (s) return s;
  if (n_q_heads < 1 || n_q_heads > 4096 || n_q_heads % kv->n_kv_heads) return CAS_ERR_INVALID;
  if (b->rows == 0 || b->batch == 0) return CAS_OK;
  if (!q || !o || !aligned16(q) || !aligned16(o)) return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < cas_paged_attn_workspace_bytes(b->rows, n_q_heads, kv->n_kv_heads))
    return CAS_ERR_BUFFER;
  const int64_t warps = (int64_t)b->rows * n_q_heads, blocks = (warps + 3) / 4;
  if (blocks > 0x7FFFFFFF) return CAS_ERR_INVALID;
  return launch_k(paged_attn_kernel, (unsigned)blocks, 128, 0, (cudaStream_t)stream, make_paged_dev(kv, b), q,
                  n_q_heads, o);
}
