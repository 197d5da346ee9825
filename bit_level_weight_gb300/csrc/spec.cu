// spec.cu - acceptance of drafted tokens by given random numbers.
//
// One CTA judges a sequence: it takes the chosen tokens' probabilities row by
// row, stops at the first rejection and draws the next token from the
// remainder by its cumulative sum, in 64 bits.
#include <cuda_runtime.h>

#include <cmath>

#include "common.cuh"

namespace cas {
namespace {

constexpr int kThreads = 1024;

struct SpecArgs {
  const float *target, *draft, *u;
  const int32_t *x, *n_draft;
  int64_t ts, ds, V;
  int batch, gamma;
  double temp;
  int32_t *n_accepted, *tokens;
  float* ratio;
};

struct Smem {
  double red[kThreads / 32];
  int64_t idx[kThreads / 32];
  double out;
  int64_t oidx;
};

__device__ __forceinline__ double clean(float l) { return l == l ? (double)l : -INFINITY; }

// largest logit and its lowest index (V when there is none above -inf)
__device__ double block_max(const float* r, int64_t V, Smem& sm, int64_t* where) {
  double best = -INFINITY;
  int64_t idx = V;
  for (int64_t i = threadIdx.x; i < V; i += kThreads) {
    const double v = clean(r[i]);
    if (v > best) best = v, idx = i;
  }
  for (int d = 16; d > 0; d >>= 1) {
    const double ov = __shfl_xor_sync(CAS_FULL, best, d);
    const int64_t oi = __shfl_xor_sync(CAS_FULL, idx, d);
    if (ov > best || (ov == best && oi < idx)) best = ov, idx = oi;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.red[threadIdx.x >> 5] = best, sm.idx[threadIdx.x >> 5] = idx;
  __syncthreads();
  best = sm.red[0], idx = sm.idx[0];
  for (int w = 1; w < kThreads / 32; ++w)
    if (sm.red[w] > best || (sm.red[w] == best && sm.idx[w] < idx)) best = sm.red[w], idx = sm.idx[w];
  *where = idx;
  return best;
}

__device__ double block_sum(double v, Smem& sm) {
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(CAS_FULL, v, d);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sm.red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int w = 0; w < kThreads / 32; ++w) v += sm.red[w];
  return v;
}

struct Row {
  const float* r;
  double m, z, temp;
  int64_t top;  // greedy index, V when the row has no mass
  __device__ double p(int64_t i, int64_t V) const {
    if (top >= V) return 0.0;
    if (temp == 0.0) return i == top ? 1.0 : 0.0;
    const double l = clean(r[i]);
    return (l == m ? 1.0 : exp((l - m) / temp)) / z;
  }
};

__device__ Row make_row(const float* r, int64_t V, double temp, Smem& sm) {
  Row w{r, 0.0, 1.0, temp, V};
  w.m = block_max(r, V, sm, &w.top);
  if (w.top < V && temp > 0.0) {
    double z = 0.0;
    for (int64_t i = threadIdx.x; i < V; i += kThreads) {
      const double l = clean(r[i]);
      z += l == w.m ? 1.0 : exp((l - w.m) / temp);
    }
    w.z = block_sum(z, sm);
  }
  return w;
}

// lowest index whose cumulative sum of r passes u * R; -1 when R is zero
__device__ int64_t draw(const Row& p, const Row* q, float u, int64_t V, Smem& sm) {
  const int64_t per = (V + kThreads - 1) / kThreads, i0 = threadIdx.x * per, i1 = min(V, i0 + per);
  double own = 0.0;
  int64_t last = -1;
  for (int64_t i = i0; i < i1; ++i) {
    const double r = max(0.0, p.p(i, V) - (q ? q->p(i, V) : 0.0));
    own += r;
    if (r > 0.0) last = i;
  }
  // exclusive prefix over the threads, by one thread after a barrier
  __shared__ double part[kThreads];
  __shared__ double total;
  __shared__ long long lastp, found;
  __syncthreads();
  part[threadIdx.x] = own;
  if (threadIdx.x == 0) lastp = -1, found = V;
  __syncthreads();
  if (last >= 0) atomicMax(&lastp, (long long)last);
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int t = 0; t < kThreads; ++t) {
      const double v = part[t];
      part[t] = s;
      s += v;
    }
    total = s;
  }
  __syncthreads();
  if (lastp < 0) return -1;
  const double goal = (u == u && u > 0.f ? (double)u : 0.0) * total;
  double c = part[threadIdx.x];
  for (int64_t i = i0; i < i1; ++i) {
    const double r = max(0.0, p.p(i, V) - (q ? q->p(i, V) : 0.0));
    c += r;
    if (r > 0.0 && c > goal) {
      atomicMin(&found, (long long)i);
      break;
    }
  }
  __syncthreads();
  return found < V ? found : lastp;
}

__global__ void __launch_bounds__(kThreads) spec_verify_kernel(SpecArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ Smem sm;
  const int b = blockIdx.x, G = a.gamma;
  const int64_t V = a.V;
  const int nd = a.n_draft ? max(0, min(G, a.n_draft[b])) : G;
  const float* T = a.target + (int64_t)b * (G + 1) * a.ts;
  int n = -1;
  for (int j = 0; j < G; ++j) {
    double ratio = 0.0;
    const int64_t x = a.x[(int64_t)b * G + j];
    if (j < nd && x >= 0 && x < V) {
      const Row p = make_row(T + j * a.ts, V, a.temp, sm);
      if (a.temp == 0.0) {
        ratio = p.p(x, V);
      } else {
        const Row q = make_row(a.draft + ((int64_t)b * G + j) * a.ds, V, a.temp, sm);
        const double pv = p.p(x, V), qv = q.p(x, V);
        ratio = pv > 0.0 ? (qv > 0.0 ? min(1.0, pv / qv) : 1.0) : 0.0;
      }
    }
    if (a.ratio && threadIdx.x == 0) a.ratio[(int64_t)b * G + j] = (float)ratio;
    const bool ok = a.temp == 0.0 ? ratio > 0.0 : a.u[(int64_t)b * (G + 1) + j] < (float)ratio;
    if (n < 0 && (j >= nd || !ok)) n = j;
  }
  if (n < 0) n = nd;
  const Row p = make_row(T + n * a.ts, V, a.temp, sm);
  int64_t next;
  if (a.temp == 0.0) {
    next = p.top < V ? p.top : -1;
  } else {
    const float u = a.u[(int64_t)b * (G + 1) + G];
    next = -1;
    if (n < nd) {
      const Row q = make_row(a.draft + ((int64_t)b * G + n) * a.ds, V, a.temp, sm);
      next = draw(p, &q, u, V, sm);
    }
    if (next < 0) next = draw(p, nullptr, u, V, sm);
  }
  if (threadIdx.x == 0) {
    a.n_accepted[b] = n;
    int32_t* t = a.tokens + (int64_t)b * (G + 1);
    for (int j = 0; j <= G; ++j) t[j] = j < n ? a.x[(int64_t)b * G + j] : j == n ? (int32_t)next : -1;
  }
}

}  // namespace
}  // namespace cas

using namespace cas;

extern "C" uint64_t cas_spec_verify_workspace_bytes(int batch, int gamma, int64_t vocab) {
  (void)batch, (void)gamma, (void)vocab;
  return 256;
}

extern "C" int cas_spec_verify(const float* target, int64_t target_stride, const float* draft, int64_t draft_stride,
                               const int32_t* x, const float* u, const int32_t* n_draft, int batch, int gamma,
                               int64_t vocab, double temperature, int32_t* n_accepted, int32_t* tokens, float* ratio,
                               void* workspace, uint64_t workspace_bytes, void* stream) {
  if (batch < 0 || batch > 65535 || gamma < 0 || gamma > 64 || vocab < 1 || vocab > 0x7FFFFFFF ||
      target_stride < vocab || !(temperature == 0.0 || (temperature >= 1e-6 && temperature <= 1e6)))
    return CAS_ERR_INVALID;
  const bool greedy = temperature == 0.0;
  if (!greedy && gamma > 0 && draft_stride < vocab) return CAS_ERR_INVALID;
  if (batch == 0) return CAS_OK;
  if (!target || !n_accepted || !tokens || (gamma > 0 && !x) || (!greedy && (!u || (gamma > 0 && !draft))))
    return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) || workspace_bytes < cas_spec_verify_workspace_bytes(batch, gamma, vocab))
    return CAS_ERR_BUFFER;
  SpecArgs a{target, draft, u,    x,           n_draft,    target_stride, draft_stride, vocab,
             batch,  gamma, temperature, n_accepted, tokens, ratio};
  return launch_k(spec_verify_kernel, batch, kThreads, 0, (cudaStream_t)stream, a);
}
