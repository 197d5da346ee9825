// rules.cu - penalties for repeated tokens, biases and grammar masks on logits
// (cas_adjust_logits in cas.h states the rules).
//
// Two kernels. mask_kernel takes the logits through with their masks alone, a piece of a
// row a CTA. rules_kernel writes the tokens again that have a count or a bias: a CTA
// takes a slice of the vocabulary of one sequence, counts the history's tokens of that
// slice in shared memory (integer atomics: the order does not matter), marks the last
// bias of each token, lists what it has found, and goes through all rows with each of
// those. What it finds does not hang on the first kernel, so it may begin while that
// one ends.
//
// What bounds it: the traffic of the logits in and out (masks of 29 x up to 7 rows of
// 151936 bf16 logits in 21.8 us: 41 MB in and 81 MB out, which partly stay in L2), then the CTAs whose
// slices hold most of a history, beside the walk of the history by every slice (30 us with 16K
// tokens each, half of them in the first slice; 14 with empty histories and no biases); a few rows, the
// launches and the chain history -> counts -> rows. In place (fp32), 29 x up to 7 rows take 60.5 us instead of 54.6
// into a new output, as masked tokens are written one by one beside those that stay, and 29.1 without masks; 5
// rows of 128256 9.4 instead of 9.2. (In one kernel, a slice of a sequence's rows a CTA, the rows' latencies add up: 48 us
// for 29 x up to 7 rows of 151936, 30 without any rule; with eight rows loaded before the
// history is counted, 84.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"

namespace cas {
namespace {

constexpr int kThreads = 256;  // of the mask kernel
// Of the rules kernel, as a slice may hold most of a history: with 256 threads a CTA 29 x 7 rows of 151936 take 70 us
// instead of 64, of up to 7 rows 48.7 instead of 48.4, 5 rows of 128256 10.5 instead of 9.2; histories that are empty
// 28 instead of 32. With 1024, 86, 69 and 9.1.
constexpr int kRuleThreads = 512;
constexpr int kGroups = 4;  // of eight tokens a thread of the mask kernel takes
// Tokens of the vocabulary a CTA of the rules kernel takes: fewer where the CTAs would not fill the GPU.
constexpr int kSliceMin = 1024, kSliceMax = 4096;
constexpr int kLoads = 4;  // of four tokens of a history that a thread has in flight
constexpr int kRowsMost = 65;
constexpr uint32_t kDrafted = 0x80000000u;

struct RuleArgs {
  cas_logit_rules r;
  const void* in;
  float* out;
  const int32_t *x, *n_draft;
  int64_t stride, out_stride, x_stride, vocab;
  int batch, rows, slice, pieces;
  bool wait_late;  // rules_kernel follows mask_kernel, which alone writes what it reads late
  bool vec;  // eight tokens whose first has a place divisible by eight lie on the bytes of one access, in both
};
// Drafted tokens of sequence b that count, as many as rows behind the first.
__device__ __forceinline__ int drafts_of(const RuleArgs& a, int b) {
  return a.n_draft ? min(max(a.n_draft[b], 0), a.rows - 1) : a.rows - 1;
}
// Words of the mask of a row, or none.
__device__ __forceinline__ const uint32_t* mask_of(const RuleArgs& a, int64_t row) {
  if (!a.r.mask) return nullptr;
  const int m = a.r.mask_row[row];
  return m >= 0 && m < a.r.n_masks ? a.r.mask + m * a.r.mask_stride : nullptr;
}
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return bf2f(v); }
// Eight logits as they are loaded.
template <class T>
struct Raw {
  uint4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) == 4)
      asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                   : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z),
                     "=r"(v[1].w)
                   : "l"(p));
    else
      v[0] = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float l[8]) const {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
      const uint32_t u[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (sizeof(T) == 4) {
          l[4 * k + i] = __uint_as_float(u[i]);
        } else {
          l[2 * i] = __uint_as_float(u[i] << 16);
          l[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
      }
    }
  }
};

// 32 bytes in one access: as two of 16, lanes 32 bytes apart, each would touch every sector
// (29 x up to 7 rows of 151936 without rules: 30 us).
__device__ __forceinline__ void store8(float* p, const float l[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(l[0]), "f"(l[1]), "f"(l[2]), "f"(l[3]),
               "f"(l[4]), "f"(l[5]), "f"(l[6]), "f"(l[7])
               : "memory");
}

// Piece blockIdx.x % pieces of row blockIdx.x / pieces.
template <class T, bool IN_PLACE>
__global__ void __launch_bounds__(kThreads) mask_kernel(const __grid_constant__ RuleArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x / a.pieces;
  const int piece = (int)(blockIdx.x - row * a.pieces), b = (int)(row / a.rows), t = threadIdx.x;
  const T* in = (const T*)a.in + row * a.stride;
  float* out = a.out + row * a.out_stride;
  const int vocab = (int)a.vocab;
  // tokens up to the first that lies on a whole access, groups of eight, and the rest; without vec all is rest
  const int head = a.vec ? min(vocab, (int)(-(row * a.stride) & 7)) : 0, groups = a.vec ? (vocab - head) >> 3 : 0;
  const int g0 = piece * (kThreads * kGroups) + t;
  if ((int)(row - (int64_t)b * a.rows) > drafts_of(a, b)) return;
  Raw<T> raw[kGroups];
  if (!IN_PLACE) {
#pragma unroll
    for (int k = 0; k < kGroups; ++k)
      if (g0 + k * kThreads < groups) raw[k].load(in + head + 8 * (int64_t)(g0 + k * kThreads));
  }
  const uint32_t* mask = mask_of(a, row);
  if (IN_PLACE && !mask) return;
#pragma unroll
  for (int k = 0; k < kGroups; ++k) {
    const int g = g0 + k * kThreads;
    if (g >= groups) break;
    const int i = head + 8 * g;
    // (a group lies in the words of its first and its last token)
    const uint32_t on = mask ? __funnelshift_r(mask[i >> 5], mask[(i + 7) >> 5], i & 31) & 0xFFu : 0xFFu;
    float l[8];
    if (!IN_PLACE) raw[k].get(l);
    if (!IN_PLACE || on == 0) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (IN_PLACE || !(on >> e & 1)) l[e] = -INFINITY;
      store8(out + i, l);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(on >> e & 1)) out[i + e] = -INFINITY;
    }
  }
  auto single = [&](int i) {
    const bool on = !mask || (mask[i >> 5] >> (i & 31) & 1);
    if (!IN_PLACE)
      out[i] = on ? widen(in[i]) : -INFINITY;
    else if (!on)
      out[i] = -INFINITY;
  };
  if (a.vec) {
    if (piece == 0 && t < head) single(t);
    if (piece == 0 && head + 8 * groups + t < vocab) single(head + 8 * groups + t);  // (seven at most)
  } else {
    const int64_t first = (int64_t)piece * (8 * kThreads * kGroups);
    for (int64_t i = first + t; i < min((int64_t)vocab, first + 8 * kThreads * kGroups); i += kThreads) single((int)i);
  }
}

// Of a token: how often it was given out, at the top whether it is drafted (and counts from its
// row on); whether the prompt has it, a byte that several threads may set.
template <class T>
__global__ void __launch_bounds__(kRuleThreads, 1024 / kRuleThreads) rules_kernel(const __grid_constant__ RuleArgs a) {
  extern __shared__ __align__(16) uint32_t sm[];
  __shared__ int listed;
  __shared__ const uint32_t* masks[kRowsMost];
  __shared__ uint32_t xs[kRowsMost];  // the drafted tokens' places in the slice
  const bool penal = a.r.history != nullptr, biased = a.r.bias_start != nullptr;
  uint32_t* count = sm;
  int* bias = reinterpret_cast<int*>(sm + a.slice);  // place of the token's last entry and one; only where there are any
  const int words = (biased ? 2 : 1) * a.slice;
  uint8_t* said = reinterpret_cast<uint8_t*>(sm + words);
  uint16_t* list = reinterpret_cast<uint16_t*>(said + a.slice);
  // (slices in order: the first often have most of the histories' tokens, and take longest)
  const int b = blockIdx.x % a.batch, t = threadIdx.x;
  const int64_t w0 = (int64_t)(blockIdx.x / a.batch) * a.slice;
  const int n = (int)min((int64_t)a.slice, a.vocab - w0);
  for (int i = t; i < words / 4 + a.slice / 16; i += kRuleThreads) reinterpret_cast<uint4*>(sm)[i] = make_uint4(0, 0, 0, 0);
  if (t == 0) listed = 0;
  if (!a.wait_late) pdl_wait();
  pdl_trigger();
  // The history's first tokens are loaded before its length is known: its row has room for max_history. Four
  // tokens a load, behind those before the first 16 bytes.
  const int32_t* h = penal ? a.r.history + (int64_t)b * a.r.history_stride : nullptr;
  const int to16 = (int)((16 - ((uintptr_t)h & 15)) & 15) / 4;
  const int4* from = reinterpret_cast<const int4*>(h + to16);
  int4 v[kLoads];
  auto take = [&](int k0, int quads) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u)
      if (k0 + u * kRuleThreads < quads) v[u] = from[k0 + u * kRuleThreads];
  };
  if (penal) take(t, (int)(max(a.r.max_history - to16, (int64_t)0) / 4));
  const int drafts = drafts_of(a, b);
  // (of all rows: a thread that saw another n_draft, changed under the kernel, finds a mask or none)
  if (t < a.rows) masks[t] = mask_of(a, (int64_t)b * a.rows + t);
  // (token ids outside the vocabulary are none of the slice's n, negative ones neither)
  auto place = [&](int32_t token) { return (uint32_t)token - (uint32_t)w0; };
  if (t < drafts) xs[t] = penal && a.x ? place(a.x[(int64_t)b * a.x_stride + t]) : 0xFFFFFFFFu;
  int all = 0, prompt = 0;
  float rep = 1.f, freq = 0.f, pres = 0.f;
  if (penal) {
    all = (int)min(max((int64_t)a.r.n_history[b], (int64_t)0), a.r.max_history);
    prompt = a.r.n_prompt ? min(max(a.r.n_prompt[b], 0), all) : 0;
    if (a.r.repetition) rep = a.r.repetition[b];
    if (a.r.frequency) freq = a.r.frequency[b];
    if (a.r.presence) pres = a.r.presence[b];
  }
  // (l / rep as a product, whose two roundings are half a step more; where 1 / rep is no normal number the quotient)
  const float inv = __fdiv_rn(1.f, rep);
  const bool divide = !(fabsf(inv) >= 1.17549435e-38f && fabsf(inv) < INFINITY);
  __syncthreads();
  if (penal) {
    auto see = [&](bool in_prompt, uint32_t w) {
      if (w < (uint32_t)n) {
        if (in_prompt)
          said[w] = 1;
        else
          atomicAdd(&count[w], 1u);
      }
    };
    // most are another slice's
    const int head = min(all, to16), quads = (all - head) / 4;
    if (t < head) see(t < prompt, place(h[t]));
    for (int k0 = t; k0 < quads; k0 += kLoads * kRuleThreads) {
      if (k0 != t) take(k0, quads);
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int k = k0 + u * kRuleThreads, i0 = head + 4 * k;
        const uint32_t w[4] = {place(v[u].x), place(v[u].y), place(v[u].z), place(v[u].w)};
        if (k < quads && min(min(w[0], w[1]), min(w[2], w[3])) < (uint32_t)n) {
          if (i0 + 3 < prompt) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (w[i] < (uint32_t)n) said[w[i]] = 1;
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) see(i0 + i < prompt, w[i]);
          }
        }
      }
    }
    const int last = head + 4 * quads + t;
    if (last < all) see(last < prompt, place(h[last]));
    if (t < drafts && xs[t] < (uint32_t)n) atomicOr(&count[xs[t]], kDrafted);
  }
  if (biased) {
    const int64_t e1 = min(max((int64_t)a.r.bias_start[b + 1], (int64_t)0), a.r.n_bias);
    for (int64_t e = max((int64_t)a.r.bias_start[b], (int64_t)0) + t; e < e1; e += kRuleThreads) {
      const uint32_t w = place(a.r.bias_token[e]);
      if (w < (uint32_t)n) atomicMax(&bias[w], (int)e + 1);
    }
  }
  __syncthreads();
  // the list: a thread looks over 16 neighbouring tokens at a time, four in a load
  for (int i0 = 16 * t; i0 < a.slice + 16 * (t & 31); i0 += 16 * kRuleThreads) {  // (whole warps)
    uint32_t found = 0;
    if (i0 < a.slice) {
      const uint4 s4 = reinterpret_cast<const uint4*>(said + i0)[0];
      const uint32_t bytes[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 c = reinterpret_cast<const uint4*>(count + i0)[q];
        uint4 e = make_uint4(0, 0, 0, 0);
        if (biased) e = reinterpret_cast<const uint4*>(bias + i0)[q];
        const uint32_t any[4] = {c.x | e.x, c.y | e.y, c.z | e.z, c.w | e.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) found |= (uint32_t)(any[k] || (bytes[q] >> (8 * k) & 0xFF)) << (4 * q + k);
      }
    }
    const int mine = __popc(found), upto = warp_incl_add(mine, t & 31);
    int at = 0;
    if ((t & 31) == 31 && upto) at = atomicAdd(&listed, upto);
    at = __shfl_sync(CAS_FULL, at, 31) + upto - mine;
    for (; found; found &= found - 1) list[at++] = (uint16_t)(i0 + __ffs(found) - 1);
  }
  __syncthreads();
  if (a.wait_late) pdl_wait();  // the masked logits are there
  const int64_t row0 = (int64_t)b * a.rows;
  const T* in = (const T*)a.in + row0 * a.stride + w0;
  float* out = a.out + row0 * a.out_stride + w0;
  const int found = listed;
  // A slice may hold most of a history's tokens (frequent ones often have low ids): two tokens of a thread
  // and eight rows are loaded together, with the words of their masks.
  constexpr int kTokens = 2, kRows = 8;
  for (int k0 = t; k0 < found; k0 += kTokens * kRuleThreads) {
    int at[kTokens], e[kTokens];
    uint32_t c[kTokens];
    bool seen[kTokens];
    float add[kTokens];
#pragma unroll
    for (int u = 0; u < kTokens; ++u) {
      const int k = k0 + u * kRuleThreads;
      at[u] = k < found ? list[k] : -1;
      c[u] = k < found ? count[at[u]] : 0;
      seen[u] = k < found && said[at[u]];
      e[u] = k < found && biased ? bias[at[u]] : 0;
      add[u] = e[u] ? a.r.bias_value[e[u] - 1] : 0.f;
    }
    for (int j0 = 0; j0 <= drafts; j0 += kRows) {
      T l[kTokens][kRows];
      uint32_t on[kTokens][kRows];
#pragma unroll
      for (int u = 0; u < kTokens; ++u)
#pragma unroll
        for (int r = 0; r < kRows; ++r)
          if (at[u] >= 0 && j0 + r <= drafts) {
            l[u][r] = in[(j0 + r) * a.stride + at[u]];
            const uint32_t* mask = masks[j0 + r];
            on[u][r] = mask ? mask[(w0 + at[u]) >> 5] : 0xFFFFFFFFu;
          }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const int j = j0 + r;
        if (j > drafts) break;
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
          const uint32_t told = c[u] & ~kDrafted;
          if (at[u] >= 0 && (told || seen[u] || e[u]) && (on[u][r] >> (at[u] & 31) & 1)) {
            float x = widen(l[u][r]);
            if (told || seen[u]) x = x > 0.f ? (divide ? __fdiv_rn(x, rep) : x * inv) : x * rep;
            if (told) x = x - freq * (float)told - pres;
            out[j * a.out_stride + at[u]] = e[u] ? x + add[u] : x;
          }
          if ((c[u] & kDrafted) && j < drafts && xs[j] == (uint32_t)at[u]) ++c[u];
        }
      }
    }
  }
}

}  // namespace
}  // namespace cas

using namespace cas;

extern "C" int cas_adjust_logits(const void* logits, int logits_type, int64_t stride, int batch, int rows, int64_t vocab,
                                 const int32_t* x, int64_t x_stride, const int32_t* n_draft,
                                 const cas_logit_rules* rules, float* out, int64_t out_stride, void* stream) {
  if (batch < 0 || batch > 65535 || rows < 0 || rows > kRowsMost || vocab < 1 || vocab > 0x7FFFFFFF ||
      (logits_type != CAS_T_F32 && logits_type != CAS_T_BF16) || !rules)
    return CAS_ERR_INVALID;
  if (batch == 0 || rows == 0) return CAS_OK;
  const cas_logit_rules& r = *rules;
  if (!logits || !out || stride < vocab || out_stride < vocab || (x && x_stride < rows - 1)) return CAS_ERR_INVALID;
  if (r.history ? !r.n_history || r.max_history < 0 || r.max_history > 0x3FFFFFFF || r.history_stride < r.max_history
                : r.repetition || r.frequency || r.presence)
    return CAS_ERR_INVALID;
  if (r.bias_start && (!r.bias_token || !r.bias_value || r.n_bias < 0 || r.n_bias > 0x7FFFFFFF)) return CAS_ERR_INVALID;
  if (r.mask && (!r.mask_row || r.n_masks < 1 || r.mask_stride < (vocab + 31) / 32)) return CAS_ERR_INVALID;
  const bool same = (const void*)out == logits;
  const uint64_t size = logits_type == CAS_T_F32 ? 4 : 2, ia = (uint64_t)(uintptr_t)logits, oa = (uint64_t)(uintptr_t)out;
  const uint64_t steps = (uint64_t)batch * rows - 1;
  if (same ? logits_type != CAS_T_F32 || stride != out_stride
           : ia < oa + (steps * out_stride + vocab) * 4 && oa < ia + (steps * stride + vocab) * size)
    return CAS_ERR_INVALID;
  RuleArgs a{};
  a.r = r;
  a.in = logits, a.out = out, a.x = x, a.n_draft = n_draft, a.stride = stride, a.out_stride = out_stride;
  a.x_stride = x_stride, a.vocab = vocab, a.rows = rows, a.batch = batch;
  a.vec = ia % (8 * size) == 0 && oa % 32 == 0 && (stride - out_stride) % 8 == 0;
  const cudaStream_t st = (cudaStream_t)stream;
  const bool bf16 = logits_type == CAS_T_BF16, more = r.history || r.bias_start;
  if (!same || r.mask) {
    a.pieces = (int)((vocab + 8 * kThreads * kGroups - 1) / (8 * kThreads * kGroups));
    const int64_t blocks = (int64_t)batch * rows * a.pieces;
    if (blocks > 0x7FFFFFFF) return CAS_ERR_INVALID;
    const auto kernel = bf16 ? mask_kernel<uint16_t, false> : same ? mask_kernel<float, true> : mask_kernel<float, false>;
    if (const int e = launch_k(kernel, (unsigned)blocks, kThreads, 0, st, a)) return e;
    a.wait_late = true;
  }
  if (!more) return CAS_OK;
  a.slice = kSliceMax;
  while (a.slice > kSliceMin && (vocab + a.slice - 1) / a.slice * batch < 4 * (int64_t)sm_count()) a.slice /= 2;
  const int64_t grid = (vocab + a.slice - 1) / a.slice * batch;
  if (grid > 0x7FFFFFFF) return CAS_ERR_INVALID;
  const size_t smem = (size_t)a.slice * (r.bias_start ? 11 : 7);
  // directly behind our own kernel: its launch may overlap that kernel's tail
  return launch_with(a.wait_late || launch_overlap(), bf16 ? rules_kernel<uint16_t> : rules_kernel<float>, (unsigned)grid,
                     kRuleThreads, smem, st, a);
}
