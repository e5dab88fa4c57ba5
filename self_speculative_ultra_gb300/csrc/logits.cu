// Logits of a batch's rows under biases, repetition penalties and masks, and the
// token counts that the penalties read.
//
//   x = logit + bias[v]
//   x = x > 0 ? x / repetition : x * repetition         where v was seen
//   x = x - frequency c - presence (c > 0)               c: how often
//   x = masked_value                                     where v is not allowed
//
// "Seen" and c: the sequence's own (a bit and a count a token, kept from step to
// step) and, for the node of a draft tree, the drafted tokens on its path.
#include <cuda_fp16.h>

#include "logits.cuh"
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kThreads = 256;
constexpr int kSlice = 4096;           // tokens of a block

template <typename T>
__device__ __forceinline__ float widen(const T& x);
template <>
__device__ __forceinline__ float widen<float>(const float& x) { return x; }
template <>
__device__ __forceinline__ float widen<__nv_bfloat16>(const __nv_bfloat16& x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float widen<__half>(const __half& x) { return __half2float(x); }

// What a slice's tokens have beside the sequence's own state: a bit a token, and
// where it is set a word: the place of its bias in the list + 1 (16 bits), and how
// often the node's path holds it.
struct Extra {
  uint32_t bit[kSlice / 32];
  uint32_t word[kSlice];
  int seq;
};

template <typename T>
__global__ void __launch_bounds__(kThreads)
logits_kernel(const LogitsArgs a, int n_slices, int32_t* status) {
  __shared__ Extra ex;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / n_slices, v0 = blockIdx.x % n_slices * kSlice;
  const int words = (a.V + 31) / 32;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) ex.seq = 0x7FFFFFFF;
  for (int i = tid; i < kSlice / 32; i += kThreads) ex.bit[i] = 0u;
  __syncthreads();
  // the row's sequence: the first that holds it
  for (int s = tid; s < a.n_seq; s += kThreads) {
    const int a0 = a.cu_q[s], a1 = a.cu_q[s + 1];
    if (blockIdx.x == 0 && (a0 < 0 || a1 < a0 || a1 > a.n)) set_status(status, TS_ERR_INVALID_ARG);
    if (row >= a0 && row < a1) atomicMin(&ex.seq, s);
  }
  __syncthreads();
  const int s = ex.seq;
  if (s == 0x7FFFFFFF) return;             // behind the last sequence: left as it is
  // ------------------------------------------------------ biases and the node's path
  const int32_t* ids = a.bias_ids + (int64_t)s * a.n_bias;
  auto mark = [&](int id) {
    ex.word[id - v0] = 0u;
    atomicOr(&ex.bit[(id - v0) >> 5], 1u << (id & 31));
  };
  auto here = [&](int id) { return id >= v0 && id < min(v0 + kSlice, a.V); };
  for (int i = tid; i < a.n_bias; i += kThreads) {
    const int id = ids[i];
    if (v0 == 0 && (id < -1 || id >= a.V)) set_status(status, TS_ERR_INVALID_ARG);
    if (here(id)) mark(id);
  }
  int drafted[2] = {-1, -1};
  if (a.tokens && warp == 0) {
    const int q0 = max(a.cu_q[s], 0), node = row - q0;
    const int nodes = min(min(a.cu_q[s + 1], a.n) - q0, kTreeNodes);
    if (min(a.cu_q[s + 1], a.n) - q0 > kTreeNodes && lane == 0)
      set_status(status, TS_ERR_INVALID_ARG);
    TreeBits tree;
    tree.build(a.parents + q0, nodes, lane, status);
    const unsigned long long on = node < kTreeNodes ? tree.of(node) : 0ull;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = lane + 32 * i;
      if (at == 0 || !(on >> at & 1)) continue;     // the root is in the history
      const int id = a.tokens[q0 + at];
      if (id < 0 || id >= a.V) set_status(status, TS_ERR_INVALID_ARG);
      else if (here(id)) {
        drafted[i] = id;
        mark(id);
      }
    }
  }
  __syncthreads();
  // of equal ids the last of the list counts
  for (int i = tid; i < a.n_bias; i += kThreads)
    if (here(ids[i])) atomicMax(&ex.word[ids[i] - v0], (uint32_t)i + 1u);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (drafted[i] >= 0) atomicAdd(&ex.word[drafted[i] - v0], 1u << 16);
  __syncthreads();
  // ------------------------------------------------------ the slice
  float rep = a.repetition ? a.repetition[s] : 1.f;
  if (!(rep > 0.f)) {
    if (v0 == 0 && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
    rep = 1.f;
  }
  const float freq = a.frequency ? a.frequency[s] : 0.f;
  const float pres = a.presence ? a.presence[s] : 0.f;
  int mr = a.mask ? (a.mask_rows ? a.mask_rows[row] : row) : -1;
  if (mr < -1 || (a.mask && mr >= a.n_masks)) {
    if (v0 == 0 && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
    mr = -1;
  }
  const T* in = static_cast<const T*>(a.logits) + row * a.row_stride;
  float* out = a.out + row * a.out_stride;
  for (int v = v0 + tid; v < min(v0 + kSlice, a.V); v += kThreads) {
    float x = widen<T>(in[v]);
    const uint32_t bit = 1u << (v & 31);
    bool met = a.seen && (a.seen[(int64_t)s * words + (v >> 5)] & bit);
    int c = met && a.counts ? a.counts[(int64_t)s * a.V + v] : 0;
    if (ex.bit[(v - v0) >> 5] & bit) {
      const uint32_t w = ex.word[v - v0];
      if (w & 0xFFFFu) x += a.bias[(int64_t)s * a.n_bias + (w & 0xFFFFu) - 1];
      if (w >> 16) {
        met = true;
        c += (int)(w >> 16);
      }
    }
    if (met) {
      x = x > 0.f ? __fdiv_rn(x, rep) : x * rep;
      x = __fsub_rn(x, __fmul_rn(freq, (float)c));
      if (c > 0) x -= pres;
    }
    if (mr >= 0 && !(a.mask[(int64_t)mr * words + (v >> 5)] & bit)) x = a.masked_value;
    out[v] = x;
  }
}

__global__ void __launch_bounds__(kThreads)
token_counts_kernel(const int32_t* __restrict__ tokens, const int32_t* __restrict__ lens,
                    int n_seq, int stride, int per_seq, int V, int32_t* __restrict__ counts,
                    int32_t* __restrict__ seen, int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.x / per_seq, i = blockIdx.x % per_seq * kThreads + threadIdx.x;
  const int n = lens[s];
  if (i == 0 && (n < 0 || n > stride)) set_status(status, TS_ERR_INVALID_ARG);
  if (i >= min(n, stride)) return;
  const int id = tokens[(int64_t)s * stride + i];
  if (id < 0 || id >= V) {
    set_status(status, TS_ERR_INVALID_ARG);
    return;
  }
  atomicOr(&seen[(int64_t)s * ((V + 31) / 32) + (id >> 5)], 1 << (id & 31));
  if (counts) atomicAdd(&counts[(int64_t)s * V + id], 1);
}

}  // namespace

int launch_logits(const LogitsArgs& a, int type, int32_t* status, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const int n_slices = (a.V + kSlice - 1) / kSlice;
  pdl_config(&cfg, attr, dim3((unsigned)((int64_t)a.n * n_slices)), dim3(kThreads), 0, st);
  cudaLaunchKernelEx(&cfg,
                     type == 0   ? logits_kernel<float>
                     : type == 1 ? logits_kernel<__nv_bfloat16>
                                 : logits_kernel<__half>,
                     a, n_slices, status);
  return launch_status("logits_kernel");
}

int launch_token_counts(const int32_t* tokens, const int32_t* lens, int n_seq, int stride, int V,
                        int32_t* counts, int32_t* seen, bool reset, bool prompt, int32_t* status,
                        cudaStream_t st) {
  if (reset) {
    cudaMemsetAsync(seen, 0, (size_t)n_seq * ((V + 31) / 32) * 4, st);
    if (counts) cudaMemsetAsync(counts, 0, (size_t)n_seq * V * 4, st);
  }
  if (stride == 0) return launch_status("token counts");
  const int per_seq = (stride + kThreads - 1) / kThreads;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)((int64_t)per_seq * n_seq)), dim3(kThreads), 0, st);
  cudaLaunchKernelEx(&cfg, token_counts_kernel, tokens, lens, n_seq, stride, per_seq, V,
                     prompt ? (int32_t*)nullptr : counts, seen, status);
  return launch_status("token_counts_kernel");
}

}  // namespace ts
