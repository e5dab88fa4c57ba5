// The accepted rows of draft trees move to the end of their sequences in a
// paged cache, every layer in one launch.
//
//   row L + path[t] -> row L + t, t = 1 .. n_path - 1, L = seq_len - q_len
//
// A tree's rows are a few hundred bytes each: one launch, bound by its chain of
// loads (lengths and path, page table, rows).  A small block takes one (layer,
// sequence, KV head), so that thousands stand on the SMs at once.  Nothing is
// written before the whole path and its pages are known to be good; then the rows
// go a few at a time in rising order: the source of a row lies at or behind it, so
// what a later one reads has not been written yet, and within a turn all are read
// before any is written.
// Key bounds: a page that starts inside the tree starts over with the committed
// rows, which drops what rejected rows had left there; the page in front, whose
// older rows are not read here, is widened.  32 layers and 16 streams of 8 KV
// heads: 6.2 us, in blocks of 256 threads that hold a whole path in registers 15.4.
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kThreads = 64;
static_assert(kThreads >= kTreeNodes, "a thread looks up one row of the path");

template <typename T>
__device__ __forceinline__ void fold(uint4& lo, uint4& hi, const uint4& v) {
  using T2 = typename Pair<T>::T2;
  T2* l = reinterpret_cast<T2*>(&lo);
  T2* h = reinterpret_cast<T2*>(&hi);
  const T2* x = reinterpret_cast<const T2*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    l[i] = __hmin2_nan(l[i], x[i]);
    h[i] = __hmax2_nan(h[i], x[i]);
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
paged_commit_kernel(const PagedBatch b, const CommitArgs a, int32_t* status) {
  constexpr int V16 = D / 8, kRows = kThreads / V16;     // rows a turn
  // where row L + path[t] lies and where row L + t does, in 16-byte chunks
  __shared__ int64_t from[kTreeNodes], to[kTreeNodes];
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x % a.Hkv, s = blockIdx.x / a.Hkv % b.n_seq;
  const int layer = blockIdx.x / a.Hkv / b.n_seq;
  const SeqSpan sp = seq_span(b, s);
  const int n = a.n_path[s];
  const int step = tid < a.path_stride ? a.path[(int64_t)s * a.path_stride + tid] : 0;
  uint4* k = static_cast<uint4*>(a.k_pages[layer]);
  uint4* v = static_cast<uint4*>(a.v_pages[layer]);
  const int L = sp.kl - sp.ql;
  const bool owns = sp.ql > 0 && !sp.bad;
  bool bad = sp.bad || (owns && (n < 1 || n > min(sp.ql, a.path_stride) || L < 0));
  if (owns && !bad && tid < n) {
    // the root stays (its path entry is not looked at)
    const int src = tid == 0 ? 0 : step;
    if (src < tid || src >= sp.ql) {
      bad = true;
    } else {
      const int in = (1 << b.page_shift) - 1;
      const int32_t* table = b.table + (int64_t)s * b.max_pages;
      const int64_t p = table[(L + src) >> b.page_shift], q = table[(L + tid) >> b.page_shift];
      bad = p < 0 || p >= b.n_pages || q < 0 || q >= b.n_pages;
      from[tid] = (((p * a.Hkv + h) << b.page_shift) + ((L + src) & in)) * V16;
      to[tid] = (((q * a.Hkv + h) << b.page_shift) + ((L + tid) & in)) * V16;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
  if (blockIdx.x == s * a.Hkv && tid == 0 && a.new_lens)
    a.new_lens[s] = owns && !bad ? L + n : b.seq_lens[s];
  if (bad || !owns) return;
  const int x = tid % V16;
  for (int t0 = 1; t0 < n; t0 += kRows) {
    const int t = t0 + tid / V16;
    uint4 kr, vr;
    if (t < n) {
      kr = k[from[t] + x];
      vr = v[from[t] + x];
    }
    __syncthreads();
    if (t < n) {
      k[to[t] + x] = kr;
      v[to[t] + x] = vr;
    }
  }
  if (!a.key_min) return;
  __syncthreads();
  const int first = L >> b.page_shift, pages = ((L + n - 1) >> b.page_shift) - first + 1;
  for (int e = tid; e < pages * V16; e += kThreads) {
    const int start = (first + e / V16) << b.page_shift;
    const int t0 = max(start - L, 0), t1 = min(start + (1 << b.page_shift) - L, n);
    uint4 lo = k[to[t0] + x], hi = lo;
#pragma unroll 4
    for (int t = t0 + 1; t < t1; ++t) fold<T>(lo, hi, k[to[t] + x]);
    // the page's bounds, from the place of its row t0
    const int64_t at = (to[t0] / V16 >> b.page_shift) * V16 + x;
    uint4* mn = static_cast<uint4*>(a.key_min[layer]) + at;
    uint4* mx = static_cast<uint4*>(a.key_max[layer]) + at;
    if (start < L) {
      uint4 spare = lo;
      fold<T>(lo, spare, *mn);
      spare = hi;
      fold<T>(spare, hi, *mx);
    }
    *mn = lo;
    *mx = hi;
  }
}

}  // namespace

template <typename T>
static int go_commit(const PagedBatch& b, const CommitArgs& a, int n_layers, int d, int32_t* status,
                     cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)((int64_t)n_layers * b.n_seq * a.Hkv)), dim3(kThreads), 0,
             st);
  if (d == 128) cudaLaunchKernelEx(&cfg, paged_commit_kernel<T, 128>, b, a, status);
  else cudaLaunchKernelEx(&cfg, paged_commit_kernel<T, 64>, b, a, status);
  return launch_status("paged_commit_kernel");
}

int launch_paged_commit(const PagedBatch& b, const CommitArgs& a, int n_layers, int d, bool fp16,
                        int32_t* status, cudaStream_t st) {
  return fp16 ? go_commit<__half>(b, a, n_layers, d, status, st)
              : go_commit<__nv_bfloat16>(b, a, n_layers, d, status, st);
}

}  // namespace ts
