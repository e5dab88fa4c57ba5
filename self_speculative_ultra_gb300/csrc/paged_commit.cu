// The accepted rows of draft trees move to the end of their sequences in a
// paged cache, every layer in one launch.
//
//   row L + path[t] -> row L + t, t = 1 .. n_path - 1, L = seq_len - q_len
//
// A tree's rows are a few hundred bytes each: one launch, bound by its chain of
// loads (lengths and path, page table, rows).  A block takes one (layer,
// sequence, KV head): it holds all of the head's rows that move, so every source
// is read before a destination is written, whatever their order.
// Key bounds: a page that starts inside the tree starts over with the committed
// rows, which drops what rejected rows had left there; the page in front, whose
// older rows are not read here, is widened.
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kThreads = 256;

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
  constexpr int V16 = D / 8;
  constexpr int kEach = ((kTreeNodes - 1) * V16 + kThreads - 1) / kThreads;
  __shared__ uint4 rows[kTreeNodes][V16];        // committed keys, for the bounds
  const int tid = threadIdx.x;
  griddep_wait();
  griddep_launch_dependents();
  const int h = blockIdx.x % a.Hkv, s = blockIdx.x / a.Hkv % b.n_seq;
  const int layer = blockIdx.x / a.Hkv / b.n_seq;
  const SeqSpan sp = seq_span(b, s);
  const int n = a.n_path[s];
  const int L = sp.kl - sp.ql;
  const bool owns = sp.ql > 0 && !sp.bad;
  bool bad = sp.bad || (owns && (n < 1 || n > min(sp.ql, a.path_stride) || L < 0));
  // a row's place in the pool, in 16-byte chunks; -1: its page is not there
  auto place = [&](int r) -> int64_t {
    const int64_t ph = b.table[(int64_t)s * b.max_pages + (r >> b.page_shift)];
    if (ph < 0 || ph >= b.n_pages) return -1;
    return ((((ph * a.Hkv + h) << b.page_shift)) + (r & ((1 << b.page_shift) - 1))) * V16;
  };
  const int moved = owns && !bad ? (n - 1) * V16 : 0;
  uint4* k = static_cast<uint4*>(a.k_pages[layer]);
  uint4* v = static_cast<uint4*>(a.v_pages[layer]);
  uint4 kr[kEach], vr[kEach];
  int64_t to[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int e = tid + i * kThreads, t = e / V16 + 1, x = e % V16;
    to[i] = -1;
    if (e < moved) {
      const int from = a.path[(int64_t)s * a.path_stride + t];
      if (from < t || from >= sp.ql) {
        bad = true;
      } else {
        const int64_t src = place(L + from), dst = place(L + t);
        if (src < 0 || dst < 0) {
          bad = true;
        } else {
          kr[i] = k[src + x];
          vr[i] = v[src + x];
          to[i] = dst + x;
        }
      }
    }
  }
  const bool bounds = a.key_min != nullptr;
  if (bounds && owns && !bad && tid < V16) {
    const int64_t root = place(L);
    if (root < 0) bad = true;
    else rows[0][tid] = k[root + tid];
  }
  bad = __syncthreads_or(bad);               // every source is read
  if (bad && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
  if (blockIdx.x == (int64_t)s * a.Hkv && tid == 0 && a.new_lens)
    a.new_lens[s] = owns && !bad ? L + n : b.seq_lens[s];
  if (bad || !owns) return;
#pragma unroll
  for (int i = 0; i < kEach; ++i)
    if (to[i] >= 0) {
      k[to[i]] = kr[i];
      v[to[i]] = vr[i];
      const int e = tid + i * kThreads;
      if (bounds) rows[e / V16 + 1][e % V16] = kr[i];
    }
  if (!bounds) return;
  __syncthreads();
  const int first = L >> b.page_shift, pages = ((L + n - 1) >> b.page_shift) - first + 1;
  for (int e = tid; e < pages * V16; e += kThreads) {
    const int pg = first + e / V16, x = e % V16, start = pg << b.page_shift;
    const int64_t ph = b.table[(int64_t)s * b.max_pages + pg];    // seen above
    const int t0 = max(start - L, 0), t1 = min(start + (1 << b.page_shift) - L, n);
    uint4 lo = rows[t0][x], hi = lo;
    for (int t = t0 + 1; t < t1; ++t) fold<T>(lo, hi, rows[t][x]);
    const int64_t at = (ph * a.Hkv + h) * V16 + x;
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
