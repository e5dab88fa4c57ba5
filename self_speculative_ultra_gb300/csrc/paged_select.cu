// Choice of pages by a bound on their scores.
//
// A page's key bounds (element-wise minimum and maximum of its rows) give an
// upper bound of the scores any of its keys can reach with the query heads of
// a KV head's group:
//   score(page) = sum_h sum_c max(q_hc mn_c, q_hc mx_c)
//               = sum_c (sum_h q_hc+) mx_c + (sum_h q_hc-) mn_c,
// one product of 2 d numbers a page and KV head whatever the group's size.
// Kept: the first n_sink and the last n_recent pages a token sees and the
// n_top best between them, by (score desc, page asc).
//
// The scores decide which whole numbers come out, so they must not depend on
// the order of a sum: they are formed to about 2^-45 and rounded to fp32
// once.  Query sums are split into a part of 12 bits, whose product with a
// 16-bit element is exact in fp32, and the rest; the exact products are added
// with the rounding error of every addition kept beside the sum (Knuth's
// two-sum).
//
// Two launches: scores (memory bound: 4 d bytes a page and KV head; 8 lanes a
// page, packed fp32 pairs), then per (token, KV head) a radix selection of
// the n_top-th key and an ordered write.
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace ts {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kPickThreads = 512;
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
static_assert(kPickThreads / 32 <= 32, "one warp scans the warps' sums");
constexpr int kPickSmemKeys = 48 * 1024;     // larger candidate lists stay in the workspace
constexpr uint32_t kLowest = 0x007FFFFFu;    // float_key(-inf)

// s + e += p, the sum's rounding error kept in e
__device__ __forceinline__ void two_sum(uint64_t& s, uint64_t& e, uint64_t p) {
  const uint64_t t = ptx::add2(s, p);
  const uint64_t bb = ptx::sub2(t, s);
  e = ptx::add2(e, ptx::add2(ptx::sub2(s, ptx::sub2(t, bb)), ptx::sub2(p, bb)));
  s = t;
}
__device__ __forceinline__ void two_sum1(float& s, float& e, float p) {
  const float t = __fadd_rn(s, p);
  const float bb = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, bb)), __fsub_rn(p, bb)));
  s = t;
}

// What one token chooses from: pages [lo, hi) compete for n_top places (none
// when every visible page is kept).
struct Span {
  int vis, lo, hi;
};
__device__ __forceinline__ Span span_of(const SeqSpan& sp, int t, int shift, int n_top, int n_sink,
                                        int n_recent) {
  const int p = sp.kl - sp.ql + (t - sp.q0);      // the token's row
  Span r;
  r.vis = p < 0 ? 0 : (p >> shift) + 1;
  r.lo = r.hi = 0;
  if ((int64_t)r.vis > (int64_t)n_top + n_sink + n_recent) {
    r.lo = n_sink;
    r.hi = r.vis - n_recent;
  }
  return r;
}

template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads)
paged_score_kernel(const PagedBatch b, const T* __restrict__ q, const T* __restrict__ key_min,
                   const T* __restrict__ key_max, int Hq, int Hkv, int n_top, int n_sink,
                   int n_recent, int per_block, uint32_t* __restrict__ keys, int32_t* status) {
  // query sums: [positive, negative][12-bit part, rest][column]
  __shared__ __align__(16) float qs[2][2][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.y, kv = blockIdx.z, G = Hq / Hkv;
  griddep_wait();
  griddep_launch_dependents();
  const int s = warp_find_seq(b, t, lane);
  if (s < 0) return;
  const SeqSpan sp = seq_span(b, s);
  if (blockIdx.x == 0 && kv == 0 && tid == 0 && sp.bad) set_status(status, TS_ERR_INVALID_ARG);
  const Span w = span_of(sp, t, b.page_shift, n_top, n_sink, n_recent);
  const int p0 = w.lo + (int)blockIdx.x * per_block;
  const int p1 = min(w.hi, p0 + per_block);
  if (p0 >= p1) return;
  for (int c = tid; c < D; c += kScoreThreads) {
    float up = 0.f, upe = 0.f, dn = 0.f, dne = 0.f;
    for (int g = 0; g < G; ++g) {
      const float x = Pair<T>::one(q[((int64_t)t * Hq + kv * G + g) * D + c]);
      two_sum1(up, upe, fmaxf(x, 0.f));
      two_sum1(dn, dne, fminf(x, 0.f));
    }
    // 12 leading bits: the product with an 11-bit element is exact
    const float uh = __uint_as_float(__float_as_uint(up) & 0xFFFFF000u);
    const float dh = __uint_as_float(__float_as_uint(dn) & 0xFFFFF000u);
    qs[0][0][c] = uh;
    qs[0][1][c] = (up - uh) + upe;
    qs[1][0][c] = dh;
    qs[1][1][c] = (dn - dh) + dne;
  }
  __syncthreads();
  // lane: page lane / 8 of the warp's four, 16-byte chunks sub and sub + 8
  constexpr int kCh = D / 64;
  const int sub = lane & 7;
  uint64_t uh[kCh][4], ul[kCh][4], dh[kCh][4], dl[kCh][4];
#pragma unroll
  for (int x = 0; x < kCh; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = (sub + 8 * x) * 8 + 2 * i;
      uh[x][i] = *reinterpret_cast<const uint64_t*>(&qs[0][0][c]);
      ul[x][i] = *reinterpret_cast<const uint64_t*>(&qs[0][1][c]);
      dh[x][i] = *reinterpret_cast<const uint64_t*>(&qs[1][0][c]);
      dl[x][i] = *reinterpret_cast<const uint64_t*>(&qs[1][1][c]);
    }
  const int32_t* trow = b.table + (int64_t)s * b.max_pages;
  uint32_t* out = keys + ((int64_t)t * Hkv + kv) * b.max_pages;
  // a page's rows are on their way while the page before is summed, its pool
  // page while the one before that is
  struct Rows {
    uint4 mx[kCh], mn[kCh];
    bool ok;
  };
  auto pool_page = [&](int pg) { return pg < p1 ? trow[pg] : 0; };
  auto ask = [&](int pg, int ph) {
    Rows r;
    r.ok = pg < p1;
    if (ph < 0 || ph >= b.n_pages) {
      if (sub == 0) set_status(status, TS_ERR_INVALID_ARG);
      r.ok = false;
    }
    const int64_t row = ((int64_t)(r.ok ? ph : 0) * Hkv + kv) * (D / 8);
    const uint4* mx = reinterpret_cast<const uint4*>(key_max) + row;
    const uint4* mn = reinterpret_cast<const uint4*>(key_min) + row;
#pragma unroll
    for (int x = 0; x < kCh; ++x) {
      r.mx[x] = __ldg(mx + sub + 8 * x);
      r.mn[x] = __ldg(mn + sub + 8 * x);
    }
    return r;
  };
  const int first = p0 + warp * 4 + (lane >> 3);
  constexpr int kEach = kScoreThreads / 8;           // pages a trip
  Rows next = ask(first, pool_page(first));
  int ph_next = pool_page(first + kEach);
  for (int base = p0; base < p1; base += kEach) {    // the same trips for every lane
    const int pg = base + (first - p0);
    const Rows r = next;
    if (base + kEach < p1) {
      next = ask(pg + kEach, ph_next);
      ph_next = pool_page(pg + 2 * kEach);
    }
    uint64_t sum = 0, err = 0, sum2 = 0, err2 = 0;
#pragma unroll
    for (int x = 0; x < kCh; ++x) {
      const uint32_t wx[4] = {r.mx[x].x, r.mx[x].y, r.mx[x].z, r.mx[x].w};
      const uint32_t wn[4] = {r.mn[x].x, r.mn[x].y, r.mn[x].z, r.mn[x].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 fx = Pair<T>::unpack(wx[k]), fn = Pair<T>::unpack(wn[k]);
        const uint64_t px = ptx::f2(fx.x, fx.y), pn = ptx::f2(fn.x, fn.y);
        two_sum(sum, err, ptx::mul2(uh[x][k], px));
        err = ptx::fma2(ul[x][k], px, err);
        two_sum(sum2, err2, ptx::mul2(dh[x][k], pn));
        err2 = ptx::fma2(dl[x][k], pn, err2);
      }
    }
    two_sum(sum, err, sum2);
    err = ptx::add2(err, err2);
    float s0, s1, e0, e1;
    ptx::f2_split(sum, s0, s1);
    ptx::f2_split(err, e0, e1);
    e0 += e1;
    two_sum1(s0, e0, s1);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) {
      const float so = __shfl_xor_sync(0xffffffffu, s0, o);
      const float eo = __shfl_xor_sync(0xffffffffu, e0, o);
      e0 += eo;
      two_sum1(s0, e0, so);
    }
    const float score = s0 + e0;
    if (sub == 0 && pg < p1)
      out[pg] = r.ok && isfinite(score) ? float_key(score) : kLowest;   // not finite: last
  }
}

__global__ void __launch_bounds__(kPickThreads)
paged_pick_kernel(const PagedBatch b, const uint32_t* __restrict__ keys, int Hkv, int n_top,
                  int n_sink, int n_recent, int smem_keys, int32_t* __restrict__ pages,
                  int32_t* __restrict__ counts) {
  extern __shared__ uint32_t held[];
  __shared__ int hist[kBins];
  __shared__ int scan_gt[kPickThreads / 32], scan_eq[kPickThreads / 32];
  __shared__ uint32_t s_low, s_high, s_bin;
  __shared__ int s_need, s_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, kv = blockIdx.y;
  const int N = n_sink + n_top + n_recent;
  griddep_wait();
  griddep_launch_dependents();
  const int s = warp_find_seq(b, t, lane);
  if (s < 0) return;
  const SeqSpan sp = seq_span(b, s);
  const Span w = span_of(sp, t, b.page_shift, n_top, n_sink, n_recent);
  int32_t* out = pages + ((int64_t)t * Hkv + kv) * N;
  if (tid == 0) counts[(int64_t)t * Hkv + kv] = min(w.vis, N);
  if (w.lo == w.hi) {
    // every visible page fits (w.hi > w.lo otherwise: vis > N)
    for (int i = tid; i < N; i += kPickThreads) out[i] = i < w.vis ? i : -1;
    return;
  }
  for (int i = tid; i < n_sink; i += kPickThreads) out[i] = i;
  for (int i = tid; i < n_recent; i += kPickThreads) out[n_sink + n_top + i] = w.hi + i;
  if (n_top == 0) return;
  const int m = w.hi - w.lo;                       // candidates; m > n_top
  const uint32_t* src = keys + ((int64_t)t * Hkv + kv) * b.max_pages + w.lo;
  const uint32_t* key = src;
  if (tid == 0) {
    s_low = 0xFFFFFFFFu;
    s_high = 0u;
  }
  __syncthreads();
  uint32_t low = 0xFFFFFFFFu, high = 0u;
  for (int i = tid; i < m; i += kPickThreads) {
    const uint32_t x = src[i];
    if (m <= smem_keys) held[i] = x;
    low = min(low, x);
    high = max(high, x);
  }
  if (m <= smem_keys) key = held;
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  if (lane == 0) {
    atomicMin(&s_low, low);
    atomicMax(&s_high, high);
  }
  __syncthreads();
  // The n_top-th largest key, 11 bits a pass from the highest bit in which the
  // keys differ (scores share sign and exponent: their leading bits would put
  // them all in one bin).  The keys x - low of the bin found so far lie in
  // [at, at + 2^shift); `need` of them are kept, and all if there are no more.
  low = s_low;
  int shift = 32 - __clz(s_high - low);              // 0: all keys are equal
  uint32_t at = 0;
  int need = n_top, in_bin = m;
  while (shift > 0 && need < in_bin) {
    const int step = min(shift, kBinBits), down = shift - step;
    for (int i = tid; i < kBins; i += kPickThreads) hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kPickThreads) {
      const uint32_t d = key[i] - low - at;          // wraps for smaller keys
      if (shift == 32 || d >> shift == 0) atomicAdd(&hist[d >> down], 1);
    }
    __syncthreads();
    // thread: four bins, largest first
    int c[kBins / kPickThreads], sum = 0;
#pragma unroll
    for (int i = 0; i < kBins / kPickThreads; ++i) {
      c[i] = hist[kBins - 1 - (tid * (kBins / kPickThreads) + i)];
      sum += c[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) scan_gt[warp] = inc;
    __syncthreads();
    int above = inc - sum;
    {
      const int x = lane < warp ? scan_gt[lane] : 0;
      above += warp_sum_int(x);
    }
    if (above < need && need <= above + sum) {
#pragma unroll
      for (int i = 0; i < kBins / kPickThreads; ++i) {
        if (above < need && need <= above + c[i]) {
          s_bin = kBins - 1 - (tid * (kBins / kPickThreads) + i);
          s_need = need - above;
          s_in = c[i];
        }
        above += c[i];
      }
    }
    __syncthreads();
    at += s_bin << down;
    need = s_need;
    in_bin = s_in;
    shift = down;
  }
  // kept: keys above the bin, and the bin's first `need` (of equal keys, or all
  // of it); thread tid owns a run of candidates, so ranks follow from one scan
  auto above_bin = [&](uint32_t x) {
    const uint32_t d = x - low;
    return d >= at && shift < 32 && (d - at) >> shift != 0;
  };
  auto of_bin = [&](uint32_t x) {
    const uint32_t d = x - low;
    return d >= at && (shift == 32 || (d - at) >> shift == 0);
  };
  const int per = (m + kPickThreads - 1) / kPickThreads;
  const int i0 = min(tid * per, m), i1 = min(i0 + per, m);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = key[i];
    gt += above_bin(x);
    eq += of_bin(x);
  }
  int ig = gt, ie = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, ig, o), y = __shfl_up_sync(0xffffffffu, ie, o);
    if (lane >= o) {
      ig += x;
      ie += y;
    }
  }
  if (lane == 31) {
    scan_gt[warp] = ig;
    scan_eq[warp] = ie;
  }
  __syncthreads();
  int g = ig - gt, q = ie - eq;                    // before this thread's run
  g += warp_sum_int(lane < warp ? scan_gt[lane] : 0);
  q += warp_sum_int(lane < warp ? scan_eq[lane] : 0);
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = key[i];
    const bool over = above_bin(x), same = of_bin(x);
    if (over || (same && q < need)) out[n_sink + g + min(q, need)] = w.lo + i;
    g += over;
    q += same;
  }
}

}  // namespace

size_t paged_select_ws_bytes(int n, int Hkv, int max_pages) {
  return align_up((size_t)n * Hkv * max_pages * sizeof(uint32_t), 256);
}

int launch_paged_select(const PagedBatch& b, const void* q, const void* key_min,
                        const void* key_max, int Hq, int Hkv, int d, bool fp16, int n_top,
                        int n_sink, int n_recent, int32_t* pages, int32_t* counts, void* ws,
                        int32_t* status, cudaStream_t st) {
  uint32_t* keys = static_cast<uint32_t*>(ws);
  // pages a block: enough that the query sums and the first loads' latency are
  // spread over several trips of 16 pages, while the SMs have blocks to overlap
  int per_block = 256;
  while (per_block > 32 &&
         (int64_t)b.n * Hkv * ((b.max_pages + per_block - 1) / per_block) < 4 * kGb300Sms)
    per_block >>= 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  auto score = [&](auto kern, auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    pdl_config(&cfg, attr,
               dim3((b.max_pages + per_block - 1) / per_block, b.n, Hkv), dim3(kScoreThreads), 0,
               st);
    cudaLaunchKernelEx(&cfg, kern, b, static_cast<const T*>(q), static_cast<const T*>(key_min),
                       static_cast<const T*>(key_max), Hq, Hkv, n_top, n_sink, n_recent, per_block,
                       keys, status);
  };
  if (fp16)
    d == 128 ? score(paged_score_kernel<__half, 128>, (__half*)nullptr)
             : score(paged_score_kernel<__half, 64>, (__half*)nullptr);
  else
    d == 128 ? score(paged_score_kernel<__nv_bfloat16, 128>, (__nv_bfloat16*)nullptr)
             : score(paged_score_kernel<__nv_bfloat16, 64>, (__nv_bfloat16*)nullptr);
  int rc = launch_status("paged_score_kernel");
  if (rc) return rc;
  const int smem_keys = b.max_pages < kPickSmemKeys ? b.max_pages : kPickSmemKeys;
  cudaFuncSetAttribute(paged_pick_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       kPickSmemKeys * 4);
  pdl_config(&cfg, attr, dim3(b.n, Hkv), dim3(kPickThreads), (size_t)smem_keys * 4, st);
  cudaLaunchKernelEx(&cfg, paged_pick_kernel, b, (const uint32_t*)keys, Hkv, n_top, n_sink,
                     n_recent, smem_keys, pages, counts);
  return launch_status("paged_pick_kernel");
}

}  // namespace ts
