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
// The scores decide which whole numbers come out, so the choice must not hang
// on the order of a sum: it is that of the sums formed to about 2^-45 and
// rounded to fp32 once.  But only pages near the cut need them so well:
//   scores  every page's sum and its size S = sum |u| |m|, on the tensor cores
//           (memory bound: 4 d bytes a page and KV head).  The sum is off by less
//           than e = (76 + G) 2^-24 S: products are exact, a chain of two products
//           has 32 additions, each taken to be off by at most 2^-23 of what is summed
//           (an assumption: a truncating fp32 adder; nothing documents what the matrix
//           instruction adds in, and choices among scores that differ by its rounding
//           are tested), behind it come 7 roundings to fp32, the query sums' G and the
//           score's own.
//   pick    per (token, KV head) the n_top-th largest of them, T.  With e the
//           largest such error, a page above T + 2 e is kept and one below
//           T - 2 e is not, whatever the errors; when more are left
//           than places, the pages between are formed well (query sums split
//           into a part of 12 bits, whose product with a 16-bit element is
//           exact in fp32, and the rest; the rounding error of every addition
//           kept beside the sum, Knuth's two-sum) and ranked again.  With
//           scores that are not made to tie that is rarely a page.  (One page of very
//           large bounds widens e for all, and many may have to be formed.)
// Forming every page's sum well made the first kernel bound by fp32 arithmetic:
// 39 us for 16 streams of up to 3200 pages (8 KV heads, d = 128), which take 38
// now with both kernels.  (Plain sums on the fp32 pipes took ~90 instructions a
// page: 41.5 us, at d = 64 27.6 for 23.0.)
#include "paged.cuh"
#include "tc_ptx.cuh"

namespace ts {

namespace {

constexpr int kScoreThreads = 128;
constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kBinBits = 11, kBins = 1 << kBinBits;
constexpr int kPickSmemKeys = 48 * 1024;     // larger candidate lists stay in the workspace
constexpr uint32_t kLowest = 0x007FFFFFu;    // float_key(-inf)
constexpr uint32_t kKept = 0xFFFFFFFFu, kDropped = 0u;   // beyond every score's key
constexpr int kPickList = 64;                // close pages ranked against each other
static_assert(kPickWarps <= 32, "one warp scans the warps' sums");

// s + e += p, the sum's rounding error kept in e
__device__ __forceinline__ void two_sum(float& s, float& e, float p) {
  const float t = __fadd_rn(s, p);
  const float bb = __fsub_rn(t, s);
  e = __fadd_rn(e, __fadd_rn(__fsub_rn(s, __fsub_rn(t, bb)), __fsub_rn(p, bb)));
  s = t;
}

// x where it is above 0; a NaN stays one (its pages' scores are not finite)
__device__ __forceinline__ float positive(float x) { return x <= 0.f ? 0.f : x; }

__device__ __forceinline__ float key_float(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
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

// C += A B for 16 pages (rows of A) and 16 columns of their bounds.
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                    uint32_t a3, uint2 b) {
  if (Pair<T>::kFp16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b.x), "r"(b.y));
}

// The first 8 (bf16) or 11 (fp16) bits of x as a T; x becomes the rest.
template <typename T>
__device__ __forceinline__ T lead_bits(float& x) {
  T h;
  if constexpr (Pair<T>::kFp16) h = __float2half_rn(x);
  else h = __ushort_as_bfloat16((unsigned short)(__float_as_uint(x) >> 16));
  x -= Pair<T>::one(h);
  return h;
}

// Per page: .x the score's key, .y its size S (fp32 bits).
//
// A warp takes 16 pages a trip.  Their bounds are the rows of A, read as 16-byte
// words: lane (g, c) = (lane / 4, lane % 4) reads columns 8 (c + 4 x) .. + 7 of
// pages g and g + 8, and as a product does not mind the order of its columns,
// these words are the operand as they lie.  B's columns 0, 1, 2 hold the query
// sums in three parts of T's bits, which together are exact to fp32 (fp16: but
// for 2^-25, where the largest is brought to 2^13 .. 2^14).  Column 3 holds the
// size's |u|: its leading part, and in fp16 2^-7 more, so that e covers what the
// parts lose (76 * 2^-24 * 2^-7 > 2^-25).
template <typename T, int D>
__global__ void __launch_bounds__(kScoreThreads, 3)
paged_score_kernel(const PagedBatch b, const T* __restrict__ q, const T* __restrict__ key_min,
                   const T* __restrict__ key_max, int Hq, int Hkv, int n_top, int n_sink,
                   int n_recent, int per_block, uint2* __restrict__ scores, int32_t* status) {
  constexpr int kX = D / 32, kWarps = kScoreThreads / 32;
  __shared__ __align__(16) T parts[2][4][D];    // query sums' positive, negative parts
  __shared__ float s_top[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.y, kv = blockIdx.z, G = Hq / Hkv;
  const int g = lane >> 2, c = lane & 3;
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && t == 0 && kv == 0)     // every sequence's tables, once
    for (int i = tid; i < b.n_seq; i += kScoreThreads)
      if (seq_span(b, i).bad) set_status(status, TS_ERR_INVALID_ARG);
  const int s = warp_find_seq(b, t, lane);
  if (s < 0) return;
  const SeqSpan sp = seq_span(b, s);
  const Span w = span_of(sp, t, b.page_shift, n_top, n_sink, n_recent);
  const int p0 = w.lo + (int)blockIdx.x * per_block;
  const int p1 = min(w.hi, p0 + per_block);
  if (p0 >= p1) return;
  const int32_t* trow = b.table + (int64_t)s * b.max_pages;
  uint2* out = scores + ((int64_t)t * Hkv + kv) * b.max_pages;
  auto pool_page = [&](int pg) { return pg < p1 ? trow[pg] : 0; };
  int first = p0 + warp * 16;
  int ph[2] = {pool_page(first + g), pool_page(first + g + 8)};
  uint4 mx[2][kX], mn[2][kX];
  bool ok[2];
  // ask for a trip's rows; then for the pool pages of the next
  auto ask = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pg = first + g + 8 * i;
      ok[i] = pg < p1;
      if (ok[i] && (ph[i] < 0 || ph[i] >= b.n_pages)) {
        if (c == 0) set_status(status, TS_ERR_INVALID_ARG);
        ok[i] = false;
      }
      const int64_t row = ((int64_t)(ok[i] ? ph[i] : 0) * Hkv + kv) * (D / 8) + c;
#pragma unroll
      for (int x = 0; x < kX; ++x) {
        mx[i][x] = __ldg(reinterpret_cast<const uint4*>(key_max) + row + 4 * x);
        mn[i][x] = __ldg(reinterpret_cast<const uint4*>(key_min) + row + 4 * x);
      }
      ph[i] = pool_page(pg + kWarps * 16);
    }
  };
  if (first < p1) ask();
  float unscale = 1.f;
  {
    // the query sums, while the first rows are on their way
    float up = 0.f, dn = 0.f;
    if (tid < D) {
      const T* x = q + ((int64_t)t * Hq + kv * G) * D + tid;
#pragma unroll 4
      for (int h = 0; h < G; ++h) {
        const float v = Pair<T>::one(x[h * D]);
        up += positive(v);
        dn -= positive(-v);
      }
    }
    float scale = 1.f;
    if constexpr (Pair<T>::kFp16) {
      const float top = warp_max(fmaxf(up, -dn));
      if (lane == 0) s_top[warp] = top;
      __syncthreads();
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) m = fmaxf(m, s_top[i]);
      const int e = (int)(__float_as_uint(m) >> 23) - 127;
      if (m > 0.f) scale = __uint_as_float((uint32_t)(127 + 13 - e) << 23);
      unscale = 1.f / scale;
    }
    if (tid < D) {
      float u = up * scale, d = dn * scale;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        parts[0][i][tid] = lead_bits<T>(u);
        parts[1][i][tid] = lead_bits<T>(d);
      }
      constexpr float kMore = Pair<T>::kFp16 ? 0.0078125f : 0.f;
      parts[0][3][tid] = T(Pair<T>::one(parts[0][0][tid]) + kMore);
      parts[1][3][tid] = T(kMore - Pair<T>::one(parts[1][0][tid]));
    }
    __syncthreads();
  }
  uint2 uf[2][kX][2];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      const uint4 v = *reinterpret_cast<const uint4*>(&parts[p][min(g, 3)][(c + 4 * x) * 8]);
      uf[p][x][0] = make_uint2(v.x, v.y);
      uf[p][x][1] = make_uint2(v.z, v.w);
    }
  while (first < p1) {
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    float size[4] = {0.f, 0.f, 0.f, 0.f};            // sums of |u| |bound|
#pragma unroll
    for (int x = 0; x < kX; ++x) {
      // (few additions in a row: the error's bound decides how many pages near the
      // cut are formed well)
      float z[2][4] = {};
      mma<T>(z[0], mx[0][x].x, mx[1][x].x, mx[0][x].y, mx[1][x].y, uf[0][x][0]);
      mma<T>(z[1], mn[0][x].x, mn[1][x].x, mn[0][x].y, mn[1][x].y, uf[1][x][0]);
      mma<T>(z[0], mx[0][x].z, mx[1][x].z, mx[0][x].w, mx[1][x].w, uf[0][x][1]);
      mma<T>(z[1], mn[0][x].z, mn[1][x].z, mn[0][x].w, mn[1][x].w, uf[1][x][1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += z[0][i] + z[1][i];
      auto abs4 = [](const uint4& v) {
        return make_uint4(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu);
      };
      const uint4 ax0 = abs4(mx[0][x]), ax1 = abs4(mx[1][x]), an0 = abs4(mn[0][x]), an1 = abs4(mn[1][x]);
      mma<T>(size, ax0.x, ax1.x, ax0.y, ax1.y, uf[0][x][0]);
      mma<T>(size, an0.x, an1.x, an0.y, an1.y, uf[1][x][0]);
      mma<T>(size, ax0.z, ax1.z, ax0.w, ax1.w, uf[0][x][1]);
      mma<T>(size, an0.z, an1.z, an0.w, an1.w, uf[1][x][1]);
    }
    const int done = first;
    const bool read[2] = {ok[0], ok[1]};
    first += kWarps * 16;
    if (first < p1) ask();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // columns 2 c, 2 c + 1 of the products: lane c = 0 has parts 0, 1, lane 1 part 2
      // and the size
      const float a = acc[2 * i];
      const float score = ((a + acc[2 * i + 1]) + __shfl_xor_sync(0xffffffffu, a, 1)) * unscale;
      const float mag = __shfl_xor_sync(0xffffffffu, size[2 * i + 1], 1);
      const int pg = done + g + 8 * i;
      if (c == 0 && pg < p1) {
        // |u|'s leading part is at most 2^-7 of it short
        const float m = mag * unscale * 1.01f;
        const bool good = read[i] && isfinite(score) && isfinite(m);     // the others rank last
        out[pg] = make_uint2(good ? float_key(score) : kLowest, good ? __float_as_uint(m) : 0u);
      }
    }
  }
}

// The candidates' keys: in shared memory, or in the workspace (stride 2).
struct Keys {
  uint32_t* p;
  int stride;
  __device__ __forceinline__ uint32_t get(int i) const { return p[(int64_t)i * stride]; }
  __device__ __forceinline__ void set(int i, uint32_t x) const { p[(int64_t)i * stride] = x; }
};

// Where the n_top-th largest key lies: the keys x with x - low in [at, at +
// 2^shift) are the last bin, of which `need` are kept (all when it holds no
// more).
struct Cut {
  uint32_t low, at;
  int shift, need;
  __device__ __forceinline__ bool above(uint32_t x) const {
    const uint32_t d = x - low;
    return d >= at && shift < 32 && (d - at) >> shift != 0;
  }
  __device__ __forceinline__ bool in(uint32_t x) const {
    const uint32_t d = x - low;
    return d >= at && (shift == 32 || (d - at) >> shift == 0);
  }
};

struct PickSmem {
  int hist[kBins];
  int scan_a[kPickWarps], scan_b[kPickWarps];
  uint32_t low, high, bin, widest;
  int need, in;
  int listed, list[kPickList];               // close pages, and their keys formed well
  uint32_t listed_key[kPickList];
};

// Selection 11 bits a pass from the highest bit in which the keys differ
// (scores share sign and exponent: their leading bits would put them all in one
// bin).  Whole block; low and high: the block's least and largest key.
__device__ Cut find_cut(PickSmem& sm, const Keys& keys, int m, int n_top, uint32_t low,
                        uint32_t high) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Cut c{low, 0, 32 - __clz(high - low), n_top};     // shift 0: all keys are equal
  int in_bin = m;
  while (c.shift > 0 && c.need < in_bin) {
    const int step = min(c.shift, kBinBits), down = c.shift - step;
    for (int i = tid; i < kBins; i += kPickThreads) sm.hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < m; i += kPickThreads) {
      const uint32_t d = keys.get(i) - low - c.at;  // wraps for smaller keys
      if (c.shift == 32 || d >> c.shift == 0) atomicAdd(&sm.hist[d >> down], 1);
    }
    __syncthreads();
    // thread: its bins, largest first
    constexpr int kOwn = kBins / kPickThreads;
    int cnt[kOwn], sum = 0;
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      cnt[i] = sm.hist[kBins - 1 - (tid * kOwn + i)];
      sum += cnt[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sm.scan_a[warp] = inc;
    __syncthreads();
    int above = inc - sum + warp_sum_int(lane < warp ? sm.scan_a[lane] : 0);
    if (above < c.need && c.need <= above + sum) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        if (above < c.need && c.need <= above + cnt[i]) {
          sm.bin = kBins - 1 - (tid * kOwn + i);
          sm.need = c.need - above;
          sm.in = cnt[i];
        }
        above += cnt[i];
      }
    }
    __syncthreads();
    c.at += sm.bin << down;
    c.need = sm.need;
    in_bin = sm.in;
    c.shift = down;
  }
  return c;
}

// The score's key formed well, by a warp (all lanes return it).  qs: query sums
// [positive, negative][12-bit part, rest][column].
template <typename T, int D>
__device__ uint32_t exact_key(const float (*qs)[2][D], const T* mn, const T* mx, int lane) {
  float s = 0.f, e = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int c = lane + 32 * i;
    const float x = Pair<T>::one(mx[c]), n = Pair<T>::one(mn[c]);
    two_sum(s, e, __fmul_rn(qs[0][0][c], x));
    e = fmaf(qs[0][1][c], x, e);
    two_sum(s, e, __fmul_rn(qs[1][0][c], n));
    e = fmaf(qs[1][1][c], n, e);
  }
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const float so = __shfl_xor_sync(0xffffffffu, s, o), eo = __shfl_xor_sync(0xffffffffu, e, o);
    e += eo;
    two_sum(s, e, so);
  }
  const float score = s + e;
  const uint32_t k = isfinite(score) ? float_key(score) : kLowest;
  return __shfl_sync(0xffffffffu, k, 0);      // the lanes' sums may differ in the last place
}

template <typename T, int D>
__global__ void __launch_bounds__(kPickThreads)
paged_pick_kernel(const PagedBatch b, const T* __restrict__ q, const T* __restrict__ key_min,
                  const T* __restrict__ key_max, uint2* __restrict__ scores,
                  int Hq, int Hkv, int n_top, int n_sink,
                  int n_recent, int smem_keys, int32_t* __restrict__ pages,
                  int32_t* __restrict__ counts) {
  extern __shared__ uint32_t held[];
  __shared__ PickSmem sm;
  __shared__ float qs[2][2][D];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int t = blockIdx.x, kv = blockIdx.y, G = Hq / Hkv;
  const int N = n_sink + n_top + n_recent;
  // The score kernel lets this one start only when all that came before is
  // complete, so what it reads as well may be read ahead of its end.
  const int s = warp_find_seq(b, t, lane);
  const SeqSpan sp = seq_span(b, max(s, 0));
  const Span w = span_of(sp, t, b.page_shift, n_top, n_sink, n_recent);
  // the query sums, should a page have to be formed well
  for (int c = tid; c < D; c += kPickThreads) {
    float up = 0.f, upe = 0.f, dn = 0.f, dne = 0.f;
#pragma unroll 4
    for (int g = 0; g < G; ++g) {
      const float x = Pair<T>::one(q[((int64_t)t * Hq + kv * G + g) * D + c]);
      two_sum(up, upe, positive(x));
      two_sum(dn, dne, -positive(-x));
    }
    // 12 leading bits: the product with an 11-bit element is exact
    const float uh = __uint_as_float(__float_as_uint(up) & 0xFFFFF000u);
    const float dh = __uint_as_float(__float_as_uint(dn) & 0xFFFFF000u);
    qs[0][0][c] = uh;
    qs[0][1][c] = (up - uh) + upe;
    qs[1][0][c] = dh;
    qs[1][1][c] = (dn - dh) + dne;
  }
  griddep_wait();
  griddep_launch_dependents();
  if (s < 0) return;
  const int64_t unit = (int64_t)t * Hkv + kv;
  int32_t* out = pages + unit * N;
  if (tid == 0) counts[unit] = min(w.vis, N);
  if (w.lo == w.hi) {
    // every visible page fits (w.hi > w.lo otherwise: vis > N)
    for (int i = tid; i < N; i += kPickThreads) out[i] = i < w.vis ? i : -1;
    return;
  }
  for (int i = tid; i < n_sink; i += kPickThreads) out[i] = i;
  for (int i = tid; i < n_recent; i += kPickThreads) out[n_sink + n_top + i] = w.hi + i;
  if (n_top == 0) return;
  const int m = w.hi - w.lo;                       // candidates; m > n_top
  uint2* src = scores + unit * b.max_pages + w.lo;
  const bool near = m <= smem_keys;
  const Keys keys{near ? held : reinterpret_cast<uint32_t*>(src), near ? 1 : 2};
  auto bounds = [&](uint32_t low, uint32_t high, uint32_t widest) {
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    widest = __reduce_max_sync(0xffffffffu, widest);
    __syncthreads();
    if (tid == 0) {
      sm.low = 0xFFFFFFFFu;
      sm.high = sm.widest = 0u;
    }
    __syncthreads();
    if (lane == 0) {
      atomicMin(&sm.low, low);
      atomicMax(&sm.high, high);
      atomicMax(&sm.widest, widest);
    }
    __syncthreads();
  };
  uint32_t low = 0xFFFFFFFFu, high = 0u, widest = 0u;
#pragma unroll 8
  for (int i = tid; i < m; i += kPickThreads) {
    const uint2 x = src[i];
    if (near) held[i] = x.x;
    low = min(low, x.x);
    high = max(high, x.x);
    widest = max(widest, x.y);                     // magnitudes order as their bits
  }
  if (tid == 0) sm.listed = 0;
  bounds(low, high, widest);
  Cut cut = find_cut(sm, keys, m, n_top, sm.low, sm.high);
  // pages that may be on either side of the cut
  const float delta = 2.125f * (76.f + G) * 5.9604645e-8f * __uint_as_float(sm.widest);
  const uint32_t bin0 = cut.low + cut.at;
  const uint32_t bin1 = cut.shift == 32 ? 0xFFFFFFFFu : bin0 + ((1u << cut.shift) - 1u);
  const float from = key_float(bin0) - delta, to = key_float(min(bin1, sm.high)) + delta;
  auto side = [&](uint32_t x) {                    // 2: kept, 1: near the cut, 0: not kept
    const float f = key_float(x);
    return f > to ? 2 : f < from ? 0 : 1;
  };
  int over = 0, close = 0;
  for (int i = tid; i < m; i += kPickThreads) {
    const int x = side(keys.get(i));
    over += x == 2;
    if (x == 1) {
      ++close;
      const int at = atomicAdd(&sm.listed, 1);
      if (at < kPickList) sm.list[at] = i;
    }
  }
  over = __reduce_add_sync(0xffffffffu, over);
  close = __reduce_add_sync(0xffffffffu, close);
  __syncthreads();                                 // the sums' places were read in find_cut
  if (lane == 0) {
    sm.scan_a[warp] = over;
    sm.scan_b[warp] = close;
  }
  __syncthreads();
  over = warp_sum_int(lane < kPickWarps ? sm.scan_a[lane] : 0);
  close = warp_sum_int(lane < kPickWarps ? sm.scan_b[lane] : 0);
  const int32_t* trow = b.table + (int64_t)s * b.max_pages + w.lo;
  auto formed = [&](int i) {
    const int64_t row = ((int64_t)trow[i] * Hkv + kv) * D;
    return exact_key<T, D>(qs, key_min + row, key_max + row, lane);
  };
  const bool all_close = over + close <= n_top;
  const bool few = !all_close && close <= kPickList;
  if (few) {
    // rank the close ones against each other: the best take the places left
    for (int a = warp; a < close; a += kPickWarps) {
      const int i = sm.list[a];
      const uint32_t x = keys.get(i);
      // a page that ranks last has no score to form
      const uint32_t k = x == kLowest ? x : formed(i);
      if (lane == 0) sm.listed_key[a] = k;
    }
    __syncthreads();
    bool best = false;
    int mine = 0;
    if (tid < close) {
      mine = sm.list[tid];
      const uint32_t k = sm.listed_key[tid];
      int before = 0;
      for (int a = 0; a < close; ++a)
        before += sm.listed_key[a] > k || (sm.listed_key[a] == k && sm.list[a] < mine);
      best = before < n_top - over;
    }
    __syncthreads();
    if (tid < close) keys.set(mine, best ? kKept : kDropped);
    __syncthreads();
  } else if (!all_close) {
    // form all close ones well and rank everything again: kept pages first, the
    // others last
    low = 0xFFFFFFFFu;
    high = 0u;
    for (int base = warp * 32; base < m; base += kPickThreads) {
      const int i = base + lane;
      uint32_t x = i < m ? keys.get(i) : kDropped;
      const int where = i < m ? side(x) : 0;
      if (where != 1) x = where == 2 ? kKept : kDropped;
      unsigned todo = __ballot_sync(0xffffffffu, where == 1 && x != kLowest);
      while (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const uint32_t k = formed(base + l);
        if (lane == l) x = k;
      }
      if (i < m) {
        keys.set(i, x);
        low = min(low, x);
        high = max(high, x);
      }
    }
    bounds(low, high, 0u);
    cut = find_cut(sm, keys, m, n_top, sm.low, sm.high);
  }
  // ordered write; thread tid owns a run of candidates, so ranks follow from
  // one scan: all close pages where they fit, else what the second cut says
  const bool ranked = !all_close && !few;
  auto kept = [&](uint32_t x) {
    return ranked ? cut.above(x) : few ? x == kKept || (x != kDropped && side(x) == 2) : side(x) != 0;
  };
  const int per = (m + kPickThreads - 1) / kPickThreads;
  const int i0 = min(tid * per, m), i1 = min(i0 + per, m);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = keys.get(i);
    gt += kept(x);
    eq += ranked && cut.in(x);
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
  __syncthreads();
  if (lane == 31) {
    sm.scan_a[warp] = ig;
    sm.scan_b[warp] = ie;
  }
  __syncthreads();
  // kept and in the bin before this thread's run
  int g = ig - gt + warp_sum_int(lane < warp ? sm.scan_a[lane] : 0);
  int e = ie - eq + warp_sum_int(lane < warp ? sm.scan_b[lane] : 0);
  const int need = ranked ? cut.need : 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t x = keys.get(i);
    const bool is_over = kept(x), same = ranked && cut.in(x);
    if (is_over || (same && e < need)) out[n_sink + g + min(e, need)] = w.lo + i;
    g += is_over;
    e += same;
  }
}

}  // namespace

size_t paged_select_ws_bytes(int n, int Hkv, int max_pages) {
  return align_up((size_t)n * Hkv * max_pages * sizeof(uint2), 256);
}

template <typename T, int D>
static int go_select(const PagedBatch& b, const void* q, const void* key_min, const void* key_max,
                     int Hq, int Hkv, int n_top, int n_sink, int n_recent, int32_t* pages,
                     int32_t* counts, void* ws, int32_t* status, cudaStream_t st) {
  uint2* scores = static_cast<uint2*>(ws);
  const T* qt = static_cast<const T*>(q);
  const T* mn = static_cast<const T*>(key_min);
  const T* mx = static_cast<const T*>(key_max);
  // pages a block: enough that the query sums and the first loads' latency are
  // spread over several trips of 64 pages, while the SMs have blocks to overlap
  // (128, 256, 512 a block: 39.0, 38.6, 42.2 us on the 16 streams above)
  int per_block = 256;
  while (per_block > 64 &&
         (int64_t)b.n * Hkv * ((b.max_pages + per_block - 1) / per_block) < 4 * kGb300Sms)
    per_block >>= 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((b.max_pages + per_block - 1) / per_block, b.n, Hkv),
             dim3(kScoreThreads), 0, st);
  cudaLaunchKernelEx(&cfg, paged_score_kernel<T, D>, b, qt, mn, mx, Hq, Hkv, n_top, n_sink,
                     n_recent, per_block, scores, status);
  int rc = launch_status("paged_score_kernel");
  if (rc) return rc;
  const int smem_keys = b.max_pages < kPickSmemKeys ? b.max_pages : kPickSmemKeys;
  cudaFuncSetAttribute(paged_pick_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                       kPickSmemKeys * 4);
  pdl_config(&cfg, attr, dim3(b.n, Hkv), dim3(kPickThreads), (size_t)smem_keys * 4, st);
  cudaLaunchKernelEx(&cfg, paged_pick_kernel<T, D>, b, qt, mn, mx, scores, Hq,
                     Hkv, n_top, n_sink, n_recent, smem_keys, pages, counts);
  return launch_status("paged_pick_kernel");
}

int launch_paged_select(const PagedBatch& b, const void* q, const void* key_min,
                        const void* key_max, int Hq, int Hkv, int d, bool fp16, int n_top,
                        int n_sink, int n_recent, int32_t* pages, int32_t* counts, void* ws,
                        int32_t* status, cudaStream_t st) {
  auto go = [&](auto run) {
    return run(b, q, key_min, key_max, Hq, Hkv, n_top, n_sink, n_recent, pages, counts, ws, status,
               st);
  };
  if (fp16) return d == 128 ? go(go_select<__half, 128>) : go(go_select<__half, 64>);
  return d == 128 ? go(go_select<__nv_bfloat16, 128>) : go(go_select<__nv_bfloat16, 64>);
}

}  // namespace ts
