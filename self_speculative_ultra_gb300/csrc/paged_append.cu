// Rotary positions fused with the write of new tokens into a paged cache.
//
// A pair (x, y) of a query or key row at position p turns by a = p * f_c:
//   (x, y) -> ((x cos a - y sin a) * scale, (y cos a + x sin a) * scale).
// The angle is kept in turns: f_c / 2 pi as a sum of two floats, p as a sum of
// two exact floats, each product with its rounding error, so only the
// fraction of a turn is ever rounded and far positions lose nothing
// (cos(2 pi r) then comes from the half-turn functions).
//
// Memory bound: every element is read and written once.  One launch; block
// roles by index:
//   page blocks  one (touched page, chunk of KV heads): rotate the page's new
//                key rows, copy its value rows, and fold the rows' bounds
//                (element-wise minimum and maximum).  A page's new rows are
//                handled by one block, so its bounds need no atomics.
//   query blocks 16 tokens x 8 query heads.
// cos/sin are formed once per (token, pair) in shared memory and used by all
// of the block's heads.
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kThreads = 256;
constexpr int kSub = 32;        // tokens of a page block per trip
constexpr int kQTok = 16;       // tokens of a query block
constexpr int kQHeads = 8;      // heads of a query block

struct Smem {
  union {
    float2 cs[kSub][64];                 // (cos, sin) * scale
    uint4 red[kThreads][4];              // bounds: minimum (2), maximum (2)
  };
  float2 turn[64];                       // f / 2 pi = x + y
  int pos[kSub];
  int scan[kThreads / 32];
  int seq, page;
};

__device__ __forceinline__ float2 sincos_turns(int pos, float2 f, float scale) {
  // pos = hi + lo, both exact in fp32
  const float lo = (float)(pos & 4095), hi = (float)(pos - (pos & 4095));
  const float p1 = hi * f.x, p2 = lo * f.x;
  const float e = fmaf(hi, f.x, -p1) + fmaf(lo, f.x, -p2) + (hi + lo) * f.y;
  const float r = (p1 - rintf(p1)) + (p2 - rintf(p2)) + e;
  float s, c;
  sincospif(2.f * r, &s, &c);
  return make_float2(c * scale, s * scale);
}

// Rotate the unit (two 16-byte chunks a, b of one head row) in place.  In the
// half layout chunk a holds first members and b second members of 8 pairs
// starting at pair c0; interleaved, a and b hold pairs c0..c0+3, c0+4..c0+7.
template <typename T>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float2* cs, bool inter) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = Pair<T>::unpack(wa[i]), y = Pair<T>::unpack(wb[i]);
      const float2 t = cs[i], u = cs[4 + i];
      wa[i] = Pair<T>::pack(x.x * t.x - x.y * t.y, x.y * t.x + x.x * t.y);
      wb[i] = Pair<T>::pack(y.x * u.x - y.y * u.y, y.y * u.x + y.x * u.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = Pair<T>::unpack(wa[i]), y = Pair<T>::unpack(wb[i]);
      const float2 t = cs[2 * i], u = cs[2 * i + 1];
      wa[i] = Pair<T>::pack(x.x * t.x - y.x * t.y, x.y * u.x - y.y * u.y);
      wb[i] = Pair<T>::pack(y.x * t.x + x.x * t.y, y.y * u.x + x.y * u.y);
    }
  }
}

// Chunk indices of unit u (0 .. D/16 - 1) of a head row, and its first pair
// (-1: the unit lies behind the rotated part).
__device__ __forceinline__ void unit_chunks(int u, int rot, bool inter, int& ca, int& cb, int& c0) {
  const int nr = rot / 16;
  if (u < nr) {
    ca = inter ? 2 * u : u;
    cb = inter ? 2 * u + 1 : u + nr;
    c0 = 8 * u;
  } else {
    ca = 2 * u;
    cb = 2 * u + 1;
    c0 = -1;
  }
}

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
__global__ void __launch_bounds__(kThreads, 4)
paged_append_kernel(const PagedBatch b, const AppendArgs a, int n_page_blocks, int heads_per_block,
                    int32_t* status) {
  __shared__ Smem sm;
  constexpr int kUnits = D / 16;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int half = a.rot / 2;
  const bool inter = a.interleaved != 0;
  griddep_wait();
  griddep_launch_dependents();
  if (tid < half) {
    const double f = a.freqs[tid] * 0.15915494309189533577;   // 1 / (2 pi)
    const float hi = (float)f;
    sm.turn[tid] = make_float2(hi, (float)(f - (double)hi));
  }
  const T* k = static_cast<const T*>(a.k);
  const T* v = static_cast<const T*>(a.v);
  const T* q = static_cast<const T*>(a.q);

  if ((int)blockIdx.x >= n_page_blocks) {
    // ------------------------------------------------------------ queries
    const int qb = blockIdx.x - n_page_blocks;
    const int n_hc = (a.Hq + kQHeads - 1) / kQHeads;
    const int t0 = qb / n_hc * kQTok, h0 = qb % n_hc * kQHeads;
    const int nh = min(kQHeads, a.Hq - h0);
    // positions of the block's tokens: each thread looks at its sequences
    if (tid < kQTok) sm.pos[tid] = INT_MIN;
    __syncthreads();
    for (int s = tid; s < b.n_seq; s += kThreads) {
      const SeqSpan sp = seq_span(b, s);
      for (int t = max(sp.q0, t0); t < min(sp.q0 + sp.ql, t0 + kQTok); ++t)
        sm.pos[t - t0] = a.positions ? a.positions[t] : sp.kl - sp.ql + (t - sp.q0);
    }
    __syncthreads();
    for (int e = tid; e < kQTok * half; e += kThreads) {
      const int i = e / half, c = e - i * half;
      sm.cs[i][c] = sincos_turns(sm.pos[i], sm.turn[c], a.rope_scale);
    }
    __syncthreads();
    T* out = static_cast<T*>(a.q_out);
#pragma unroll 2
    for (int e = tid; e < kQTok * nh * kUnits; e += kThreads) {
      const int u = e % kUnits, h = e / kUnits % nh, i = e / (kUnits * nh);
      const int t = t0 + i;
      if (t >= b.n || sm.pos[i] == INT_MIN) continue;   // behind the last sequence
      int ca, cb, c0;
      unit_chunks(u, a.rot, inter, ca, cb, c0);
      const uint4* src = reinterpret_cast<const uint4*>(q + t * a.q_stride + (int64_t)(h0 + h) * D);
      uint4 x = src[ca], y = src[cb];
      if (c0 >= 0) rotate<T>(x, y, &sm.cs[i][c0], inter);
      uint4* dst = reinterpret_cast<uint4*>(out + ((int64_t)t * a.Hq + h0 + h) * D);
      dst[ca] = x;
      dst[cb] = y;
    }
    return;
  }

  // -------------------------------------------------------------- pages
  const int n_hc = (a.Hkv + heads_per_block - 1) / heads_per_block;
  const int slot = blockIdx.x / n_hc, h0 = blockIdx.x % n_hc * heads_per_block;
  const int nh = min(heads_per_block, a.Hkv - h0);
  // the slot-th touched page of the batch: a running count over sequences
  if (tid == 0) sm.seq = -1;
  int before = 0;
  for (int base = 0; base < b.n_seq; base += kThreads) {
    const int s = base + tid;
    int cnt = 0, first = 0;
    if (s < b.n_seq) {
      const SeqSpan sp = seq_span(b, s);
      const int a0 = max(sp.kl - sp.ql, 0);
      if (sp.ql > 0 && sp.kl > 0) {
        first = a0 >> b.page_shift;
        cnt = ((sp.kl - 1) >> b.page_shift) - first + 1;
      }
      if (blockIdx.x == 0 && (sp.bad || sp.kl < sp.ql)) set_status(status, TS_ERR_INVALID_ARG);
    }
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) sm.scan[warp] = inc;
    __syncthreads();
    int off = before, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const int x = sm.scan[w];
      if (w < warp) off += x;
      total += x;
    }
    if (slot >= off + inc - cnt && slot < off + inc) {
      sm.seq = s;
      sm.page = first + slot - (off + inc - cnt);
    }
    before += total;
    __syncthreads();
    if (slot < before && blockIdx.x != 0) break;   // uniform; block 0 checks every sequence
  }
  __syncthreads();
  const int s = sm.seq, pg = sm.page;
  if (s < 0) return;
  const SeqSpan sp = seq_span(b, s);
  const int a0 = sp.kl - sp.ql;                       // row of the first new token
  const int r0 = max(max(a0, 0), pg << b.page_shift);
  const int r1 = min(sp.kl, (pg + 1) << b.page_shift);
  const int64_t phys = b.table[(int64_t)s * b.max_pages + pg];
  if (phys < 0 || phys >= b.n_pages) {
    if (tid == 0) set_status(status, TS_ERR_INVALID_ARG);
    return;
  }
  const int ps = 1 << b.page_shift;
  T* kp = static_cast<T*>(a.k_pages);
  T* vp = static_cast<T*>(a.v_pages);
  // thread = (token lane, head, unit); the head and unit stay for all tokens,
  // so the bounds accumulate in registers
  const int combos = heads_per_block * kUnits;
  const int combo = tid % combos, tl = tid / combos, n_tl = kThreads / combos;
  const int h = combo / kUnits, u = combo % kUnits;
  int ca, cb, c0;
  unit_chunks(u, a.rot, inter, ca, cb, c0);
  uint4 loa, lob, hia, hib;
  bool any = false;
  for (int t0 = r0; t0 < r1; t0 += kSub) {
    const int m = min(kSub, r1 - t0);
    if (tid < m) {
      const int t = sp.q0 + (t0 + tid - a0);
      sm.pos[tid] = a.positions ? a.positions[t] : t0 + tid;
    }
    __syncthreads();
    for (int e = tid; e < m * half; e += kThreads) {
      const int i = e / half, c = e - i * half;
      sm.cs[i][c] = sincos_turns(sm.pos[i], sm.turn[c], a.rope_scale);
    }
    __syncthreads();
    if (h < nh) {
#pragma unroll 2
      for (int i = tl; i < m; i += n_tl) {
        const int64_t t = sp.q0 + (t0 + i - a0);
        const uint4* ks = reinterpret_cast<const uint4*>(k + t * a.k_stride + (int64_t)(h0 + h) * D);
        const uint4* vs = reinterpret_cast<const uint4*>(v + t * a.v_stride + (int64_t)(h0 + h) * D);
        uint4 x = ks[ca], y = ks[cb];
        const uint4 va = vs[2 * u], vb = vs[2 * u + 1];
        if (c0 >= 0) rotate<T>(x, y, &sm.cs[i][c0], inter);
        const int64_t row = ((phys * a.Hkv + h0 + h) << b.page_shift) + ((t0 + i) & (ps - 1));
        uint4* kd = reinterpret_cast<uint4*>(kp + row * D);
        uint4* vd = reinterpret_cast<uint4*>(vp + row * D);
        kd[ca] = x;
        kd[cb] = y;
        vd[2 * u] = va;
        vd[2 * u + 1] = vb;
        if (!any) {
          loa = hia = x;
          lob = hib = y;
          any = true;
        } else {
          fold<T>(loa, hia, x);
          fold<T>(lob, hib, y);
        }
      }
    }
    __syncthreads();
  }
  if (!a.key_min) return;
  // token lanes beyond the page's rows hold nothing; lane 0 always does
  sm.red[tid][0] = loa;
  sm.red[tid][1] = lob;
  sm.red[tid][2] = hia;
  sm.red[tid][3] = hib;
  __syncthreads();
  if (tid < combos && h < nh) {
    // lanes that saw a row: the longest trip had min(kSub, rows) tokens
    const int live = min(n_tl, min(kSub, r1 - r0));
    for (int j = 1; j < live; ++j) {
      const uint4* o = sm.red[j * combos + tid];
      fold<T>(loa, hia, o[0]);
      fold<T>(lob, hib, o[1]);
      fold<T>(loa, hia, o[2]);
      fold<T>(lob, hib, o[3]);
    }
    uint4* mn = reinterpret_cast<uint4*>(static_cast<T*>(a.key_min) + (phys * a.Hkv + h0 + h) * D);
    uint4* mx = reinterpret_cast<uint4*>(static_cast<T*>(a.key_max) + (phys * a.Hkv + h0 + h) * D);
    if (r0 > (pg << b.page_shift)) {       // rows in front were held before
      fold<T>(loa, hia, mn[ca]);
      fold<T>(lob, hib, mn[cb]);
      fold<T>(loa, hia, mx[ca]);
      fold<T>(lob, hib, mx[cb]);
    }
    mn[ca] = loa;
    mn[cb] = lob;
    mx[ca] = hia;
    mx[cb] = hib;
  }
}

}  // namespace

int launch_paged_append(const PagedBatch& b, const AppendArgs& a, int d, bool fp16,
                        int32_t* status, cudaStream_t st) {
  // touched pages: at most one a token, and ql / ps + 2 a sequence
  const int64_t slots = imin64(b.n, (b.n >> b.page_shift) + 2 * (int64_t)b.n_seq);
  // KV heads of a page block: more heads share the block's cos/sin, fewer
  // heads fill the SMs when few pages are touched
  int hpb = 4;
  while (hpb > 1 && (hpb > a.Hkv || slots * ((a.Hkv + hpb - 1) / hpb) < 4 * kGb300Sms)) hpb >>= 1;
  const int64_t page_blocks = slots * ((a.Hkv + hpb - 1) / hpb);
  const int64_t q_blocks =
      (int64_t)((b.n + kQTok - 1) / kQTok) * ((a.Hq + kQHeads - 1) / kQHeads);
  const int64_t blocks = page_blocks + q_blocks;
  if (blocks > INT32_MAX)
    return fail(TS_ERR_UNSUPPORTED, "ts_paged_rope_append: %lld blocks in one launch",
                (long long)blocks);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)blocks), dim3(kThreads), 0, st);
  auto go = [&](auto kern) {
    cudaLaunchKernelEx(&cfg, kern, b, a, (int)page_blocks, hpb, status);
  };
  if (fp16)
    d == 128 ? go(paged_append_kernel<__half, 128>) : go(paged_append_kernel<__half, 64>);
  else
    d == 128 ? go(paged_append_kernel<__nv_bfloat16, 128>)
             : go(paged_append_kernel<__nv_bfloat16, 64>);
  return launch_status("paged_append_kernel");
}

}  // namespace ts
