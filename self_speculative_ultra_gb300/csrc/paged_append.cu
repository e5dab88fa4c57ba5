// Rotary positions fused with the write of new tokens into a paged cache.
//
// A pair (x, y) of a query or key row at position p turns by a = p * f_c:
//   (x, y) -> ((x cos a - y sin a) * scale, (y cos a + x sin a) * scale).
// The angle is kept in turns: f_c / 2 pi as a sum of two floats, p as a sum of
// two exact floats, each product with its rounding error, so only the
// fraction of a turn is ever rounded and far positions lose nothing.
//
// Memory bound: every element is read and written once (9.9K tokens, 32/32
// heads, half of 128 columns rotated: 41 us, 5.95 TB/s).  One launch; block
// roles by index:
//   page blocks  one (touched page, chunk of KV heads): rotate the page's new
//                key rows, copy its value rows, and fold the rows' bounds
//                (element-wise minimum and maximum).  A page's new rows are
//                handled by one block, so its bounds need no atomics.
//   query blocks 16 tokens x 8 query heads.
// cos/sin are formed once per (token, pair) in shared memory and used by all
// of the block's heads, while the rows they turn are on their way to registers.
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kThreads = 256;
constexpr int kSub = 32;        // most tokens of a page block per trip
constexpr int kQTok = 16;       // tokens of a query block
constexpr int kQHeads = 8;      // heads of a query block, at d = 128

struct Smem {
  union {
    // (cos, sin) * scale of pair c: half c % 2 of cs[.][c % 8 / 2][c / 8], so
    // that neighbouring units read neighbouring 16-byte words
    float4 cs[kSub][4][8];
    uint4 red[kThreads][4];              // bounds: minimum (2), maximum (2)
  };
  float2 turn[64];                       // f / 2 pi = x + y
  int pos[kQTok];
  int scan[kThreads / 32];
  int seq, page;
};

__device__ __forceinline__ float2 sincos_turns(int pos, float2 f, float scale) {
  // pos = hi + lo, both exact in fp32
  const float lo = (float)(pos & 4095), hi = (float)(pos - (pos & 4095));
  const float p1 = hi * f.x, p2 = lo * f.x;
  const float e = fmaf(hi, f.x, -p1) + fmaf(lo, f.x, -p2) + (hi + lo) * f.y;
  const float r0 = (p1 - rintf(p1)) + (p2 - rintf(p2)) + e;
  // within half a turn the hardware's sine and cosine are good to 2^-21, far
  // below half a step of a 16-bit output (9.9K tokens, 32/32 heads of 128 rotated
  // columns: 42.1 us, with the accurate ones 46.3)
  float s, c;
  __sincosf((r0 - rintf(r0)) * 6.283185307179586f, &s, &c);
  return make_float2(c * scale, s * scale);
}

// Rotate unit u (two 16-byte chunks a, b of one head row) in place.  In the
// half layout chunk a holds first members and b second members of 8 pairs
// starting at pair 8 u; interleaved, a and b hold pairs 8 u .. + 3, + 4 .. + 7.
template <typename T>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float4 (*cs)[8], int u, bool inter) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
  const float4 t[4] = {cs[0][u], cs[1][u], cs[2][u], cs[3][u]};
  if (inter) {
    auto turn = [](uint32_t w, float c, float s) {
      const float2 x = Pair<T>::unpack(w);
      return Pair<T>::pack(x.x * c - x.y * s, x.y * c + x.x * s);
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wa[2 * i] = turn(wa[2 * i], t[i].x, t[i].y);
      wa[2 * i + 1] = turn(wa[2 * i + 1], t[i].z, t[i].w);
      wb[2 * i] = turn(wb[2 * i], t[2 + i].x, t[2 + i].y);
      wb[2 * i + 1] = turn(wb[2 * i + 1], t[2 + i].z, t[2 + i].w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = Pair<T>::unpack(wa[i]), y = Pair<T>::unpack(wb[i]);
      wa[i] = Pair<T>::pack(x.x * t[i].x - y.x * t[i].y, x.y * t[i].z - y.y * t[i].w);
      wb[i] = Pair<T>::pack(y.x * t[i].x + x.x * t[i].y, y.y * t[i].z + x.y * t[i].w);
    }
  }
}

// Chunk indices of unit u (0 .. D/16 - 1) of a head row; false: the unit lies
// behind the rotated part.
__device__ __forceinline__ bool unit_chunks(int u, int rot, bool inter, int& ca, int& cb) {
  const int nr = rot / 16;
  const bool turned = u < nr;
  ca = turned && !inter ? u : 2 * u;
  cb = turned && !inter ? u + nr : 2 * u + 1;
  return turned;
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
__global__ void __launch_bounds__(kThreads, 3)
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
    constexpr int kHeads = kQHeads * 128 / D;
    const int n_hc = (a.Hq + kHeads - 1) / kHeads;
    const int t0 = qb / n_hc * kQTok, h0 = qb % n_hc * kHeads;
    const int nh = min(kHeads, a.Hq - h0);
    // a thread's rows, asked for first (a token of no sequence has a row too)
    constexpr int kEach = kQTok * kQHeads * 8 / kThreads;   // units a thread
    const int n_units = kQTok * nh * kUnits;
    uint4 xa[kEach], xb[kEach];
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = tid + i * kThreads;
      const int u = e % kUnits, h = e / kUnits % nh, t = t0 + e / (kUnits * nh);
      if (e < n_units && t < b.n) {
        int ca, cb;
        const bool turned = unit_chunks(u, a.rot, inter, ca, cb);
        const uint4* src = reinterpret_cast<const uint4*>(q + t * a.q_stride + (int64_t)(h0 + h) * D);
        xa[i] = src[ca];
        xb[i] = src[cb];
      }
    }
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
      reinterpret_cast<float2*>(&sm.cs[i][(c & 7) >> 1][c >> 3])[c & 1] =
          sincos_turns(sm.pos[i], sm.turn[c], a.rope_scale);
    }
    __syncthreads();
    T* out = static_cast<T*>(a.q_out);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int e = tid + i * kThreads;
      const int u = e % kUnits, h = e / kUnits % nh, at = e / (kUnits * nh), t = t0 + at;
      if (e >= n_units || t >= b.n || sm.pos[at] == INT_MIN) continue;   // of no sequence
      int ca, cb;
      const bool turned = unit_chunks(u, a.rot, inter, ca, cb);
      if (turned) rotate<T>(xa[i], xb[i], sm.cs[at], u, inter);
      uint4* dst = reinterpret_cast<uint4*>(out + ((int64_t)t * a.Hq + h0 + h) * D);
      dst[ca] = xa[i];
      dst[cb] = xb[i];
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
  int ca, cb;
  const bool turned = unit_chunks(u, a.rot, inter, ca, cb);
  uint4 loa, lob, hia, hib;
  bool any = false;
  constexpr int kEach = 2;               // tokens of a trip a thread
  const int per_trip = min(kSub, kEach * n_tl);
  for (int t0 = r0; t0 < r1; t0 += per_trip) {
    const int m = min(per_trip, r1 - t0);
    uint4 kx[kEach], ky[kEach], vx[kEach], vy[kEach];
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int i = tl + x * n_tl;
      if (h < nh && i < m) {
        const int64_t t = sp.q0 + (t0 + i - a0);
        const uint4* ks = reinterpret_cast<const uint4*>(k + t * a.k_stride + (int64_t)(h0 + h) * D);
        const uint4* vs = reinterpret_cast<const uint4*>(v + t * a.v_stride + (int64_t)(h0 + h) * D);
        kx[x] = ks[ca];
        ky[x] = ks[cb];
        vx[x] = vs[2 * u];
        vy[x] = vs[2 * u + 1];
      }
    }
    __syncthreads();                     // the trip before is done with cos/sin
    for (int e = tid; e < m * half; e += kThreads) {
      const int i = e / half, c = e - i * half;
      const int pos = a.positions ? a.positions[sp.q0 + (t0 + i - a0)] : t0 + i;
      reinterpret_cast<float2*>(&sm.cs[i][(c & 7) >> 1][c >> 3])[c & 1] =
          sincos_turns(pos, sm.turn[c], a.rope_scale);
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int i = tl + x * n_tl;
      if (h < nh && i < m) {
        if (turned) rotate<T>(kx[x], ky[x], sm.cs[i], u, inter);
        const int64_t row = ((phys * a.Hkv + h0 + h) << b.page_shift) + ((t0 + i) & (ps - 1));
        uint4* kd = reinterpret_cast<uint4*>(kp + row * D);
        uint4* vd = reinterpret_cast<uint4*>(vp + row * D);
        kd[ca] = kx[x];
        kd[cb] = ky[x];
        vd[2 * u] = vx[x];
        vd[2 * u + 1] = vy[x];
        if (!any) {
          loa = hia = kx[x];
          lob = hib = ky[x];
          any = true;
        } else {
          fold<T>(loa, hia, kx[x]);
          fold<T>(lob, hib, ky[x]);
        }
      }
    }
  }
  if (!a.key_min) return;
  __syncthreads();
  // token lanes beyond the page's rows hold nothing; lane 0 always does
  sm.red[tid][0] = loa;
  sm.red[tid][1] = lob;
  sm.red[tid][2] = hia;
  sm.red[tid][3] = hib;
  __syncthreads();
  if (tid < combos && h < nh) {
    const int live = min(n_tl, min(per_trip, r1 - r0));   // lanes that saw a row
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
  int hpb = 4 * 128 / d;
  while (hpb > 1 && (hpb > a.Hkv || slots * ((a.Hkv + hpb - 1) / hpb) < 4 * kGb300Sms)) hpb >>= 1;
  const int64_t page_blocks = slots * ((a.Hkv + hpb - 1) / hpb);
  const int q_heads = kQHeads * 128 / d;
  const int64_t q_blocks =
      (int64_t)((b.n + kQTok - 1) / kQTok) * ((a.Hq + q_heads - 1) / q_heads);
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
