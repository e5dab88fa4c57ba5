// Attention of few query rows over a paged cache: the next token of a batch
// of streams (or a few tokens each), and its sparse form over per-token page
// lists.
//
//   s_ij = q_i . k_j / sqrt(d),  o_i = softmax_j(s) . v,  lse_i = ln sum exp(s)
//
// over the rows j <= seq_len - q_len + i of the sequence (dense), or those of
// them in the token's listed pages (sparse).
//
// Memory bound: K and V are read once, 4 d bytes a key and KV head.  The
// query rows of a KV head (new tokens x group) are packed into blocks of 16,
// so a key tile is read once for all of them.  A unit is one block of rows of
// one KV head; all units' keys, in trips of 128, form one line of work that is
// cut into equal stretches, one a SM, whatever the lengths: a unit that a cut
// falls into is joined by a second kernel.  A CTA's four warps work on their
// own 32-key tiles of a trip: each streams its tiles through its own ring of
// asynchronous copies, which runs on across units, and runs the online softmax
// by itself, without a CTA-wide barrier; the four states are joined at the
// unit's end in shared memory.
// Q.K^T and P.V use 16x8x16 matrix instructions: 16 rows never fill a tensor
// core tile, so the copy engine's 128-row tiles would only pad.  P is split
// into a 16-bit value and its 16-bit remainder (two products), so P.V sees a
// weight to 16 bits (bf16), or to 22 (fp16) but for 2^-33 of the largest weight
// of its 32 keys (see moved()).
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTileKeys = 32;              // keys of a warp's tile
constexpr int kStep = kWarps * kTileKeys;  // keys a CTA takes per trip
constexpr int kStages = 2;
constexpr int kMinTrips = 2;               // trips a CTA takes at least
constexpr int kMostCluster = 8;            // CTAs of a cluster
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Ring {
  static constexpr int kRow = D * 2;
  static constexpr int kTile = kTileKeys * kRow;
  static constexpr int kStage = 2 * kTile;                 // K tile, V tile
  static constexpr int kStates = kWarps * kStages * kStage;  // the warps' states at a unit's end
  static constexpr int kBytes = kStates + kWarps * 16 * (D + 2) * 4;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool fill) {
  const int n = fill ? 16 : 0;            // 0: sixteen zero bytes
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n));
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
template <typename T>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  if (Pair<T>::kFp16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                 "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Where the reference m of P = 2^(x - m) stands for 32 keys whose largest
// exponent is y.  In bf16 it is the running maximum.  fp16 has nothing below
// 2^-24: against a maximum far above (a first key that draws most of the
// attention) the tail's weights would round to 0 while their sum counts them.
// So there the reference goes with the keys, up and down: it stays while their
// largest P is 2^8 .. 2^15 and is set for 2^12 else, and a weight is off by at
// most 2^-25 in these units.  O and l are held in the same units; `least` keeps
// them below 2^120 (2^64 for a reference that falls, 2^15 a weight, 2^25 keys,
// |v| < 2^16), and what lies below it is 2^-64 of what was seen before.
constexpr float kTop = 15.f, kAt = 12.f, kLow = 8.f, kFall = 64.f;
template <bool kFp16>
__device__ __forceinline__ float moved(float m, float& least, float y) {
  if (!kFp16) return fmaxf(m, y);
  if (y > m + kTop || (y < m + kLow && y != -INFINITY)) {
    m = fmaxf(y - kAt, least);
    least = fmaxf(least, m - kFall);
  }
  return m;
}

// 16-byte chunk c of tile row r, swizzled so that the eight rows of an 8x8
// matrix fall into different banks
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// What the first kernel leaves for the second: unit `first of a stretch's last,
// cut unit`, its rows, and how many stretches hold a part of it.
struct CutUnit {
  int tok0, kv, r0, nr;
  int parts;             // 0: the stretch ends with a whole unit
  int pad[3];
};

// A unit: a block of 16 packed rows of one KV head, and the keys it walks.
struct Unit {
  int s, kv, r0, nr;     // nr = 0: nothing to do
  int tok0, see0;        // row R is token tok0 + R / G and sees rows up to see0 + R / G
  int n_keys;            // in list order
  const int32_t* list;   // sparse: the listed pages
};

template <bool kSparse>
__device__ __forceinline__ Unit make_unit(const PagedBatch& b, const RowsArgs& a, int owner, int kv,
                                          int rb, int lane, int32_t* status) {
  Unit u;
  const int G = a.Hq / a.Hkv;
  u.kv = kv;
  u.r0 = rb * 16;
  u.list = nullptr;
  u.nr = 0;
  u.n_keys = 0;
  u.tok0 = u.see0 = 0;
  u.s = kSparse ? warp_find_seq(b, owner, lane) : owner;
  if (u.s < 0) return u;                     // a token behind the last sequence
  const SeqSpan sp = seq_span(b, u.s);
  u.tok0 = kSparse ? owner : sp.q0;
  u.see0 = sp.kl - sp.ql + (kSparse ? owner - sp.q0 : 0);
  const int rows = kSparse ? G : min(sp.ql, a.max_q) * G;
  u.nr = max(0, min(16, rows - u.r0));
  if (u.nr == 0) {                           // a shorter sequence: no row, nothing to walk
    u.tok0 = u.r0 = 0;
    return u;
  }
  if (kSparse) {
    int cnt = a.counts[(int64_t)owner * a.Hkv + kv];
    if (cnt < 0 || cnt > a.n_sel) {
      set_status(status, TS_ERR_INVALID_ARG);
      cnt = cnt < 0 ? 0 : a.n_sel;
    }
    u.list = a.pages + ((int64_t)owner * a.Hkv + kv) * a.n_sel;
    u.n_keys = u.see0 < 0 ? 0 : cnt << b.page_shift;
  } else {
    u.n_keys = max(0, u.see0 + (u.r0 + u.nr - 1) / G + 1);
  }
  return u;
}

// Trips a sequence's units take each in the dense form (at least one where
// there are tokens: rows without a key are written too).
__device__ __forceinline__ int seq_trips(const SeqSpan& sp) {
  return sp.ql > 0 ? max(1, (sp.kl + kStep - 1) / kStep) : 0;
}

// Stretches a line of `total` trips is cut into: all of the grid's CTAs, as far
// as each gets kMinTrips.
__device__ __forceinline__ int stretches(long long total) {
  const long long n = total / kMinTrips;
  return (int)(n < 1 ? 1 : n < gridDim.x ? n : gridDim.x);
}

// Four columns of row r over the warps' states.
template <int D>
__device__ __forceinline__ float4 join_warps(const float* so, const float2* sml, int r, int c4,
                                             float& m, float& l) {
  m = -INFINITY;
  l = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sml[w * 16 + r].x);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (m != -INFINITY) {
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 x = sml[w * 16 + r];
      const float f = ex2(x.x - m);
      const float4 v = *reinterpret_cast<const float4*>(so + (w * 16 + r) * D + c4 * 4);
      l += f * x.y;
      acc.x += f * v.x;
      acc.y += f * v.y;
      acc.z += f * v.z;
      acc.w += f * v.w;
    }
  }
  return acc;
}

template <typename T, int D>
__device__ __forceinline__ void write_row(const RowsArgs& a, const Unit& u, int r, int c4,
                                          const float4& acc, float m, float l) {
  const int G = a.Hq / a.Hkv, R = u.r0 + r;
  const int64_t row = (int64_t)(u.tok0 + R / G) * a.Hq + u.kv * G + R % G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + row * D + c4 * 4) =
      make_uint2(Pair<T>::pack(acc.x * inv, acc.y * inv), Pair<T>::pack(acc.z * inv, acc.w * inv));
  if (a.lse && c4 == 0) a.lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// Clusters: the barrier, and loads from the shared memory of CTA `rank`.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t far_addr(const void* p, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 far_float4(const void* p, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(far_addr(p, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float2 far_float2(const void* p, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(far_addr(p, rank))
               : "memory");
  return v;
}

template <typename T, int D, bool kSparse>
__global__ void __launch_bounds__(kThreads, 1)
paged_rows_kernel(const PagedBatch b, const RowsArgs a, int n_rb, int unit_trips, int cluster,
                  float* __restrict__ part_o, float2* __restrict__ part_ml,
                  CutUnit* __restrict__ cuts, int32_t* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ long long s_sum[kWarps];
  __shared__ long long s_before;
  __shared__ int s_first;
  using R = Ring<D>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = a.Hq / a.Hkv;
  const int ps = 1 << b.page_shift;
  const int c = blockIdx.x;
  griddep_wait();
  griddep_launch_dependents();

  // ------------------------------------------------------ this CTA's stretch
  // Trips [w0, w1) of the line; `owner` (sequence or token), KV head and row
  // block of its first unit, and the unit's first trip on the line.
  long long total, w0, w1, unit_at;
  // (With `cluster` > 0 the line is one unit and its CTAs are a cluster.)
  int C, owner, sub;                           // sub = kv * n_rb + row block
  const int subs = a.Hkv * n_rb;
  if (cluster > 0) {
    const int u = c / cluster, rank = c % cluster;
    owner = u / subs;
    sub = u % subs;
    C = gridDim.x;
    unit_at = 0;
    const SeqSpan sp = kSparse ? SeqSpan{} : seq_span(b, owner);
    if (!kSparse) {
      unit_trips = seq_trips(sp);
      if (sub == 0 && rank == 0 && tid == 0 && (sp.bad || sp.ql > a.max_q))
        set_status(status, TS_ERR_INVALID_ARG);
    } else if (c == 0) {
      for (int s = tid; s < b.n_seq; s += kThreads)
        if (seq_span(b, s).bad) set_status(status, TS_ERR_INVALID_ARG);
    }
    total = unit_trips;
    w0 = total * rank / cluster;
    w1 = total * (rank + 1) / cluster;
  } else if (kSparse) {
    total = (long long)b.n * subs * unit_trips;
    C = stretches(total);
    w0 = total * c / C;
    w1 = total * (c + 1) / C;
    const long long u = w0 / unit_trips;
    owner = (int)(u / subs);
    sub = (int)(u % subs);
    unit_at = u * unit_trips;
    if (c == 0)
      for (int s = tid; s < b.n_seq; s += kThreads)
        if (seq_span(b, s).bad) set_status(status, TS_ERR_INVALID_ARG);
  } else {
    long long mine = 0;
    for (int s = tid; s < b.n_seq; s += kThreads) {
      const SeqSpan sp = seq_span(b, s);
      if (c == 0 && (sp.bad || sp.ql > a.max_q)) set_status(status, TS_ERR_INVALID_ARG);
      mine += seq_trips(sp);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    if (lane == 0) s_sum[warp] = mine;
    __syncthreads();
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) total += s_sum[w];
    total *= subs;
    C = stretches(total);
    w0 = total * c / C;
    w1 = total * (c + 1) / C;
    // the sequence that holds trip w0: one warp walks the running count
    if (warp == 0) {
      long long before = 0;
      for (int base = 0; base < b.n_seq; base += 32) {
        const int s = base + lane;
        const long long t = s < b.n_seq ? (long long)seq_trips(seq_span(b, s)) * subs : 0;
        long long inc = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long x = __shfl_up_sync(0xffffffffu, inc, o);
          if (lane >= o) inc += x;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, w0 < before + inc && c < C);
        if (hit) {
          const int f = __ffs(hit) - 1;
          if (lane == f) {
            s_first = s;
            s_before = before + inc - t;
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, inc, 31);
      }
    }
    __syncthreads();
    owner = sub = 0;
    unit_at = 0;
    if (c < C && w0 < w1) {
      owner = s_first;
      unit_trips = seq_trips(seq_span(b, owner));
      sub = (int)((w0 - s_before) / unit_trips);
      unit_at = s_before + (long long)sub * unit_trips;
    }
  }
  if (cluster == 0) {
    if (tid == 0) cuts[c].parts = 0;
    if (c >= C || w0 >= w1) return;
  } else if (total == 0) {
    return;                                    // the whole cluster
  }
  const float sl2 = kLog2e / sqrtf((float)D);

  // A place on the line: a unit, and the trips [k, k1) of it in this stretch.
  struct Place {
    int owner, sub, trips;
    long long at;          // the unit's first trip on the line
    Unit u;
    int k, k1;
  };
  auto enter = [&](Place& p) {
    p.u = make_unit<kSparse>(b, a, p.owner, p.sub / n_rb, p.sub % n_rb, lane, status);
    p.k = (int)(w0 > p.at ? w0 - p.at : 0);
    p.k1 = (int)imin64(p.trips, w1 - p.at);
  };
  // the next unit of the stretch (false: its end)
  auto leave = [&](Place& p) -> bool {
    p.at += p.trips;
    if (p.at >= w1) return false;
    if (++p.sub == subs) {
      p.sub = 0;
      ++p.owner;
      if (!kSparse) {
        // sequences without new tokens take no trips
        while ((p.trips = seq_trips(seq_span(b, p.owner))) == 0) ++p.owner;
      }
    }
    enter(p);
    return true;
  };

  const uint32_t ring = smem_addr(smem) + warp * (kStages * R::kStage);
  constexpr int kCh = D / 8;                       // 16-byte chunks a row
  constexpr int kRowsPer = 32 / kCh;               // rows a warp copies at once
  // The pages a unit walks, 32 at a time, one a lane: `lp` in the sequence, `ph`
  // in the pool (-1: not there).  The window behind is on its way meanwhile:
  // its list entries are asked for when a window begins, its table entries one
  // trip later, and neither is looked at before it is needed.
  struct Pages {
    int lp, ph, lp2, ph2;
    int base;               // first page of the window
    bool half;              // lp2 asked for, ph2 not yet
  } pg;
  auto ask_lp = [&](const Unit& u, int base) -> int {
    const int i = base + lane;
    if (i >= (u.n_keys + ps - 1) >> b.page_shift) return -1;
    return kSparse ? u.list[i] : i;
  };
  auto seen_lp = [&](const Unit& u, int base, int lp) -> int {
    // in the sparse form a listed page may lie anywhere
    if (kSparse && base + lane < (u.n_keys + ps - 1) >> b.page_shift &&
        (lp < 0 || lp > (u.see0 >> b.page_shift))) {
      set_status(status, TS_ERR_INVALID_ARG);
      return -1;
    }
    return lp;
  };
  auto ask_ph = [&](const Unit& u, int lp) -> int {
    return lp < 0 ? -1 : b.table[(int64_t)u.s * b.max_pages + lp];
  };
  auto seen_ph = [&](int lp, int ph) -> int {
    if (lp >= 0 && (ph < 0 || ph >= b.n_pages)) {
      set_status(status, TS_ERR_INVALID_ARG);
      return -1;
    }
    return ph;
  };
  auto window_at = [&](const Unit& u, int k) { return (k * kStep >> b.page_shift) & ~31; };
  auto open_pages = [&](const Unit& u, int k) {
    pg.base = window_at(u, k);
    pg.lp = seen_lp(u, pg.base, ask_lp(u, pg.base));
    pg.lp2 = ask_lp(u, pg.base + 32);
    pg.ph = seen_ph(pg.lp, ask_ph(u, pg.lp));
    pg.half = true;
  };
  auto second_half = [&](const Unit& u) {
    pg.lp2 = seen_lp(u, pg.base + 32, pg.lp2);
    pg.ph2 = ask_ph(u, pg.lp2);
    pg.half = false;
  };
  // the window of trip k (the trips of a unit come in order)
  auto pages_for = [&](const Unit& u, int k) {
    if (window_at(u, k) != pg.base) {
      if (pg.half) second_half(u);
      pg.base += 32;
      pg.lp = pg.lp2;
      pg.ph = seen_ph(pg.lp2, pg.ph2);
      pg.lp2 = ask_lp(u, pg.base + 32);
      pg.half = true;
    } else if (pg.half) {
      second_half(u);
    }
  };
  // A warp's 32-key tile lies in one page, or in two of 16 rows.
  struct Tile {
    int lp0, lp1;           // pages in the sequence; -1: not readable
  };
  // a lane copies 16-byte chunk lane % kCh of rows lane / kCh + x * kRowsPer;
  // within a page its addresses are one base and constant steps
  const uint32_t lane_bytes = (lane / kCh) * (D * 2) + (lane % kCh) * 16;
  const char* kbase = static_cast<const char*>(a.k_pages) + lane_bytes;
  const char* vbase = static_cast<const char*>(a.v_pages) + lane_bytes;
  const int64_t page_bytes = (int64_t)a.Hkv * ps * (D * 2);
  auto fetch = [&](const Unit& u, int k, uint32_t stage) -> Tile {
    const int j = k * kStep + warp * kTileKeys;
    const int src = (j >> b.page_shift) - pg.base;
    const int two = b.page_shift == 4 ? src + 1 : src;
    const int ph0 = __shfl_sync(0xffffffffu, pg.ph, src);
    const int ph1 = __shfl_sync(0xffffffffu, pg.ph, two & 31);
    Tile t;
    t.lp0 = __shfl_sync(0xffffffffu, pg.lp, src);
    t.lp1 = __shfl_sync(0xffffffffu, pg.lp, two & 31);
    if (ph0 < 0) t.lp0 = -1;
    if (ph1 < 0) t.lp1 = -1;
    const uint32_t st = ring + stage * R::kStage;
    const int in_page = j & (ps - 1);
    const int64_t head_bytes = (int64_t)u.kv * ps * (D * 2);
    // rows behind the last visible one are filled with zeros: whatever their
    // page holds there must not reach P.V
    int live0 = t.lp0 < 0 ? 0 : u.n_keys - j, live1 = t.lp1 < 0 ? 0 : u.n_keys - j;
    if (kSparse) {
      live0 = min(live0, u.see0 + 1 - (t.lp0 << b.page_shift) - in_page);
      live1 = min(live1, u.see0 + 1 - (t.lp1 << b.page_shift) - in_page +
                             (b.page_shift == 4 ? 16 : 0));
    }
    const int64_t o0 = (int64_t)max(ph0, 0) * page_bytes + head_bytes + in_page * (D * 2);
    // rows 16.. of the tile: the next 16 of the page, or the second page's
    const int64_t o1 =
        b.page_shift == 4 ? (int64_t)max(ph1, 0) * page_bytes + head_bytes - 16 * (D * 2) : o0;
    const int r0l = lane / kCh;
#pragma unroll
    for (int x = 0; x < kTileKeys / kRowsPer; ++x) {
      const int r = x * kRowsPer + r0l;
      const bool second = x * kRowsPer >= 16;
      const bool live = r < (second ? live1 : live0);
      // a row that is not read still needs a valid address
      const int64_t off = (second ? o1 : o0) + x * (kRowsPer * D * 2);
      const int64_t at = live ? off : -(int64_t)lane_bytes;
      const uint32_t dst = chunk_off<D>(r, lane % kCh);
      cp16(st + dst, kbase + at, live);
      cp16(st + R::kTile + dst, vbase + at, live);
    }
    return t;
  };

  // The copies run kStages - 1 trips ahead of the products, on their own place.
  Place ahead{owner, sub, unit_trips, unit_at, {}, 0, 0};
  enter(ahead);
  Place now = ahead;
  bool more = w0 < w1;                  // a cluster may have more CTAs than trips
  if (!more) now.k1 = now.k;
  Tile held[kStages];           // tiles whose copies are on their way, oldest first
  if (more) open_pages(ahead.u, ahead.k);
  uint32_t put = 0, got = 0;    // trips copied, trips used
  auto push = [&](Tile& into) {
    if (more) {
      pages_for(ahead.u, ahead.k);
      into = fetch(ahead.u, ahead.k, put % kStages);
      ++put;
      if (++ahead.k == ahead.k1) {
        more = leave(ahead);
        if (more) open_pages(ahead.u, ahead.k);
      }
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) push(held[i]);

  const int ra = lane >> 2, rb8 = ra + 8;      // the rows of this thread's accumulators
  float* so = reinterpret_cast<float*>(smem + R::kStates);          // [warp][16][D]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * 16 * D);    // [warp][16]
  while (true) {
    const Unit& u = now.u;
    const int lim_a = ra < u.nr ? u.see0 + (u.r0 + ra) / G : -1;
    const int lim_b = rb8 < u.nr ? u.see0 + (u.r0 + rb8) / G : -1;
    // below this key every live row sees everything (rows without a query only
    // ever feed accumulators that are not written)
    const int free_to = u.see0 + u.r0 / G + 1;
    float oacc[D / 8][4];
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) oacc[i][x] = 0.f;
    float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;
    float least_a = -INFINITY, least_b = -INFINITY;
    // query fragments (16 x 16 blocks), straight from global memory
    uint32_t qf[D / 16][4];
    {
      auto row_ptr = [&](int r) {
        const int RR = u.r0 + max(0, min(r, u.nr - 1));
        return reinterpret_cast<const uint32_t*>(
            static_cast<const T*>(a.q) + ((int64_t)(u.tok0 + RR / G) * a.Hq + u.kv * G + RR % G) * D);
      };
      const uint32_t* pa = row_ptr(ra);
      const uint32_t* pb = row_ptr(rb8);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qf[ks][0] = pa[ks * 8 + (lane & 3)];
        qf[ks][1] = pb[ks * 8 + (lane & 3)];
        qf[ks][2] = pa[ks * 8 + 4 + (lane & 3)];
        qf[ks][3] = pb[ks * 8 + 4 + (lane & 3)];
      }
    }
    for (; now.k < now.k1; ++now.k, ++got) {
      __syncwarp();                       // every lane is done with the stage refilled now
      push(held[kStages - 1]);
      const Tile cur = held[0];
#pragma unroll
      for (int x = 0; x + 1 < kStages; ++x) held[x] = held[x + 1];
      cp_wait<kStages - 1>();
      __syncwarp();
      const int j = now.k * kStep + warp * kTileKeys;
      if (j >= u.n_keys) continue;        // nothing of this trip is this warp's
      const uint32_t kt = ring + (got % kStages) * R::kStage, vt = kt + R::kTile;
      // S = Q K^T: 16 rows x 32 keys
      float c[4][4];
#pragma unroll
      for (int nb = 0; nb < 4; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) c[nb][x] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
#pragma unroll
        for (int nn = 0; nn < 2; ++nn) {
          uint32_t kb[4];
          const int r = nn * 16 + (lane >> 4) * 8 + (lane & 7);
          ldsm4(kt + chunk_off<D>(r, ks * 2 + ((lane >> 3) & 1)), kb);
          mma<T>(c[2 * nn], qf[ks], kb[0], kb[1]);
          mma<T>(c[2 * nn + 1], qf[ks], kb[2], kb[3]);
        }
      // keys a row does not see: behind its own position, behind the range, or
      // in a page that could not be read
      const bool bad = cur.lp0 < 0 || cur.lp1 < 0;
      const int top = kSparse ? (max(cur.lp0, cur.lp1) << b.page_shift) + ps : j + kTileKeys;
      if (bad || top > free_to || j + kTileKeys > u.n_keys) {
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = nb * 8 + (lane & 3) * 2 + x;
            int key = j + r;
            const bool none = key >= u.n_keys || (nb < 2 ? cur.lp0 : cur.lp1) < 0;
            if (kSparse) key = ((nb < 2 ? cur.lp0 : cur.lp1) << b.page_shift) + (key & (ps - 1));
            if (none || key > lim_a) c[nb][x] = -INFINITY;
            if (none || key > lim_b) c[nb][2 + x] = -INFINITY;
          }
      }
      // online softmax over the rows ra (c[.][0..1]) and rb8 (c[.][2..3])
      float xa = -INFINITY, xb = -INFINITY;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        xa = fmaxf(xa, fmaxf(c[nb][0], c[nb][1]));
        xb = fmaxf(xb, fmaxf(c[nb][2], c[nb][3]));
      }
#pragma unroll
      for (int o = 1; o < 4; o <<= 1) {
        xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, o));
        xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, o));
      }
      const float na = moved<Pair<T>::kFp16>(ma, least_a, xa * sl2);
      const float nb_ = moved<Pair<T>::kFp16>(mb, least_b, xb * sl2);
      // nothing seen so far: reference 0 keeps 2^(-inf) = 0
      const float refa = na == -INFINITY ? 0.f : na, refb = nb_ == -INFINITY ? 0.f : nb_;
      const float fa = ex2(ma - refa), fb = ex2(mb - refb);
      ma = na;
      mb = nb_;
      float sa = 0.f, sb = 0.f;
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        c[nb][0] = ex2(fmaf(c[nb][0], sl2, -refa));
        c[nb][1] = ex2(fmaf(c[nb][1], sl2, -refa));
        c[nb][2] = ex2(fmaf(c[nb][2], sl2, -refb));
        c[nb][3] = ex2(fmaf(c[nb][3], sl2, -refb));
        sa += c[nb][0] + c[nb][1];
        sb += c[nb][2] + c[nb][3];
      }
      la = la * fa + sa;
      lb = lb * fb + sb;
      if (__any_sync(0xffffffffu, fa != 1.f || fb != 1.f)) {
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
          oacc[n][0] *= fa;
          oacc[n][1] *= fa;
          oacc[n][2] *= fb;
          oacc[n][3] *= fb;
        }
      }
      // O += P V, P as a 16-bit value and its remainder
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float p0 = c[2 * kk + (x >> 1)][(x & 1) * 2], p1 = c[2 * kk + (x >> 1)][(x & 1) * 2 + 1];
          hi[x] = Pair<T>::pack(p0, p1);
          const float2 back = Pair<T>::unpack(hi[x]);
          lo[x] = Pair<T>::pack(p0 - back.x, p1 - back.y);
        }
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
          uint32_t vb[4];
          const int r = kk * 16 + ((lane >> 3) & 1) * 8 + (lane & 7);
          ldsm4t(vt + chunk_off<D>(r, n * 2 + (lane >> 4)), vb);
          mma<T>(oacc[2 * n], hi, vb[0], vb[1]);
          mma<T>(oacc[2 * n + 1], hi, vb[2], vb[3]);
          mma<T>(oacc[2 * n], lo, vb[0], vb[1]);
          mma<T>(oacc[2 * n + 1], lo, vb[2], vb[3]);
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      la += __shfl_xor_sync(0xffffffffu, la, o);
      lb += __shfl_xor_sync(0xffffffffu, lb, o);
    }
    // a sum that is NaN counts in the joins, whatever the maximum saw
    if (la != la) ma = INFINITY;
    if (lb != lb) mb = INFINITY;
    // -------------------------------------------------------- join the warps
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
      const int col = n * 8 + (lane & 3) * 2;
      *reinterpret_cast<float2*>(so + (warp * 16 + ra) * D + col) = make_float2(oacc[n][0], oacc[n][1]);
      *reinterpret_cast<float2*>(so + (warp * 16 + rb8) * D + col) = make_float2(oacc[n][2], oacc[n][3]);
    }
    if ((lane & 3) == 0) {
      sml[warp * 16 + ra] = make_float2(ma, la);
      sml[warp * 16 + rb8] = make_float2(mb, lb);
    }
    __syncthreads();
    const bool starts = now.at >= w0, ends = now.at + now.trips <= w1;
    if (cluster > 0) {
      // ------------------------------------------------- join the cluster's CTAs
      // Each leaves its state where its ring was; then each reads the others'
      // for its share of the columns.
      cp_wait<0>();
      __syncthreads();
      float* jo = reinterpret_cast<float*>(smem);                      // [16][D]
      float2* jml = reinterpret_cast<float2*>(jo + 16 * D);            // [16]
      for (int e = tid; e < u.nr * (D / 4); e += kThreads) {
        const int r = e / (D / 4), c4 = e % (D / 4);
        float m, l;
        const float4 acc = join_warps<D>(so, sml, r, c4, m, l);
        *reinterpret_cast<float4*>(jo + r * D + c4 * 4) = acc;
        if (c4 == 0) jml[r] = make_float2(m, l);
      }
      cluster_sync();
      const int rank = c % cluster;
      for (int e = tid * cluster + rank; e < u.nr * (D / 4); e += kThreads * cluster) {
        const int r = e / (D / 4), c4 = e % (D / 4);
        float2 ml[kMostCluster];
        float4 v[kMostCluster];
#pragma unroll
        for (int i = 0; i < kMostCluster; ++i)
          if (i < cluster) {
            ml[i] = far_float2(jml + r, i);
            v[i] = far_float4(jo + r * D + c4 * 4, i);
          }
        float m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < kMostCluster; ++i)
          if (i < cluster) m = fmaxf(m, ml[i].x);
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (m != -INFINITY) {
#pragma unroll
          for (int i = 0; i < kMostCluster; ++i)
            if (i < cluster) {
              const float f = ex2(ml[i].x - m);
              l += f * ml[i].y;
              acc.x += f * v[i].x;
              acc.y += f * v[i].y;
              acc.z += f * v[i].z;
              acc.w += f * v[i].w;
            }
        }
        write_row<T, D>(a, u, r, c4, acc, m, l);
      }
      cluster_sync();                     // nobody leaves while its state is read
      return;
    }
    // a part that does not hold the unit's first trip takes the stretch's slot
    // 0, one that does slot 1; the latter's stretch says what is to be joined
    const int64_t slot = (int64_t)c * 2 + (starts ? 1 : 0);
    constexpr int kQuads = D / 4;
    for (int e = tid; e < u.nr * kQuads; e += kThreads) {
      const int r = e / kQuads, c4 = e % kQuads;
      float m, l;
      const float4 acc = join_warps<D>(so, sml, r, c4, m, l);
      if (starts && ends) {
        write_row<T, D>(a, u, r, c4, acc, m, l);
      } else {
        *reinterpret_cast<float4*>(part_o + (slot * 16 + r) * D + c4 * 4) = acc;
        if (c4 == 0) part_ml[slot * 16 + r] = make_float2(m, l);
      }
    }
    if (tid == 0 && starts && !ends && u.nr > 0) {
      CutUnit x{};
      x.tok0 = u.tok0;
      x.kv = u.kv;
      x.r0 = u.r0;
      x.nr = u.nr;
      // the stretch that holds the unit's last trip z: the last whose start is
      // at or before z
      const long long z = now.at + now.trips - 1;
      int q = (int)((z * C) / total);
      while (q + 1 < C && total * (q + 1) / C <= z) ++q;
      while (total * q / C > z) --q;
      x.parts = q - c + 1;
      cuts[c] = x;
    }
    if (!leave(now)) break;
    __syncthreads();                      // the states are read before the next unit's
  }
  cp_wait<0>();
}

// Joins cut units: CTA c the one that stretch c starts and does not end.  Four
// columns of a row a thread; the loads of O do not wait for one another.
template <typename T, int D>
__global__ void __launch_bounds__(512)
paged_rows_merge(const CutUnit* __restrict__ cuts, const float* __restrict__ part_o,
                 const float2* __restrict__ part_ml, int Hq, int Hkv, T* o, float* lse) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, G = Hq / Hkv;
  constexpr int kQuads = D / 4, kAtOnce = 8;
  const int r = threadIdx.x / kQuads, c4 = threadIdx.x % kQuads;
  // part i: stretch c's slot 1, then slot 0 of the stretches behind it.  The
  // first parts are asked for before their number is known (every slot up to
  // the grid's is there to be read): one round trip for most units.
  auto at = [&](int i) { return ((int64_t)(i == 0 ? 2 * c + 1 : 2 * (c + i))) * 16 + r; };
  const int most = min(kAtOnce, (int)gridDim.x - c);
  float2 ml[kAtOnce];
  float4 v[kAtOnce];
  auto ask = [&](int i0, int n) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (i < n) {
        ml[i] = part_ml[at(i0 + i)];
        v[i] = *reinterpret_cast<const float4*>(part_o + at(i0 + i) * D + c4 * 4);
      }
  };
  ask(0, most);
  const CutUnit x = cuts[c];
  if (r >= x.nr || x.parts == 0) return;
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < x.parts; i0 += kAtOnce) {
    const int n = min(kAtOnce, x.parts - i0);
    if (i0 > 0) ask(i0, n);
    float mn = m;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (i < n) mn = fmaxf(mn, ml[i].x);
    if (mn == -INFINITY) continue;                  // no key so far
    const float f0 = exp2f(m - mn);
    l *= f0;
    acc.x *= f0;
    acc.y *= f0;
    acc.z *= f0;
    acc.w *= f0;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (i < n) {
        const float f = exp2f(ml[i].x - mn);        // 0 for a part without a key
        l += f * ml[i].y;
        acc.x += f * v[i].x;
        acc.y += f * v[i].y;
        acc.z += f * v[i].z;
        acc.w += f * v[i].w;
      }
    m = mn;
  }
  const int RR = x.r0 + r;
  const int64_t row = (int64_t)(x.tok0 + RR / G) * Hq + x.kv * G + RR % G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint2*>(o + row * D + c4 * 4) =
      make_uint2(Pair<T>::pack(acc.x * inv, acc.y * inv), Pair<T>::pack(acc.z * inv, acc.w * inv));
  if (lse && c4 == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace

// One CTA a SM (the rings fill its shared memory).  Few units of few trips take
// a cluster of CTAs each, which join in shared memory: no second kernel and no
// workspace, worth ~4 trips (3 streams of up to 4096 rows: 9.0 -> 7.4 us).  Else
// the line of all units is cut into stretches of at least kMinTrips.
RowsPlan rows_plan(int64_t units, int rows, int d, int64_t max_keys) {
  constexpr int64_t kJoinTrips = 4;
  RowsPlan p{};
  p.n_rb = (rows + 15) / 16;
  p.unit_trips = (int)imax64(1, (max_keys + kStep - 1) / kStep);
  units *= p.n_rb;
  const int64_t trips = units * p.unit_trips;
  int64_t size = kMostCluster;
  while (size > 1 && (units * size > kGb300Sms || size > p.unit_trips)) size >>= 1;
  if (units * size <= kGb300Sms &&
      (p.unit_trips + size - 1) / size <= imax64(trips / kGb300Sms, kMinTrips) + kJoinTrips) {
    p.cluster = (int)size;
    p.grid = (int)(units * size);
    return p;
  }
  p.grid = (int)imax64(1, imin64(kGb300Sms, trips / kMinTrips));
  p.cuts_bytes = align_up((size_t)p.grid * sizeof(CutUnit), 256);
  p.part_bytes = (size_t)p.grid * 2 * 16 * d * sizeof(float);
  p.ws_bytes = p.cuts_bytes + p.part_bytes + align_up((size_t)p.grid * 2 * 16 * sizeof(float2), 256);
  return p;
}

template <typename T, int D>
static int go_rows(const PagedBatch& b, const RowsArgs& a, const RowsPlan& p, void* ws,
                   int32_t* status, cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  CutUnit* cuts = reinterpret_cast<CutUnit*>(w);
  float* part_o = reinterpret_cast<float*>(w + p.cuts_bytes);
  float2* part_ml = reinterpret_cast<float2*>(w + p.cuts_bytes + p.part_bytes);
  const bool sparse = a.pages != nullptr;
  auto kern = sparse ? paged_rows_kernel<T, D, true> : paged_rows_kernel<T, D, false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kBytes);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  pdl_config(&cfg, attr, dim3(p.grid), dim3(kThreads), Ring<D>::kBytes, st);
  if (p.cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  cudaLaunchKernelEx(&cfg, kern, b, a, p.n_rb, p.unit_trips, p.cluster, part_o, part_ml, cuts,
                     status);
  int rc = launch_status("paged_rows_kernel");
  if (rc || p.cluster > 0) return rc;
  // sparse units are cut by the host's numbers: none where the CTAs divide them
  if (rc || p.grid == 1 || (sparse && (int64_t)b.n * a.Hkv * p.n_rb % p.grid == 0)) return rc;
  pdl_config(&cfg, attr, dim3(p.grid), dim3(16 * (D / 4)), 0, st);
  cudaLaunchKernelEx(&cfg, paged_rows_merge<T, D>, (const CutUnit*)cuts, (const float*)part_o,
                     (const float2*)part_ml, a.Hq, a.Hkv, static_cast<T*>(a.o), a.lse);
  return launch_status("paged_rows_merge");
}

int launch_paged_rows(const PagedBatch& b, const RowsArgs& a, const RowsPlan& p, int d, bool fp16,
                      void* ws, int32_t* status, cudaStream_t st) {
  if (fp16)
    return d == 128 ? go_rows<__half, 128>(b, a, p, ws, status, st)
                    : go_rows<__half, 64>(b, a, p, ws, status, st);
  return d == 128 ? go_rows<__nv_bfloat16, 128>(b, a, p, ws, status, st)
                  : go_rows<__nv_bfloat16, 64>(b, a, p, ws, status, st);
}

}  // namespace ts
