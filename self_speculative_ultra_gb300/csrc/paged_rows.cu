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
// so a key tile is read once for all of them; the keys are split over CTAs.
// A CTA's four warps work on their own 32-key tiles: each warp streams its
// tiles through its own ring of asynchronous copies and runs the online
// softmax by itself, without a CTA-wide barrier in the loop; the four states
// are joined at the end in shared memory, the splits by a second kernel.
// Q.K^T and P.V use 16x8x16 matrix instructions: 16 rows never fill a tensor
// core tile, so the copy engine's 128-row tiles would only pad.  P is split
// into a 16-bit value and its 16-bit remainder (two products), so P.V sees P
// to 16 bits or more and the only rounding to 16 bits is the output's.
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kWarps = 4;
constexpr int kCtas = 1;                   // CTAs a SM
constexpr int kThreads = kWarps * 32;
constexpr int kTileKeys = 32;              // keys of a warp's tile
constexpr int kStep = kWarps * kTileKeys;  // keys a CTA takes per trip
constexpr int kStages = 3;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

template <int D>
struct Ring {
  static constexpr int kRow = D * 2;
  static constexpr int kTile = kTileKeys * kRow;
  static constexpr int kStage = 2 * kTile;                 // K tile, V tile
  static constexpr int kBytes = kWarps * kStages * kStage;
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

// 16-byte chunk c of tile row r, swizzled so that the eight rows of an 8x8
// matrix fall into different banks
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int r, int c) {
  return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// Partials of row (t, head) and split s: O (fp32, scaled to the split's own
// maximum) at ((t * Hq + head) * n_split + s) * D, (m, l) likewise.
template <typename T, int D, bool kSparse>
__global__ void __launch_bounds__(kThreads, kCtas)
paged_rows_kernel(const PagedBatch b, const RowsArgs a, int n_rb, int n_split, int keys_per_split,
                  float* __restrict__ part_o, float2* __restrict__ part_ml, int32_t* status) {
  extern __shared__ __align__(128) uint8_t smem[];
  using R = Ring<D>;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = blockIdx.x % n_split;
  const int unit = blockIdx.x / n_split;       // sequence (dense) or token (sparse)
  const int kv = blockIdx.y / n_rb, rb = blockIdx.y % n_rb;
  const int G = a.Hq / a.Hkv;
  const int ps = 1 << b.page_shift;
  griddep_wait();
  griddep_launch_dependents();
  const int s = kSparse ? warp_find_seq(b, unit, lane) : unit;
  if (s < 0) return;                           // a token behind the last sequence
  const SeqSpan sp = seq_span(b, s);
  const bool first_cta = split == 0 && blockIdx.y == 0 && tid == 0;
  if (first_cta && (sp.bad || (!kSparse && sp.ql > a.max_q)))
    set_status(status, TS_ERR_INVALID_ARG);
  // rows of this block: R = r0 .. r0 + nr - 1; row R is token tok0 + R / G,
  // head kv * G + R % G, and sees rows up to see0 + R / G
  const int tok0 = kSparse ? unit : sp.q0;
  const int see0 = kSparse ? sp.kl - sp.ql + (unit - sp.q0) : sp.kl - sp.ql;
  const int rows = kSparse ? G : min(sp.ql, a.max_q) * G;
  const int r0 = rb * 16;
  if (r0 >= rows) return;
  const int nr = min(16, rows - r0);
  const int32_t* list = nullptr;
  int n_keys;                                  // keys to walk, in list order
  if (kSparse) {
    int cnt = a.counts[(int64_t)unit * a.Hkv + kv];
    if (cnt < 0 || cnt > a.n_sel) {
      if (split == 0 && rb == 0 && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
      cnt = cnt < 0 ? 0 : a.n_sel;
    }
    list = a.pages + ((int64_t)unit * a.Hkv + kv) * a.n_sel;
    n_keys = see0 < 0 ? 0 : cnt << b.page_shift;
  } else {
    n_keys = max(0, see0 + (r0 + nr - 1) / G + 1);
  }
  const int j0 = (int)imin64((int64_t)split * keys_per_split, n_keys);
  // the last split takes whatever the host's bound on the lengths left out
  const int j1 = split == n_split - 1 ? n_keys : (int)imin64((int64_t)j0 + keys_per_split, n_keys);
  const float sl2 = kLog2e / sqrtf((float)D);

  // the two rows of this thread's accumulators
  const int ra = lane >> 2, rb8 = ra + 8;
  const int lim_a = ra < nr ? see0 + (r0 + ra) / G : -1;
  const int lim_b = rb8 < nr ? see0 + (r0 + rb8) / G : -1;
  // below this key every live row sees everything (rows without a query only
  // ever feed accumulators that are not written)
  const int free_to = see0 + r0 / G + 1;

  float oacc[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) oacc[i][x] = 0.f;
  float ma = -INFINITY, mb = -INFINITY, la = 0.f, lb = 0.f;

  if (j0 < j1) {
    // query fragments (16 x 16 blocks), straight from global memory
    uint32_t qf[D / 16][4];
    {
      auto row_ptr = [&](int r) {
        const int RR = r0 + min(r, nr - 1);
        return reinterpret_cast<const uint32_t*>(
            static_cast<const T*>(a.q) + ((int64_t)(tok0 + RR / G) * a.Hq + kv * G + RR % G) * D);
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
    const uint32_t ring = smem_addr(smem) + warp * (kStages * R::kStage);
    const int n_tiles = (j1 - j0 + kStep - 1) / kStep;
    const int32_t* trow = b.table + (int64_t)s * b.max_pages;
    // page of list position j: logical page and where its rows start (-1: none)
    auto page_at = [&](int j, int& logical) -> int64_t {
      logical = -1;
      if (j >= j1) return -1;
      const int lp = kSparse ? list[j >> b.page_shift] : j >> b.page_shift;
      if (kSparse && (lp < 0 || lp > (see0 >> b.page_shift))) {
        set_status(status, TS_ERR_INVALID_ARG);
        return -1;
      }
      const int64_t ph = trow[lp];
      if (ph < 0 || ph >= b.n_pages) {
        set_status(status, TS_ERR_INVALID_ARG);
        return -1;
      }
      logical = lp;
      return ph;
    };
    // A 32-key tile lies in one page, or in two of 16 rows.
    struct Tile {
      int64_t ph0, ph1;
      int lp0, lp1;
    };
    auto look = [&](int i) {
      Tile t;
      const int j = j0 + i * kStep + warp * kTileKeys;
      t.ph0 = page_at(j, t.lp0);
      t.ph1 = t.ph0;
      t.lp1 = t.lp0;
      if (b.page_shift == 4) t.ph1 = page_at(j + 16, t.lp1);
      return t;
    };
    constexpr int kCh = D / 8;                       // 16-byte chunks a row
    constexpr int kRowsPer = 32 / kCh;               // rows a warp copies at once
    // a lane copies 16-byte chunk lane % kCh of rows lane / kCh + x * kRowsPer;
    // within a page its addresses are one base and constant steps
    const uint32_t lane_bytes = (lane / kCh) * (D * 2) + (lane % kCh) * 16;
    const char* kbase = static_cast<const char*>(a.k_pages) + lane_bytes;
    const char* vbase = static_cast<const char*>(a.v_pages) + lane_bytes;
    const int64_t page_bytes = (int64_t)a.Hkv * ps * (D * 2);
    const int64_t head_bytes = (int64_t)kv * ps * (D * 2);
    auto fetch = [&](int i, const Tile& t) {
      if (i < n_tiles) {
        const int j = j0 + i * kStep + warp * kTileKeys;
        const uint32_t st = ring + (i % kStages) * R::kStage;
        const int in_page = j & (ps - 1);
        // rows behind the last visible one are filled with zeros: whatever
        // their page holds there must not reach P.V
        int live0 = t.ph0 < 0 ? 0 : j1 - j, live1 = t.ph1 < 0 ? 0 : j1 - j;
        if (kSparse) {
          live0 = min(live0, see0 + 1 - (t.lp0 << b.page_shift) - in_page);
          live1 = min(live1, see0 + 1 - (t.lp1 << b.page_shift) - in_page +
                                 (b.page_shift == 4 ? 16 : 0));
        }
        const int64_t o0 = max(t.ph0, (int64_t)0) * page_bytes + head_bytes + in_page * (D * 2);
        // rows 16.. of the tile: the next 16 of the page, or the second page's
        const int64_t o1 = b.page_shift == 4
                               ? max(t.ph1, (int64_t)0) * page_bytes + head_bytes - 16 * (D * 2)
                               : o0;
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
      }
      cp_commit();
    };
    // tiles in flight, and the logical pages of the tile in hand
    Tile ahead[kStages];
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      ahead[i] = look(i);
      fetch(i, ahead[i]);
    }
    Tile next = look(kStages - 1);
    for (int i = 0; i < n_tiles; ++i) {
      const Tile cur = ahead[0];
      __syncwarp();                       // every lane is done with the stage refilled now
      fetch(i + kStages - 1, next);
#pragma unroll
      for (int x = 0; x + 2 < kStages; ++x) ahead[x] = ahead[x + 1];
      ahead[kStages - 2] = next;
      next = look(i + kStages);
      cp_wait<kStages - 1>();
      __syncwarp();
      const int j = j0 + i * kStep + warp * kTileKeys;
      if (j >= j1) continue;              // this warp's share of the last trip is empty
      const uint32_t kt = ring + (i % kStages) * R::kStage, vt = kt + R::kTile;
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
      const bool bad = cur.ph0 < 0 || cur.ph1 < 0;
      const int top = kSparse ? (max(cur.lp0, cur.lp1) << b.page_shift) + ps : j + kTileKeys;
      if (bad || top > free_to || j + kTileKeys > j1) {
#pragma unroll
        for (int nb = 0; nb < 4; ++nb)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int r = nb * 8 + (lane & 3) * 2 + x;
            int key = j + r;
            bool none = key >= j1 || (nb < 2 ? cur.ph0 : cur.ph1) < 0;
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
      const float na = fmaxf(ma, xa * sl2), nb_ = fmaxf(mb, xb * sl2);
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
    cp_wait<0>();
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      la += __shfl_xor_sync(0xffffffffu, la, o);
      lb += __shfl_xor_sync(0xffffffffu, lb, o);
    }
  }

  // ---------------------------------------------------------- join the warps
  __syncthreads();
  float* so = reinterpret_cast<float*>(smem);                       // [warp][16][D]
  float2* sml = reinterpret_cast<float2*>(so + kWarps * 16 * D);    // [warp][16]
  static_assert(kWarps * 16 * (D + 2) * 4 <= R::kBytes, "the states must fit the ring");
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
  constexpr int kQuads = D / 4;
  for (int e = tid; e < nr * kQuads; e += kThreads) {
    const int r = e / kQuads, c4 = e % kQuads;
    float m = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sml[w * 16 + r].x);
    float l = 0.f;
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
    const int RR = r0 + r;
    const int64_t row = (int64_t)(tok0 + RR / G) * a.Hq + kv * G + RR % G;
    if (n_split == 1) {
      const float inv = l > 0.f ? 1.f / l : 0.f;
      *reinterpret_cast<uint2*>(static_cast<T*>(a.o) + row * D + c4 * 4) =
          make_uint2(Pair<T>::pack(acc.x * inv, acc.y * inv), Pair<T>::pack(acc.z * inv, acc.w * inv));
      if (a.lse && c4 == 0) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
    } else {
      const int64_t at = row * n_split + split;
      if (l > 0.f) *reinterpret_cast<float4*>(part_o + at * D + c4 * 4) = acc;
      if (c4 == 0) part_ml[at] = make_float2(m, l);
    }
  }
}

// Joins the splits of every row: a warp a row, each lane D/32 columns.  The
// lanes hold one split's weight each; the loads of O do not wait for one
// another.
template <typename T, int D>
__global__ void __launch_bounds__(128)
paged_rows_merge(const PagedBatch b, const float* __restrict__ part_o,
                 const float2* __restrict__ part_ml, int Hq, int n_split, int max_q, T* o,
                 float* lse) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int t = (int)(row / Hq);
  if (t >= b.n) return;
  const float2* ml = part_ml + row * n_split;
  const float2 first = lane < n_split ? ml[lane] : make_float2(-INFINITY, 0.f);
  const int s = warp_find_seq(b, t, lane);
  if (s < 0) return;
  if (max_q > 0 && t - seq_span(b, s).q0 >= max_q) return;   // no partials were made
  float m = first.x;
  for (int i = lane + 32; i < n_split; i += 32) m = fmaxf(m, ml[i].x);
  m = warp_max(m);
  constexpr int kPer = D / 32;
  float acc[kPer], l = 0.f;
#pragma unroll
  for (int x = 0; x < kPer; ++x) acc[x] = 0.f;
  if (m != -INFINITY) {
    const float* po = part_o + row * n_split * D + lane * kPer;
    for (int base = 0; base < n_split; base += 32) {
      const float2 x = base == 0 ? first
                                 : base + lane < n_split ? ml[base + lane] : make_float2(-INFINITY, 0.f);
      const float w = x.y > 0.f ? exp2f(x.x - m) : 0.f;      // an empty split left no O
      l += w * x.y;
      const int n = min(32, n_split - base);
#pragma unroll 8
      for (int i = 0; i < n; ++i) {
        const float f = __shfl_sync(0xffffffffu, w, i);
        float v[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) v[y] = 0.f;
        if (f > 0.f) {
          if (kPer == 4) {
            const float4 u = *reinterpret_cast<const float4*>(po + (int64_t)(base + i) * D);
            v[0] = u.x;
            v[1] = u.y;
            v[2 % kPer] = u.z;
            v[3 % kPer] = u.w;
          } else {
            const float2 u = *reinterpret_cast<const float2*>(po + (int64_t)(base + i) * D);
            v[0] = u.x;
            v[1] = u.y;
          }
        }
#pragma unroll
        for (int y = 0; y < kPer; ++y) acc[y] += f * v[y];
      }
    }
  }
  l = warp_sum(l);
  const float inv = l > 0.f ? 1.f / l : 0.f;
  uint32_t* dst = reinterpret_cast<uint32_t*>(o + row * D + lane * kPer);
#pragma unroll
  for (int x = 0; x < kPer / 2; ++x) dst[x] = Pair<T>::pack(acc[2 * x] * inv, acc[2 * x + 1] * inv);
  if (lse && lane == 0) lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

// units x 16-row blocks x splits CTAs, one a SM (their rings fill its shared
// memory): the split count that minimises waves x (trips + a fixed cost).
RowsPlan rows_plan(int64_t units, int n, int Hq, int rows, int d, int64_t max_keys) {
  constexpr double kFixedTrips = 6.0;  // ~2 us
  RowsPlan p{};
  p.n_rb = (rows + 15) / 16;
  const int64_t base = units * p.n_rb;
  const int64_t trips = imax64(1, (max_keys + kStep - 1) / kStep);
  double best = 1e300;
  int64_t best_per = trips;
  for (int64_t ns = 1; ns <= imin64(trips, 256); ++ns) {
    const int64_t per = (trips + ns - 1) / ns;
    const int64_t used = (trips + per - 1) / per;
    const int64_t waves = (base * used + kCtas * kGb300Sms - 1) / (kCtas * kGb300Sms);
    const double cost = (double)waves * ((double)per + kFixedTrips);
    if (cost < best - 1e-9) {
      best = cost;
      best_per = per;
    }
  }
  p.keys_per_split = (int)(best_per * kStep);
  p.n_split = (int)((trips + best_per - 1) / best_per);
  if (p.n_split > 1) {
    p.part_bytes = align_up((size_t)n * Hq * p.n_split * d * sizeof(float), 256);
    p.ml_bytes = align_up((size_t)n * Hq * p.n_split * sizeof(float2), 256);
  }
  p.ws_bytes = p.part_bytes + p.ml_bytes;
  return p;
}

template <typename T, int D>
static int go_rows(const PagedBatch& b, const RowsArgs& a, const RowsPlan& p, void* ws,
                   int32_t* status, cudaStream_t st) {
  float* part_o = static_cast<float*>(ws);
  float2* part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + p.part_bytes);
  const bool sparse = a.pages != nullptr;
  const int units = sparse ? b.n : b.n_seq;
  auto kern = sparse ? paged_rows_kernel<T, D, true> : paged_rows_kernel<T, D, false>;
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ring<D>::kBytes);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  pdl_config(&cfg, attr, dim3((unsigned)units * p.n_split, a.Hkv * p.n_rb), dim3(kThreads),
             Ring<D>::kBytes, st);
  cudaLaunchKernelEx(&cfg, kern, b, a, p.n_rb, p.n_split, p.keys_per_split, part_o, part_ml,
                     status);
  int rc = launch_status("paged_rows_kernel");
  if (rc || p.n_split == 1) return rc;
  const int64_t rows = (int64_t)b.n * a.Hq;
  pdl_config(&cfg, attr, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st);
  cudaLaunchKernelEx(&cfg, paged_rows_merge<T, D>, b, (const float*)part_o, (const float2*)part_ml,
                     a.Hq, p.n_split, sparse ? 0 : a.max_q, static_cast<T*>(a.o), a.lse);
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
