// Shared pieces of the paged-cache operators: the batch description, bounds
// of what device-side tables may say, 16-bit type traits, launchers.
//
// A paged cache holds K and V as [n_pages, Hkv, page_size, d]; row p of
// sequence s sits in page page_table[s][p / page_size], row p % page_size.
// A batch packs the new tokens of n_seq sequences: sequence s owns tokens
// [cu_q[s], cu_q[s+1]) and has seq_lens[s] rows, the new ones included, so
// its i-th new token stands at row seq_lens[s] - q_len + i.
#pragma once

#include <cuda_fp16.h>

#include "ts_common.cuh"

namespace ts {

struct PagedBatch {
  const int32_t* cu_q;       // [n_seq + 1]
  const int32_t* seq_lens;   // [n_seq]
  const int32_t* table;      // [n_seq, max_pages]
  int n;                     // token rows of the batch's tensors
  int n_seq;
  int max_pages;
  int page_shift;            // log2(page_size), 4..7
  int64_t n_pages;
};

// ---------------------------------------------------------------- device side
struct SeqSpan {
  int q0, ql;   // first token, new tokens
  int kl;       // rows, the new ones included
  bool bad;     // the tables said something out of their range
};

// One sequence's span, clamped so that no index derived from it leaves the
// batch's tensors or the page table.
__device__ __forceinline__ SeqSpan seq_span(const PagedBatch& b, int s) {
  const int a0 = b.cu_q[s], a1 = b.cu_q[s + 1], kl = b.seq_lens[s];
  const int64_t cap = (int64_t)b.max_pages << b.page_shift;
  SeqSpan r;
  r.q0 = min(max(a0, 0), b.n);
  const int q1 = min(max(a1, r.q0), b.n);
  r.ql = q1 - r.q0;
  r.kl = (int)imin64(imax64(kl, 0), cap);
  r.bad = a0 < 0 || a1 < a0 || a1 > b.n || kl != r.kl;
  return r;
}

// The sequence that owns token t (-1: none), searched by a whole warp.
__device__ __forceinline__ int warp_find_seq(const PagedBatch& b, int t, int lane) {
  for (int base = 0; base < b.n_seq; base += 32) {
    const int s = base + lane;
    const bool before = s < b.n_seq && t < b.cu_q[s + 1];
    const unsigned hit = __ballot_sync(0xffffffffu, before);
    if (hit) {
      const int f = base + __ffs(hit) - 1;
      return t >= b.cu_q[f] ? f : -1;
    }
  }
  return -1;
}

// The draft tree of one sequence: which nodes are ancestors of which.  Lane i
// holds node i's ancestor-or-self bits (below 32: nodes only look back) and node
// 32 + i's.  Built by a warp by pointer jumping, a round for every doubling of
// the depth (a [1, 3, 3, 3] tree takes two), instead of a chain of loads.
constexpr int kTreeNodes = 64;
struct TreeBits {
  uint32_t low;           // node lane
  uint32_t up_lo, up_hi;  // node 32 + lane

  // parents: of the sequence's first `nodes` tokens.  A parent that is not an
  // earlier node (-1 of the first) is reported, and its node becomes a root.
  __device__ __forceinline__ void build(const int32_t* parents, int nodes, int lane,
                                        int32_t* status) {
    int p0 = lane < nodes ? parents[lane] : -1;
    int p1 = 32 + lane < nodes ? parents[32 + lane] : -1;
    bool bad = false;
    if (lane < nodes && (lane == 0 ? p0 != -1 : p0 < 0 || p0 >= lane)) {
      bad = true;
      p0 = -1;
    }
    if (32 + lane < nodes && (p1 < 0 || p1 >= 32 + lane)) {
      bad = true;
      p1 = -1;
    }
    if (bad) set_status(status, TS_ERR_INVALID_ARG);
    low = 1u << lane;
    up_lo = 0u;
    up_hi = 1u << lane;
    while (__any_sync(0xffffffffu, p0 >= 0 || p1 >= 0)) {
      const uint32_t a = __shfl_sync(0xffffffffu, low, p0 & 31);
      const int pa = __shfl_sync(0xffffffffu, p0, p0 & 31);
      const uint32_t b = __shfl_sync(0xffffffffu, low, p1 & 31);
      const int pb = __shfl_sync(0xffffffffu, p0, p1 & 31);
      const uint32_t c = __shfl_sync(0xffffffffu, up_lo, p1 & 31);
      const uint32_t d = __shfl_sync(0xffffffffu, up_hi, p1 & 31);
      const int pc = __shfl_sync(0xffffffffu, p1, p1 & 31);
      if (p0 >= 0) {
        low |= a;
        p0 = pa;
      }
      if (p1 >= 32) {
        up_lo |= c;
        up_hi |= d;
        p1 = pc;
      } else if (p1 >= 0) {
        up_lo |= b;
        p1 = pb;
      }
    }
  }
  // node i's bits, a node a lane; called by the whole warp
  __device__ __forceinline__ unsigned long long of(int i) const {
    const uint32_t a = __shfl_sync(0xffffffffu, low, i & 31);
    const uint32_t b = __shfl_sync(0xffffffffu, up_lo, i & 31);
    const uint32_t c = __shfl_sync(0xffffffffu, up_hi, i & 31);
    return i < 32 ? a : ((unsigned long long)c << 32 | b);
  }
};

// 16-bit element types.
template <typename T>
struct Pair;
template <>
struct Pair<__nv_bfloat16> {
  using T2 = __nv_bfloat162;
  static constexpr bool kFp16 = false;
  __device__ static __forceinline__ float2 unpack(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ static __forceinline__ float one(const __nv_bfloat16& x) { return __bfloat162float(x); }
};
template <>
struct Pair<__half> {
  using T2 = __half2;
  static constexpr bool kFp16 = true;
  __device__ static __forceinline__ float2 unpack(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ static __forceinline__ uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
  __device__ static __forceinline__ float one(const __half& x) { return __half2float(x); }
};

// ---------------------------------------------------------------- launchers
struct AppendArgs {
  const void *q, *k, *v;                       // rows of n tokens
  int64_t q_stride, k_stride, v_stride;        // elements between tokens
  void *q_out, *k_pages, *v_pages;
  void *key_min, *key_max;                     // [n_pages, Hkv, d] or NULL
  const int32_t* positions;                    // [n] or NULL
  const double* freqs;                         // [rot / 2], radians a position
  float rope_scale;
  int rot, Hq, Hkv, interleaved;
};
int launch_paged_append(const PagedBatch& b, const AppendArgs& a, int d, bool fp16,
                        int32_t* status, cudaStream_t st);

// Attention of few query rows a KV head (new tokens x group), keys split over
// CTAs, its sparse form over per-token page lists, and its form for draft trees.
struct RowsPlan {
  int n_rb;            // blocks of 16 query rows
  int unit_trips;      // trips of 128 keys a unit, by the host's bound
  int grid;
  int cluster;         // CTAs a unit, joined on chip (0: stretches of the line)
  size_t cuts_bytes, part_bytes, ws_bytes;
};
RowsPlan rows_plan(int64_t units, int rows, int d, int64_t max_keys, bool tree = false);
struct RowsArgs {
  const void *q, *k_pages, *v_pages;
  const int32_t *pages, *counts;   // sparse form: [n, Hkv, n_sel], [n, Hkv]; else NULL
  int n_sel;
  const int32_t* parents;          // draft trees: [n], else NULL
  int Hq, Hkv, max_q;
  void* o;
  float* lse;
};
int launch_paged_rows(const PagedBatch& b, const RowsArgs& a, const RowsPlan& p, int d, bool fp16,
                      void* ws, int32_t* status, cudaStream_t st);

struct CommitArgs {
  void *const *k_pages, *const *v_pages;       // [n_layers] on the device
  void *const *key_min, *const *key_max;       // [n_layers] on the device, or NULL
  const int32_t *path, *n_path;                // [n_seq, path_stride], [n_seq]
  int path_stride, Hkv;
  int32_t* new_lens;                           // [n_seq] or NULL
};
int launch_paged_commit(const PagedBatch& b, const CommitArgs& a, int n_layers, int d, bool fp16,
                        int32_t* status, cudaStream_t st);

size_t paged_select_ws_bytes(int n, int Hkv, int max_pages);
int launch_paged_select(const PagedBatch& b, const void* q, const void* key_min,
                        const void* key_max, int Hq, int Hkv, int d, bool fp16, int n_top,
                        int n_sink, int n_recent, int32_t* pages, int32_t* counts, void* ws,
                        int32_t* status, cudaStream_t st);

}  // namespace ts
