// Logits of a batch's rows under biases, repetition penalties and masks, and the
// token counts that the penalties read.
//
//   x = logit + bias[v]
//   x = (x > 0 ? x * (1 / repetition) : x * repetition)
//       - (frequency c + presence (c > 0))     where v was met; c: how often
//   x = masked_value                            where v is not allowed
//
// "Seen" and c: the sequence's own (a bit and a count a token, kept from step to
// step) and, for the node of a draft tree, the drafted tokens on its path.
#include <cuda_fp16.h>

#include <type_traits>

#include "logits.cuh"
#include "paged.cuh"

namespace ts {

namespace {

constexpr int kThreads = 128;
constexpr int kEach = 16;              // values of a thread
constexpr int kSlice = kThreads * kEach;   // values of a block
constexpr int kMostRun = 16, kBlocksPerSm = 6;
constexpr int kAddThreads = 256;

// kG neighbouring values as they lie in memory, and in fp32.
template <int kBytes>
struct RawOf;
template <>
struct RawOf<2> { using type = unsigned short; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<8> { using type = uint2; };
template <>
struct RawOf<16> { using type = uint4; };
template <typename T, int kG, typename Raw>
__device__ __forceinline__ void widen(const Raw& raw, float* x) {
  if constexpr (sizeof(T) == 4) {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < kG; ++i) x[i] = __uint_as_float(w[i]);
  } else if constexpr (kG == 1) {
    x[0] = Pair<T>::unpack(raw).x;
  } else {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw);
#pragma unroll
    for (int i = 0; i < kG / 2; ++i) {
      const float2 y = Pair<T>::unpack(w[i]);
      x[2 * i] = y.x;
      x[2 * i + 1] = y.y;
    }
  }
}
template <int kG>
struct FloatsOf { using type = float4; };
template <>
struct FloatsOf<2> { using type = float2; };
template <>
struct FloatsOf<1> { using type = float; };

// The sequence whose rows hold `row` (-1: none), searched by a whole warp in 32
// steps at once: one round of loads up to 31 sequences, two up to 1023.
__device__ __forceinline__ int find_seq(const LogitsArgs& a, int row, int lane) {
  // even batches: the sequence stands where its share of the rows does
  const int guess = (int)((int64_t)row * a.n_seq / a.n);
  const int g0 = a.cu_q[guess], g1 = a.cu_q[guess + 1];
  if (row >= g0 && row < g1) return guess;
  int lo = 0, hi = a.n_seq + 1;        // offsets up to lo are at most row, from hi on above it
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + (lane + 1) * step;
    const unsigned in = __ballot_sync(0xffffffffu, at < hi && a.cu_q[at] <= row);
    // (offsets that fall may leave holes: up to the first one counts)
    const int steps = in == 0xffffffffu ? 32 : __ffs(~in) - 1;
    lo += steps * step;
    hi = min(hi, lo + step);
  }
  return lo < a.n_seq && a.cu_q[lo] <= row && row < a.cu_q[lo + 1] ? lo : -1;
}

// What a token's count takes off, and x under the penalties.  x / repetition is
// x times its reciprocal, off by half a step more than the quotient: the division
// and its branches took three quarters of the kernel's instructions (1024 rows of
// 128256 values: 235 us).
__device__ __forceinline__ float taken(float freq, float pres, int c) {
  const float p = __fmul_rn(freq, (float)c);
  return c > 0 ? __fadd_rn(p, pres) : p;
}
__device__ __forceinline__ float penalised(float x, float inv, float rep, float less) {
  return __fsub_rn(__fmul_rn(x, x > 0.f ? inv : rep), less);
}

// One block takes a slice of the vocabulary for a run of rows.  A thread owns the
// same tokens in every row and keeps what they have from their sequence (bits,
// penalties) in registers, gathered once a sequence; rows then need no barrier, and
// the next row's values and mask are on their way while one is worked on.  Every
// value goes through the penalties' arithmetic and is selected by its bit: the
// tokens met lie anywhere, so branches around single ones only diverge.
// Memory bound: a value is read and written once, and a mask's bit a row.  1024
// rows of 128256 bf16 values under masks, biases and drafted paths: 135 us, 5.9
// TB/s (0.88 of a copy); 64 fp32 rows of 151936: 17 us; four rows of 32000: 2.7.
// What a row costs besides its values (addresses, masks, the path) is shared by a
// thread's 16, what a sequence costs by up to 16 rows: with 8 values a thread 163
// us, with 32 152, in blocks of 256 threads (three a SM) 153, with 8 rows 157.
struct State {
  float less[kSlice];                      // what a token's count takes off
  uint32_t bias[kSlice];                   // a token's bias; its place in the list + 1 before
  unsigned long long path[kTreeNodes];     // nodes on each node's path
  unsigned long long same[kTreeNodes];     // nodes with the same token
  unsigned long long here;                 // nodes whose token is in the slice
  int token[kTreeNodes];                   // drafted tokens, from the slice's first
  int before[kTreeNodes];                  // how often they were generated before
  float saved[kTreeNodes];                 // `less` of a drafted token while a row counts it
};
static_assert(sizeof(State) <= 48 * 1024, "more shared memory has to be asked for");

// kG: neighbouring values of a thread that its rows allow to go together (4, 2 or 1;
// single values want 96 registers, and in the 80 of six blocks a SM take 434 us for
// 164 on 1024 rows of 128255, though 7.8 for 9.5 where 48 rows of 32003 are 768 blocks
// for the 760 places of five a SM).
template <typename T, int kG>
__global__ void __launch_bounds__(kThreads, kG == 1 ? 5 : kBlocksPerSm)
logits_kernel(const LogitsArgs a, int n_slices, int run, int32_t* status) {
  extern __shared__ __align__(16) uint8_t smem[];
  State& st = *reinterpret_cast<State*>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = blockIdx.x % n_slices * kSlice, v1 = min(v0 + kSlice, a.V);
  const int row0 = blockIdx.x / n_slices * run, row1 = min(row0 + run, a.n);
  const int words = (a.V + 31) / 32;
  griddep_wait();
  griddep_launch_dependents();
  // value e of this thread: its token, from the slice's first
  auto slot = [&](int e) {
    return (e / kG * kThreads + tid) * kG + e % kG;
  };
  uint32_t valid = 0;                      // values inside the slice
#pragma unroll
  for (int e = 0; e < kEach; ++e) valid |= (uint32_t)(v0 + slot(e) < v1) << e;
  // A row of bits: a warp's tokens take kEach words, one a lane; then each thread
  // picks the bits of its own.
  const int my_word = lane / kG * (kThreads * kG / 32) + warp * kG + lane % kG;
  const bool has_word = lane < kEach && (v0 >> 5) + my_word < words;
  auto ask_bits = [&](const int32_t* w) -> uint32_t {
    return has_word ? (uint32_t)w[(v0 >> 5) + my_word] : 0u;
  };
  constexpr uint32_t kBits = (1u << kG) - 1u;
  auto own_bits = [&](uint32_t w) -> uint32_t {
    uint32_t r = 0;
#pragma unroll
    for (int e = 0; e < kEach; e += kG) {
      const uint32_t x = __shfl_sync(0xffffffffu, w, e + lane * kG / 32);
      r |= (x >> lane * kG % 32 & kBits) << e;
    }
    return r;
  };
  using Raw = typename RawOf<kG * sizeof(T)>::type;
  using Floats = typename FloatsOf<kG>::type;
  Raw raw[kEach / kG];                     // the next row's values
  auto ask = [&](int row) {
    const T* in = static_cast<const T*>(a.logits) + row * a.row_stride + v0;
#pragma unroll
    for (int e = 0; e < kEach; e += kG)
      if (valid >> e & 1u) raw[e / kG] = __ldcs(reinterpret_cast<const Raw*>(in + slot(e)));
  };
  // Rows of no sequence are left as they are, and their masks are not looked at.  The
  // last rows end at the largest offset: where offsets fall, it is not the last.  (Of
  // the last 32; a loop here, or a branch, costs the rows' loop below 6 registers: 145
  // us for 136 on 1024 rows of 128256, 26 for 17.7 on 64 sequences' rows.)
  const int first = a.cu_q[0];
  const int end = min(row1, __reduce_max_sync(0xffffffffu, a.cu_q[max(a.n_seq - lane, 0)]));
  auto mask_row = [&](int row) -> int {
    if ((!a.mask && !a.mask_rows) || row >= end) return -1;
    const int mr = a.mask_rows ? a.mask_rows[row] : row;
    if (mr >= -1 && mr < a.n_masks) return mr;
    if (v0 == 0 && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
    return -1;
  };
  auto ask_mask = [&](int mr) -> uint32_t {
    return mr < 0 ? 0xFFFFFFFFu : ask_bits(a.mask + (int64_t)mr * words);
  };
  ask(row0);
  int mr = row0 + 1 < first ? -1 : mask_row(row0 + 1);
  uint32_t may_next = ask_mask(row0 < first ? -1 : mask_row(row0));
  if (blockIdx.x == 0)
    for (int s = tid; s < a.n_seq; s += kThreads) {
      const int a0 = a.cu_q[s], a1 = a.cu_q[s + 1];
      if (a0 < 0 || a1 < a0 || a1 > a.n) set_status(status, TS_ERR_INVALID_ARG);
    }
  int q0 = 0, q1 = row0;                   // the rows of the sequence at hand
  uint32_t met = 0, biased = 0;            // its bits of this thread's tokens
  float rep = 1.f, inv = 1.f, freq = 0.f, pres = 0.f;
  bool tree = false;
  for (int row = row0; row < end; ++row) {
    if (row >= q1) {
      // ---------------------------------------------------- a sequence begins
      const int s = find_seq(a, row, lane);
      if (s < 0) {
        // in front of the first sequence (whose offset is read again: in a register
        // over the loop it is one too many, 153 us for 146 at even vocabularies)
        const int begin = a.cu_q[0];
        if (begin <= row || begin >= end) return;
        ask(begin);
        may_next = ask_mask(mask_row(begin));
        mr = mask_row(begin + 1);
        row = begin - 1;
        continue;
      }
      q0 = max(a.cu_q[s], 0);
      q1 = a.cu_q[s + 1];
      rep = a.repetition ? a.repetition[s] : 1.f;
      freq = a.frequency ? a.frequency[s] : 0.f;
      pres = a.presence ? a.presence[s] : 0.f;
      const uint32_t word = a.seen ? ask_bits(a.seen + (int64_t)s * words) : 0u;
      if (!(rep >= 0x1p-64f && rep <= 0x1p64f)) {
        if (v0 == 0 && tid == 0) set_status(status, TS_ERR_INVALID_ARG);
        rep = 1.f;
      }
      inv = __fdiv_rn(1.f, rep);
      const int32_t* ids = a.bias_ids + (int64_t)s * a.n_bias;
      if (row > row0 && (a.n_bias > 0 || a.tokens)) __syncthreads();   // done with the one before
      if (a.n_bias > 0) {
#pragma unroll
        for (int e = 0; e < kEach; ++e) st.bias[slot(e)] = 0u;
        __syncthreads();
        for (int i = tid; i < a.n_bias; i += kThreads) {
          const int id = ids[i];
          if (v0 == 0 && (id < -1 || id >= a.V)) set_status(status, TS_ERR_INVALID_ARG);
          // of equal ids the last of the list counts
          if (id >= v0 && id < v1) atomicMax(&st.bias[id - v0], (uint32_t)i + 1u);
        }
      }
      if (a.tokens && warp < 3) {
        // three warps gather a part each of what the paths need
        const int nodes = min(min(q1, a.n) - q0, kTreeNodes);
        if (warp == 0) {
          if (min(q1, a.n) - q0 > kTreeNodes && lane == 0) set_status(status, TS_ERR_INVALID_ARG);
          TreeBits bits;
          bits.build(a.parents + q0, nodes, lane, status);
          st.path[lane] = bits.of(lane);
          st.path[lane + 32] = bits.of(lane + 32);
        } else {
          int id[2];
          bool here[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = lane + 32 * i;
            const bool one = at > 0 && at < nodes;           // the root is in the history
            id[i] = one ? a.tokens[q0 + at] : v0 - 1;
            here[i] = id[i] >= v0 && id[i] < v1;
            if (one && (id[i] < 0 || id[i] >= a.V)) set_status(status, TS_ERR_INVALID_ARG);
          }
          if (warp == 1) {
            const unsigned lo = __ballot_sync(0xffffffffu, here[0]);
            const unsigned hi = __ballot_sync(0xffffffffu, here[1]);
            const unsigned long long all = (unsigned long long)hi << 32 | lo;
            unsigned long long same[2] = {0, 0};
            for (unsigned long long left = all; left; left &= left - 1) {
              const int i = __ffsll(left) - 1;
              const int x = __shfl_sync(0xffffffffu, i < 32 ? id[0] : id[1], i & 31);
              if (id[0] == x) same[0] |= 1ull << i;
              if (id[1] == x) same[1] |= 1ull << i;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              st.token[lane + 32 * i] = id[i] - v0;
              st.same[lane + 32 * i] = same[i];
            }
            if (lane == 0) st.here = all;
          } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const bool known =
                  here[i] && a.counts &&
                  ((uint32_t)a.seen[(int64_t)s * words + (id[i] >> 5)] >> (id[i] & 31) & 1u);
              st.before[lane + 32 * i] = known ? a.counts[(int64_t)s * a.V + id[i]] : 0;
            }
          }
        }
      }
      // this thread's tokens: their counts, all asked for at once
      met = own_bits(word) & valid;
      const int32_t* counts = a.counts ? a.counts + (int64_t)s * a.V + v0 : nullptr;
      int c[kEach];
#pragma unroll
      for (int e = 0; e < kEach; ++e) c[e] = 0;
      if (counts) {
#pragma unroll
        for (int e = 0; e < kEach; e += kG)
          if (met >> e & kBits) {
            const Floats y = *reinterpret_cast<const Floats*>(counts + slot(e));   // as bits
            const int* w = reinterpret_cast<const int*>(&y);
#pragma unroll
            for (int i = 0; i < kG; ++i) c[e + i] = w[i];
          }
      }
#pragma unroll
      for (int e = 0; e < kEach; ++e) st.less[slot(e)] = taken(freq, pres, c[e]);
      if (a.n_bias > 0 || a.tokens) __syncthreads();
      tree = a.tokens && st.here != 0;
      biased = 0;
      if (a.n_bias > 0) {
        const float* bias = a.bias + (int64_t)s * a.n_bias;
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
          const uint32_t i = st.bias[slot(e)];
          if (i) {
            biased |= 1u << e;
            st.bias[slot(e)] = __float_as_uint(bias[i - 1]);
          }
        }
      }
    }
    // ------------------------------------------------------ one row
    float x[kEach];
#pragma unroll
    for (int e = 0; e < kEach; e += kG) widen<T, kG>(raw[e / kG], x + e);
    const uint32_t may = own_bits(may_next);
    if (row + 1 < end) {
      ask(row + 1);
      may_next = ask_mask(mr);
      mr = mask_row(row + 2);
    }
    if (biased) {
#pragma unroll
      for (int e = 0; e < kEach; ++e)
        if (biased >> e & 1u) x[e] += __uint_as_float(st.bias[slot(e)]);
    }
    // Tokens drafted on this row's path: their owners count them in for the row.
    uint32_t do_now = met;
    unsigned long long changed = 0;
    if (tree) {
      const unsigned long long drafted = row - q0 < kTreeNodes ? st.path[row - q0] & st.here : 0ull;
      for (unsigned long long left = drafted; left; left &= left - 1) {
        const int at = __ffsll(left) - 1, t = st.token[at];
        if (t / kG % kThreads != tid) continue;
        const uint32_t bit = 1u << (t / (kG * kThreads) * kG + t % kG);
        const unsigned long long same = drafted & st.same[at];
        if (same & ((1ull << at) - 1)) continue;             // an earlier node took it
        st.saved[at] = st.less[t];
        st.less[t] = taken(freq, pres, st.before[at] + __popcll(same));
        changed |= 1ull << at;
        do_now |= bit;
      }
    }
#pragma unroll
    for (int g = 0; g < kEach; g += 4) {
      if (!__any_sync(0xffffffffu, do_now >> g & 15u)) continue;
      float less[4];
#pragma unroll
      for (int i = 0; i < 4; i += kG)
        *reinterpret_cast<Floats*>(less + i) = *reinterpret_cast<const Floats*>(&st.less[slot(g + i)]);
#pragma unroll
      for (int e = g; e < g + 4; ++e) {
        const float y = penalised(x[e], inv, rep, less[e - g]);
        x[e] = do_now >> e & 1u ? y : x[e];
      }
    }
    for (; changed; changed &= changed - 1) {
      const int at = __ffsll(changed) - 1;
      st.less[st.token[at]] = st.saved[at];
    }
    float* out = a.out + row * a.out_stride + v0;
#pragma unroll
    for (int e = 0; e < kEach; ++e)
      if (!(may >> e & 1u)) x[e] = a.masked_value;
#pragma unroll
    for (int e = 0; e < kEach; e += kG)
      if (valid >> e & 1u)
        *reinterpret_cast<Floats*>(out + slot(e)) = *reinterpret_cast<const Floats*>(x + e);
  }
}

// Counts added to a state: an atomic a token and count, a bit only where it is not
// set yet (a stream's frequent tokens share a few words).
__global__ void __launch_bounds__(kAddThreads)
token_counts_kernel(const int32_t* __restrict__ tokens, const int32_t* __restrict__ lens,
                    int stride, int per_seq, int V, int32_t* __restrict__ counts, int32_t* seen,
                    int32_t* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.x / per_seq, i = blockIdx.x % per_seq * kAddThreads + threadIdx.x;
  const int n = lens[s];
  if (i == 0 && (n < 0 || n > stride)) set_status(status, TS_ERR_INVALID_ARG);
  if (i >= min(n, stride)) return;
  const int id = tokens[(int64_t)s * stride + i];
  if (id < 0 || id >= V) {
    set_status(status, TS_ERR_INVALID_ARG);
    return;
  }
  int32_t* word = &seen[(int64_t)s * ((V + 31) / 32) + (id >> 5)];
  const int32_t bit = (int32_t)(1u << (id & 31));
  if (!(*(volatile int32_t*)word & bit)) atomicOr(word, bit);
  if (counts) atomicAdd(&counts[(int64_t)s * V + id], 1);
}

// A state that starts over: a block counts one share of the vocabulary in shared
// memory over all of the sequence's tokens and writes it whole, so nothing is
// cleared first and nothing is counted in memory.  Shares go round by 32 tokens (a
// word of bits), since frequent tokens lie together.  8 streams of up to 100K
// tokens: 13.8 us; in contiguous shares 15, with clears and atomics in memory 31,
// with a warp's equal tokens matched first 58.
constexpr int kCountThreads = 1024;
constexpr int kMostShare = 48 * 1024;  // counts in shared memory
__global__ void __launch_bounds__(kCountThreads)
token_recount_kernel(const int32_t* __restrict__ tokens, const int32_t* __restrict__ lens,
                     int stride, int shares_log, int V, int prompt,
                     int32_t* __restrict__ counts, int32_t* __restrict__ seen, int32_t* status) {
  extern __shared__ int hist[];
  const int tid = threadIdx.x, lane = tid & 31;
  const int s = blockIdx.x >> shares_log, share = blockIdx.x & ((1 << shares_log) - 1);
  const int words = (V + 31) / 32;
  const int mine_words = (words - share + (1 << shares_log) - 1) >> shares_log;
  griddep_wait();
  griddep_launch_dependents();
  for (int v = tid; v < mine_words * 32; v += kCountThreads) hist[v] = 0;
  const int n = min(max(lens[s], 0), stride);
  if (share == 0 && tid == 0 && n != lens[s]) set_status(status, TS_ERR_INVALID_ARG);
  __syncthreads();
  const int32_t* mine = tokens + (int64_t)s * stride;
  // four neighbours a load where the rows allow it; the next are on their way while
  // these are counted
  constexpr int kAtOnce = 4;
  const bool whole = stride % 4 == 0 && reinterpret_cast<uintptr_t>(tokens) % 16 == 0;
  int4 id[kAtOnce], then[kAtOnce];
  auto ask = [&](int base, int4 (&to)[kAtOnce]) {
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int i = base + (x * kCountThreads + tid) * 4;
      to[x] = make_int4(-1, -1, -1, -1);
      if (whole && i + 4 <= n) {
        to[x] = *reinterpret_cast<const int4*>(mine + i);
      } else {
        if (i < n) to[x].x = mine[i];
        if (i + 1 < n) to[x].y = mine[i + 1];
        if (i + 2 < n) to[x].z = mine[i + 2];
        if (i + 3 < n) to[x].w = mine[i + 3];
      }
    }
  };
  auto count = [&](int x, int i) {
    if ((unsigned)x >= (unsigned)V) {
      if (share == 0 && i < n) set_status(status, TS_ERR_INVALID_ARG);
    } else if ((x >> 5 & ((1 << shares_log) - 1)) == share) {
      atomicAdd(&hist[(x >> (5 + shares_log) << 5) | (x & 31)], 1);
    }
  };
  ask(0, id);
  for (int base = 0; base < n; base += kCountThreads * kAtOnce * 4) {
    ask(base + kCountThreads * kAtOnce * 4, then);
#pragma unroll
    for (int x = 0; x < kAtOnce; ++x) {
      const int i = base + (x * kCountThreads + tid) * 4;
      count(id[x].x, i);
      count(id[x].y, i + 1);
      count(id[x].z, i + 2);
      count(id[x].w, i + 3);
      id[x] = then[x];
    }
  }
  __syncthreads();
  // a warp a word of 32 tokens
  int32_t* row = counts ? counts + (int64_t)s * V : nullptr;
  int32_t* bits = seen + (int64_t)s * words;
  for (int w = tid >> 5; w < mine_words; w += kCountThreads / 32) {
    const int at = (w << shares_log) + share, v = at * 32 + lane;
    const int c = hist[w * 32 + lane];
    const unsigned word = __ballot_sync(0xffffffffu, c > 0);
    if (lane == 0) bits[at] = (int32_t)word;
    if (row && v < V) row[v] = prompt ? 0 : c;
  }
}

}  // namespace

template <typename T>
static int go_logits(const LogitsArgs& a, int32_t* status, cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const int n_slices = (a.V + kSlice - 1) / kSlice;
  // rows a block takes in a run: one as long as the SMs are not full
  const int64_t blocks = (int64_t)a.n * n_slices;
  const int run = (int)imax64(1, imin64(kMostRun, blocks / (kGb300Sms * kBlocksPerSm)));
  // four or two values at once where every row starts on a boundary of as many (1024
  // bf16 rows of 128256, 128254 and 128255 values: 135, 148 and 164 us)
  auto fits = [&](int g) {
    auto one = [&](const void* p, int64_t stride, size_t size) {
      return reinterpret_cast<uintptr_t>(p) % (g * size) == 0 && stride % g == 0;
    };
    return a.V % g == 0 && one(a.logits, a.n > 1 ? a.row_stride : 0, sizeof(T)) &&
           one(a.out, a.n > 1 ? a.out_stride : 0, 4) && one(a.counts, 0, 4);
  };
  const int g = fits(4) ? 4 : fits(2) ? 2 : 1;
  pdl_config(&cfg, attr, dim3((unsigned)((a.n + run - 1) / run * n_slices)),
             dim3(kThreads), sizeof(State), st);
  auto kern = g == 4 ? logits_kernel<T, 4> : g == 2 ? logits_kernel<T, 2> : logits_kernel<T, 1>;
  cudaLaunchKernelEx(&cfg, kern, a, n_slices, run, status);
  return launch_status("logits_kernel");
}

int launch_logits(const LogitsArgs& a, int type, int32_t* status, cudaStream_t st) {
  return type == 0   ? go_logits<float>(a, status, st)
         : type == 1 ? go_logits<__nv_bfloat16>(a, status, st)
                     : go_logits<__half>(a, status, st);
}

int launch_token_counts(const int32_t* tokens, const int32_t* lens, int n_seq, int stride, int V,
                        int32_t* counts, int32_t* seen, bool reset, bool prompt, int32_t* status,
                        cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  if (reset) {
    // shares that shared memory holds, and enough for the SMs while they keep 4096
    // tokens
    const int words = (V + 31) / 32;
    int shares_log = 0;
    auto share_words = [&] { return (words + (1 << shares_log) - 1) >> shares_log; };
    while (share_words() * 32 > kMostShare ||
           ((n_seq << (shares_log + 1)) <= kGb300Sms && share_words() * 32 >= 8192))
      ++shares_log;
    cudaFuncSetAttribute(token_recount_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kMostShare * 4);
    pdl_config(&cfg, attr, dim3((unsigned)(n_seq << shares_log)), dim3(kCountThreads),
               (size_t)share_words() * 128, st);
    cudaLaunchKernelEx(&cfg, token_recount_kernel, tokens, lens, stride, shares_log, V, (int)prompt,
                       counts, seen, status);
    return launch_status("token_recount_kernel");
  }
  const int per_seq = (stride + kAddThreads - 1) / kAddThreads;
  pdl_config(&cfg, attr, dim3((unsigned)((int64_t)per_seq * n_seq)), dim3(kAddThreads), 0, st);
  cudaLaunchKernelEx(&cfg, token_counts_kernel, tokens, lens, stride, per_seq, V,
                     prompt ? (int32_t*)nullptr : counts, seen, status);
  return launch_status("token_counts_kernel");
}

}  // namespace ts
