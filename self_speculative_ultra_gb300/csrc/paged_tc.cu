// Attention of chunks of new tokens over a paged cache on the 5th-generation
// tensor cores (tcgen05).
//
//   s_ij = q_i . k_j / sqrt(d), j <= seq_len - q_len + i
//   o_i = softmax_j(s) . v,  lse_i = ln sum_j exp(s_ij)
//
// or, where the new tokens are the nodes of a draft tree, over the rows in front
// of the tree and those of the node's ancestors and itself.
// The query rows of a KV head (row R = new token R / G, head kv * G + R % G)
// are cut into tiles of 256, two groups of 128.  A chunk over a long cache is
// bound by the tensor cores (4 d flops a row and key); the softmax stands between
// the two products, so the groups alternate: while one group's scores are
// exponentiated the tensor core works for the other.  2048 tokens over 100K rows,
// 32/8 heads, d = 128: 1.93 ms, 1760 TFLOP/s; over 32K rows, 12/2 heads: 245 us, in
// fp16 250, at d = 64 177 and 180 us (the best of a few calls in a row; called for
// seconds on end, at the power cap, the first two take 2.15 ms and 266 us).
//
// A draft tree has at most 64 nodes, so its rows are one tile of 256 (or a few), and
// the call stands between HBM and the tensor cores: a step reads 64 KB at d = 128,
// 1.47 us at an even share of the copy bandwidth, and takes 1.5 us of products.  A
// node's ancestors are 64 bits a row, laid over the one or two key tiles that hold
// the tree; all other tiles are as in a chunk.  A tile of at most 128 rows is one
// group, which takes both S tiles in turn (0.9 us a step for 1.5).  Where every tree
// is one tile there is no plan (see Line).  64 nodes over 100K rows, 32/8 heads: 80
// us, 5.2 TB/s with start and join (90 back to back for seconds, at the power cap); 12
// trees of 25 nodes over 24K rows, 40/8 heads: 189 us (6.4 TB/s), of 51 nodes 229, of
// 64 (a tile of 256 rows and one of 64, which read the keys twice) 364 to 371.
//
// Three launches.  The plan (one CTA) lists the work from the device-side
// lengths in order of falling cost: the tiles of whole rounds over the SMs as
// they are, the rest cut along the keys into pieces where it pays.  The
// attention kernel keeps one CTA a SM; its copy warp takes the next item off
// the list when the last copies of the one before are due, so that copies run
// ahead across items.  The third kernel joins the pieces of cut tiles.
//
// Per 128-key tile of an item:
//   warps 0, 2   copy K (2 stages) and V (3 stages), one box a page and
//                64-column panel, each lane one box; 128-byte swizzle
//   warp 1       S_g = Q_g K^T (M = N = 128, fp32 in TMEM); when the softmax
//                has written P_g over S_g, O_g += P_g V with P read from TMEM (at
//                d = 64 that is warp 3's)
//   warps 4..7   the item's query rows into shared memory; rows of V behind
//                the sequence's last are cleared (0 * NaN would reach O)
//   warps 8..15  softmax, one thread a row: all 128 scores in registers,
//                P = 2^(s log2e / sqrt(d) - m) against a reference m that moves
//                only when a tile's row sum of P exceeds 2^15 (or in fp16 falls
//                below 2^-7, see kHead); sums in fp32.  P is rounded once, to
//                the type of V, since the tensor core takes both operands of a
//                product in one 16-bit type: off by half a step a weight, as the
//                output's own rounding is, and averaged over the keys.  (The call
//                over a contiguous cache has P in fp16 and turns a bf16 V into fp16
//                for it, which bounds |v|; here V keeps its type and range.)
// At the end of an item the softmax warps write O / l (or the piece's O, m, l
// in fp32); the next item's first scores are formed meanwhile.
//
// Every wait is bounded; on expiry the CTA reports TS_ERR_TIMEOUT, waits for
// its own copies and products, frees its TMEM and returns.
#include <cuda.h>
#include <cstddef>

#include "paged.cuh"
#include "paged_tc.cuh"
#include "tc_ptx.cuh"

namespace ts {

namespace {

constexpr int kNk = 128;               // keys a tile
constexpr int kM = kTcRows;            // query rows a tile
constexpr int kRing = 4;               // barriers in turn for a group's tiles
constexpr int kThreads = 512;
constexpr int kRegsLow = 64, kRegsSoftmax = 192;
static_assert(2 * 128 * kRegsLow + 2 * 128 * kRegsSoftmax == kThreads * 128,
              "the register split must use exactly the launch's registers");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFastSum = 32768.0f;
// Where the reference m of P = 2^(x - m) stands.  In bf16 it is the largest
// exponent x at its last move, and only rises.  fp16 has nothing below 2^-24:
// against a maximum far above (a first key that draws most of the attention) the
// tail's weights would round to 0 while their sum counts them.  So there it is
// set kHead below the largest (128 weights of 2^7 sum to 2^14), and falls too,
// where a row's 128 weights sum to less than kLeastSum: above that they lose at
// most 128 * 2^-25 = 2^-11 of their sum beside their own half steps.  It falls by
// kFall at most and only while l is below kFallSum, which keeps O and l in fp32's
// range (2^40 * 2^64, |v| < 2^16); 128 keys that it does not follow are less
// than 2^-47 of what was seen.  A tile that moves it is loaded and exponentiated
// twice: one sink moves it once (2048 tokens over 32K rows: 260 us with and without),
// scores that swing by tens of nats every 128 keys at every tile (387 us).
constexpr float kHead = 7.f, kLeastSum = 1.f / 128.f, kFall = 64.f, kFallSum = 1.1e12f;
constexpr long long kDrainCycles = 1ll << 31;
constexpr uint32_t kNegInf = 0xFF800000u;

struct Header {
  int n_entries;      // entries of the list; an entry is one item a KV head
  int n_cut;          // cut tiles
  int taken;          // items taken off the list behind each CTA's first
};

// -------------------------------------------------------------------- plan
constexpr int kPlanThreads = 1024;
constexpr int kPlanTiles = 2048;
constexpr int kPlanParts = 512;      // more than a tile is ever cut into

__device__ __forceinline__ int tile_steps(const SeqSpan& sp, int rows, int tile, int G) {
  const int last = min((tile + 1) * kM, rows) - 1;
  const int vis = sp.kl - sp.ql + last / G + 1;
  return vis <= 0 ? 0 : (vis + kNk - 1) / kNk;
}

// A tile of one group (at most 128 rows) carries this bit beside its number.  Where
// one group takes both S tiles (draft trees at d = 128) a step of it costs less
// than one of two groups: 1720 cycles for 2870 with K and V in L2.
constexpr int kSoloBit = 1 << 30, kSoloEighths = 5;

// Pieces of a tile of `steps` key tiles when a piece takes at most `per`.
__device__ __forceinline__ int pieces_of(int steps, int per) {
  return steps <= per ? 1 : (steps + per - 1) / per;
}

__global__ void __launch_bounds__(kPlanThreads)
paged_plan_kernel(const PagedBatch b, int Hkv, int G, int D, int max_q, int solo, int max_tiles,
                  int max_entries, int max_slots, Header* hdr, int4* tiles, int4* entries, int* slots, int4* cuts,
                  int32_t* status) {
  // the tiles as found and in order: in shared memory where they fit (every
  // pass over them otherwise waits for L2, and the plan is all latency)
  extern __shared__ int4 near_tiles[];
  if (max_tiles <= kPlanTiles) tiles = near_tiles;
  int4* sorted = tiles + max_tiles;
  __shared__ int first[kPlanThreads + 1];    // tiles before each sequence of the trip
  __shared__ int seq_rows[kPlanThreads];
  __shared__ int scan[32];
  __shared__ int s_max;
  __shared__ unsigned long long s_total, s_keys;
  __shared__ float est[32];
  __shared__ int est_per[32], est_whole[32];
  __shared__ int hist[256];
  __shared__ int at[kPlanParts];
  __shared__ int s_slots, s_cut, s_most, s_entries;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) {
    s_max = 0;
    s_total = s_keys = 0;
  }
  for (int i = tid; i < 256; i += kPlanThreads) hist[i] = 0;
  // a tile (sequence, number and bit, steps): what it costs, in steps of two groups
  auto price = [&](const int4& t) { return t.y & kSoloBit ? (t.z * solo + 7) >> 3 : t.z; };
  int n_tiles = 0;
  for (int base = 0; base < b.n_seq; base += kPlanThreads) {
    const int s = base + tid;
    int cnt = 0, rows = 0;
    unsigned long long keys = 0;
    if (s < b.n_seq) {
      const SeqSpan sp = seq_span(b, s);
      if (sp.bad || sp.ql > max_q) set_status(status, TS_ERR_INVALID_ARG);
      rows = min(sp.ql, max_q) * G;
      cnt = (rows + kM - 1) / kM;
      if (cnt) keys = sp.kl;
    }
    int inc = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    const int mine_w = scan[lane];
    const int total = warp_sum_int(mine_w);
    const int off = warp_sum_int(lane < warp ? mine_w : 0);
    first[tid] = off + inc - cnt;
    seq_rows[tid] = rows;
    if (tid == 0) first[kPlanThreads] = total;
    __syncthreads();
    unsigned long long mine = 0;
    int top = 0;
    for (int i = tid; i < total; i += kPlanThreads) {
      // the last sequence of the trip that starts at or before tile i
      int lo = 0, hi = kPlanThreads - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      const int sq = base + lo, t = i - first[lo];
      const int steps = tile_steps(seq_span(b, sq), seq_rows[lo], t, G);
      const int4 tile = make_int4(sq, seq_rows[lo] - t * kM <= 128 ? t | kSoloBit : t, steps, 0);
      if (n_tiles + i < max_tiles) tiles[n_tiles + i] = tile;
      mine += price(tile);
      top = max(top, price(tile));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      mine += __shfl_xor_sync(0xffffffffu, mine, o);
      keys += __shfl_xor_sync(0xffffffffu, keys, o);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) {
      atomicAdd(&s_keys, keys);
      atomicAdd(&s_total, mine);
      atomicMax(&s_max, top);
    }
    n_tiles += total;
    __syncthreads();
  }
  n_tiles = min(n_tiles, max_tiles);
  const int longest = max(s_max, 1);
  // counts of the classes -> where each class starts
  auto starts = [&]() {
    int c[8], sum = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = hist[lane * 8 + i];
      sum += c[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += x;
    }
    int at = inc - sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      hist[lane * 8 + i] = at;
      at += c[i];
    }
    if (lane == 31) s_entries = at;
  };
  // tiles by falling cost (256 classes)
  const float class_of = 255.f / longest;
  auto bucket = [&](int steps) { return 255 - min(255, (int)(steps * class_of)); };
  for (int i = tid; i < n_tiles; i += kPlanThreads) atomicAdd(&hist[bucket(price(tiles[i]))], 1);
  __syncthreads();
  if (warp == 0) starts();
  __syncthreads();
  // Where tiles may be cut, those of a class stay in the order of the batch: which
  // are cut, and where, must not hang on which warp comes first, or the sums'
  // rounding would.  One warp, 32 tiles a trip.
  const bool may_cut = (long long)n_tiles * Hkv < 16 * kGb300Sms && longest > 1 && max_slots > 0;
  if (!may_cut) {
    for (int i = tid; i < n_tiles; i += kPlanThreads) {
      const int4 t = tiles[i];
      sorted[atomicAdd(&hist[bucket(price(t))], 1)] = t;
    }
  } else if (warp == 0) {
    for (int base = 0; base < n_tiles; base += 32) {
      const int i = base + lane;
      const int4 t = i < n_tiles ? tiles[i] : make_int4(0, 0, 0, 0);
      const int c = i < n_tiles ? bucket(price(t)) : 256;
      const unsigned same = __match_any_sync(0xffffffffu, c);
      const int to = (c < 256 ? hist[c] : 0) + __popc(same & ((1u << lane) - 1u));
      __syncwarp();
      if (c < 256) {
        sorted[to] = t;
        if (lane == 31 - __clz(same)) hist[c] = to + 1;
      }
      __syncwarp();
    }
  }
  __syncthreads();
  // Which tiles to cut, and how far: the first `whole` of the order stay, the
  // others go into pieces of at most `per` steps.  Candidates: no cut, and
  // whole rounds over the SMs (none, all, all but one) x 8 to 15 piece lengths.
  // A candidate's time in key steps is at least its work spread evenly, and at
  // least what its longest chain takes.  Pieces of about one length go in
  // rounds, behind the rounds of whole tiles; others end half a piece ragged.
  // A piece costs kFixed steps more (first copies, last product, epilogue),
  // a cut one kCut for its partial rows.
  constexpr float kFixed = 3.f, kCut = 2.f;
  const int C = kGb300Sms;
  int whole = n_tiles, per = longest, stretch = 0;
  if (may_cut) {
    const int rounds = n_tiles * Hkv / C;
    float best = INFINITY;
    int best_whole = n_tiles, best_per = longest;
    // one candidate a warp: 16 without whole tiles (the first without a cut),
    // 8 behind all and 8 behind all but one round
    int w = n_tiles, p = longest;
    const int kind = warp < 16 ? 0 : warp < 24 ? 1 : 2;
    const int keep = kind == 0 ? 0 : rounds + 1 - kind;
    const bool valid = warp == 0 || kind == 0 || keep > 0;
    if (valid && warp > 0) {
      w = min(n_tiles, keep * C / Hkv);
      if (w < n_tiles) {
        constexpr unsigned char kParts[16] = {1, 2, 3, 4, 5, 6, 7, 8, 10, 13, 17, 24, 36, 54, 76, 120};
        const int parts = kParts[kind == 0 ? warp : (warp & 7) + 1];
        // no tile of the rest is longer than its first's class (a step more for
        // the class's rounding)
        const int top = min(longest, price(sorted[w]) + longest / 255 + 2);
        p = (top + parts - 1) / parts;
      }
    }
    // pieces_of without its division (the quotient put right, as the slots are
    // counted by it); the lengths only feed the estimate
    const float inv = 1.f / p;
    int n_pieces = 0, n_cut = 0;
    float low = longest, high = 0.f;
    for (int i = w + lane; i < n_tiles; i += 32) {
      const int steps = price(sorted[i]);
      int np = (int)(steps * inv);
      np += np * p < steps;
      np -= (np - 1) * p >= steps;
      np = max(np, 1);
      n_pieces += np;
      if (np > 1) n_cut += np;
      const float len = __fdividef((float)steps, (float)np);
      low = fminf(low, len);
      high = fmaxf(high, len);
    }
    const float shortest = -warp_max(-low), widest = warp_max(high);
    n_pieces = __reduce_add_sync(0xffffffffu, n_pieces);
    n_cut = __reduce_add_sync(0xffffffffu, n_cut);
    const float cost = kFixed + (n_cut ? kCut : 0.f);
    const float even = ((float)s_total * Hkv + (float)(n_pieces + w) * Hkv * kFixed +
                        (float)n_cut * Hkv * kCut) / C;
    // longest chain of whole tiles: k + 1 of them where the order's item
    // k C is the k-th to follow
    float chain = 0.f;
    if (lane * C < w * Hkv) chain = (lane + 1) * (price(sorted[lane * C / Hkv]) + kFixed);
    chain = warp_max(chain);
    const float pieces = (float)((n_pieces * Hkv + C - 1) / C) * (widest + cost);
    float e = fmaxf(even, chain) + (n_cut ? kCut : 0.f);
    if (w < n_tiles) {
      const bool equal = w == 0 || price(sorted[w - 1]) * 10 >= price(sorted[0]) * 9;
      if (!equal || shortest * 10.f < widest * 9.f)
        e = fmaxf(e, even + 0.5f * widest);
      else
        e = fmaxf(e, (w ? (float)((w * Hkv + C - 1) / C) * (price(sorted[0]) + kFixed) : 0.f) + pieces);
    }
    if (valid && (long long)n_cut * Hkv <= max_slots) {
      best = e;
      best_whole = w;
      best_per = p;
    }
    if (lane == 0) {
      est[warp] = best;
      est_per[warp] = best_per;
      est_whole[warp] = best_whole;
    }
    __syncthreads();
    // the least, of equals the first warp's
    best = est[lane];
    int from = lane;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float x = __shfl_xor_sync(0xffffffffu, best, o);
      const int f = __shfl_xor_sync(0xffffffffu, from, o);
      if (x < best || (x == best && f < from)) {
        best = x;
        from = f;
      }
    }
    whole = est_whole[from];
    per = est_per[from];
    // Or, where pieces of about one length would leave a round half empty, cut
    // evenly: the tiles in a line, in equal stretches, as many a KV head as it
    // has SMs.  The stretches stand at different keys, so K and V have to stay in
    // L2.  (2048 tokens over 32K rows, 2 KV heads: 257 us in pieces, 244 in
    // stretches; tiles of many lengths fill the SMs better by themselves: 9 mixed
    // streams take 6 % longer in stretches, 10 draft trees over 3K to 24K rows too.)
    const unsigned heads = C / Hkv;
    if (heads > 0 && price(sorted[n_tiles - 1]) * 10 >= longest * 9 && s_keys * Hkv * D * 4 <= (64ull << 20) &&
        (long long)(n_tiles + heads) * Hkv <= max_slots) {
      // at most 16 C tiles of 2^18 steps: below 2^31
      const int even = (int)(((unsigned)s_total + heads - 1) / heads);
      if (even + 3.f * kFixed + 2.f * kCut < best) stretch = even;
    }
  }
  if (stretch > 0) {
    // The list: the stretches' parts of tiles, the longest first (a CTA that ends
    // a short one early takes the longest left, so two together make a stretch).
    // sorted[i].w: where tile i starts on the line, which is measured in cost.
    __syncthreads();
    if (tid < 256) hist[tid] = 0;
    if (tid == 0) s_slots = s_cut = 0;
    int before = 0;
    for (int base = 0; base < n_tiles; base += kPlanThreads) {
      const int i = base + tid, z = i < n_tiles ? price(sorted[i]) : 0;
      int inc = z;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      const int mine_w = scan[lane];
      if (i < n_tiles) sorted[i].w = before + inc - z;
      const int ahead = warp_sum_int(lane < warp ? mine_w : 0);
      if (i < n_tiles) sorted[i].w += ahead;
      before += warp_sum_int(mine_w);
      __syncthreads();
    }
    const float part_class = 255.f / stretch;
    auto cls = [&](int len) { return 255 - min(255, (int)(len * part_class)); };
    // part p of tile t at [w, w + price): from the p-th cut at or before it, in steps;
    // returns its cost
    auto part = [&](const int4& t, int p, int& k0, int& k1) {
      const int at = t.w, z = price(t), cut = (at / stretch + p) * stretch;
      const int c0 = max(cut, at) - at, c1 = min(cut + stretch, at + z) - at;
      const int eighths = t.y & kSoloBit ? solo : 8;
      k0 = min(c0 * 8 / eighths, t.z);
      k1 = c1 == z ? t.z : min(c1 * 8 / eighths, t.z);
      return c1 - c0;
    };
    auto parts = [&](const int4& t) {
      return t.z == 0 ? 1 : (t.w + price(t) - 1) / stretch - t.w / stretch + 1;
    };
    for (int i = tid; i < n_tiles; i += kPlanThreads) {
      const int4 t = sorted[i];
      const int np = parts(t);
      for (int p = 0; p < np; ++p) {
        int k0, k1;
        atomicAdd(&hist[cls(part(t, p, k0, k1))], 1);
      }
    }
    __syncthreads();
    if (warp == 0) starts();
    __syncthreads();
    for (int i = tid; i < n_tiles; i += kPlanThreads) {
      const int4 t = sorted[i];
      const int np = parts(t);
      int slot = -1;
      if (np > 1) {
        slot = atomicAdd(&s_slots, np);
        cuts[atomicAdd(&s_cut, 1)] = make_int4(t.x, t.y & ~kSoloBit, slot, np);
      }
      for (int p = 0; p < np; ++p) {
        int k0, k1;
        const int e = atomicAdd(&hist[cls(part(t, p, k0, k1))], 1);
        if (e >= max_entries) continue;
        entries[e] = make_int4(t.x, t.y & ~kSoloBit, k0, k1);
        slots[e] = slot < 0 ? -1 : slot + p;
      }
    }
    __syncthreads();
  } else {
    // The list: whole tiles, then the others' pieces, first pieces first, so that
    // neighbours in time read the same keys.  at[p]: where the p-th pieces go.
    __syncthreads();
    if (tid < kPlanParts) at[tid] = 0;
    if (tid == 0) s_slots = s_cut = s_most = 0;
    __syncthreads();
    for (int i = tid; i < n_tiles; i += kPlanThreads) {
      const int4 t = sorted[i];
      if (i < whole) {
        if (i < max_entries) {
          entries[i] = make_int4(t.x, t.y & ~kSoloBit, 0, t.z);
          slots[i] = -1;
        }
        continue;
      }
      const int np = pieces_of(price(t), per);
      atomicAdd(&at[np - 1], 1);          // tiles of np pieces, for now
      atomicMax(&s_most, np);
      int slot = -1;
      if (np > 1) {
        slot = atomicAdd(&s_slots, np);
        cuts[atomicAdd(&s_cut, 1)] = make_int4(t.x, t.y & ~kSoloBit, slot, np);
      }
      sorted[i].w = slot;
    }
    __syncthreads();
    const int most = s_most;
    if (warp == 0) {
      // tiles that have a p-th piece: sums from the back; then where they start
      int n_p[kPlanParts / 32], sum = 0;
#pragma unroll
      for (int x = kPlanParts / 32 - 1; x >= 0; --x) {
        sum += at[lane * (kPlanParts / 32) + x];
        n_p[x] = sum;
      }
      int behind = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_down_sync(0xffffffffu, behind, o);
        if (lane + o < 32) behind += x;
      }
      behind -= sum;                      // tiles whose last piece is a later lane's
      sum = 0;
#pragma unroll
      for (int x = 0; x < kPlanParts / 32; ++x) {
        n_p[x] += behind;
        sum += n_p[x];
      }
      int before = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += x;
      }
      if (lane == 31) s_entries = whole + before;
      before += whole - sum;
#pragma unroll
      for (int x = 0; x < kPlanParts / 32; ++x) {
        at[lane * (kPlanParts / 32) + x] = before;
        before += n_p[x];
      }
    }
    __syncthreads();
    for (int u = tid; u < (n_tiles - whole) * most; u += kPlanThreads) {
      const int i = whole + u / most, p = u % most;
      const int4 t = sorted[i];
      const int np = pieces_of(price(t), per);
      if (p >= np) continue;
      const int len = (t.z + np - 1) / np, e = atomicAdd(&at[p], 1);
      if (e >= max_entries) continue;
      entries[e] = make_int4(t.x, t.y & ~kSoloBit, min(p * len, t.z), min((p + 1) * len, t.z));
      slots[e] = t.w < 0 ? -1 : t.w + p;
    }
  }
  if (tid == 0) {
    hdr->n_entries = min(s_entries, max_entries);
    hdr->n_cut = s_cut;
    hdr->taken = 0;
  }
}

// -------------------------------------------------------------------- attention
// One item: a tile's key steps [k0, k0 + n) for one KV head.
struct Item {
  int kv, slot;
  int q0, r0, rows;     // first token, the tile's first row, rows of the sequence
  int see0;             // row R sees keys up to see0 + R / G
  int kl;
  int k0, n;            // first key step, steps; n < 0: the list is at its end
  int n_g[2];           // steps each group needs
  int s;
};

constexpr int kNext = 4;

constexpr int kMostStages = 4;

struct Aux {
  uint64_t k_full[kMostStages], v_full[kMostStages], v_empty[kMostStages];
  // a V tile that reaches behind the sequence's rows lands on v_tail, and
  // v_clear follows when the rows behind are cleared (v_full only counts it)
  uint64_t v_tail[kMostStages], v_clear[kMostStages];
  // a group's tiles take these in turn: a tile's turn comes again only when
  // every waiter has seen its last
  uint64_t s_full[2][kRing], p_ready[2][kRing], o_done[2][kRing];
  uint64_t solo_done[kRing];                      // P V of the tiles of one-group items
  uint64_t q_full, q_empty, drain[2];
  uint64_t next_full[kNext], next_empty[kNext];   // items handed to the other warps
  uint32_t tmem_base;
  volatile int32_t abort_flag;
  Item next[kNext];
};

template <int D>
struct Layout {
  static constexpr int kPanel = 128 * 128;
  static constexpr int kTile = 128 * D * 2;
  static constexpr int kSK = D == 64 ? 4 : 2, kSV = D == 64 ? 4 : 3;   // ring depths
  // score tiles in TMEM beside the two O tiles (512 columns in all)
  static constexpr int kScores = D == 64 ? 3 : 2;
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kSK * kTile;
  static constexpr int kAux = kV + kSV * kTile;
  static constexpr int kBytes = kAux + (int)sizeof(Aux);
  static constexpr uint32_t kTmemCols = 512;
  __host__ __device__ static constexpr uint32_t obase(int g) { return (uint32_t)(g * D); }
  __host__ __device__ static constexpr uint32_t sbase(int i) { return (uint32_t)(2 * D + i * kNk); }
};

struct Work {
  Header* hdr;
  const int4* entries;
  const int* slots;
  int4* line_cuts;      // of trees of one tile (see Line)
  bool by_tile;         // line_cuts by tile, else by the CTA that starts one
};

// -------------------------------------------------------------------- a line of trees
// Where every tree is one tile, nothing is gained from a list: a tile's keys are
// read by nobody else, so pieces need no order in time.  The tiles (sequence, KV
// head) stand on a line, each as long as it costs, and CTA c takes the c-th of C
// equal stretches of it, which it finds from the lengths by itself; a tile that
// cuts fall into is joined as in the plan's list.  That saves the plan's launch (64
// nodes over 100K rows 91 -> 80 us, nine short streams 33 -> 22).  The host sees to
// it that the line is shorter than 2^31.
// The first copy waits for all of this, and for its instructions too, which a new
// kernel fetches from afar: a warp does it alone, in few of them.
constexpr int kLineFixed = 3;   // what a tile costs beside its steps, in steps
constexpr int kLineLeast = 3;   // a stretch is at least as long

// The tile of a tree's rows: its steps, and its length on the line.
template <int D>
struct TreeTile {
  int q0, nodes, see0, kl, steps;
  bool bad;
  int eighths;                  // what a step costs
  __device__ __forceinline__ int price() const { return (steps * eighths + 7) >> 3; }
  __device__ __forceinline__ int length() const { return nodes > 0 ? price() + kLineFixed : 0; }
  // steps in front of the tile's place c
  __device__ __forceinline__ int steps_at(int c) const {
    return c >= length() ? steps : c <= kLineFixed ? 0 : min((c - kLineFixed) * 8 / eighths, steps);
  }
  __device__ __forceinline__ void set(const PagedBatch& b, int s, int max_q, int G) {
    q0 = nodes = see0 = kl = 0;       // behind the batch (all lanes' are shuffled)
    bad = false;
    if (s >= b.n_seq) return;
    const SeqSpan sp = seq_span(b, s);
    bad = sp.bad || sp.ql > max_q;
    q0 = sp.q0;
    nodes = min(sp.ql, max_q);
    see0 = sp.kl - sp.ql;
    kl = sp.kl;
    finish(G);
  }
  __device__ __forceinline__ void finish(int G) {
    steps = (max(see0 + nodes, 0) + kNk - 1) / kNk;        // the last node sees up to its own row
    eighths = D == 128 && nodes * G <= 128 ? kSoloEighths : 8;
  }
};

struct Line {
  uint32_t each, more;          // the first `more` stretches are each + 1 long, the others each
  uint32_t w0, len;             // this CTA's stretch
  int s;                        // the sequence that holds w0, and where it starts
  uint32_t at;
  __device__ __forceinline__ void cut(uint32_t total) {
    const uint32_t C = max(1u, min(total / kLineLeast, gridDim.x)), c = blockIdx.x;
    each = total / C;
    more = total - each * C;
    w0 = each * c + min(c, more);
    len = c < C ? each + (c < more) : 0;
  }
};

// The line, found by the whole CTA.
template <int D>
__device__ __forceinline__ Line find_line(const PagedBatch& b, int Hkv, int G, int max_q,
                                          int32_t* status) {
  __shared__ uint32_t sums[kThreads / 32], s_at;
  __shared__ int s_seq;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto length = [&](int s, bool report) -> uint32_t {
    TreeTile<D> t;
    t.set(b, s, max_q, G);
    if (report && t.bad) set_status(status, TS_ERR_INVALID_ARG);
    return (uint32_t)Hkv * t.length();
  };
  const uint32_t first = length(tid, blockIdx.x == 0);
  uint32_t mine = first;
  for (int s = tid + kThreads; s < b.n_seq; s += kThreads) mine += length(s, blockIdx.x == 0);
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) sums[warp] = mine;
  if (tid == 0) {
    s_seq = 0;
    s_at = 0;
  }
  __syncthreads();
  uint32_t total = 0;
  for (int w = 0; w < kThreads / 32; ++w) total += sums[w];
  Line r;
  r.cut(total);
  uint32_t before = 0;
  for (int base = 0; base < b.n_seq && before <= r.w0; base += kThreads) {
    const uint32_t x = base == 0 ? first : length(base + tid, false);
    uint32_t inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    __syncthreads();
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    uint32_t at = before + inc - x;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) at += sums[w];
      before += sums[w];
    }
    if (x > 0 && r.w0 >= at && r.w0 - at < x) {
      s_seq = base + tid;
      s_at = at;
    }
  }
  __syncthreads();
  r.s = s_seq;
  r.at = s_at;
  return r;
}

// The stretch's items in turn: part of a tile each.  A warp walks; the tiles of 32
// sequences are its lanes'.  Up to 32 sequences' line is its own work, without a
// barrier.
template <int D>
struct LineWalk {
  TreeTile<D> mine, t;          // of sequence base + lane; the tile ahead
  int base, s, kv, c0;          // c0: where the stretch enters it
  int left;                     // what is left of the stretch
  int each, more;               // of the stretches behind this one
  int rest;                     // of the item's tile behind the stretch; -1: none that it starts
  __device__ __forceinline__ void take(const PagedBatch& b, int max_q, int G, int lane) {
    if (s - base >= 32) {
      base = s;
      mine.set(b, base + lane, max_q, G);
    }
    t.q0 = __shfl_sync(0xffffffffu, mine.q0, s - base);
    t.nodes = __shfl_sync(0xffffffffu, mine.nodes, s - base);
    t.see0 = __shfl_sync(0xffffffffu, mine.see0, s - base);
    t.kl = __shfl_sync(0xffffffffu, mine.kl, s - base);
    t.finish(G);
  }
  __device__ __forceinline__ void begin(const PagedBatch& b, Line l, int Hkv, int G, int max_q,
                                        int lane, int32_t* status) {
    base = b.n_seq > 32 ? l.s : 0;
    mine.set(b, base + lane, max_q, G);
    if (b.n_seq <= 32) {
      if (blockIdx.x == 0 && mine.bad) set_status(status, TS_ERR_INVALID_ARG);
      const uint32_t x = mine.length();
      uint32_t inc = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      l.cut(__shfl_sync(0xffffffffu, inc, 31) * (uint32_t)Hkv);
      // the last that starts at or before w0 and has tokens
      const unsigned in = __ballot_sync(0xffffffffu, x > 0 && (inc - x) * Hkv <= l.w0);
      l.s = in ? 31 - __clz(in) : 0;
      l.at = __shfl_sync(0xffffffffu, inc - x, l.s) * (uint32_t)Hkv;
    }
    left = l.len;
    each = (int)l.each;
    more = max((int)l.more - (int)blockIdx.x - 1, 0);
    s = l.s;
    kv = c0 = 0;
    if (left == 0) return;
    take(b, max_q, G, lane);
    // w0 lies in this sequence (bounded all the same, here and below: lengths that
    // change under the call must neither leave the pool nor keep the warp)
    const uint32_t length = max(t.length(), 1), in = l.w0 - l.at;
    kv = min(in / length, (uint32_t)Hkv - 1u);
    c0 = min(in - kv * length, length - 1u);
  }
  // n < 0: the stretch is at its end
  __device__ __forceinline__ Item next(const PagedBatch& b, int Hkv, int G, int max_q, int lane) {
    Item w;
    w.n = -1;
    bool some = false;
    while (!some && left > 0) {
      const int length = max(t.length(), 1), c1 = min(c0 + left, length);
      const int k0 = t.steps_at(c0), k1 = t.steps_at(c1);
      const bool starts = t.steps > 0 ? k0 == 0 : c0 == 0, ends = k1 == t.steps;
      some = k0 < k1 || (t.steps == 0 && starts);              // else between two tiles' steps
      left -= c1 - c0;
      c0 = 0;
      rest = !starts ? -1 : ends ? 0 : length - c1;
      w.kv = kv;
      w.s = s;
      w.q0 = t.q0;
      w.r0 = 0;
      w.rows = t.nodes * G;
      w.see0 = t.see0;
      w.kl = t.kl;
      w.k0 = k0;
      w.n = some ? k1 - k0 : -1;
      w.slot = starts && ends ? -1 : 2 * (int)blockIdx.x + (starts ? 1 : 0);
      // group 0 ends with the node of its last row
      const int vis = t.see0 + min(127 / G, t.nodes - 1) + 1;
      w.n_g[0] = max(min(vis <= 0 ? 0 : (vis + kNk - 1) / kNk, k1) - k0, 0);
      w.n_g[1] = w.rows > 128 ? k1 - k0 : 0;
      if (++kv == Hkv) {
        kv = 0;
        // (a sequence without tokens has no length; while the stretch goes on there
        // is one with)
        while (left > 0) {
          if (++s >= b.n_seq) left = 0;
          take(b, max_q, G, lane);
          if (t.nodes > 0) break;
        }
      }
    }
    return w;
  }
  // Where the item's pieces lie, if the tile starts with it: with the CTAs up to the
  // one where it ends (0: it is whole).
  __device__ __forceinline__ void note(const Work& work, const Item& w, int Hkv) const {
    if (rest < 0) return;
    int parts = 0;
    if (rest > 0)
      parts = 1 + (rest <= (int64_t)more * (each + 1)
                       ? (rest + each) / (each + 1)
                       : more + (rest - more * (each + 1) + each - 1) / each);
    if (work.by_tile || parts > 0)
      work.line_cuts[work.by_tile ? w.s * Hkv + w.kv : (int)blockIdx.x] =
          make_int4(w.q0, w.rows | w.kv << 16, (int)blockIdx.x, parts);
  }
};

__device__ __forceinline__ Item load_item(const PagedBatch& b, const Work& w, int i, int Hkv, int G,
                                          int max_q) {
  Item it;
  const int e = i / Hkv;
  it.kv = i - e * Hkv;
  const int4 x = __ldcg(&w.entries[e]);
  it.slot = __ldcg(&w.slots[e]);
  it.s = x.x;
  const SeqSpan sp = seq_span(b, x.x);
  it.q0 = sp.q0;
  it.r0 = x.y * kM;
  it.rows = min(sp.ql, max_q) * G;
  it.see0 = sp.kl - sp.ql;
  it.kl = sp.kl;
  it.k0 = x.z;
  it.n = x.w - x.z;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int a = it.r0 + g * 128;
    int steps = 0;
    if (a < it.rows) {
      const int vis = it.see0 + (min(a + 128, it.rows) - 1) / G + 1;
      steps = vis <= 0 ? 0 : (vis + kNk - 1) / kNk;
    }
    it.n_g[g] = max(0, min(steps, x.w) - x.z);
  }
  return it;
}

// A group's turn as the place of its barrier in [2][kRing] and the parity of its round.
__device__ __forceinline__ uint32_t use_of(uint32_t g, uint32_t turn) {
  static_assert(kRing == 4, "three bits for the place");
  return g * kRing + turn % kRing + (turn / kRing % 2) * 8;
}

__device__ __forceinline__ void give_up(Aux* aux, int32_t* status) {
  aux->abort_flag = 1;
  set_status(status, TS_ERR_TIMEOUT);
}

// The next item as the copy warp handed it on; false: a wait ran out.
__device__ __forceinline__ bool take_item(Aux* aux, uint32_t& count, Item& w, int lane,
                                          long long limit) {
  const uint32_t at = count % kNext;
  const bool got = ptx::mbar_wait(&aux->next_full[at], (count / kNext) & 1u, limit);
  if (!__all_sync(0xffffffffu, got)) return false;
  w = aux->next[at];
  __syncwarp();
  if (lane == 0) ptx::mbar_arrive(&aux->next_empty[at]);
  ++count;
  return true;
}

__device__ __forceinline__ float fmax32(const uint32_t* r) {
  float a = ptx::max3(__uint_as_float(r[0]), __uint_as_float(r[1]), __uint_as_float(r[2]));
  float c = ptx::max3(__uint_as_float(r[3]), __uint_as_float(r[4]), __uint_as_float(r[5]));
#pragma unroll
  for (int x = 6; x < 30; x += 4) {
    a = ptx::max3(a, __uint_as_float(r[x]), __uint_as_float(r[x + 1]));
    c = ptx::max3(c, __uint_as_float(r[x + 2]), __uint_as_float(r[x + 3]));
  }
  return ptx::max3(a, c, fmaxf(__uint_as_float(r[30]), __uint_as_float(r[31])));
}

// Keys 32 c .. 32 c + 31 of a tile as bits, for a row that sees all keys before
// the tile's key `base` (which may lie in front of the tile or behind it) and
// behind it the tree's nodes `nodes`.
__device__ __forceinline__ uint32_t tree_word(unsigned long long nodes, int base, int c) {
  const int first = 32 * c - base;             // the word's first key as a node
  if (first >= 64) return 0u;
  if (first >= 0) return (uint32_t)(nodes >> first);
  if (first <= -32) return 0xFFFFFFFFu;
  return (uint32_t)(nodes << -first) | ((1u << -first) - 1u);
}

// What the new tokens are: a chunk, the nodes of trees whose tiles the plan lists, or
// of trees of one tile on a line.
enum Kind { kChunk, kTreeList, kTreeLine };

template <typename T, int D, Kind kKind>
__global__ void __launch_bounds__(kThreads, 1)
paged_tc_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                const PagedBatch b, const T* __restrict__ q, int Hq, int Hkv, int max_q,
                const int32_t* __restrict__ parents,
                const Work work, T* __restrict__ o, float* __restrict__ lse,
                float* __restrict__ part_o, float2* __restrict__ part_ml, long long wait_limit,
                int32_t* status) {
  using Ly = Layout<D>;
  constexpr bool kTree = kKind != kChunk, kOnLine = kKind == kTreeLine;
  constexpr int kSK = Ly::kSK, kSV = Ly::kSV, kScores = Ly::kScores;
  extern __shared__ __align__(1024) uint8_t sm[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = Hq / Hkv;
  if ((ptx::smem_u32(sm) & 1023u) != 0) {      // the swizzle needs 1024-byte aligned tiles
    if (tid == 0) set_status(status, TS_ERR_CUDA);
    return;
  }
  uint8_t* sq = sm + Ly::kQ;
  uint8_t* sk = sm + Ly::kK;
  uint8_t* sv = sm + Ly::kV;
  Aux* aux = reinterpret_cast<Aux*>(sm + Ly::kAux);
  if (tid == 0) {
    for (int i = 0; i < kSK; ++i) {
      ptx::mbar_init(&aux->k_full[i], 1);
    }
    for (int i = 0; i < kSV; ++i) {
      ptx::mbar_init(&aux->v_full[i], 1);
      ptx::mbar_init(&aux->v_empty[i], 1);
      ptx::mbar_init(&aux->v_tail[i], 1);
      ptx::mbar_init(&aux->v_clear[i], 4);
    }
    ptx::mbar_init(&aux->q_full, 4);
    ptx::mbar_init(&aux->q_empty, 1);
    for (int g = 0; g < 2; ++g) {
      for (int i = 0; i < kRing; ++i) {
        ptx::mbar_init(&aux->s_full[g][i], 1);
        ptx::mbar_init(&aux->p_ready[g][i], 4);
        ptx::mbar_init(&aux->o_done[g][i], 1);
      }
    }
    for (int i = 0; i < kRing; ++i) ptx::mbar_init(&aux->solo_done[i], 1);
    ptx::mbar_init(&aux->drain[0], 1);
    ptx::mbar_init(&aux->drain[1], 1);
    for (int i = 0; i < kNext; ++i) {
      ptx::mbar_init(&aux->next_full[i], 1);
      // warps 1, 2, 4..7, 8..15, and 3 where it has work
      ptx::mbar_init(&aux->next_empty[i], (kScores == 2 ? 2 : 3) + 4 + 8);
    }
    aux->abort_flag = 0;
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(&aux->tmem_base, Ly::kTmemCols);
    ptx::tmem_relinquish();
  }
  if (kOnLine && tid == 0) {
    ptx::prefetch_map(&tmap_k);
    ptx::prefetch_map(&tmap_v);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = aux->tmem_base;
  griddep_wait();
  griddep_launch_dependents();
  Line line{};
  int n_items = 0;
  if constexpr (kOnLine) {
    if (!work.by_tile && tid == 0) work.line_cuts[blockIdx.x] = make_int4(0, 0, 0, 0);
    if (b.n_seq > 32) line = find_line<D>(b, Hkv, G, max_q, status);
  } else {
    n_items = __ldcg(&work.hdr->n_entries) * Hkv;
  }
  const int ps = 1 << b.page_shift;

  if (warp < 8) {
    ptx::regs_dec<kRegsLow>();
    if (warp == 0 || warp == 2) {
      // ------------------------------------------------------------ copies
      // warp 0 copies K, warp 2 V; lane: page `box` of the tile, both panels.
      // (Small pages make many boxes, and a box costs its warp's lanes a turn
      // each: one warp for both took 7 % longer at pages of 16 rows.)
      const bool is_k = warp == 0;
      const uint32_t depth = is_k ? kSK : kSV;
      const CUtensorMap* map = is_k ? &tmap_k : &tmap_v;
      uint64_t* full = is_k ? aux->k_full : aux->v_full;
      const uint32_t ring = ptx::smem_u32(is_k ? sk : sv);
      const int boxes = kNk >> b.page_shift;
      const uint64_t pol = ptx::l2_evict_first_policy();
      uint32_t it = 0, done = 0;          // key tiles so far; copies issued
      uint32_t base_g[2] = {0, 0};        // tiles of each group before this item
      // A stage is free when its tile's last product is complete, which that
      // product's own barrier says: its group and turn, 4 bits a stage.  (A barrier
      // of the stage's own would be one more commit between products.)  The barrier
      // cannot pass its next round unseen, since that needs a later tile of this
      // ring; and its last round is over, since products end in order.
      uint32_t uses = 0;
      uint32_t tail_on = 0, tail_par = 0; // a stage's v_tail was used; parity of its last use
      bool ok = true;
      auto ids = [&](const Item& w, int step) -> int64_t {
        // the page of this lane's box, -1: behind the sequence
        const int key = (w.k0 + step) * kNk + (lane << b.page_shift);
        if (step >= w.n || lane >= boxes || key >= w.kl) return -1;
        int64_t ph = b.table[(int64_t)w.s * b.max_pages + (key >> b.page_shift)];
        if (ph < 0 || ph >= b.n_pages) {
          set_status(status, TS_ERR_INVALID_ARG);
          ph = 0;                          // any page: the sequence's outputs are unspecified
        }
        return ph;
      };
      int taken = blockIdx.x;             // warp 0: the next item; the first is the CTA's own
      LineWalk<D> walk;
      if constexpr (kOnLine) {
        if (is_k) walk.begin(b, line, Hkv, G, max_q, lane, status);
      }
      for (uint32_t count = 0; ok;) {
        Item w;
        if (is_k) {
          const int i = __shfl_sync(0xffffffffu, taken, 0);
          const uint32_t at = count % kNext;
          if (count >= kNext)
            ok = ptx::mbar_wait(&aux->next_empty[at], (count / kNext - 1) & 1u, wait_limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          w.n = -1;
          if constexpr (kOnLine) w = walk.next(b, Hkv, G, max_q, lane);
          else if (i < n_items) w = load_item(b, work, i, Hkv, G, max_q);
          if (lane == 0) {
            aux->next[at] = w;
            ptx::mbar_arrive(&aux->next_full[at]);
          }
          ++count;
        } else {
          ok = take_item(aux, count, w, lane, wait_limit);
        }
        if (!ok || w.n < 0) break;
        int64_t next = ids(w, 0);
        if (kOnLine && is_k && lane == 0 && w.n == 0) walk.note(work, w, Hkv);
        if (!kOnLine && w.n == 0 && lane == 0 && is_k) taken = gridDim.x + atomicAdd(&work.hdr->taken, 1);
        for (int k = 0; ok && k < w.n; ++k, ++it) {
          // the next item is taken as late as its latency allows
          if (!kOnLine && is_k && k == max(0, w.n - 2) && lane == 0)
            taken = gridDim.x + atomicAdd(&work.hdr->taken, 1);
          const int64_t ph = next;
          next = ids(w, k + 1);
          const int row = (int)(((ph < 0 ? 0 : ph) * Hkv + w.kv) << b.page_shift);
          const uint32_t bytes = (uint32_t)__popc(__ballot_sync(0xffffffffu, ph >= 0)) *
                                 (uint32_t)(ps * D * 2);
          const uint32_t st = it % depth;
          if (it >= depth) {
            if (kScores == 2 && !is_k) {
              ok = ptx::mbar_wait(&aux->v_empty[st], (it / depth - 1) & 1u, wait_limit);
            } else {
              const uint32_t x = uses >> (4 * st);
              uint64_t* last = is_k ? &aux->s_full[0][0] : &aux->o_done[0][0];
              ok = ptx::mbar_wait(last + (x & 7u), (x >> 3) & 1u, wait_limit);
            }
          }
          const uint32_t g = k < w.n_g[1] ? 1u : 0u, turn = (g ? base_g[1] : base_g[0]) + k;
          uses = (uses & ~(15u << (4 * st))) | use_of(g, turn) << (4 * st);
          ok = __all_sync(0xffffffffu, ok && aux->abort_flag == 0);
          if (!ok) break;
          const bool tail = !is_k && (w.k0 + k + 1) * kNk > w.kl;
          uint64_t* land = tail ? &aux->v_tail[st] : &full[st];
          if (tail) {
            tail_par = (tail_on >> st) & 1u ? tail_par ^ (1u << st) : tail_par;
            tail_on |= 1u << st;
          }
          if (lane == 0) {
            ptx::mbar_arrive_expect_tx(land, bytes);
            if (tail) ptx::mbar_arrive(&full[st]);
          }
          __syncwarp();
          if (ph >= 0)
            for (int p = 0; p < D / 64; ++p)
              ptx::tma_load_2d_at(ring + st * Ly::kTile + p * Ly::kPanel + lane * ps * 128, map,
                                  land, p * 64, row, pol);
          if (kOnLine && is_k && lane == 0 && k == 0) walk.note(work, w, Hkv);
          ++done;
        }
        base_g[0] += w.n_g[0];
        base_g[1] += w.n_g[1];
      }
      if (!ok) give_up(aux, status);
      // every copy issued must land before the CTA exits
      if (lane == 0) {
        for (uint32_t t = done > depth ? done - depth : 0; t < done; ++t)
          ptx::mbar_wait(&full[t % depth], (t / depth) & 1u, kDrainCycles);
        for (int t = 0; t < kSV; ++t)
          if ((tail_on >> t) & 1u)
            ptx::mbar_wait(&aux->v_tail[t], (tail_par >> t) & 1u, kDrainCycles);
      }
    } else if (warp == 1 || (kScores > 2 && warp == 3)) {
      // ------------------------------------------------------------ products
      // The whole warp walks the loop, and one lane issues under a predicate.
      // Everything an instruction's operands come from is the same in all lanes,
      // and is made so for the compiler too (broadcasts of lane 0): it then keeps
      // them in uniform registers.  The queue in front of the tensor core is
      // short, so what this warp spends between products leaves it idle: issued
      // by one lane of a divergent warp a step took 3.6 K cycles, in a branch of
      // the elected lane 2.9 K, under a predicate 2.6 K (2182 and 1974 us for 2048
      // tokens over 100K rows, 8B shape, with the softmax as it was then).
      constexpr uint32_t idesc_qk = Pair<T>::kFp16 ? ptx::idesc_f16_f32(128, kNk, false)
                                                   : ptx::idesc_bf16_f32(128, kNk, false);
      constexpr uint32_t idesc_pv = Pair<T>::kFp16 ? ptx::idesc_f16_f32(128, D, true)
                                                   : ptx::idesc_bf16_f32(128, D, true);
      auto same = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
      const uint32_t base = same(ptx::smem_u32(sm));
      const uint32_t tm = same(tmem);
      const uint32_t lead = ptx::elect_one() ? 1u : 0u;
      const uint32_t bars = base + Ly::kAux;
      const uint64_t qd0 = ptx::sdesc_sw128(base + Ly::kQ, 16, 1024);
      const uint64_t kd0 = ptx::sdesc_sw128(base + Ly::kK, 16, 1024);
      const uint64_t vd0 = ptx::sdesc_sw128(base + Ly::kV, Ly::kPanel, 1024);
      constexpr uint32_t kTile16 = Ly::kTile >> 4;
      uint32_t it = 0, items = 0, clear_par = 0, count = 0;
      uint32_t base0 = 0, base1 = 0;      // tiles of each group before this item
      uint32_t outs_g[2] = {0, 0};        // items ended
      uint32_t ops = 0, at = 0, uses = 0; // ops so far; S tile of the next; who used each last
      uint32_t solo = 0;                  // tiles of one-group items so far
      bool ok = true;
      auto commit = [&](uint32_t off) { ptx::mma_commit_if(lead, bars + off); };
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        const bool got = __all_sync(0xffffffffu, ptx::mbar_wait(bar, parity & 1u, wait_limit));
        ptx::tc_fence_after();
        return got;
      };
      while (ok) {
        Item w;
        ok = take_item(aux, count, w, lane, wait_limit);
        if (!ok) break;
        const int n = (int)same(w.n), n0 = (int)same(w.n_g[0]), n1 = (int)same(w.n_g[1]);
        const bool tail = same((w.k0 + w.n) * kNk > w.kl) != 0;   // of the item's last tile
        if (n < 0) break;
        if (n == 0) continue;
        if (warp == 1) ok = wait(&aux->q_full, items);
        if constexpr (kScores == 2) {
          // S tile g is group g's: its next scores go behind its P V, in the order
          // of one warp's products.  (S tiles in turn took 5 % longer on 2048
          // tokens over 100K rows, in turn and two warps, as below, 11 %.)
          auto scores_to = [&](int g, uint32_t t, uint32_t to) {
            const uint64_t a0 = qd0 + (uint64_t)(g * kTile16);
            const uint64_t b0 = kd0 + (uint64_t)((t % kSK) * kTile16);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = (ks >> 2) * (Ly::kPanel >> 4) + (ks & 3) * 2;
              ptx::mma_ss_if(lead, to, a0 + off, b0 + off, idesc_qk, ks > 0 ? 1u : 0u);
            }
            commit(offsetof(Aux, s_full) + (g * kRing + ((g ? base1 : base0) + (t - it)) % kRing) * 8);
          };
          auto scores = [&](int g, uint32_t t) { scores_to(g, t, tm + Ly::sbase(g)); };
          ok = ok && wait(&aux->k_full[it % kSK], it / kSK);
          if (!ok) break;
          if (kTree && n1 == 0) {
            // One group alone takes both S tiles in turn: its next scores are formed
            // while it works on these.  (P V of the tile before is then not implied by
            // a tile's scores: solo_done tells it.)
            scores(0, it);
            if (n > 1) {
              ok = wait(&aux->k_full[(it + 1) % kSK], (it + 1) / kSK);
              if (!ok) break;
              scores_to(0, it + 1, tm + Ly::sbase(1));
            }
            if (n <= 2) commit(offsetof(Aux, q_empty));
            for (int k = 0; k < n; ++k, ++solo) {
              const uint32_t t = it + k, stV = t % kSV, turn = base0 + k;
              const uint32_t s0 = tm + 2 * D + (k & 1) * kNk;
              ok = wait(&aux->v_full[stV], t / kSV);
              if (ok && tail && k + 1 == n) {
                ok = wait(&aux->v_clear[stV], clear_par >> stV);
                clear_par ^= 1u << stV;
              }
              ok = ok && wait(&aux->p_ready[0][turn % kRing], turn / kRing);
              if (!ok) break;
              const uint64_t b0 = vd0 + (uint64_t)(stV * kTile16);
              const uint32_t acc = k > 0 ? 1u : 0u;
#pragma unroll
              for (int ks = 0; ks < kNk / 16; ++ks)
                ptx::mma_ts_if(lead, tm + Ly::obase(0), s0 + 8 * ks, b0 + (uint64_t)(ks * 128),
                               idesc_pv, ks > 0 ? 1u : acc);
              commit(offsetof(Aux, solo_done) + (solo % kRing) * 8);
              commit(offsetof(Aux, v_empty) + stV * 8);
              if (k + 1 == n) commit(offsetof(Aux, o_done) + (outs_g[0]++ % kRing) * 8);
              if (k + 2 < n) {
                ok = wait(&aux->k_full[(t + 2) % kSK], (t + 2) / kSK);
                if (!ok) break;
                scores_to(0, t + 2, s0);
                if (k + 3 == n) commit(offsetof(Aux, q_empty));
              }
            }
            if (!ok) break;
            it += n;
            base0 += n0;
            ++items;
            continue;
          }
          if (n0 > 0) scores(0, it);
          if (n1 > 0) scores(1, it);
          if (n == 1) commit(offsetof(Aux, q_empty));
          for (int k = 0; k < n; ++k) {
            const uint32_t t = it + k, stV = t % kSV;
            ok = wait(&aux->v_full[stV], t / kSV);
            if (ok && tail && k + 1 == n) {
              ok = wait(&aux->v_clear[stV], clear_par >> stV);
              clear_par ^= 1u << stV;
            }
            if (!ok) break;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int ng = g == 0 ? n0 : n1;
              if (ok && k < ng) {
                const uint32_t turn = (g ? base1 : base0) + k;
                ok = wait(&aux->p_ready[g][turn % kRing], turn / kRing);
                if (ok) {
                  const uint64_t b0 = vd0 + (uint64_t)(stV * kTile16);
#pragma unroll
                  for (int ks = 0; ks < kNk / 16; ++ks)
                    ptx::mma_ts_if(lead, tm + Ly::obase(g), tm + Ly::sbase(g) + 8 * ks,
                                   b0 + (uint64_t)(ks * 128), idesc_pv, (ks > 0 || k > 0) ? 1u : 0u);
                  if (k + 1 == ng) commit(offsetof(Aux, o_done) + (g * kRing + outs_g[g]++ % kRing) * 8);
                  if (k + 1 < ng) {
                    ok = wait(&aux->k_full[(t + 1) % kSK], (t + 1) / kSK);
                    if (ok) scores(g, t + 1);
                  }
                }
              }
            }
            if (!ok) break;
            commit(offsetof(Aux, v_empty) + stV * 8);
            if (k + 2 == n) commit(offsetof(Aux, q_empty));
          }
        } else {
          // The item's products in pairs, by tile and group: op i writes its scores
          // to S tile i % kScores and, once they are P, multiplies them by V.  The
          // scores of op i + kScores go behind the P V of op i, so every group has
          // its next scores while it works on these.
          // Warp 1 forms the scores, warp 3 the products with V: what a warp does
          // between two products is longer than a product at d = 64 (one warp for
          // both: 195 us for 179 on 2048 tokens over 32K rows, 12/2 heads).  Op i of
          // the item: while both groups have tiles, theirs in turn; then the rest of
          // one's.  The ops of all items take the S tiles in turn, and scores go
          // where the P V of three ops before is complete.
          const int both = 2 * min(n0, n1), total = n0 + n1, rest = n1 > n0 ? 1 : 0;
          if (warp == 1) {
            for (int i = 0; ok && i < total; ++i) {
              const bool two = i < both;
              const uint32_t g = two ? i & 1 : rest, k = two ? i >> 1 : i - (both >> 1), t = it + k;
              const uint32_t turn = (g ? base1 : base0) + k;
              if (!two || g == 0) ok = wait(&aux->k_full[t % kSK], t / kSK);
              if (ops >= kScores) {
                const uint32_t x = uses >> (4 * at);
                ok = ok && wait(&aux->o_done[0][0] + (x & 7u), (x >> 3) & 1u);
              }
              if (!ok) break;
              uses = (uses & ~(15u << (4 * at))) | use_of(g, turn) << (4 * at);
              const uint64_t a0 = qd0 + (uint64_t)(g * kTile16);
              const uint64_t b0 = kd0 + (uint64_t)((t % kSK) * kTile16);
              const uint32_t d0 = tm + 2 * D + at * kNk;
#pragma unroll
              for (int ks = 0; ks < D / 16; ++ks) {
                const uint32_t off = (ks >> 2) * (Ly::kPanel >> 4) + (ks & 3) * 2;
                ptx::mma_ss_if(lead, d0, a0 + off, b0 + off, idesc_qk, ks > 0 ? 1u : 0u);
              }
              commit(offsetof(Aux, s_full) + (g * kRing + turn % kRing) * 8);
              if (i + 1 == total) commit(offsetof(Aux, q_empty));
              ++ops;
              at = at + 1 == kScores ? 0 : at + 1;
            }
          } else {
            for (int i = 0; ok && i < total; ++i) {
              const bool two = i < both;
              const uint32_t g = two ? i & 1 : rest, k = two ? i >> 1 : i - (both >> 1), t = it + k;
              const uint32_t turn = (g ? base1 : base0) + k, bar = g * kRing + turn % kRing;
              const uint32_t stV = t % kSV;
              if (!two || g == 0) {
                ok = wait(&aux->v_full[stV], t / kSV);
                if (ok && tail && (int)k + 1 == n) {
                  ok = wait(&aux->v_clear[stV], clear_par >> stV);
                  clear_par ^= 1u << stV;
                }
              }
              ok = ok && wait(&aux->p_ready[0][0] + bar, turn / kRing);
              if (!ok) break;
              const uint64_t b0 = vd0 + (uint64_t)(stV * kTile16);
              const uint32_t s0 = tm + 2 * D + at * kNk, d0 = tm + g * D;
              const uint32_t acc = k > 0 ? 1u : 0u;
#pragma unroll
              for (int ks = 0; ks < kNk / 16; ++ks)
                ptx::mma_ts_if(lead, d0, s0 + 8 * ks, b0 + (uint64_t)(ks * 128), idesc_pv,
                               ks > 0 ? 1u : acc);
              commit(offsetof(Aux, o_done) + bar * 8);
              at = at + 1 == kScores ? 0 : at + 1;
            }
          }
        }
        it += n;
        base0 += n0;
        base1 += n1;
        ++items;
      }
      if (!ok) give_up(aux, status);
      // this warp's products end before TMEM is freed
      commit(offsetof(Aux, drain) + (warp >> 1) * 8);
      ptx::mbar_wait(&aux->drain[warp >> 1], 0, kDrainCycles);
    } else if (warp >= 4) {
      // ------------------------------------------------------------ query rows, V tails
      const int t = tid - 128;
      constexpr int kCh = D / 8;
      uint32_t it = 0, items = 0, tail_par = 0, count = 0;
      bool ok = true;
      while (ok) {
        Item w;
        ok = take_item(aux, count, w, lane, wait_limit);
        if (!ok || w.n < 0) break;
        if (w.n == 0) continue;
        if (items > 0) ok = ptx::mbar_wait(&aux->q_empty, (items - 1) & 1u, wait_limit);
        ok = __all_sync(0xffffffffu, ok && !aux->abort_flag);
        if (!ok) break;
        // thread: 16-byte chunk c of every kHop-th row; (token, head) of its row
        // advance without a division a row
        constexpr int kHop = 128 / kCh;
        const int c = t % kCh;
        int R = w.r0 + t / kCh, tok = R / G, head = R - tok * G;
        const int dt = kHop / G, dh = kHop - dt * G;
        const T* src = q + ((int64_t)w.q0 * Hq + w.kv * G) * D + c * 8;
        const uint32_t dst = ptx::smem_u32(sq) + (c >> 3) * Ly::kPanel;
#pragma unroll 8
        for (int r = t / kCh; r < kM; r += kHop) {
          const bool live = R < w.rows;
          const T* from = live ? src + ((int64_t)tok * Hq + head) * D : q;
          const int n = live ? 16 : 0;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                           dst + (r >> 7) * Ly::kTile + (r & 127) * 128 + (((c & 7) ^ (r & 7)) << 4)),
                       "l"(from), "r"(n));
          R += kHop;
          tok += dt;
          head += dh;
          if (head >= G) {
            head -= G;
            ++tok;
          }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->q_full);
        // the item's last tile, where it reaches behind the sequence's rows
        const int last = w.k0 + w.n - 1;
        if ((last + 1) * kNk > w.kl) {
          const uint32_t st = (it + w.n - 1) % kSV;
          ok = ptx::mbar_wait(&aux->v_tail[st], (tail_par >> st) & 1u, wait_limit);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tail_par ^= 1u << st;
          const int keep = w.kl - last * kNk;      // rows [keep, 128) are cleared
          for (int e = t; e < (kNk - keep) * kCh; e += 128) {
            const int r = keep + e / kCh, c = e % kCh;
            *reinterpret_cast<uint4*>(sv + st * Ly::kTile + (c >> 3) * Ly::kPanel +
                                      r * 128 + ((c & 7) << 4)) = make_uint4(0, 0, 0, 0);
          }
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&aux->v_clear[st]);
        }
        it += w.n;
        ++items;
      }
      if (!ok) give_up(aux, status);
    }
  } else {
    ptx::regs_inc<kRegsSoftmax>();
    // ------------------------------------------------------------ softmax
    const int g = (warp - 8) >> 2;
    const int tr = (warp & 3) * 32 + lane;       // row of the group
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t o_addr = tmem + lane_off + Ly::obase(g);
    const float sl2 = kLog2e / sqrtf((float)D);
    const uint64_t sl2x2 = ptx::f2(sl2, sl2);
    uint32_t tiles = 0, outs = 0, count = 0, ops = 0, solos = 0;
    bool ok = true;
    while (ok) {
      Item w;
      ok = take_item(aux, count, w, lane, wait_limit);
      if (!ok || w.n < 0) break;
      const int wr0 = w.r0 + g * 128 + (warp & 3) * 32;     // the warp's first row
      const bool warp_rows = wr0 < w.rows;
      const int R = w.r0 + g * 128 + tr;
      const bool valid = R < w.rows;
      const int lim = w.see0 + (valid ? R : w.rows - 1) / G;   // last key this row sees
      const int lim0 = w.see0 + min(wr0, w.rows - 1) / G;      // least of the warp
      unsigned long long nodes = 0;                            // a tree's: those this row sees
      if constexpr (kTree) {
        TreeBits tree;
        tree.build(parents + w.q0, (w.rows + G - 1) / G, lane, status);
        nodes = tree.of((valid ? R : w.rows - 1) / G);
      }
      const int n_mine = g == 0 ? w.n_g[0] : w.n_g[1];
      const bool solo = kTree && kScores == 2 && w.n_g[1] == 0;   // one group, both S tiles
      float m_used = -INFINITY, l = 0.f;
      for (int k = 0; k < n_mine; ++k, ++tiles, solos += solo) {
        bool got = !aux->abort_flag && ptx::mbar_wait(&aux->s_full[g][tiles % kRing], (tiles / kRing) & 1u, wait_limit);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        if (!warp_rows) {        // padding rows: their P feeds O rows that are never written
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&aux->p_ready[g][tiles % kRing]);
          continue;
        }
        // this tile's place among the item's products
        const uint32_t op = kScores == 2 ? (solo ? k & 1 : g)
                                         : ops + min(k, w.n_g[0]) + min(k, w.n_g[1]) +
                                               (g == 1 && k < w.n_g[0] ? 1 : 0);
        const uint32_t s_addr = tmem + lane_off + Ly::sbase(op % kScores);
        const int key0 = (w.k0 + k) * kNk;
        // warp-uniform
        const bool edge = kTree ? key0 + kNk > w.see0 : key0 + kNk > lim0 + 1;
        uint32_t r[kNk];
        auto load_s = [&]() {
          ptx::tc_fence_after();
#pragma unroll
          for (int c = 0; c < kNk / 32; ++c)
            ptx::tmem_ld32(s_addr + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * c));
          ptx::tmem_ld_wait();
          if (edge) {
            if constexpr (kTree) {
#pragma unroll
              for (int c = 0; c < kNk / 32; ++c) {
                const uint32_t see = tree_word(nodes, w.see0 - key0, c);
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if (!(see >> x & 1u)) r[32 * c + x] = kNegInf;
              }
            } else {
              const int vis = lim + 1 - key0;
#pragma unroll
              for (int x = 0; x < kNk; ++x)
                if (x >= vis) r[x] = kNegInf;
            }
          }
        };
        // P against mref, packed in place: the pair of keys 32c + 2i, 32c + 2i + 1
        // in r[32c + i]; returns the row sum of P before rounding
        auto exp_pack = [&](float mref, uint32_t (&lo)[32], uint32_t (&hi)[32]) -> float {
          const uint64_t negm = ptx::f2(-mref, -mref);
          auto chunk_exp = [&](int c, float (&pe)[32]) {
            const uint32_t* x = r + 32 * c;
#pragma unroll
            for (int y = 0; y < 16; ++y)
              ptx::f2_split(ptx::fma2(ptx::f2(__uint_as_float(x[2 * y]), __uint_as_float(x[2 * y + 1])),
                                      sl2x2, negm),
                            pe[2 * y], pe[2 * y + 1]);
#pragma unroll
            for (int y = 0; y < 32; ++y) pe[y] = ptx::ex2(pe[y]);
          };
          uint64_t acc[2 * (kNk / 32)];
          float pa[32], pb[32];
          chunk_exp(0, pa);
#pragma unroll
          for (int c = 0; c < kNk / 32; ++c) {
            float (&cur)[32] = (c & 1) ? pb : pa;
            float (&nxt)[32] = (c & 1) ? pa : pb;
            if (c + 1 < kNk / 32) chunk_exp(c + 1, nxt);
            uint32_t* x = (c < 2 ? lo : hi) + 16 * (c & 1);
            uint64_t s0 = ptx::f2(cur[0], cur[1]), s1 = ptx::f2(cur[2], cur[3]);
#pragma unroll
            for (int y = 2; y < 16; y += 2) {
              s0 = ptx::add2(s0, ptx::f2(cur[2 * y], cur[2 * y + 1]));
              s1 = ptx::add2(s1, ptx::f2(cur[2 * y + 2], cur[2 * y + 3]));
            }
#pragma unroll
            for (int y = 0; y < 16; ++y) x[y] = Pair<T>::pack(cur[2 * y], cur[2 * y + 1]);
            acc[2 * c] = s0;
            acc[2 * c + 1] = s1;
          }
          const uint64_t s = ptx::add2(ptx::add2(ptx::add2(acc[0], acc[1]), ptx::add2(acc[2], acc[3])),
                                       ptx::add2(ptx::add2(acc[4], acc[5]), ptx::add2(acc[6], acc[7])));
          float x, y;
          ptx::f2_split(s, x, y);
          return x + y;
        };
        // the reference moves only when it has to: a row sum of at most 2^15
        // means every P is at most 2^15, finite in either type
        auto put = [&](const uint32_t (&lo)[32], const uint32_t (&hi)[32]) {
          ptx::tmem_st32(s_addr, lo);
          ptx::tmem_st32(s_addr + 32, hi);
        };
        bool fast = m_used != -INFINITY, stored = false;
        float lt = 1.f;
        if (__all_sync(0xffffffffu, fast)) {
          uint32_t lo[32], hi[32];
          load_s();
          lt = exp_pack(m_used, lo, hi);
          fast = lt <= kFastSum;
          // (a row that sees none of the tile's keys stays)
          if (Pair<T>::kFp16 && lt < kLeastSum) {
            bool none = lim < key0;
            if constexpr (kTree)
              none = key0 >= w.see0 && (key0 - w.see0 >= 64 || nodes >> (key0 - w.see0) == 0);
            fast = l >= kFallSum || (edge && none);
          }
          if (__all_sync(0xffffffffu, fast)) {
            put(lo, hi);
            l += lt;
            stored = true;
          }
        } else {
          fast = false;
        }
        bool move = false;
        float f = 1.f;
        if (!stored) {
          uint32_t lo[32], hi[32];
          load_s();
          const float ms = fmaxf(fmaxf(fmax32(&r[0]), fmax32(&r[32])),
                                 fmaxf(fmax32(&r[64]), fmax32(&r[96]))) * sl2;
          float to = ms;
          move = !fast && ms > m_used;
          if constexpr (Pair<T>::kFp16) {
            to = fmaxf(ms - kHead, m_used - kFall);
            move = !fast && (to > m_used || lt < 1.f);
          }
          f = move ? ptx::ex2(m_used - to) : 1.f;
          if (move) {
            l *= f;
            m_used = to;
          }
          lt = exp_pack(m_used == -INFINITY ? 0.f : m_used, lo, hi);   // nothing seen: 2^-inf = 0
          if (lt != lt) m_used = INFINITY;     // a join drops no NaN; the warp's others go on as they were
          put(lo, hi);
          l += lt;
        }
        ptx::tmem_st_wait();
        if (k > 0 && __any_sync(0xffffffffu, move)) {
          // O may be rescaled once the P V of the tile before is complete.  With
          // an S tile a group this tile's scores went behind it; else it is asked
          if constexpr (kScores > 2) {
            const uint32_t last = tiles - 1;
            bool done = ptx::mbar_wait(&aux->o_done[g][last % kRing], (last / kRing) & 1u, wait_limit);
            if (!__all_sync(0xffffffffu, done)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
          } else if (solo) {
            const uint32_t last = solos - 1;
            bool done = ptx::mbar_wait(&aux->solo_done[last % kRing], (last / kRing) & 1u, wait_limit);
            if (!__all_sync(0xffffffffu, done)) {
              ok = false;
              break;
            }
            ptx::tc_fence_after();
          }
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t x[16];
            ptx::tmem_ld16(o_addr + c * 16, x);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int y = 0; y < 16; ++y) x[y] = __float_as_uint(__uint_as_float(x[y]) * f);
            ptx::tmem_st16(o_addr + c * 16, x);
          }
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&aux->p_ready[g][tiles % kRing]);
      }
      if (!ok) break;
      ops = (ops + w.n_g[0] + w.n_g[1]) % kScores;
      // ------------------------------------------------------------ the item's output
      if (n_mine > 0) {
        // with an S tile a group, o_done counts items, not tiles
        const uint32_t last = kScores > 2 ? tiles - 1 : outs++;
        bool got = !aux->abort_flag &&
                   ptx::mbar_wait(&aux->o_done[g][last % kRing], (last / kRing) & 1u, wait_limit);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
      }
      if (!warp_rows) continue;
      const int64_t row = (int64_t)(w.q0 + R / G) * Hq + w.kv * G + R % G;
      const bool cut = w.slot >= 0;
      const int64_t piece = kOnLine ? w.slot : (int64_t)w.slot * Hkv + w.kv;
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t x[32];
        if (n_mine > 0) {
          ptx::tmem_ld32(o_addr + c * 32, x);
          ptx::tmem_ld_wait();
        } else {
#pragma unroll
          for (int y = 0; y < 32; ++y) x[y] = 0u;
        }
        if (!valid) continue;
        // a row that has seen nothing has P = 0 and l = 0: O = 0
        if (cut) {
          // a piece's O by column quads, rows inside: a warp's stores are contiguous
          uint4* dst = reinterpret_cast<uint4*>(part_o) + piece * (kM * D / 4) + (c * 8) * kM + g * 128 + tr;
#pragma unroll
          for (int y = 0; y < 8; ++y)
            dst[y * kM] = make_uint4(x[4 * y], x[4 * y + 1], x[4 * y + 2], x[4 * y + 3]);
        } else {
          auto h2 = [&](int y) {
            return Pair<T>::pack(__uint_as_float(x[y]) * inv, __uint_as_float(x[y + 1]) * inv);
          };
          uint4* dst = reinterpret_cast<uint4*>(o + row * D + c * 32);
#pragma unroll
          for (int y = 0; y < 4; ++y)
            dst[y] = make_uint4(h2(8 * y), h2(8 * y + 2), h2(8 * y + 4), h2(8 * y + 6));
        }
      }
      if (valid) {
        if (cut) part_ml[piece * kM + g * 128 + tr] = make_float2(m_used, l);
        else if (lse) lse[row] = l == 0.f ? -INFINITY : (m_used + log2f(l)) * kLn2;
      }
      // O has been read before this warp's next P is announced
      ptx::tc_fence_before();
    }
    if (!ok) give_up(aux, status);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, Ly::kTmemCols);
  }
}

// -------------------------------------------------------------------- join
// (kLine: n_line cut tiles of trees, by tile or by the CTA that starts one, whose
// parts lie with the CTAs behind it.)
// The rows of cut tiles, 32 neighbouring rows at a time, a row a lane and
// kPart columns a thread: a piece's O lies by column quads, rows inside, so a
// warp's loads are contiguous.  A CTA's warps take the D / kPart column parts of
// the rows, or where there are CTAs enough, the pieces of one part among them.
// (Few rows are many pieces of few tiles: smaller CTAs, so that all are there at once.)
constexpr int merge_warps(bool line) { return line ? 4 : 8; }
template <typename T, int D, bool kLine>
__global__ void __launch_bounds__(merge_warps(kLine) * 32, kLine ? 4 : 2)
paged_tc_merge(const PagedBatch b, const Header* __restrict__ hdr, const int4* __restrict__ cuts,
               int n_line, bool by_tile, int n_ctas, int Hq, int Hkv, int max_q, const float* __restrict__ part_o,
               const float2* __restrict__ part_ml, T* __restrict__ o, float* __restrict__ lse) {
  constexpr int kWarps = merge_warps(kLine), kPart = 16, kQuads = kPart / 4, kParts = D / kPart;
  __shared__ float4 s_o[kWarps][kQuads][32];
  __shared__ float2 s_ml[kWarps][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, G = Hq / Hkv;
  // units: (cut tile, KV head, 32 rows, part)
  const int64_t total = (kLine ? n_line : (int64_t)__ldcg(&hdr->n_cut) * Hkv) * (kM / 32) * kParts;
  const bool shared = total <= gridDim.x;
  const int64_t first = shared ? blockIdx.x : (int64_t)blockIdx.x * kWarps + warp;
  const int64_t hop = shared ? gridDim.x : (int64_t)gridDim.x * kWarps;
  for (int64_t u = first; u < total; u += hop) {
    const int part = (int)(u % kParts), r = (int)(u / kParts % (kM / 32)) * 32 + lane;
    const int64_t at = u / kParts / (kM / 32);
    const int4 c = __ldcg(&cuts[kLine ? at : at / Hkv]);
    int kv, q0, R;
    bool live;
    if constexpr (kLine) {
      // first token, rows and KV head, CTA, pieces.  By tile, a sequence without tokens
      // wrote none, and one whose CTA gave up may not have: the entry only says where
      // the pieces lie, if it says so within the workspace.
      kv = c.y >> 16;
      q0 = c.x;
      int rows = c.y & 0xFFFF;
      if (by_tile) {
        const SeqSpan sp = seq_span(b, (int)(at / Hkv));
        kv = (int)(at % Hkv);
        q0 = sp.q0;
        rows = min(sp.ql, max_q) * G;
      }
      R = r;
      live = r < rows && c.w > 0 && c.z >= 0 && c.z < n_ctas && c.w <= n_ctas - c.z;
    } else {
      // sequence, tile, slot, pieces
      const SeqSpan sp = seq_span(b, c.x);
      kv = (int)(at % Hkv);
      q0 = sp.q0;
      R = c.y * kM + r;
      live = R < min(sp.ql, max_q) * G;
    }
    if (!__any_sync(0xffffffffu, live)) continue;        // the same for the CTA's warps, if shared
    const int i0 = shared ? warp : 0, di = shared ? kWarps : 1;
    float4 acc[kQuads];
    float l = 0.f, m = -INFINITY;
#pragma unroll
    for (int x = 0; x < kQuads; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](float mi, float li, const float4 (&v)[kQuads]) {
      const float mn = fmaxf(m, mi);
      if (mn == -INFINITY) return;                       // no key so far
      const float f0 = exp2f(m - mn), f = exp2f(mi - mn);
      l = l * f0 + f * li;
#pragma unroll
      for (int x = 0; x < kQuads; ++x) {
        acc[x].x = acc[x].x * f0 + f * v[x].x;
        acc[x].y = acc[x].y * f0 + f * v[x].y;
        acc[x].z = acc[x].z * f0 + f * v[x].z;
        acc[x].w = acc[x].w * f0 + f * v[x].w;
      }
      m = mn;
    };
    // four pieces' loads together (rows behind the tile's last are there to be
    // read, and go nowhere)
    constexpr int kAtOnce = 4;
    for (int ib = i0; ib < c.w; ib += kAtOnce * di) {
      float2 ml[kAtOnce];
      float4 v[kAtOnce][kQuads];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int i = ib + j * di;
        if (i < c.w) {
          const int64_t piece = kLine ? (i == 0 ? 2 * (int64_t)c.z + 1 : 2 * (int64_t)(c.z + i))
                                      : (int64_t)(c.z + i) * Hkv + kv;
          ml[j] = __ldcg(&part_ml[piece * kM + r]);
          const float4* p = reinterpret_cast<const float4*>(part_o) + piece * (kM * D / 4) +
                            (int64_t)(part * kQuads) * kM + r;
#pragma unroll
          for (int x = 0; x < kQuads; ++x) v[j][x] = __ldcg(p + x * kM);
        }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (ib + j * di < c.w) add(ml[j].x, ml[j].y, v[j]);
    }
    if (shared) {
#pragma unroll
      for (int x = 0; x < kQuads; ++x) s_o[warp][x][lane] = acc[x];
      s_ml[warp][lane] = make_float2(m, l);
      __syncthreads();
      if (warp > 0) continue;                            // one unit a CTA: no trip follows
      for (int w = 1; w < kWarps; ++w) {
        float4 v[kQuads];
#pragma unroll
        for (int x = 0; x < kQuads; ++x) v[x] = s_o[w][x][lane];
        const float2 ml = s_ml[w][lane];
        add(ml.x, ml.y, v);
      }
    }
    if (!live) continue;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const int64_t row = (int64_t)(q0 + R / G) * Hq + kv * G + R % G;
    uint4* dst = reinterpret_cast<uint4*>(o + row * D + part * kPart);
#pragma unroll
    for (int x = 0; x < kQuads; x += 2)
      dst[x / 2] = make_uint4(Pair<T>::pack(acc[x].x * inv, acc[x].y * inv),
                              Pair<T>::pack(acc[x].z * inv, acc[x].w * inv),
                              Pair<T>::pack(acc[x + 1].x * inv, acc[x + 1].y * inv),
                              Pair<T>::pack(acc[x + 1].z * inv, acc[x + 1].w * inv));
    if (lse && part == 0) lse[row] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
  }
}

// -------------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// The pool as rows of d: a box is one page's 64-column panel.
int pool_map(CUtensorMap* map, const void* base, const PagedBatch& b, int Hkv, int d, bool fp16) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(TS_ERR_CUDA, "cuTensorMapEncodeTiled is unavailable");
  const int ps = 1 << b.page_shift;
  cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)b.n_pages * Hkv * ps};
  cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  cuuint32_t box[2] = {64, (cuuint32_t)ps};
  cuuint32_t estr[2] = {1, 1};
  const CUresult r =
      fn(map, fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2,
         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(TS_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return TS_OK;
}

template <typename T, int D>
int go_tc(const PagedBatch& b, const TcArgs& a, const TcPlan& p, char* ws, int32_t* status,
          cudaStream_t st) {
  CUtensorMap mk, mv;
  int rc = pool_map(&mk, a.k_pages, b, a.Hkv, D, Pair<T>::kFp16);
  if (!rc) rc = pool_map(&mv, a.v_pages, b, a.Hkv, D, Pair<T>::kFp16);
  if (rc) return rc;
  auto kern = p.line      ? paged_tc_kernel<T, D, kTreeLine>
              : a.parents ? paged_tc_kernel<T, D, kTreeList>
                          : paged_tc_kernel<T, D, kChunk>;
  // the warps' register split adds up to 128 registers a thread at launch; any
  // other count would leave the softmax warps waiting for registers
  cudaFuncAttributes fa{};
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess || fa.numRegs != 128)
    return fail(TS_ERR_CUDA, "paged attention compiled to %d registers a thread; its register "
                "split needs 128", fa.numRegs);
  cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
  Header* hdr = reinterpret_cast<Header*>(ws);
  int4* tiles = reinterpret_cast<int4*>(ws + p.tiles_at);
  int4* entries = reinterpret_cast<int4*>(ws + p.entries_at);
  int* slots = reinterpret_cast<int*>(ws + p.slots_at);
  int4* cuts = reinterpret_cast<int4*>(ws + p.cuts_at);
  float* part_o = reinterpret_cast<float*>(ws + p.part_at);
  float2* part_ml = reinterpret_cast<float2*>(ws + p.ml_at);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  const Work work{hdr, entries, slots, cuts, p.line && p.line_cuts < p.grid};
  if (!p.line) {
    const size_t near = p.max_tiles <= kPlanTiles ? (size_t)p.max_tiles * 2 * sizeof(int4) : 0;
    cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                         kPlanTiles * 2 * sizeof(int4));
    pdl_config(&cfg, attr, dim3(1), dim3(kPlanThreads), near, st);
    cudaLaunchKernelEx(&cfg, paged_plan_kernel, b, a.Hkv, a.Hq / a.Hkv, D, a.max_q,
                       a.parents && D == 128 ? kSoloEighths : 8, p.max_tiles,
                       p.max_entries, p.max_slots, hdr, tiles, entries, slots, cuts, status);
    rc = launch_status("paged_plan_kernel");
    if (rc) return rc;
  }
  pdl_config(&cfg, attr, dim3(p.grid), dim3(kThreads), Layout<D>::kBytes, st);
  cudaLaunchKernelEx(&cfg, kern, mk, mv, b, static_cast<const T*>(a.q), a.Hq, a.Hkv, a.max_q,
                     a.parents, work, static_cast<T*>(a.o), a.lse, part_o, part_ml, wait_limit_cycles(), status);
  rc = launch_status("paged_tc_kernel");
  if (rc || p.max_slots == 0) return rc;
  pdl_config(&cfg, attr, dim3(p.merge_grid), dim3(merge_warps(p.line) * 32), 0, st);
  cudaLaunchKernelEx(&cfg, p.line ? paged_tc_merge<T, D, true> : paged_tc_merge<T, D, false>, b,
                     (const Header*)hdr, (const int4*)cuts, p.line_cuts, work.by_tile, p.grid, a.Hq,
                     a.Hkv, a.max_q, (const float*)part_o, (const float2*)part_ml, static_cast<T*>(a.o),
                     a.lse);
  return launch_status("paged_tc_merge");
}

}  // namespace

TcPlan tc_plan(int n, int n_seq, int Hq, int Hkv, int d, int max_q, int64_t max_kv, int64_t cap,
               bool tree) {
  TcPlan p{};
  const int64_t G = Hq / Hkv;
  // tiles: a sequence's rows rounded up to whole tiles
  const int64_t per_seq = (max_q * G + kM - 1) / kM;
  const int64_t tiles = imin64(n * G / kM + n_seq, per_seq * n_seq);
  // partial rows of cut tiles: at most six pieces a SM, and no more than the
  // tiles have key steps
  const int64_t steps = imax64(1, (max_kv + kNk - 1) / kNk);
  int64_t slots = imin64(6 * kGb300Sms / Hkv, tiles * steps);
  if (steps == 1 || tiles * Hkv >= 16 * kGb300Sms) slots = 0;
  p.max_tiles = (int)tiles;
  p.max_slots = (int)(slots * Hkv);
  p.max_entries = (int)(tiles + slots);
  p.grid = (int)imin64(kGb300Sms, (int64_t)p.max_entries * Hkv);
  // units of 32 rows and 16 columns, eight warps a CTA; a cut tile has at least
  // two pieces
  p.merge_grid = (int)imin64(8 * kGb300Sms, imax64(1, slots * Hkv * (kM / 32) * (d / 16) / 2));
  size_t at = 256;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += align_up(bytes, 256);
    return r;
  };
  const int64_t units = (int64_t)n_seq * Hkv;
  if (tree && max_q * G <= kM && units < (int64_t(1) << 31) / (cap / kNk + 1 + kLineFixed)) {
    p.line = true;
    p.grid = (int)imax64(1, imin64(kGb300Sms, units * (steps + kLineFixed) / kLineLeast));
    p.line_cuts = (int)imin64(units, p.grid);
    p.max_slots = p.grid > 1 ? 2 * p.grid : 0;
    p.merge_grid = (int)imin64(8 * kGb300Sms, (int64_t)p.line_cuts * (kM / 32) * (d / 16));
    p.cuts_at = take((size_t)p.grid * sizeof(int4));
    p.part_at = take((size_t)p.max_slots * kM * d * sizeof(float));
    p.ml_at = take((size_t)p.max_slots * kM * sizeof(float2));
    p.ws_bytes = at;
    return p;
  }
  p.tiles_at = take((size_t)tiles * 2 * sizeof(int4));
  p.entries_at = take((size_t)p.max_entries * sizeof(int4));
  p.slots_at = take((size_t)p.max_entries * sizeof(int));
  p.cuts_at = take((size_t)(slots / 2 + 1) * sizeof(int4));
  p.part_at = take((size_t)p.max_slots * kM * d * sizeof(float));
  p.ml_at = take((size_t)p.max_slots * kM * sizeof(float2));
  p.ws_bytes = at;
  return p;
}

int launch_paged_tc(const PagedBatch& b, const TcArgs& a, const TcPlan& p, int d, bool fp16,
                    void* ws, int32_t* status, cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  if (fp16)
    return d == 128 ? go_tc<__half, 128>(b, a, p, w, status, st)
                    : go_tc<__half, 64>(b, a, p, w, status, st);
  return d == 128 ? go_tc<__nv_bfloat16, 128>(b, a, p, w, status, st)
                  : go_tc<__nv_bfloat16, 64>(b, a, p, w, status, st);
}

}  // namespace ts
