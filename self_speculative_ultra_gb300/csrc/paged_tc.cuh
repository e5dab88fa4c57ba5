// Chunk attention over a paged cache on the tensor cores (paged_tc.cu): plan
// and launcher.
#pragma once

#include "paged.cuh"

namespace ts {

constexpr int kTcRows = 256;   // query rows a tile

struct TcPlan {
  int max_tiles, max_entries;
  int max_slots;               // partial tiles, KV heads included (0: nothing is cut)
  int grid, merge_grid;
  size_t tiles_at, entries_at, slots_at, cuts_at, part_at, ml_at, ws_bytes;
};
TcPlan tc_plan(int n, int n_seq, int Hq, int Hkv, int d, int max_q, int64_t max_kv);

struct TcArgs {
  const void *q, *k_pages, *v_pages;
  int Hq, Hkv, max_q;
  void* o;
  float* lse;
};
int launch_paged_tc(const PagedBatch& b, const TcArgs& a, const TcPlan& p, int d, bool fp16,
                    void* ws, int32_t* status, cudaStream_t st);

}  // namespace ts
