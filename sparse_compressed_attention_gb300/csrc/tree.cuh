// What the kernels of the tree attention share: the call's arguments, a row's
// key list and the cache row behind each position of the list.
//
// The keys of a row are numbered entries first (ne), then the committed
// tokens of the window (nw), then the drafted ancestors (nd).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace v4 {

constexpr int kPlanWords = 8;

struct TreeArgs {
  const void* q;
  const int32_t* plan;
  const void* tok_cache;
  const int32_t* tok_table;
  const void* ent_cache;
  const int32_t* ent_table;
  const int32_t* ent_len;
  const int32_t* idx;
  const float* sink;
  const float* inv_freq;
  long long tok_slots, ent_slots;
  int n_rows, tok_blocks, tok_page, ent_blocks, ent_page;
  void* o;
  float* lse;
  int* status;
  int B, H, D, R, ratio, window, K;
  float scale;
};

// A planned row.  live = false: padding, or a plan row that cannot be used
// (flagged).
struct TreeRow {
  int b, node, t, L;
  int nv;                 // visible entries
  int ne, lo, nw;         // list: entry positions, first window token, window tokens
  bool live;
};

__device__ __forceinline__ TreeRow tree_row(const TreeArgs& a, int row) {
  const int4 w = *reinterpret_cast<const int4*>(a.plan + (size_t)row * kPlanWords);
  TreeRow r;
  r.b = w.x;
  r.node = w.y;
  r.t = w.z;
  r.L = w.w;
  r.live = r.b >= 0 && r.b < a.B && r.t >= 0 && r.L >= 0 && r.node >= 0 && r.node < V4_TREE_MAX_NODES;
  if (!r.live) {
    if (r.b != -1) set_status(a.status, kStatusBadIndex);
    r.nv = r.ne = r.lo = r.nw = 0;
    return r;
  }
  r.nv = 0;
  if (a.ratio > 0) {
    // (t + 1) / ratio without the overflow at the largest position
    const int by_pos = (int)(((unsigned)r.t + 1u) / (unsigned)a.ratio);
    const long long held = (long long)a.ent_blocks * a.ent_page;
    int len = a.ent_len[r.b];
    if (len < 0) { set_status(a.status, kStatusBadIndex); len = 0; }
    if (len > held) { set_status(a.status, kStatusBadIndex); len = (int)held; }
    r.nv = min(by_pos, len);
  }
  r.ne = a.K > 0 ? a.K : r.nv;
  // committed tokens u < min(L, t + 1), u > t - W
  int hi = r.L <= r.t ? r.L : r.t + 1;
  const long long held = (long long)a.tok_blocks * a.tok_page;
  if (a.window != 0 && hi > held) {               // the table ends before the tokens do
    set_status(a.status, kStatusBadIndex);
    hi = (int)held;
  }
  r.lo = a.window < 0 ? 0 : max(0, r.t - a.window + 1);
  r.nw = a.window == 0 ? 0 : max(0, hi - r.lo);
  return r;
}

// The drafted keys of a row: bit j of mask[4] that is in the window.  Called
// by lane j of 128 threads or in a loop; returns whether node j is a key.
__device__ __forceinline__ bool tree_draft_key(const TreeArgs& a, const TreeRow& r, int row, int j, uint32_t word) {
  if (a.window == 0 || !((word >> (j & 31)) & 1u)) return false;
  const int at = row - r.node + j;                    // the sequence's rows are consecutive
  if (at < 0 || at >= a.n_rows) { set_status(a.status, kStatusBadIndex); return false; }
  const int4 w = *reinterpret_cast<const int4*>(a.plan + (size_t)at * kPlanWords);
  if (w.x != r.b || w.y != j) { set_status(a.status, kStatusBadIndex); return false; }
  const long long d = (long long)r.t - w.z;
  return d >= 0 && (a.window < 0 || d < a.window);
}

// Row of a paged cache for logical row `at` of sequence b, -1 (flagged) where
// the table or the cache does not hold it.
__device__ __forceinline__ long long paged_row(const int32_t* table, int blocks, int page, long long slots, int b,
                                               long long at, int* status) {
  const long long blk = at / page;
  if (at < 0 || blk >= blocks) { set_status(status, kStatusBadIndex); return -1; }
  const int pg = table[(size_t)b * blocks + blk];
  const long long s = (long long)pg * page + (at - blk * page);
  if (pg < 0 || s >= slots) { set_status(status, kStatusBadIndex); return -1; }
  return s;
}

// Entry slot k of a row (k < ne): the cache row, -1 where the slot is unused
// or not visible.
__device__ __forceinline__ long long tree_entry_row(const TreeArgs& a, const TreeRow& r, int row, int k) {
  int s = k;
  if (a.K > 0) {
    s = a.idx[(size_t)row * a.K + k];
    if (s < 0 || s >= r.nv) {
      if (s != -1) set_status(a.status, kStatusBadIndex);
      return -1;
    }
  }
  return paged_row(a.ent_table, a.ent_blocks, a.ent_page, a.ent_slots, r.b, s, a.status);
}

__device__ __forceinline__ long long tree_token_row(const TreeArgs& a, const TreeRow& r, long long at) {
  return paged_row(a.tok_table, a.tok_blocks, a.tok_page, a.tok_slots, r.b, at, a.status);
}

bool tree_tc_supported(const v4_config& c);
size_t tree_tc_workspace();
// q4: the caches hold 4-bit rows
cudaError_t launch_tree_tc(const TreeArgs& a, bool q4, void* workspace, cudaStream_t st);

}  // namespace v4
