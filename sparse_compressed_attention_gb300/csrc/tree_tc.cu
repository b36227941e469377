// Tree attention on the 5th-generation tensor cores (tcgen05, TMEM
// accumulators) for the DeepSeek-V4-Flash shapes: 64-head slices of one 512-d
// latent that is key and value, last 64 dims rotated, bf16 storage.
//
// Work.  An item is (row, 64-head slice); its keys (entries, committed window
// tokens, drafted ancestors) are numbered and cut into tiles of 128.  Lengths
// live on the device, so every block computes the same prefix sum of the
// items' tile counts and takes an equal share of all tiles: a long row is
// split over many blocks, a block walks several short rows.  A block that
// holds an item whole writes its output; pieces of a cut item leave their
// unnormalised sums, maxima and denominators in the workspace, and the join
// kernel merges them.  The cut depends on the lengths alone, so results repeat
// bit for bit.
//
// Per tile (one block, M = 128 keys or dims, N = 64 heads):
//   S^T[key, head]  = K_tile . Q^T             (K = 512, + 64 for q's low part)
//   P^T             = exp2(S^T c - m_head), rounded to bf16 like the keys that it
//                     multiplies: two terms would be 32 more products of 100 a tile.
//                     The output's error grows from 1.0 to at most 1.3 roundings of
//                     a bf16 output (selected trees 0.0017 -> 0.0021 relative)
//   O^T[dim, head] += K_tile^T . P^T           (4 x M = 128 dims)
// The rotated 64 dims of q are kept as two bf16 terms (high and low), so the
// logits, and with them lse, carry no rounding of the rotation; it costs 4
// products of 68.  m is a running maximum that is only raised when a logit
// exceeds it by more than 8 (a factor of 256, well inside bf16 P and fp32 sums):
// the O^T rescale through registers is then rare, and a vote of one
// barrier is all that a tile pays for it.
//
// Roles (448 threads): warp 0 shares out the work, loads query rows and the
// whole tiles of page runs (TMA boxes of up to a page: every entry, or every
// token), warp 1 issues the products, warps 2-3 and 12-13 look up key rows
// and gather the rest (16-byte cp.async, masked rows zero-filled so that
// nothing a mask hides is ever read), warps 4-11 softmax and output (two per
// TMEM lane quarter, 32 heads each).
//
// What bounds it.  A block takes a tile in 2.8 us when the keys come out of L2,
// in boxes or gathered (rows of 16 to 32 tiles, one to a block).  1.8 us of it are
// the 68 products, 54.3 cycles each at N = 64; the softmax lies between the S and
// the O products of the same tile, and only one tile fits beside the query rows,
// so its slots are filled again as the O products release them.  Where all 152
// blocks read keys of their own, 128 KB a tile meet HBM: 2.9 us a tile in boxes
// (6.8 TB/s, the copy rate), 4.1 gathered.  Beside the tiles a block pays 12 us
// for its first piece (launch, shares, look-ups, first tile, output, the empty
// join), 4 for each further one, and a call in which rows are cut 9 for parts
// and join.  The CUDA-core kernel's times are in brackets, tiles are a block's:
//   1 row, 512 selected entries + window        16 us     [246]     1 tile
//   32 x up to 8 nodes, selected                51 us     [2196]    7
//   8 x 8 nodes over 7812 entries each          99 us     [9681]    27
//   16 rows over all of up to 49152 tokens      91 us     [19127]   20
//   4 x 16 nodes over 32768 tokens              358 us    [40543]   109, 35% tensor pipe
// (the last reads 134 MB of keys, more than L2 holds: one sequence with 64 nodes
// takes 323).  Tried and not faster: 16 softmax warps, another split of the
// registers, the softmax in paired fp32 operations or with its exponentials ahead
// of the vote, TMEM allocated before the shares, rows asked two tiles ahead.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "sm100.cuh"
#include "tree.cuh"
#include "turn.cuh"

namespace v4 {

using namespace sm100;

namespace {

constexpr int kH = 64, kD = 512, kR = 64;
constexpr int kThreads = 448;
constexpr int kSoftThreads = 256;                 // warps 4-11
constexpr int kSoftWarps = kSoftThreads / 32;
constexpr int kGatherWarps = 4;                   // 32 key rows each
constexpr int kTile = 128;
constexpr int kSlots = 8;                         // K-blocks of 64 dims: one tile
constexpr int kPairs = kSlots / 2;
constexpr uint32_t kSlotBytes = kTile * 128;
constexpr uint32_t kQBlockBytes = kH * 128;
constexpr uint32_t kPBytes = kTile * kH * 2;
constexpr int kMaxCtas = 152;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;                     // how far (log2) a logit may exceed m

constexpr uint32_t OFF_Q = 0;                                     // 8 K-blocks, then q's low part
constexpr uint32_t OFF_SLOT = OFF_Q + 9 * kQBlockBytes;           // 73728
constexpr uint32_t OFF_P = OFF_SLOT + kSlots * kSlotBytes;        // 204800
constexpr uint32_t OFF_CTL = OFF_P + kPBytes;                     // 221184

// A row's key list in tiles.
struct Tiles {
  int n;                                 // all of them, 0: the row is not live
  int dense;                             // leading ones that are whole page runs
  int seq;
};

// A block's piece of an item.
struct alignas(16) Piece {               // two 16-byte words: it is copied through shared memory
  int row, hs, tile0, tiles;
  int done;
  int dense;                             // leading tiles that arrive as whole page runs (TMA)
  int part;                              // workspace part of a cut item, -1: the item is whole
  int seq;
};

struct Ctl {
  // K-blocks go in pairs, as an M-block of O releases them
  uint64_t full_g[kPairs], full_t[kPairs], empty[kPairs];   // gathered / page-run pair landed, pair released
  uint64_t valid_full[2];
  uint64_t q_full, q_ready, q_empty;
  uint64_t s_full[2], p_ready[2];
  uint64_t o_full, o_empty;
  uint64_t info_full[2], info_empty[2];
  uint64_t fin;
  Piece info[2];
  uint32_t valid[2][kGatherWarps];       // bit per key row of a tile
  float2 cs[2][kR / 2];                  // cos/sin of the piece's position
  alignas(16) float m[kH];               // shift of each head (log2 units), read four at a time
  float hmax[4][kH];
  float fac[kH];
  float part_l[4][kH];
  float inv[kH];
  int scan[kThreads / 32];
  int start_item, start_unit;            // where this block's share begins
  Tiles start_tiles;
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmemBytes = OFF_CTL + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory budget");

// Workspace: parts of cut items (two a block: the item its share begins
// inside, the item it ends inside), then for each block the item that begins
// there and is cut.
struct PartHead {
  float m[kH], l[kH];
};
constexpr size_t kPartFloats = (size_t)kH * kD;
constexpr size_t kPartBytes = kPartFloats * 4 + sizeof(PartHead);

struct Args {
  TreeArgs t;
  int HS, items;
  int box;                               // rows of a page run that one TMA box takes, 0: gather everything
  int dense_tok;                         // the runs are token pages (else entry pages)
  char* parts;
  int4* cuts;                            // per block: the item that goes on behind its end (or -1), that item's first and last block
};

// Tiles of a row.
__device__ __forceinline__ Tiles tree_tiles(const Args& p, int row) {
  const TreeArgs& a = p.t;
  const TreeRow r = tree_row(a, row);
  if (!r.live) return Tiles{0, 0, 0};
  const int4 w = *reinterpret_cast<const int4*>(a.plan + (size_t)row * kPlanWords + 4);
  const int nd = a.window == 0 ? 0 : __popc(w.x) + __popc(w.y) + __popc(w.z) + __popc(w.w);
  const long long nk = (long long)r.ne + r.nw + nd;
  return Tiles{nk == 0 ? 1 : (int)((nk + kTile - 1) / kTile), p.box ? (p.dense_tok ? r.nw : r.ne) / kTile : 0, r.b};
}

// Node of the i-th set bit.
__device__ __forceinline__ int nth_node(const int4 w, int i) {
  const uint32_t m[4] = {(uint32_t)w.x, (uint32_t)w.y, (uint32_t)w.z, (uint32_t)w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int n = __popc(m[k]);
    if (i < n) {
      uint32_t b = m[k];
      for (; i > 0; --i) b &= b - 1;
      return 32 * k + __ffs(b) - 1;
    }
    i -= n;
  }
  return -1;
}

// Cache row behind position `at` of a row's key list; null where there is no key.
__device__ __forceinline__ const bf16* key_row(const TreeArgs& a, const TreeRow& r, const int4 bits, int row,
                                               long long at) {
  if (at < r.ne) {
    const long long s = tree_entry_row(a, r, row, (int)at);
    return s < 0 ? nullptr : reinterpret_cast<const bf16*>(a.ent_cache) + s * kD;
  }
  at -= r.ne;
  long long u;
  if (at < r.nw) {
    u = r.lo + at;
  } else {
    if (a.window == 0 || at - r.nw >= V4_TREE_MAX_NODES) return nullptr;
    const int j = nth_node(bits, (int)(at - r.nw));
    if (j < 0 || !tree_draft_key(a, r, row, j, 0xFFFFFFFFu)) return nullptr;
    u = (long long)r.L + j;
  }
  const long long s = tree_token_row(a, r, u);
  return s < 0 ? nullptr : reinterpret_cast<const bf16*>(a.tok_cache) + s * kD;
}

// 16 bytes of global memory, or zeros, into shared memory.
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
      "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
      "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15])), "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])),
      "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])),
      "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
      "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])),
      "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])),
      "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
      : "memory");
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Barrier of n threads that also tells whether any of them saw `p`.
__device__ __forceinline__ bool bar_any(int id, int n, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)p), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// One arrival for a warp once all its lanes are here: a barrier takes arrivals
// one by one, and 256 of them lie between a tile's softmax and its products.
__device__ __forceinline__ void warp_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Every lane of a warp waits for itself (and acquires for itself).  One lane
// polling for the others woke 0.4 us later: 574 against 456 us for 16 nodes
// over 32768 tokens.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, Ctl* c, int* status) {
  const bool ok = mbar_wait(bar, parity, &c->abort, status);
  return __all_sync(0xffffffffu, ok);
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Five butterfly rounds over a warp: lane L is left with the fold of r[L] over
// the lanes.
template <typename F>
__device__ __forceinline__ float fold_lanes(float* r, int lane, F f) {
#pragma unroll
  for (int o = 16, w = 16; o >= 1; o >>= 1, w >>= 1) {
    const bool hi = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float send = hi ? r[i] : r[w + i];
      const float keep = hi ? r[w + i] : r[i];
      r[i] = f(keep, __shfl_xor_sync(0xffffffffu, send, o));
    }
  }
  return r[0];
}

// What a sink (log2 units) adds to a denominator whose shift m is at least as
// large: nothing at -inf, one where it is the shift itself (+inf among them),
// NaN for a NaN, which the maximum has dropped.
__device__ __forceinline__ float sink_mass(float s2, float m) {
  return s2 == -INFINITY ? 0.f : s2 == m ? 1.f : ex2_approx(s2 - m);
}

// Units of a share: each item is one unit (its query rows and output) plus
// its tiles.  Block c of the grid takes units [c * share, (c + 1) * share).
__device__ __forceinline__ int share_of(int total, int ctas) { return (total + ctas - 1) / ctas; }

__global__ void __launch_bounds__(kThreads, 1)
tree_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_pages, const Args p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Ctl* c = reinterpret_cast<Ctl*>(smem + OFF_CTL);
  const TreeArgs& a = p.t;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if ((smem_u32(smem) & 1023u) != 0) {          // swizzled operands need 1 KB alignment
    wait_previous();
    if (threadIdx.x == 0) {
      set_status(a.status, V4_ERR_UNSUPPORTED);
      p.cuts[blockIdx.x] = make_int4(-1, -1, -1, 0);        // nothing for the join
    }
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kPairs; ++i) {
      mbar_init(&c->full_g[i], 32 * kGatherWarps);
      mbar_init(&c->full_t[i], 1);
      mbar_init(&c->empty[i], 1);
    }
    mbar_init(&c->q_full, 1);
    mbar_init(&c->q_ready, kSoftWarps);
    mbar_init(&c->q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->valid_full[i], kGatherWarps);
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->p_ready[i], kSoftWarps);
      mbar_init(&c->info_full[i], 1);
      mbar_init(&c->info_empty[i], 1 + kSoftWarps + kGatherWarps);
    }
    mbar_init(&c->o_full, 1);
    mbar_init(&c->o_empty, kSoftWarps);
    mbar_init(&c->fin, 1);
    c->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_pages);
  }

  wait_previous();                              // nothing of global memory is read before

  // ---- this block's share: prefix sum of the items' units
  const int per = (p.items + kThreads - 1) / kThreads;
  const int i0 = threadIdx.x * per, i1 = min(i0 + per, p.items);
  int mine = 0;
  Tiles first = {0, 0, 0};
  for (int i = i0; i < i1; ++i) {
    const Tiles t = tree_tiles(p, i / p.HS);
    if (i == i0) first = t;
    mine += t.n ? t.n + 1 : 0;
  }
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += v;
  }
  if (lane == 31) c->scan[warp] = upto;
  __syncthreads();
  int before = upto - mine, total = 0;
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += c->scan[w];
    total += c->scan[w];
  }
  const int share = share_of(total, gridDim.x);
  const int s0 = min(blockIdx.x * share, total), s1 = min(s0 + share, total);
  if (s0 >= s1) {                                // nothing for this block
    if (threadIdx.x == 0) p.cuts[blockIdx.x] = make_int4(-1, -1, -1, 0);
    return;
  }
  if (before <= s0 && s0 < before + mine) {
    int at = before;
    for (int i = i0; i < i1; ++i) {
      const Tiles t = i == i0 ? first : tree_tiles(p, i / p.HS);
      const int u = t.n ? t.n + 1 : 0;
      if (s0 < at + u) {
        c->start_item = i;
        c->start_unit = at;
        c->start_tiles = t;
        break;
      }
      at += u;
    }
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ shares and query rows
    int item = c->start_item, unit = c->start_unit, qc = 0, g = 0;
    bool ok = true;
    int4 cut = make_int4(-1, -1, -1, 0);         // the item that goes on in the next block
    auto next_piece = [&]() -> Piece {
      Piece pc = {0, 0, 0, 0, 1, 0, -1, 0};
      while (item < p.items && unit < s1) {
        const Tiles t = item == c->start_item ? c->start_tiles : tree_tiles(p, item / p.HS);
        const int n = t.n;
        const int base = unit + 1;               // unit of the item's tile 0
        const int lo = max(s0, base), hi = min(s1, base + n);
        if (n > 0 && lo < hi) {
          pc.done = 0;
          pc.row = item / p.HS;
          pc.hs = item % p.HS;
          pc.tile0 = lo - base;
          pc.tiles = hi - lo;
          pc.dense = min(max(t.dense - pc.tile0, 0), pc.tiles);
          // a share that begins behind tile 0 leaves its part in the block's
          // first place, one that begins with it in the second
          pc.seq = t.seq;
          pc.part = pc.tiles == n ? -1 : 2 * (int)blockIdx.x + (lo > base ? 0 : 1);
          if (base + n > s1) cut = make_int4(item, base / share, (base + n - 1) / share, 0);
        }
        unit += n ? n + 1 : 0;
        ++item;
        if (!pc.done) break;
      }
      return pc;
    };
    auto publish = [&](const Piece& pc, int q) {
      if (lane == 0) {
        const int is = q & 1;
        if (q >= 2) ok = mbar_wait(&c->info_empty[is], ((q >> 1) - 1) & 1, &c->abort, a.status);
        if (ok) {
          c->info[is] = pc;
          mbar_arrive(&c->info_full[is]);
        }
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
    };
    // lane: box lane & 15 of K-block 2 m + (lane >> 4), m in the order in which the
    // O products release them
    const int box = lane & 15, odd = lane >> 4;
    const int boxes = p.box ? kTile / p.box : 0;
    const int32_t* table = p.dense_tok ? a.tok_table : a.ent_table;
    const int blocks = p.dense_tok ? a.tok_blocks : a.ent_blocks, page = p.dense_tok ? a.tok_page : a.ent_page;
    const int slots = (int)(p.dense_tok ? a.tok_slots : a.ent_slots);
    Piece pc = next_piece();
    publish(pc, 0);
    while (ok && !pc.done) {
      if (lane == 0) {
        if (qc >= 1) ok = mbar_wait(&c->q_empty, (qc - 1) & 1, &c->abort, a.status);
        if (ok) mbar_expect_tx(&c->q_full, 8 * kQBlockBytes);
      }
      ok = __shfl_sync(0xffffffffu, (int)ok, 0);
      if (!ok) break;
      if (lane < 8)
        tma_load_2d(smem + OFF_Q + lane * kQBlockBytes, &map_q, 64 * lane, pc.row * a.H + kH * pc.hs, &c->q_full);
      // the next piece is described while this one's tiles load
      Piece nxt = {0, 0, 0, 0, 1, 0, -1, 0};
      if (pc.dense == 0) {
        nxt = next_piece();
        publish(nxt, qc + 1);
      }
      for (int j = 0; j < pc.dense && ok; ++j) {
        // cache row of this lane's box, looked up before the slots are free; a
        // page that the table does not hold reads zeros (its rows are masked)
        int y = slots;
        if (box < boxes) {
          const long long at = (long long)(pc.tile0 + j) * kTile + box * p.box;
          const long long blk = at / page;
          const int pg = blk < blocks ? table[(size_t)pc.seq * blocks + blk] : -1;
          const long long r = (long long)pg * page + (at - blk * page);
          if (pg >= 0 && r < slots) y = (int)r;
        }
        for (int m = kPairs - 1; m >= 0 && ok; --m) {
          const int kb = 2 * m + odd;
          if (g >= 1) ok = mbar_wait(&c->empty[m], (g - 1) & 1, &c->abort, a.status);
          if (!ok) break;
          if (lane == 0) mbar_expect_tx(&c->full_t[m], 2 * kSlotBytes);
          if (box < boxes)
            tma_load_2d(smem + OFF_SLOT + kb * kSlotBytes + box * p.box * 128, &map_pages, 64 * kb, y, &c->full_t[m]);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++g;
        if (j == 0) {
          nxt = next_piece();
          publish(nxt, qc + 1);
        }
      }
      // gathered tiles: their slot releases are awaited too, a parity wait being
      // unambiguous one phase ahead only
      for (int j = pc.dense; j < pc.tiles && ok; ++j) {
        for (int m = kPairs - 1; m >= 0 && ok; --m)
          if (g >= 1) ok = warp_wait(&c->empty[m], (g - 1) & 1, c, a.status);
        ++g;
      }
      pc = nxt;
      ++qc;
    }
    if (lane == 0) p.cuts[blockIdx.x] = cut;
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    // The whole warp walks the tiles and one elected lane issues: with warp-uniform
    // control and operands the descriptors stay in uniform registers.  The same
    // loop inside `if (lane == 0)` moved each of them there for every product
    // (402 against 371 us for 16 nodes over 32768 tokens).
    {
      const bool lead = elect_one();               // issues for the converged warp
      const uint32_t id1 = idesc_bf16_f32(128, 64, 0, 0);
      const uint32_t id2 = idesc_bf16_f32(128, 64, 1, 1);
      const uint64_t dA1 = smem_desc(smem_u32(smem + OFF_SLOT), 16, 1024, kLayoutSW128);
      const uint64_t dQ = smem_desc(smem_u32(smem + OFF_Q), 16, 1024, kLayoutSW128);
      const uint64_t dA2 = smem_desc(smem_u32(smem + OFF_SLOT), kSlotBytes, 1024, kLayoutSW128);
      const uint64_t dP = smem_desc(smem_u32(smem + OFF_P), 128, 2048, kLayoutNone);
      const uint32_t hA1 = (uint32_t)(dA1 >> 32), hQ = (uint32_t)(dQ >> 32), hA2 = (uint32_t)(dA2 >> 32),
                     hP = (uint32_t)(dP >> 32);
      const uint32_t a1 = (uint32_t)dA1, q1 = (uint32_t)dQ, a2 = (uint32_t)dA2, p2 = (uint32_t)dP;
      const auto desc = [](uint32_t hi, uint32_t lo) { return ((uint64_t)hi << 32) | lo; };
      int qc = 0, g = 0, gg = 0, gt = 0;            // all tiles, gathered ones, page runs
      bool ok = true;
      while (ok) {
        const int is = qc & 1;
        ok = warp_wait(&c->info_full[is], (qc >> 1) & 1, c, a.status);
        if (!ok) break;
        const Piece pc = c->info[is];
        __syncwarp();
        if (lead) mbar_arrive(&c->info_empty[is]);
        if (pc.done) break;
        ok = warp_wait(&c->q_ready, qc & 1, c, a.status);
        tc_fence_after();
        for (int j = 0; j < pc.tiles && ok; ++j) {
          const int sb = g & 1;
          const uint32_t s_tmem = tmem + 64 * sb;
          // K-blocks as they land, two at a time (the O products release them in
          // pairs), the rotated dims' pair first: their second products then run
          // while the others land.  TMA writes need no proxy fence.
          const bool dense = j < pc.dense;
          uint64_t* full = dense ? c->full_t : c->full_g;
          const uint32_t par = (dense ? gt : gg) & 1;
#pragma unroll
          for (int m = kPairs - 1; m >= 0; --m) {
            ok = ok && warp_wait(&full[m], par, c, a.status);
            if (!dense) fence_proxy_async_smem();     // cp.async writes -> tensor-core reads
            if (lead) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                umma_f16_ss(s_tmem, desc(hA1, a1 + (((2 * m + ks / 4) * kSlotBytes + 32 * (ks & 3)) >> 4)),
                            desc(hQ, q1 + (((2 * m + ks / 4) * kQBlockBytes + 32 * (ks & 3)) >> 4)), id1,
                            m < kPairs - 1 || ks > 0);
              if (m == kPairs - 1)                    // the rotated dims once more, against q's low part
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  umma_f16_ss(s_tmem, desc(hA1, a1 + ((7 * kSlotBytes + 32 * ks) >> 4)),
                              desc(hQ, q1 + ((8 * kQBlockBytes + 32 * ks) >> 4)), id1, 1u);
            }
          }
          if (dense) ++gt; else ++gg;
          if (lead) {
            umma_commit(&c->s_full[sb]);
            if (j == pc.tiles - 1) umma_commit(&c->q_empty);
          }
          __syncwarp();
          if (!ok) break;
          ok = warp_wait(&c->p_ready[sb], (g >> 1) & 1, c, a.status);
          if (ok && j == 0 && qc >= 1) ok = warp_wait(&c->o_empty, (qc - 1) & 1, c, a.status);
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int m = kPairs - 1; m >= 0; --m) {
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                umma_f16_ss(tmem + 128 + 64 * m, desc(hA2, a2 + ((2 * m * kSlotBytes + 2048 * ks) >> 4)),
                            desc(hP, p2 + ((256 * ks) >> 4)), id2, (j > 0 || ks > 0) ? 1u : 0u);
              umma_commit(&c->empty[m]);
            }
          }
          __syncwarp();
          ++g;
        }
        if (lead) umma_commit(&c->o_full);
        ++qc;
      }
      if (lead) umma_commit(&c->fin);                        // every product completes before TMEM is released
      mbar_wait(&c->fin, 0, &c->abort, a.status, 200000000ull);
    }
    __syncwarp();
  } else if (warp < 4 || warp >= 12) {
    // ------------------------------------------------------------ key rows
    const int gw = warp < 4 ? warp - 2 : warp - 10;
    const int chunk = lane & 7;
    int qc = 0, g = 0;
    bool ok = true;
    while (ok) {
      const int is = qc & 1;
      ok = warp_wait(&c->info_full[is], (qc >> 1) & 1, c, a.status);
      const Piece pc = c->info[is];
      warp_arrive(&c->info_empty[is], lane);
      if (!ok || pc.done) break;
      const TreeRow r = tree_row(a, pc.row);
      const int4 bits = *reinterpret_cast<const int4*>(a.plan + (size_t)pc.row * kPlanWords + 4);
      // lane i looks after key row 32 gw + i of a tile
      auto look_up = [&](int j) {
        return key_row(a, r, bits, pc.row, (long long)(pc.tile0 + j) * kTile + 32 * gw + lane);
      };
      const bf16* next = look_up(0);
      for (int j = 0; j < pc.tiles && ok; ++j) {
        const bf16* src = next;
        const uint32_t live = __ballot_sync(0xffffffffu, src != nullptr);
        if (lane == 0) {
          // tile g - 2's bits have been read: its O products completed before
          // this warp could fill the slots of tile g - 1
          c->valid[g & 1][gw] = live;
          mbar_arrive(&c->valid_full[g & 1]);
        }
        const bf16* rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          rows[i] = reinterpret_cast<const bf16*>(
              __shfl_sync(0xffffffffu, (unsigned long long)src, 4 * i + (lane >> 3)));
        for (int m = kPairs - 1; m >= 0; --m) {
          if (g >= 1) ok = warp_wait(&c->empty[m], (g - 1) & 1, c, a.status);
          if (!ok) break;
          if (j < pc.dense) continue;               // arrives as page runs
          const uint32_t d0 = smem_u32(smem + OFF_SLOT + 2 * m * kSlotBytes);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int row = 32 * gw + 4 * i + (lane >> 3);
            const bool key = rows[i] != nullptr;
            const bf16* from = key ? rows[i] + m * 128 + chunk * 8 : reinterpret_cast<const bf16*>(a.q);
            const uint32_t to = d0 + row * 128 + ((chunk ^ (row & 7)) << 4);
            cp_async_16_or_zero(to, from, key);
            cp_async_16_or_zero(to + kSlotBytes, from + (key ? 64 : 0), key);
          }
          cp_async_mbar_arrive(&c->full_g[m]);
        }
        // Rows of the next tile are looked up while this one is in use, and asked
        // into L2: only one tile fits in shared memory, too few bytes in flight to
        // cover the latency of HBM (16 ragged rows over all their tokens: 105 us
        // without, 93 with).
        if (j + 1 < pc.tiles) {
          next = look_up(j + 1);
          if (next != nullptr)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(next), "r"(kD * 2) : "memory");
        }
        ++g;
      }
      ++qc;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else {
    // ------------------------------------------------------------ softmax and output
    const int ts = threadIdx.x - 128;         // 0..255
    const int quarter = warp & 3;             // TMEM lane quarter
    const int hh = (warp - 4) >> 2;           // head half
    const int h0 = 32 * hh;
    const int krow = 32 * quarter + lane;     // key row / dim row owned in TMEM
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const float c1 = a.scale * kLog2e;
    const uint64_t F = ts < kR / 2 ? turn_fraction(a.inv_freq[ts]) : 0;
    const auto fmax2 = [](float x, float y) { return fmaxf(x, y); };
    const auto fadd2 = [](float x, float y) { return x + y; };

    // The next piece, unless a warp's wait for it gave up: what that one has read
    // is none, and addresses nothing.
    auto next_piece = [&](int qc, Piece& pc) -> bool {
      const int is = qc & 1;
      const bool ok = warp_wait(&c->info_full[is], (qc >> 1) & 1, c, a.status);
      pc = c->info[is];
      const bool last = !ok || pc.done;
      warp_arrive(&c->info_empty[is], lane);
      if (!last && ts < kR / 2) {
        float cs, sn;
        turn_cos_sin(a.plan[(size_t)pc.row * kPlanWords + 2], F, &cs, &sn);
        c->cs[is][ts] = make_float2(cs, sn);
      }
      return !bar_any(1, kSoftThreads, last);
    };
    // Rotate the last 64 dims of each head (four threads a head), as a high
    // and a low bf16 term.
    auto setup_query = [&](int qc) {
      const int h = ts >> 2, part = ts & 3;
      warp_wait(&c->q_full, qc & 1, c, a.status);
      uint8_t* hi_row = smem + OFF_Q + 7 * kQBlockBytes + h * 128;
      uint8_t* lo_row = smem + OFF_Q + 8 * kQBlockBytes + h * 128;
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        const int ch = 2 * part + cc;                        // 16-byte chunk of dims 448..511
        const int at = (ch ^ (h & 7)) * 16;
        uint4 u = *reinterpret_cast<uint4*>(hi_row + at), v;
        __nv_bfloat162* hv = reinterpret_cast<__nv_bfloat162*>(&u);
        __nv_bfloat162* lv = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 cs = c->cs[qc & 1][4 * ch + i];
          float2 f = __bfloat1622float2(hv[i]);
          rot_pair(f.x, f.y, cs.x, cs.y);
          hv[i] = __floats2bfloat162_rn(f.x, f.y);
          const float2 b = __bfloat1622float2(hv[i]);
          lv[i] = __floats2bfloat162_rn(f.x - b.x, f.y - b.y);
        }
        *reinterpret_cast<uint4*>(hi_row + at) = u;
        *reinterpret_cast<uint4*>(lo_row + at) = v;
      }
      fence_proxy_async_smem();
      warp_arrive(&c->q_ready, lane);
    };

    int qc = 0, g = 0;
    Piece pc;
    bool more = next_piece(0, pc);
    if (more) setup_query(0);
    while (more) {
      float lsum[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) lsum[i] = 0.f;
      for (int j = 0; j < pc.tiles; ++j) {
        const int sb = g & 1;
        warp_wait(&c->valid_full[sb], (g >> 1) & 1, c, a.status);
        const bool valid = (c->valid[sb][quarter] >> lane) & 1u;
        warp_wait(&c->s_full[sb], (g >> 1) & 1, c, a.status);
        tc_fence_after();
        // x = logit (log2 units) minus the head's shift, the exponent's argument
        float x[32];
        tmem_ld32(tmem + lane_base + 64 * sb + h0, x);
        tmem_wait_ld();
        bool raise = j == 0;
        if (j > 0) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(&c->m[h0 + i]);
            x[i] = fmaf(x[i], c1, -m4.x);
            x[i + 1] = fmaf(x[i + 1], c1, -m4.y);
            x[i + 2] = fmaf(x[i + 2], c1, -m4.z);
            x[i + 3] = fmaf(x[i + 3], c1, -m4.w);
            top = fmaxf(fmaxf(top, fmaxf(x[i], x[i + 1])), fmaxf(x[i + 2], x[i + 3]));
          }
          raise = bar_any(2 + hh, 128, valid && top > kRaise);
        }
        if (raise) {
          // set this half's shifts to the running maximum (a piece's first tile,
          // rarely a later one) and rescale
          if (j > 0) {
            tmem_ld32(tmem + lane_base + 64 * sb + h0, x);      // the logits again
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = valid ? x[i] * c1 : -INFINITY;
          const float mine = fold_lanes(x, lane, fmax2);
          const int hd = h0 + lane;
          const float old = j == 0 ? -INFINITY : c->m[hd];
          c->hmax[quarter][hd] = mine;
          named_bar_sync(2 + hh, 128);            // every warp has also read the old shifts
          const float m = fmaxf(fmaxf(fmaxf(c->hmax[0][hd], c->hmax[1][hd]), fmaxf(c->hmax[2][hd], c->hmax[3][hd])), old);
          c->m[hd] = m;                           // the same value from each of the half's warps
          c->fac[hd] = old == m ? 1.f : ex2_approx(old - m);
          __syncwarp();
          if (j > 0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) lsum[i] *= c->fac[h0 + i];
            for (int mb = 0; mb < 4; ++mb) {      // the products into O^T so far completed before S
              tmem_ld32(tmem + lane_base + 128 + 64 * mb + h0, x);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) x[i] *= c->fac[h0 + i];
              tmem_st32(tmem + lane_base + 128 + 64 * mb + h0, x);
            }
          }
          tmem_ld32(tmem + lane_base + 64 * sb + h0, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            const float4 m4 = *reinterpret_cast<const float4*>(&c->m[h0 + i]);
            x[i] = fmaf(x[i], c1, -m4.x);
            x[i + 1] = fmaf(x[i + 1], c1, -m4.y);
            x[i + 2] = fmaf(x[i + 2], c1, -m4.z);
            x[i + 3] = fmaf(x[i + 3], c1, -m4.w);
          }
        }
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const float p0 = valid ? ex2_approx(x[i]) : 0.f;
          const float p1 = valid ? ex2_approx(x[i + 1]) : 0.f;
          // denominators from the unrounded values: the roundings of P average
          // out in the output, and lse stays exact to fp32
          lsum[i] += p0;
          lsum[i + 1] += p1;
          pk[i / 2] = pack_bf16x2(p0, p1);
        }
        // P^T [8-head column block][key].  One buffer: this tile's S completing
        // implies that the previous tile's O products have completed.
        uint8_t* prow = smem + OFF_P + krow * 16 + (4 * hh) * 2048;
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          *reinterpret_cast<uint4*>(prow + cc * 2048) =
              make_uint4(pk[4 * cc], pk[4 * cc + 1], pk[4 * cc + 2], pk[4 * cc + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(&c->p_ready[sb], lane);
        ++g;
      }
      // denominators of this piece, and its shifts
      c->part_l[quarter][h0 + lane] = fold_lanes(lsum, lane, fadd2);
      named_bar_sync(1, kSoftThreads);
      float m_row = 0.f, l_row = 0.f;
      if (ts < kH) {
        m_row = c->m[ts];
        l_row = (c->part_l[0][ts] + c->part_l[1][ts]) + (c->part_l[2][ts] + c->part_l[3][ts]);
      }
      const Piece cur = pc;
      const int par = qc & 1;
      // the next piece's queries go first, so that its first products overlap
      // this piece's output
      more = next_piece(qc + 1, pc);
      if (more) setup_query(qc + 1);

      const size_t orow = (size_t)cur.row * a.H + kH * cur.hs;
      PartHead* head = nullptr;
      float* part = nullptr;
      if (cur.part >= 0) {
        char* at = p.parts + (size_t)cur.part * kPartBytes;
        part = reinterpret_cast<float*>(at);
        head = reinterpret_cast<PartHead*>(at + kPartFloats * 4);
        if (ts < kH) {
          head->m[ts] = m_row;
          head->l[ts] = l_row;
        }
      } else {
        if (ts < kH) {
          float m = m_row, l = l_row, f = 1.f;
          if (a.sink != nullptr) {
            const float s2 = a.sink[kH * cur.hs + ts] * kLog2e;
            m = fmaxf(m_row, s2);
            f = m_row == m ? 1.f : ex2_approx(m_row - m);
            l = l_row * f + sink_mass(s2, m);
          }
          c->inv[ts] = l == 0.f ? 0.f : f / l;
          if (a.lse) a.lse[orow + ts] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
        }
        named_bar_sync(1, kSoftThreads);
      }
      warp_wait(&c->o_full, par, c, a.status);
      tc_fence_after();
      bf16* opair = reinterpret_cast<bf16*>(a.o) + (orow + h0 + (lane & 1)) * kD + (krow & ~1);
      for (int m = 0; m < 4; ++m) {
        float v[32];
        tmem_ld32(tmem + lane_base + 128 + 64 * m + h0, v);
        tmem_wait_ld();
        if (m == 3) {
          tc_fence_before();
          warp_arrive(&c->o_empty, lane);
        }
        if (part != nullptr) {
#pragma unroll
          for (int i = 0; i < 32; ++i) part[(size_t)(h0 + i) * kD + 128 * m + krow] = v[i];
          continue;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] *= c->inv[h0 + i];
        if (m == 3 && quarter >= 2) {             // dims 448..511 turn back; the pair's partner is the next lane
          const float2 cs = c->cs[par][(krow - 64) >> 1];
          const bool odd = lane & 1;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float other = __shfl_xor_sync(0xffffffffu, v[i], 1);
            v[i] = odd ? v[i] * cs.x - other * cs.y : v[i] * cs.x + other * cs.y;
          }
        }
        // two heads at a time: lanes of a pair of dims exchange, the even one
        // stores both dims of the first head, the odd one of the second (half
        // the stores, and packed conversions)
#pragma unroll
        for (int i = 0; i < 32; i += 2) {
          const uint32_t own = pack_bf16x2(v[i], v[i + 1]);
          const uint32_t oth = __shfl_xor_sync(0xffffffffu, own, 1);
          *reinterpret_cast<uint32_t*>(opair + (size_t)i * kD + 128 * m) =
              (lane & 1) ? __byte_perm(oth, own, 0x7632) : __byte_perm(own, oth, 0x5410);
        }
      }
      named_bar_sync(1, kSoftThreads);            // this piece's shifts and factors are read
      ++qc;
    }
  }

  tc_fence_before();
  start_next();
  __syncthreads();
  if (c->abort && threadIdx.x == 0) {           // bulk copies that were asked for land before the block goes
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 200000) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Join of cut items: sum_s 2^(m_s - m) O_s / sum_s 2^(m_s - m) l_s over an item's
// parts.  An item in few parts is taken by the thread blocks (its first block,
// eight heads), a warp for each head with 16 dims a lane.  One in more than
// kJoinSerial parts has as many blocks behind its first that own nothing else:
// the first eight of them take one head each, a warp every eighth part, and add
// up in shared memory: one row over 131072 tokens, 147 parts, takes 62 us in both
// kernels, 100 with a block for eight heads of any item; 16 ragged rows over all
// their tokens 92 against 95.  Eight parts is where the two ways cross (four: 94).
// Launched while the attention kernel drains (programmatic dependence) and
// waits for its end before it reads anything.
// ---------------------------------------------------------------------------
constexpr int kJoinHeads = 8, kJoinSerial = 8;

__global__ void __launch_bounds__(kJoinHeads * 32) tree_join_kernel(const Args p) {
  __shared__ float4 s_o[kJoinHeads][kD / 4];
  after_previous();
  const TreeArgs& a = p.t;
  const int4 cut = p.cuts[blockIdx.x];
  const int item = cut.x, first = cut.y, last = cut.z, which = blockIdx.x - first;
  if (item < 0) return;
  const bool serial = last - first < kJoinSerial;
  if (which >= (serial ? 1 : kJoinHeads)) return;
  const int row = item / p.HS, hs = item % p.HS;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = a.plan[(size_t)row * kPlanWords + 2];
  // the first block holds the item from tile 0 (its second place), the others
  // begin inside it (their first place)
  auto place = [&](int cta) { return p.parts + (size_t)(2 * cta + (cta == first ? 1 : 0)) * kPartBytes; };
  auto head = [&](int cta) { return reinterpret_cast<const PartHead*>(place(cta) + kPartFloats * 4); };
  // one pair of dims, divided by l: the rotated ones turned back
  auto finish = [&](float x0, float x1, int dim) {
    if (dim >= kD - kR) {
      float cs, sn;
      turn_cos_sin(t, turn_fraction(a.inv_freq[(dim - (kD - kR)) / 2]), &cs, &sn);
      rot_pair(x0, x1, cs, -sn);
    }
    return pack_bf16x2(x0, x1);
  };
  if (serial) {
    const int h = blockIdx.y * kJoinHeads + warp;
    const size_t orow = (size_t)row * a.H + kH * hs + h;
    const float s2 = a.sink != nullptr ? a.sink[kH * hs + h] * kLog2e : -INFINITY;
    float m = s2;
    for (int s = first; s <= last; ++s) m = fmaxf(m, head(s)->m[h]);
    float l = sink_mass(s2, m);
    float o[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = 0.f;
    for (int s = first; s <= last; ++s) {
      const float ms = head(s)->m[h];
      const float f = ms == m ? 1.f : ex2_approx(ms - m);
      l = fmaf(head(s)->l[h], f, l);
      const float4* src =
          reinterpret_cast<const float4*>(reinterpret_cast<const float*>(place(s)) + (size_t)h * kD) + lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = src[32 * i];
        o[4 * i] = fmaf(v.x, f, o[4 * i]);
        o[4 * i + 1] = fmaf(v.y, f, o[4 * i + 1]);
        o[4 * i + 2] = fmaf(v.z, f, o[4 * i + 2]);
        o[4 * i + 3] = fmaf(v.w, f, o[4 * i + 3]);
      }
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (a.lse && lane == 0) a.lse[orow] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int dim = 128 * i + 4 * lane;
      uint2 u;
      u.x = finish(o[4 * i] * inv, o[4 * i + 1] * inv, dim);
      u.y = finish(o[4 * i + 2] * inv, o[4 * i + 3] * inv, dim + 2);
      *reinterpret_cast<uint2*>(reinterpret_cast<bf16*>(a.o) + orow * kD + dim) = u;
    }
    return;
  }
  const int h = blockIdx.y * kJoinHeads + which;
  const size_t orow = (size_t)row * a.H + kH * hs + h;
  const float s2 = a.sink != nullptr ? a.sink[kH * hs + h] * kLog2e : -INFINITY;
  float m = s2;
  for (int s = first + lane; s <= last; s += 32) m = fmaxf(m, head(s)->m[h]);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  float l = 0.f;
  for (int s = first + lane; s <= last; s += 32) {
    const float ms = head(s)->m[h];
    l = fmaf(head(s)->l[h], ms == m ? 1.f : ex2_approx(ms - m), l);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  l += sink_mass(s2, m);
  float4 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int s = first + warp; s <= last; s += kJoinHeads) {
    const float ms = head(s)->m[h];
    const float f = ms == m ? 1.f : ex2_approx(ms - m);
    const float4* src =
        reinterpret_cast<const float4*>(reinterpret_cast<const float*>(place(s)) + (size_t)h * kD) + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = src[32 * i];
      o[i].x = fmaf(v.x, f, o[i].x);
      o[i].y = fmaf(v.y, f, o[i].y);
      o[i].z = fmaf(v.z, f, o[i].z);
      o[i].w = fmaf(v.w, f, o[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s_o[warp][32 * i + lane] = o[i];
  __syncthreads();
  float2 x = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kJoinHeads; ++w) {
    const float2 v = reinterpret_cast<const float2*>(s_o[w])[threadIdx.x];
    x.x += v.x;
    x.y += v.y;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if (a.lse && threadIdx.x == 0) a.lse[orow] = l == 0.f ? -INFINITY : m * kLn2 + logf(l);
  const int dim = 2 * threadIdx.x;
  *reinterpret_cast<uint32_t*>(reinterpret_cast<bf16*>(a.o) + orow * kD + dim) = finish(x.x * inv, x.y * inv, dim);
}

}  // namespace

bool tree_tc_supported(const v4_config& c) {
  return c.dtype == V4_BF16 && c.n_heads >= kH && c.n_heads % kH == 0 && c.n_heads <= 8 * kH && c.head_dim == kD &&
         c.rope_dim == kR;
}

size_t tree_tc_workspace() {
  return (size_t)2 * kMaxCtas * kPartBytes + ((kMaxCtas * sizeof(int4) + 255) & ~(size_t)255);
}

cudaError_t launch_tree_tc(const TreeArgs& a, void* workspace, cudaStream_t st) {
  Args p;
  p.t = a;
  p.HS = a.H / kH;
  p.items = a.n_rows * p.HS;
  // Key lists begin with every entry (no selection) or with every token (no
  // entries, no window): those come page run by page run, in TMA boxes of the
  // largest power of two that divides the page (at least the 8 rows of a
  // swizzle atom).  A window or a selection starts anywhere and is gathered.
  p.dense_tok = a.ratio == 0 && a.window < 0;
  p.box = 0;
  if (p.dense_tok || (a.ratio > 0 && a.K == 0)) {
    const int page = p.dense_tok ? a.tok_page : a.ent_page;
    int box = kTile;
    while (page % box) box >>= 1;
    if (box >= 8) p.box = box;
  }
  p.parts = (char*)workspace;
  p.cuts = (int4*)((char*)workspace + (size_t)2 * kMaxCtas * kPartBytes);
  CUtensorMap mq, mp;
  if (make_tmap_bf16_2d(&mq, a.q, kD, (uint64_t)a.n_rows * a.H, 64, 64, true)) return cudaErrorInvalidValue;
  mp = mq;
  if (p.box && make_tmap_bf16_2d(&mp, p.dense_tok ? a.tok_cache : a.ent_cache, kD,
                                 (uint64_t)(p.dense_tok ? a.tok_slots : a.ent_slots), 64, p.box, true))
    return cudaErrorInvalidValue;
  static OncePerDevice once;
  static std::atomic<int> sm_count[128];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 128) return cudaErrorInvalidDevice;
  e = once.run([&] {
    int sms = 0;
    cudaError_t r = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (r != cudaSuccess) return r;
    sm_count[dev].store(sms, std::memory_order_relaxed);
    return cudaFuncSetAttribute(tree_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  const int sms = sm_count[dev].load(std::memory_order_relaxed);
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  {
    StageTiming ps(16, st);
    e = launch_overlapped(tree_tc_kernel, dim3(grid), dim3(kThreads), kSmemBytes, st, mq, mp, p);
    if (e != cudaSuccess) return e;
    note_launch();
  }
  {
    StageTiming ps(17, st);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, kH / kJoinHeads);
    cfg.blockDim = dim3(kJoinHeads * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_join_kernel, (const Args)p);
    if (e != cudaSuccess) return e;
    note_launch();
  }
  return cudaSuccess;
}

}  // namespace v4
