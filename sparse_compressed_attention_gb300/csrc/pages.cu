// Pages of a cache: giving, sharing (fork), releasing them, copying rows of one
// page to another and moving kept rows together (v4_pages_*).
//
// ref[p] counts the table entries that hold page p; a page with ref 0 is free, and
// the lowest free pages are given first, so a call's result depends on its inputs
// alone.  Counts change by integer atomics, whose order changes nothing.
#include "common.cuh"
#include "fastdiv.cuh"
#include "internal.h"

namespace v4 {

namespace {

// ---------------------------------------------------------------------------
// Giving pages.  One block: a warp counts the entries that a sequence wants, a
// block scan numbers them, the block walks ref from page 0 and lists free pages
// (kList at a time), and the warps hand them out in order.
// ---------------------------------------------------------------------------
constexpr int kGiveThreads = 1024, kGiveWarps = kGiveThreads / 32;
constexpr int kMaxSeqs = 8192;                   // sequences of a call
constexpr int kList = 8192;

struct GiveShared {
  int before[kMaxSeqs + 1];                      // wanted entries of the sequences before
  int list[kList];
  int warp_sum[kGiveWarps];
};

// Exclusive sum of v over the block's threads; the total of all in *total.
__device__ __forceinline__ int block_scan(int v, GiveShared* sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += u;
  }
  __syncthreads();
  if (lane == 31) sh->warp_sum[warp] = s;
  __syncthreads();
  int w = sh->warp_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  *total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return s - v + (warp > 0 ? before : 0);
}

// Counts of four pages; those behind the last are not free.
__device__ __forceinline__ int4 four_counts(const int* ref, int pages, int p0) {
  int4 r = make_int4(1, 1, 1, 1);
  if (p0 + 3 < pages) {
    r = *reinterpret_cast<const int4*>(ref + p0);
  } else if (p0 < pages) {
    r.x = ref[p0];
    if (p0 + 1 < pages) r.y = ref[p0 + 1];
    if (p0 + 2 < pages) r.z = ref[p0 + 2];
  }
  return r;
}

// The lowest free pages, up to `want` <= kList of them, in sh->list; *chunk is the page
// from which the walk goes on.  Ends with a barrier.
// ahead: this thread's counts of that chunk where they were asked for before, else null.
__device__ int list_free(const int* ref, int pages, int want, int* chunk, GiveShared* sh, const int4* ahead) {
  int found = 0;
  while (found < want && *chunk < pages) {
    const int p0 = *chunk + 4 * (int)threadIdx.x;
    const int4 r = ahead ? *ahead : four_counts(ref, pages, p0);
    ahead = nullptr;
    const int f[4] = {r.x == 0, r.y == 0, r.z == 0, r.w == 0};
    int all;
    int at = found + block_scan(f[0] + f[1] + f[2] + f[3], sh, &all);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (f[e] && at < want) sh->list[at] = p0 + e;
      at += f[e];
    }
    found += all;
    if (found <= want) *chunk += 4 * kGiveThreads;        // else some of it is left for the next list
  }
  __syncthreads();
  return min(found, want);
}

// count(i): entries that sequence i wants (a whole warp asks, every lane gets it).
// give(i, first, lo, hi, list): hand list[r - lo] to the wanted entries number r in
// [lo, hi), the first entry not yet served having number `first`.
template <typename Count, typename Give>
__device__ void give_pages(int n, int* ref, int pages, int* lack, int* status, GiveShared* sh, Count count, Give give) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = warp; i < n; i += kGiveWarps) {
    const int c = count(i);
    if (lane == 0) sh->before[i] = c;
  }
  __syncthreads();
  int total = 0;
  for (int i0 = 0; i0 < n; i0 += kGiveThreads) {
    const int i = i0 + (int)threadIdx.x;
    const int c = i < n ? sh->before[i] : 0;
    int all;
    const int at = total + block_scan(c, sh, &all);
    if (i < n) sh->before[i] = at;
    total += all;
  }
  if (threadIdx.x == 0) sh->before[n] = total;
  __syncthreads();
  int given = 0;                                 // numbers below have their page
  int chunk = 0;                                 // first page of the next chunk
  while (given < total) {
    const int found = list_free(ref, pages, min(kList, total - given), &chunk, sh, nullptr);
    if (found == 0) break;
    for (int i = warp; i < n; i += kGiveWarps) {
      const int lo = sh->before[i], hi = sh->before[i + 1];
      if (max(lo, given) < min(hi, given + found)) give(i, max(lo, given), given, given + found, sh->list);
    }
    given += found;
    __syncthreads();                             // the given pages' counts are seen by the next walk
  }
  if (threadIdx.x == 0) {
    if (lack) *lack = total - given;
    else if (given < total) set_status(status, kStatusBadIndex);
  }
}

struct AllocArgs {
  int32_t* table;
  const int32_t *have, *need;
  int32_t *ref, *lack;
  int* status;
  int n, blocks, page, pages;
};

__global__ void __launch_bounds__(kGiveThreads) pages_alloc_kernel(const AllocArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  GiveShared* sh = reinterpret_cast<GiveShared*>(smem);
  after_previous();
  const int lane = threadIdx.x & 31;
  // blocks [lo, hi) of a sequence
  auto range = [&](int i, int* lo, int* hi) {
    const long long have = p.have ? p.have[i] : 0, need = p.need[i];
    *lo = *hi = 0;
    if (have < 0 || need < 0 || (max(have, need) + p.page - 1) / p.page > p.blocks) {
      set_status(p.status, kStatusBadIndex);
      return;
    }
    *lo = (int)((have + p.page - 1) / p.page);
    *hi = (int)((need + p.page - 1) / p.page);
  };
  give_pages(
      p.n, p.ref, p.pages, p.lack, p.status, sh,
      [&](int i) {
        int lo, hi, c = 0;
        range(i, &lo, &hi);
        for (int k = lo; k < hi; k += 32) {
          int32_t* at = p.table + (size_t)i * p.blocks + k + lane;
          const int pg = k + lane < hi ? *at : 0;
          if (pg < -1 || pg >= p.pages) {         // no page of the pool: taken for -1
            set_status(p.status, kStatusBadIndex);
            *at = -1;
          }
          c += __popc(__ballot_sync(0xffffffffu, pg < 0 || pg >= p.pages));
        }
        return c;
      },
      [&](int i, int first, int from, int to, const int* list) {
        int lo, hi;
        range(i, &lo, &hi);
        for (int k = lo; k < hi && first < to; k += 32) {
          int32_t* at = p.table + (size_t)i * p.blocks + k + lane;
          const bool want = k + lane < hi && *at == -1;
          const uint32_t vote = __ballot_sync(0xffffffffu, want);
          const int r = first + __popc(vote & ((1u << lane) - 1u));
          if (want && r < to) {
            const int pg = list[r - from];
            *at = pg;
            p.ref[pg] = 1;
          }
          first += __popc(vote);
        }
      });
}

// ---------------------------------------------------------------------------
// Fork.  The whole pages are shared, the partly filled last ones get a free page each.
// While pages are shared a count of 0 stays 0 and others only rise, and the pages given
// are written when that is over: what is held and what is free are the counts' at the
// call's start, whatever the order of blocks.  (Without that order a page that a table
// names though its count is 0 could be shared and given out at once.)
// ---------------------------------------------------------------------------
constexpr int kForkThreads = kGiveThreads, kForkRounds = kMaxSeqs / kForkThreads;
static_assert(kMaxSeqs <= kList, "one list serves all beams");
// One launch of one cluster while its sharing blocks have two entries a thread at most, two
// launches above.  A release and a fork, one launch against two: 64 beams of 32 blocks 6.5
// and 8.8 us, 256 of 64 9.0 and 9.4, 512 of 64 13.1 and 11.2, 8192 of 64 126 and 58.
constexpr int kClusterBlocks = 8, kForkCluster = 2 * (kClusterBlocks - 1);

struct ForkArgs {
  const int32_t *table, *src, *len;
  int32_t *out, *ref, *copies, *lack;
  int* status;
  long long items;                               // n * out_blocks
  int B, blocks, n, out_blocks, page, pages;
  FastDiv by_out;
};

// Whole blocks and rows of the last of beam i; false: nothing is shared.
__device__ __forceinline__ bool fork_row(const ForkArgs& p, int i, int* src, int* full, int* rest) {
  const int s = p.src[i], L = p.len[i];
  *src = s;
  *full = *rest = 0;
  if (s == -1) return false;
  const long long used = ((long long)L + p.page - 1) / p.page;
  if (s < 0 || s >= p.B || L < 0 || used > p.blocks || used > p.out_blocks) {
    set_status(p.status, kStatusBadIndex);
    return false;
  }
  *full = L / p.page;
  *rest = L - *full * p.page;
  return true;
}

// Page of block k, -1 (flagged) where it is none of the pool's or free.
__device__ __forceinline__ int fork_page(const ForkArgs& p, int src, int k) {
  const int pg = p.table[(size_t)src * p.blocks + k];
  if (pg == -1 || (pg >= 0 && pg < p.pages && p.ref[pg] > 0)) return pg;
  set_status(p.status, kStatusBadIndex);
  return -1;
}

// The share of one of `blocks` thread blocks in the whole pages and the empty entries.
__device__ __forceinline__ void fork_share(const ForkArgs& p, int block, int blocks) {
  for (long long j = (long long)block * kForkThreads + threadIdx.x; j < p.items; j += (long long)blocks * kForkThreads) {
    const int i = (int)p.by_out.div((uint32_t)j), k = (int)(j - (long long)i * p.out_blocks);
    int src, full, rest, pg = -1;
    const bool live = fork_row(p, i, &src, &full, &rest);
    if (live && k == full && rest > 0) continue;         // gets a page of its own
    if (live && k < full) {
      pg = fork_page(p, src, k);
      if (pg >= 0) atomicAdd(p.ref + pg, 1);
    }
    p.out[j] = pg;
  }
}

__global__ void __launch_bounds__(kForkThreads) pages_share_kernel(const ForkArgs p) {
  after_previous();
  fork_share(p, blockIdx.x, gridDim.x);
}

// A thread for each beam, 1024 at a time.  kCluster: one launch of one cluster, whose first
// block gives while the others share; else the second launch, behind pages_share_kernel.
template <bool kCluster>
__global__ void __launch_bounds__(kForkThreads) pages_fork_kernel(const ForkArgs p) {
  extern __shared__ __align__(16) uint8_t smem[];
  GiveShared* sh = reinterpret_cast<GiveShared*>(smem);
  const int t = threadIdx.x;
  after_previous();
  auto all_shared = [] {
    if (kCluster)
      asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  if (kCluster && blockIdx.x > 0) {
    fork_share(p, blockIdx.x - 1, gridDim.x - 1);
    __syncwarp();
    all_shared();
    return;
  }
  const int4 ahead = four_counts(p.ref, p.pages, 4 * t);         // asked for beside the beams' rows
  int old[kForkRounds], full[kForkRounds], rest[kForkRounds], at[kForkRounds];
  int wanted = 0, chunk = 0;
#pragma unroll
  for (int k = 0; k < kForkRounds; ++k) {
    const int i = k * kForkThreads + t;
    old[k] = -1;
    full[k] = rest[k] = at[k] = 0;
    if (k * kForkThreads >= p.n) continue;               // the same for all threads
    int src, want;
    if (i < p.n && fork_row(p, i, &src, &full[k], &rest[k]) && rest[k] > 0) old[k] = fork_page(p, src, full[k]);
    at[k] = wanted + block_scan(old[k] >= 0, sh, &want);
    wanted += want;
  }
  const int given = list_free(p.ref, p.pages, wanted, &chunk, sh, &ahead);
  all_shared();
#pragma unroll
  for (int k = 0; k < kForkRounds; ++k) {
    const int i = k * kForkThreads + t;
    if (i >= p.n) continue;
    const int pg = old[k] >= 0 && at[k] < given ? sh->list[at[k]] : -1;
    if (pg >= 0) p.ref[pg] = 1;
    if (rest[k] > 0) p.out[(size_t)i * p.out_blocks + full[k]] = pg;
    p.copies[3 * i] = pg >= 0 ? old[k] : -1;
    p.copies[3 * i + 1] = pg;
    p.copies[3 * i + 2] = pg >= 0 ? rest[k] : 0;
  }
  if (t == 0) {
    if (p.lack) *p.lack = wanted - given;
    else if (given < wanted) set_status(p.status, kStatusBadIndex);
  }
}

// ---------------------------------------------------------------------------
// Release: entries whose block holds no token in [lo, hi).
// ---------------------------------------------------------------------------
struct FreeArgs {
  int32_t *table, *ref;
  const int32_t *lo, *hi;
  int* status;
  long long items;
  int blocks, page, pages;
  FastDiv by_blocks;
};

__global__ void __launch_bounds__(256) pages_free_kernel(const FreeArgs p) {
  after_previous();
  const long long j = (long long)blockIdx.x * 256 + threadIdx.x;
  if (j >= p.items) return;
  const int pg = p.table[j];
  if (pg == -1) return;
  const int i = (int)p.by_blocks.div((uint32_t)j);
  const long long k = j - (long long)i * p.blocks;
  const long long lo = p.lo ? p.lo[i] : 0, hi = p.hi ? p.hi[i] : 0;
  if (k * p.page < hi && (k + 1) * p.page > lo && lo < hi) return;
  p.table[j] = -1;
  if (pg < 0 || pg >= p.pages) {
    set_status(p.status, kStatusBadIndex);
  } else if (atomicSub(p.ref + pg, 1) <= 0) {
    atomicAdd(p.ref + pg, 1);
    set_status(p.status, kStatusBadIndex);
  }
}

// ---------------------------------------------------------------------------
// Copies of rows from one page to another, in 16-byte words: a block takes 16 KB
// of a pair in one layer.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256, kCopyWords = 4;

struct CopyArgs {
  uint4* cache;
  const int32_t* copies;
  int* status;
  long long layer_words, page_words;
  int row_words, pages, page, chunks;
  FastDiv by_chunks;
};

__global__ void __launch_bounds__(kCopyThreads) pages_copy_kernel(const CopyArgs p) {
  after_previous();
  const int pair = (int)p.by_chunks.div(blockIdx.x), chunk = (int)blockIdx.x - pair * p.chunks;
  const int from = p.copies[3 * pair], to = p.copies[3 * pair + 1], rows = p.copies[3 * pair + 2];
  if (rows == 0 || (from == -1 && to == -1)) return;
  if (from < 0 || from >= p.pages || to < 0 || to >= p.pages || rows < 0 || rows > p.page) {
    set_status(p.status, kStatusBadIndex);
    return;
  }
  if (from == to) return;
  const int n = rows * p.row_words;
  const uint4* a = p.cache + blockIdx.y * p.layer_words + from * p.page_words;
  uint4* b = p.cache + blockIdx.y * p.layer_words + to * p.page_words;
  uint4 v[kCopyWords];
  const int i0 = chunk * (kCopyThreads * kCopyWords) + (int)threadIdx.x;
#pragma unroll
  for (int k = 0; k < kCopyWords; ++k)
    if (i0 + k * kCopyThreads < n) v[k] = a[i0 + k * kCopyThreads];
#pragma unroll
  for (int k = 0; k < kCopyWords; ++k)
    if (i0 + k * kCopyThreads < n) b[i0 + k * kCopyThreads] = v[k];
}

// ---------------------------------------------------------------------------
// Kept rows move together: row base + keep[i] to row base + i.  keep ascends, so a
// row never moves up, and rows are independent in every 16-byte column: a block
// takes a strip of columns of one sequence and layer and walks its rows in rounds.
// A round's words are asked for three rounds ahead by asynchronous copies (what a round writes lies below
// everything that later rounds read) and written behind a barrier that says that all
// of them have arrived.
// ---------------------------------------------------------------------------
constexpr int kKeepStages = 4;

struct KeepArgs {
  uint4* cache;
  const int32_t *table, *base, *count, *keep;
  int* status;
  long long layer_words;
  int blocks, page, pages, width, row_words, lg_strip;
  FastDiv by_page;
};

// Threads and words of a thread: many threads for long lists (half of 8 x 16000 rows of
// 1 KB in 4 layers: 88 us with 512 x 1, 106 with 128 x 2), few for short ones, where more
// blocks fit on an SM (6 of 16 rows for 32 sequences in 43 layers: 6.6 and 4.2 us).  The
// two cross somewhere above the rule's 16 rows: half of 2 n rows kept, 512 x 1 against
// 128 x 2, 32 sequences in 43 layers: n = 64 28.9 and 25.8, 256 116.5 and 121.8; 8 in 4:
// 64 3.9 and 2.8, 1024 12.7 and 11.9, 4096 47.0 and 55.8; 64 in 8: 64 11.4 and 11.1, 128 21.1
// and 21.3.
template <int kKeepThreads, int kKeepWords>
__global__ void __launch_bounds__(kKeepThreads) pages_keep_kernel(const KeepArgs p) {
  __shared__ uint4 s_ring[kKeepStages][kKeepWords][kKeepThreads];
  __shared__ int2 s_rows[kKeepStages][kKeepThreads];     // a round's rows: from, to (-1: stays)
  after_previous();
  const int b = blockIdx.x, t = threadIdx.x;
  const int n = p.count[b], base = p.base[b];
  if (n < 0 || n > p.width || base < 0) {
    if (t == 0) set_status(p.status, kStatusBadIndex);
    return;
  }
  const int strip = 1 << p.lg_strip, col0 = blockIdx.y << p.lg_strip;
  const int rows = min(kKeepThreads, (kKeepThreads * kKeepWords) >> p.lg_strip);      // of a round
  const int32_t* keep = p.keep + (size_t)b * p.width;
  const int32_t* table = p.table + (size_t)b * p.blocks;
  uint4* cache = p.cache + blockIdx.z * p.layer_words + col0;
  // A thread looks after one row of a round: its index two rounds ahead of the round's
  // copies, its pages one round ahead, so that no load of the chain is waited for.
  int next = 0, before = -1;                             // keep[i], keep[i - 1] of the next look-up
  int2 pages = make_int2(-1, -1), offset;                // pages and rows within them, from and to
  bool bad = false, here = false, moves = false;         // here: the thread has a row, which has to be held even where it stays
  auto index = [&](int round) {
    const int i = round * rows + t;
    const bool mine = t < rows && i < n;
    next = mine ? keep[i] : i;
    before = mine && i > 0 ? keep[i - 1] : -1;
  };
  auto find = [&](int round) {
    const int i = round * rows + t;
    bad = next < i || before >= next;                    // a thread without a row: next = i, before = -1
    here = t < rows && i < n && !bad;
    moves = here && next > i;
    pages = make_int2(-1, -1);
    if (here) {
      const long long at[2] = {(long long)base + next, (long long)base + i};
      int blk[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) blk[k] = at[k] < 0x7FFFFFFF ? (int)p.by_page.div((uint32_t)at[k]) : 0x7FFFFFFF;
      offset = make_int2((int)(at[0] - (long long)blk[0] * p.page), (int)(at[1] - (long long)blk[1] * p.page));
      if (blk[0] < p.blocks && blk[1] < p.blocks) pages = make_int2(table[blk[0]], table[blk[1]]);
    }
  };
  auto ask = [&](int round) {
    const int slot = round & (kKeepStages - 1);
    if (round * rows < n) {                              // the same for all threads
      int2 r = make_int2(-1, -1);
      const bool held = pages.x >= 0 && pages.x < p.pages && pages.y >= 0 && pages.y < p.pages;
      if (moves && held) r = make_int2(pages.x * p.page + offset.x, pages.y * p.page + offset.y);
      if (bad || (here && !held)) set_status(p.status, kStatusBadIndex);
      s_rows[slot][t] = r;
      __syncthreads();
      find(round + 1);
      index(round + 2);
#pragma unroll
      for (int k = 0; k < kKeepWords; ++k) {
        const int w = t + k * kKeepThreads, row = w >> p.lg_strip, col = w & (strip - 1);
        if (row >= rows || col0 + col >= p.row_words || s_rows[slot][row].y < 0) continue;
        const uint4* from = cache + (long long)s_rows[slot][row].x * p.row_words + col;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(&s_ring[slot][k][t])),
                     "l"(from)
                     : "memory");
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  index(0);
  find(0);
  index(1);
  for (int r = 0; r < kKeepStages - 1; ++r) ask(r);
  for (int r = 0; r * rows < n; ++r) {
    ask(r + kKeepStages - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(kKeepStages - 1) : "memory");
    __syncthreads();
    const int slot = r & (kKeepStages - 1);
#pragma unroll
    for (int k = 0; k < kKeepWords; ++k) {
      const int w = t + k * kKeepThreads, row = w >> p.lg_strip, col = w & (strip - 1);
      if (row >= rows || col0 + col >= p.row_words) continue;
      const int to = s_rows[slot][row].y;
      if (to >= 0) cache[(long long)to * p.row_words + col] = s_ring[slot][k][t];
    }
    __syncthreads();                                     // the round's rows are read: the slot may be taken
  }
}

cudaError_t give_shared() {
  static OncePerDevice once;
  return once.run([] {
    cudaError_t e = cudaFuncSetAttribute(pages_alloc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GiveShared));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(pages_fork_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GiveShared));
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(pages_fork_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(GiveShared));
    return e;
  });
}

}  // namespace

int pages_max_sequences() { return kMaxSeqs; }

cudaError_t launch_pages_alloc(int n, int32_t* table, int blocks, int page, const int32_t* have, const int32_t* need,
                               int32_t* ref, int pages, int32_t* lack, int* status, cudaStream_t st) {
  cudaError_t e = give_shared();
  if (e != cudaSuccess) return e;
  AllocArgs p;
  p.table = table;
  p.have = have;
  p.need = need;
  p.ref = ref;
  p.lack = lack;
  p.status = status;
  p.n = n;
  p.blocks = blocks;
  p.page = page;
  p.pages = pages;
  e = launch_overlapped(pages_alloc_kernel, dim3(1), dim3(kGiveThreads), sizeof(GiveShared), st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_pages_fork(int B, const int32_t* table, int blocks, int n, const int32_t* src, const int32_t* len,
                              int32_t* out, int out_blocks, int page, int32_t* ref, int pages, int32_t* copies,
                              int32_t* lack, int* status, cudaStream_t st) {
  cudaError_t e = give_shared();
  if (e != cudaSuccess) return e;
  ForkArgs p;
  p.table = table;
  p.src = src;
  p.len = len;
  p.out = out;
  p.ref = ref;
  p.copies = copies;
  p.lack = lack;
  p.status = status;
  p.items = (long long)n * out_blocks;
  p.B = B;
  p.blocks = blocks;
  p.n = n;
  p.out_blocks = out_blocks;
  p.page = page;
  p.pages = pages;
  p.by_out.set((uint32_t)out_blocks);
  const long long sharing = (p.items + kForkThreads - 1) / kForkThreads;       // blocks with an entry for each thread
  if (sharing <= kForkCluster) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kClusterBlocks);
    cfg.blockDim = dim3(kForkThreads);
    cfg.dynamicSmemBytes = sizeof(GiveShared);
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = kClusterBlocks;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, pages_fork_kernel<true>, (const ForkArgs)p);
    if (e == cudaSuccess) note_launch();
    return e;
  }
  e = launch_overlapped(pages_share_kernel, dim3((unsigned)(sharing < 304 ? sharing : 304)), dim3(kForkThreads), 0, st, p);
  if (e != cudaSuccess) return e;
  note_launch();
  e = launch_overlapped(pages_fork_kernel<false>, dim3(1), dim3(kForkThreads), sizeof(GiveShared), st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_pages_free(int n, int32_t* table, int blocks, int page, const int32_t* lo, const int32_t* hi,
                              int32_t* ref, int pages, int* status, cudaStream_t st) {
  FreeArgs p;
  p.table = table;
  p.ref = ref;
  p.lo = lo;
  p.hi = hi;
  p.status = status;
  p.items = (long long)n * blocks;
  p.blocks = blocks;
  p.page = page;
  p.pages = pages;
  p.by_blocks.set((uint32_t)blocks);
  const cudaError_t e =
      launch_overlapped(pages_free_kernel, dim3((unsigned)((p.items + 255) / 256)), dim3(256), 0, st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_pages_copy(void* cache, int layers, long long layer_bytes, int pages, int page, int row_bytes,
                              const int32_t* copies, int n, int* status, cudaStream_t st) {
  CopyArgs p;
  p.cache = (uint4*)cache;
  p.copies = copies;
  p.status = status;
  p.layer_words = layer_bytes / 16;
  p.row_words = row_bytes / 16;
  p.page_words = (long long)page * p.row_words;
  p.pages = pages;
  p.page = page;
  const int per = kCopyThreads * kCopyWords;
  p.chunks = (int)((p.page_words + per - 1) / per);
  p.by_chunks.set((uint32_t)p.chunks);
  const cudaError_t e = launch_overlapped(pages_copy_kernel, dim3((unsigned)(n * p.chunks), (unsigned)layers),
                                          dim3(kCopyThreads), 0, st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

cudaError_t launch_pages_compact(void* cache, int layers, long long layer_bytes, int pages, int page, int row_bytes,
                                 int n, const int32_t* table, int blocks, const int32_t* base, const int32_t* count,
                                 const int32_t* keep, int width, int* status, cudaStream_t st) {
  KeepArgs p;
  p.cache = (uint4*)cache;
  p.table = table;
  p.base = base;
  p.count = count;
  p.keep = keep;
  p.status = status;
  p.layer_words = layer_bytes / 16;
  p.blocks = blocks;
  p.page = page;
  p.pages = pages;
  p.width = width;
  p.row_words = row_bytes / 16;
  p.by_page.set((uint32_t)page);
  // strips of 1 KB, narrower while there are fewer blocks than two for each SM and a
  // strip keeps 64 bytes
  p.lg_strip = 6;
  while (p.lg_strip > 2 && ((1 << (p.lg_strip - 1)) >= p.row_words ||
                            (long long)n * layers * ((p.row_words + (1 << p.lg_strip) - 1) >> p.lg_strip) < 304))
    --p.lg_strip;
  const int strip = 1 << p.lg_strip;
  const dim3 grid((unsigned)n, (unsigned)((p.row_words + strip - 1) / strip), (unsigned)layers);
  const bool few = width <= 16;
  const cudaError_t e = launch_overlapped(few ? pages_keep_kernel<128, 2> : pages_keep_kernel<512, 1>, grid,
                                          dim3(few ? 128 : 512), 0, st, p);
  if (e == cudaSuccess) note_launch();
  return e;
}

}  // namespace v4
