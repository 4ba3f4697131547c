// zha_pages.cu -- page bookkeeping of a paged cache on the device: extend, fork,
// free and compact. Semantics are in include/zha.h.
//
// The free pages are those with reference count 0, and the r-th page a call needs
// (items, then KV heads, then blocks in order) is the r-th lowest free one. Both
// ranks are prefix sums, so that no atomic's order shows in a result. They want a few
// passes over the counts with all of a pass done before the next, so one cluster of
// up to 16 CTAs does them in one launch, with a cluster barrier between passes:
//   1  how many pages are free (in use, for compact) in each CTA's share of the
//      counts; each (item, KV head): is it valid, how many pages does it need
//   2  the shares' prefix turns every free page into list[rank]; the needs' prefix
//   3  entries and counts, with every rank known
// What moves page contents is wide: a second launch over the whole GPU, unless it is
// small enough to be done by the cluster.
// Bound: for small lists the launch and the passes' latencies (about 12 dependent accesses of
// 0.6 us: 7 us); for large ones the work of the cluster, which is at most 16 of 148 SMs: extend
// checks every block of every sequence, every CTA ranks every row and reads the needs of all
// of its item's heads, the search for duplicates walks the list once per row, and the fork's copy costs
// its instance 160 bytes of spills. The copied rows (HBM) for compact. Measured, by kernel: 48 forks of
// 128 sequences of up to 4096 tokens in 8 heads 16 us and their copies 8, all 128 extended 18; 384 forks of
// 1024 sequences 57 and 14, all extended 93; 1500 of 4000 with 2 heads 65 and 14, 121. Free, fork
// and extend of a beam of 4: 18 us on the device together; 7,300 pages of 32 KB moved in 79 us
// (6.1 TB/s of reads and writes). As three launches over the whole GPU each, extend and
// fork of the 128 took the same time on the device and 9 us more on the host.
#include <cstdio>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kPageThreads = 256;         // of the kernels over the whole GPU
constexpr int kBookThreads = 1024;        // of the cluster's CTAs
constexpr int kBookWarps = kBookThreads / 32;
constexpr int kMostCtas = 16;
// The cluster copies a fork's part-filled pages itself where a warp's page is small, and
// all of them together (a beam step of 4, 4 KB of K a page: 20.0 us on the device, without
// 20.5 and a launch more; 32 KB of K a page: 38.9 us, 24.9 without). Compact: twice the
// bytes.
constexpr int64_t kCopyHere = 256 << 10, kCopyPage = 4096;

struct PoolArgs {
  char* k;
  char* v;
  int32_t* table;
  int32_t* refs;
  int64_t n_pages, max_blocks;
  int32_t n_seqs, hkv, chunk, row_bytes;
  int32_t* status;
};

// Workspace, int32: scal[8] (total live, moves), seg[16], need, offs and copy[items *
// hkv], list[n_pages], code[n_pages] (compact).
struct PageWs {
  int32_t *scal, *seg, *need, *offs, *copy, *list, *code;
  int64_t bytes;
};

PageWs page_ws(void* base, int64_t n_pages, int64_t rows) {
  int32_t* p = static_cast<int32_t*>(base);
  PageWs w{};
  int64_t at = 0;
  auto take = [&](int64_t n) { int32_t* q = base == nullptr ? nullptr : p + at; at += round_up(n, 64); return q; };
  w.scal = take(8);
  w.seg = take(kMostCtas);
  w.need = take(rows);
  w.offs = take(rows);
  w.copy = take(rows);
  w.list = take(n_pages);
  w.code = take(n_pages);
  w.bytes = at * 4;
  return w;
}

enum { kLive = 0, kMoves = 1 };

__device__ __forceinline__ void flag(const PoolArgs& P, int bit) {
  if (P.status != nullptr) atomicOr(P.status, bit);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// All of the cluster's threads, with what they wrote to global memory. What another
// CTA wrote is then read past L1 (__ldcg).
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Exclusive prefix of v over the block's threads, and the sum of all.
template <typename I>
__device__ I block_prefix(I v, I* s_red, I* sum) {
  I x = v;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_red[warp] = x;
  __syncthreads();
  I w = s_red[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  *sum = __shfl_sync(0xffffffffu, w, kBookWarps - 1);
  return (warp == 0 ? I(0) : __shfl_sync(0xffffffffu, w, warp - 1)) + x - v;
}

__device__ __forceinline__ bool counted(int32_t refs, bool live) { return live ? refs > 0 : refs == 0; }

// a / b; 32-bit divisions take a fifth of the 64-bit ones.
__device__ __forceinline__ int64_t quotient(int64_t a, int32_t b) {
  return (a >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// This CTA's share of n things (n < 2^30), in eights.
struct Share {
  int a, b;
  __device__ explicit Share(int n) {
    const int per = (n + int(gridDim.x) * 8 - 1) / (int(gridDim.x) * 8) * 8;
    a = min(n, int(cluster_rank()) * per);
    b = min(n, a + per);
  }
};

// Which of the pages p..p + 7 below `end` count, as bits.
__device__ __forceinline__ uint32_t counted_bits(const int32_t* refs, int p, int end, bool live) {
  uint32_t bits = 0;
  if (p + 8 <= end && (reinterpret_cast<uintptr_t>(refs) & 15) == 0) {
    const int4 r[2] = {*reinterpret_cast<const int4*>(refs + p), *reinterpret_cast<const int4*>(refs + p + 4)};
#pragma unroll
    for (int i = 0; i < 2; ++i)
      bits |= (uint32_t(counted(r[i].x, live)) | uint32_t(counted(r[i].y, live)) << 1 |
               uint32_t(counted(r[i].z, live)) << 2 | uint32_t(counted(r[i].w, live)) << 3) << (4 * i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (p + i < end && counted(refs[p + i], live)) bits |= 1u << i;
  }
  return bits;
}

// Pass 1: this thread's part of the share's count. `bits` keeps the share's first
// 8192 pages' for pass 2.
__device__ int count_share(const PoolArgs& P, const Share& h, bool live, uint32_t* bits) {
  *bits = counted_bits(P.refs, h.a + int(threadIdx.x) * 8, h.b, live);
  int n = __popc(*bits);
#pragma unroll 4
  for (int p = h.a + (int(threadIdx.x) + kBookThreads) * 8; p < h.b; p += kBookThreads * 8)
    n += __popc(counted_bits(P.refs, p, h.b, live));
  return n;
}

// The sum of the CTAs' counts, and of those before this one.
__device__ int2 counts_of(const PageWs& W) {
  const int lane = threadIdx.x % 32;
  const int v = lane < int(gridDim.x) ? __ldcg(W.seg + lane) : 0;
  return make_int2(__reduce_add_sync(0xffffffffu, v),
                   __reduce_add_sync(0xffffffffu, lane < int(cluster_rank()) ? v : 0));
}

// Pass 2: f(page, counted, exclusive rank) for the share's pages.
template <typename F>
__device__ void rank_share(const PoolArgs& P, const Share& h, bool live, uint32_t bits, int base, int* s_red, F f) {
  for (int q = h.a; q < h.b; q += kBookThreads * 8) {
    const int p = q + int(threadIdx.x) * 8;
    if (q > h.a) bits = counted_bits(P.refs, p, h.b, live);
    int sum;
    int rank = base + block_prefix(int(__popc(bits)), s_red, &sum);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (p + i >= h.b) break;
      const bool c = (bits >> i) & 1u;
      f(p + i, c, rank);
      rank += c;
    }
    base += sum;
  }
}

// (All loads of a round before its stores: the compiler may not move them there.)
__device__ __forceinline__ void copy_bytes(char* to, const char* from, int64_t n, int id, int step) {
  constexpr int kRound = 8;
  const uint4* f = reinterpret_cast<const uint4*>(from);
  uint4* t = reinterpret_cast<uint4*>(to);
  for (int64_t i = id; i < n / 16; i += kRound * step) {
    uint4 x[kRound];
#pragma unroll
    for (int j = 0; j < kRound; ++j)
      if (i + j * step < n / 16) x[j] = f[i + j * step];
#pragma unroll
    for (int j = 0; j < kRound; ++j)
      if (i + j * step < n / 16) t[i + j * step] = x[j];
  }
}
__device__ __forceinline__ void copy_rows(const PoolArgs& P, int32_t to, int32_t from, int64_t rows, int id, int step) {
  const int64_t f = int64_t(from) * P.chunk * P.row_bytes, t = int64_t(to) * P.chunk * P.row_bytes;
  copy_bytes(P.k + t, P.k + f, rows * P.row_bytes, id, step);
  copy_bytes(P.v + t, P.v + f, rows * P.row_bytes, id, step);
}

// ---- extend and fork ----------------------------------------------------------
// One warp: how many pages row (item, head) needs, -1: refused. `list`: the sequences
// that the call changes.
template <bool kFork>
__device__ int row_need(const PoolArgs& P, const int32_t* src, const int32_t* list, const int64_t* tokens, int n_items,
                        int item, int g, int lane) {
  const int32_t d = list[item], s = kFork ? src[item] : d;
  const int64_t n = tokens[item];
  bool twice = false;
  for (int j = lane; j < (kFork ? n_items : item); j += 32) {
    const int32_t x = list[j];
    twice |= (j < item && x == d) || (kFork && x == s);
  }
  twice = __any_sync(0xffffffffu, twice);
  int bad = 0;
  if (d < 0 || d >= P.n_seqs || s < 0 || s >= P.n_seqs || twice) bad = ZHA_DEV_BAD_SEQUENCE;
  else if (n < 0 || n > P.max_blocks * P.chunk) bad = ZHA_DEV_BAD_LENGTH;
  int need = 0;
  if (bad == 0) {
    const int64_t full = quotient(n, P.chunk), blocks = full + (full * P.chunk != n);
    const int32_t* row = P.table + (int64_t(s) * P.hkv + g) * P.max_blocks;
    int miss = 0;
    bool wrong = false, taken = false;
#pragma unroll 4
    for (int64_t b = lane; b < blocks; b += 32) {
      const int32_t e = row[b];
      miss += e < 0;
      wrong |= e >= P.n_pages || (e >= 0 && P.refs[e] <= 0);
    }
    if (kFork) {
      const int32_t* to = P.table + (int64_t(d) * P.hkv + g) * P.max_blocks;
#pragma unroll 4
      for (int64_t b = lane; b < P.max_blocks; b += 32) taken |= to[b] >= 0;
    }
    miss = __reduce_add_sync(0xffffffffu, miss);
    wrong = __any_sync(0xffffffffu, wrong);
    taken = __any_sync(0xffffffffu, taken);
    if (kFork) {
      if (taken) bad = ZHA_DEV_BAD_SEQUENCE;
      else if (wrong || miss) bad = ZHA_DEV_BAD_PAGE;
      need = blocks != full;
    } else {
      if (wrong) bad = ZHA_DEV_BAD_PAGE;
      need = miss;
    }
  }
  if (bad && lane == 0) flag(P, bad);
  return bad ? -1 : need;
}

// One warp: the pages list[at], ... go to row (item, head) = idx.
template <bool kFork>
__device__ void fill_row(const PoolArgs& P, const PageWs& W, const int32_t* src, int32_t dst, int64_t n, int item, int g,
                         int idx, int at, bool copy_here, int lane) {
  int32_t* row = P.table + (int64_t(dst) * P.hkv + g) * P.max_blocks;
  const int64_t full = quotient(n, P.chunk), rest = n - full * P.chunk;
  if (!kFork) {
    const int64_t blocks = full + (rest != 0);
#pragma unroll 2
    for (int64_t b0 = 0; b0 < blocks; b0 += 32) {
      const int64_t b = b0 + lane;
      const bool miss = b < blocks && row[b] < 0;
      const uint32_t all = __ballot_sync(0xffffffffu, miss);
      if (miss) {
        const int32_t page = __ldcg(W.list + at + __popc(all & ((1u << lane) - 1)));
        row[b] = page;
        P.refs[page] = 1;
      }
      at += __popc(all);
    }
    return;
  }
  const int32_t* from = P.table + (int64_t(src[item]) * P.hkv + g) * P.max_blocks;
  const int32_t page = rest ? __ldcg(W.list + at) : -1;
#pragma unroll 2
  for (int64_t b = lane; b < full + (rest != 0); b += 32) {
    int32_t e = page;
    if (b < full) {
      e = from[b];
      atomicAdd(&P.refs[e], 1);
    }
    row[b] = e;
  }
  if (rest == 0) return;
  if (lane == 0) P.refs[page] = 1;
  if (copy_here) copy_rows(P, page, from[full], rest, lane, 32);
  else if (lane == 0) W.copy[idx] = page;
}

template <bool kFork>
__global__ void __launch_bounds__(kBookThreads)
    pages_items_kernel(PoolArgs P, PageWs W, const int32_t* src, const int32_t* dst, const int64_t* tokens, int n_items,
                       bool copy_here) {
  constexpr int kKeep = 1024;                                // of the list, and of this CTA's rows' offsets
  __shared__ int s_red[kBookWarps];
  __shared__ int64_t s_red64[kBookWarps];
  __shared__ int32_t s_list[kKeep], s_offs[kKeep];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, rows = n_items * P.hkv;
  const Share pages(int(P.n_pages)), mine(rows);
  const int32_t* list = n_items <= kKeep ? s_list : dst;
  int32_t* offs = mine.b - mine.a <= kKeep ? s_offs : W.offs + mine.a;
  if (n_items <= kKeep && threadIdx.x < n_items) s_list[threadIdx.x] = dst[threadIdx.x];
  uint32_t bits;
  const int n = count_share(P, pages, false, &bits);
  __syncthreads();
  for (int r = mine.a + warp; r < mine.b; r += kBookWarps) {
    const int item = r / P.hkv, need = row_need<kFork>(P, src, list, tokens, n_items, item, r - item * P.hkv, lane);
    if (lane == 0) {
      W.need[r] = need;
      if (kFork) W.copy[r] = -1;
    }
  }
  int sum;
  block_prefix(n, s_red, &sum);
  if (threadIdx.x == 0) W.seg[cluster_rank()] = sum;
  cluster_sync();
  const int2 have = counts_of(W);
  rank_share(P, pages, false, bits, have.y, s_red, [&](int p, bool c, int rank) {
    if (c) W.list[rank] = p;
  });
  // Every CTA ranks all needs and keeps its rows' offsets; a refused head refuses its
  // item (offset -1). Sums may pass 31 bits where no pool could serve them: they are
  // kept in 64, and an offset that does not fit belongs to a call that changes nothing.
  int64_t carry = 0;
  for (int r0 = 0; r0 < rows; r0 += kBookThreads) {
    const int r = r0 + threadIdx.x;
    int64_t v = 0, all;
    bool ok = false;
    if (r < rows) {
      ok = true;
      const int i0 = r / P.hkv * P.hkv;
#pragma unroll 4
      for (int g = 0; g < P.hkv; ++g) ok &= __ldcg(W.need + i0 + g) >= 0;
      v = ok ? __ldcg(W.need + r) : 0;
    }
    const int64_t at = carry + block_prefix(v, s_red64, &all);
    if (r >= mine.a && r < mine.b) offs[r - mine.a] = ok ? int32_t(min64(at, INT32_MAX)) : -1;
    carry += all;
  }
  cluster_sync();
  if (carry > have.x) {
    if (cluster_rank() == 0 && threadIdx.x == 0) flag(P, ZHA_DEV_NO_PAGES);
    return;
  }
  for (int r = mine.a + warp; r < mine.b; r += kBookWarps) {
    const int at = offs[r - mine.a], item = r / P.hkv;
    if (at >= 0) fill_row<kFork>(P, W, src, list[item], tokens[item], item, r - item * P.hkv, r, at, copy_here, lane);
  }
}

// The part-filled pages of a fork, one CTA per row.
__global__ void __launch_bounds__(kPageThreads)
    pages_copy_kernel(PoolArgs P, PageWs W, const int32_t* src, const int64_t* tokens) {
  pdl_trigger();
  pdl_wait();
  const int32_t to = W.copy[blockIdx.x];
  if (to < 0) return;
  const int item = blockIdx.x / P.hkv, g = blockIdx.x % P.hkv;
  const int64_t n = tokens[item];
  const int32_t from = P.table[(int64_t(src[item]) * P.hkv + g) * P.max_blocks + n / P.chunk];
  copy_rows(P, to, from, n % P.chunk, threadIdx.x, kPageThreads);
}

// ---- free ------------------------------------------------------------------
__global__ void __launch_bounds__(kPageThreads)
    pages_free_kernel(PoolArgs P, const int32_t* seqs, const int64_t* keep) {
  pdl_trigger();
  pdl_wait();
  const int item = blockIdx.x / P.hkv, g = blockIdx.x % P.hkv;
  const int32_t s = seqs[item];
  const int64_t kept = keep != nullptr ? keep[item] : 0;
  if (s < 0 || s >= P.n_seqs || kept < 0) {
    if (threadIdx.x == 0) flag(P, kept < 0 ? ZHA_DEV_BAD_LENGTH : ZHA_DEV_BAD_SEQUENCE);
    return;
  }
  int32_t* row = P.table + (int64_t(s) * P.hkv + g) * P.max_blocks;
  const int64_t first = kept / P.chunk + (kept % P.chunk != 0);
  for (int64_t b = first + threadIdx.x; b < P.max_blocks; b += kPageThreads) {
    // exchanged, so that a sequence listed twice gives its pages up once
    const int32_t e = atomicExch(&row[b], -1);
    if (e < 0) continue;
    if (e >= P.n_pages) {
      flag(P, ZHA_DEV_BAD_PAGE);
    } else if (atomicSub(&P.refs[e], 1) <= 0) {
      atomicAdd(&P.refs[e], 1);
      flag(P, ZHA_DEV_BAD_PAGE);
    }
  }
}

// ---- compact ---------------------------------------------------------------
// With n pages in use: code[p] = p for a page that stays, -1 for a free one, and
// -2 - r for one that moves, r = its rank among the moving pages from the end. list[k]
// = the k-th hole below n; list[n_pages - 1 - r] = the moving page r. There are
// as many holes as moves, at most n_pages / 2, so the two ends do not meet.
__device__ void move_pages(const PoolArgs& P, const PageWs& W, int32_t* page_map, int32_t* n_live) {
  const int moves = __ldcg(W.scal + kMoves), threads = blockDim.x;
  auto place = [&](int32_t code) { return code < -1 ? __ldcg(W.list + moves - 1 - (-2 - code)) : code; };
  auto from_of = [&](int64_t k) { return __ldcg(W.list + P.n_pages - 1 - (moves - 1 - k)); };
  // 4 KB of K or V a warp and step, so that few large pages fill the GPU evenly
  // (a page a block: 7 rounds for the work of 6.2 at 7,300 pages).
  constexpr int kPart = 4096;
  const int64_t page_bytes = int64_t(P.chunk) * P.row_bytes;
  const int half = int((page_bytes + kPart - 1) / kPart), parts = 2 * half, lane = threadIdx.x % 32;
  const int64_t warps = int64_t(gridDim.x) * (threads / 32);
  for (int64_t u = int64_t(blockIdx.x) * (threads / 32) + threadIdx.x / 32; u < int64_t(moves) * parts; u += warps) {
    const int64_t k = quotient(u, parts);
    const int part = int(u - k * parts), at = part % half * kPart;
    const int64_t to = __ldcg(W.list + k) * page_bytes + at, from = from_of(k) * page_bytes + at;
    char* pool = part < half ? P.k : P.v;
    copy_bytes(pool + to, pool + from, min64(kPart, page_bytes - at), lane, 32);
  }
  const int64_t cells = int64_t(P.n_seqs) * P.hkv * P.max_blocks, step = int64_t(gridDim.x) * threads;
  const int64_t id = int64_t(blockIdx.x) * threads + threadIdx.x;
  for (int64_t k = id; k < moves; k += step) {
    const int32_t to = __ldcg(W.list + k), from = from_of(k);
    P.refs[to] = P.refs[from];
    P.refs[from] = 0;
  }
#pragma unroll 4
  for (int64_t i = id; i < cells; i += step) {
    const int32_t e = P.table[i];
    if (e < 0 || e >= P.n_pages) continue;
    const int32_t to = place(__ldcg(W.code + e));
    if (to < 0) flag(P, ZHA_DEV_BAD_PAGE);
    if (to != e) P.table[i] = to;
  }
  if (page_map != nullptr)
    for (int64_t p = id; p < P.n_pages; p += step) page_map[p] = place(__ldcg(W.code + p));
  if (n_live != nullptr && id == 0) *n_live = __ldcg(W.scal + kLive);
}

__global__ void __launch_bounds__(kBookThreads)
    pages_plan_kernel(PoolArgs P, PageWs W, int32_t* page_map, int32_t* n_live, bool move_here) {
  __shared__ int s_red[kBookWarps];
  pdl_trigger();
  pdl_wait();
  const Share pages(int(P.n_pages));
  uint32_t bits;
  int sum;
  block_prefix(count_share(P, pages, true, &bits), s_red, &sum);
  if (threadIdx.x == 0) W.seg[cluster_rank()] = sum;
  cluster_sync();
  const int2 counts = counts_of(W);
  const int n = counts.x;
  rank_share(P, pages, true, bits, counts.y, s_red, [&](int p, bool live, int rank) {
    int32_t code = -1;
    if (live) {
      code = int32_t(p);
      if (p >= n) {
        const int r = n - 1 - rank;
        code = -2 - r;
        W.list[P.n_pages - 1 - r] = int32_t(p);
      }
    } else if (p < n) {
      W.list[p - rank] = int32_t(p);
    }
    W.code[p] = code;
    if (p == n - 1) W.scal[kMoves] = n - rank - live;      // holes below n
  });
  if (cluster_rank() == 0 && threadIdx.x == 0) {
    W.scal[kLive] = n;
    if (n == 0) W.scal[kMoves] = 0;
  }
  if (!move_here) return;
  cluster_sync();
  move_pages(P, W, page_map, n_live);
}

__global__ void __launch_bounds__(kPageThreads)
    pages_move_kernel(PoolArgs P, PageWs W, int32_t* page_map, int32_t* n_live) {
  pdl_trigger();
  pdl_wait();
  move_pages(P, W, page_map, n_live);
}

zha_status pool_args(const zha_config* cfg, const zha_page_pool* pool, const char* who, PoolArgs* out) {
  static thread_local char msg[160];
  auto bad = [&](zha_status st, const char* what) {
    snprintf(msg, sizeof msg, "%s: %s", who, what);
    return zha_report_error(st, msg);
  };
  Geom G;
  zha_status st = zha_geometry(cfg, &G);
  if (st != ZHA_OK) return st;
  if (pool == nullptr) return bad(ZHA_ERR_INVALID, "pool is NULL");
  if (pool->reserved != 0) return bad(ZHA_ERR_INVALID, "reserved must be 0");
  if (pool->k == nullptr || pool->v == nullptr || reinterpret_cast<uintptr_t>(pool->k) % 16 != 0 ||
      reinterpret_cast<uintptr_t>(pool->v) % 16 != 0)
    return bad(ZHA_ERR_INVALID, "K and V must be non-NULL 16-byte aligned device pointers");
  if (pool->block_table == nullptr || pool->refs == nullptr || reinterpret_cast<uintptr_t>(pool->block_table) % 4 != 0 ||
      reinterpret_cast<uintptr_t>(pool->refs) % 4 != 0)
    return bad(ZHA_ERR_INVALID, "block_table and refs must be non-NULL device pointers");
  constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
  if (pool->n_pages < 1 || pool->max_blocks < 1 || pool->n_seqs < 1 || pool->n_seqs > 65535)
    return bad(ZHA_ERR_INVALID, "n_pages and max_blocks must be >= 1, n_seqs 1..65535");
  if (pool->n_pages > kMaxRows / G.chunk || pool->max_blocks > kMaxRows || G.hkv > 65536)
    return bad(ZHA_ERR_UNSUPPORTED, "more than 2^31 - 512 token slots in the pool, or max_blocks or heads out of range");
  PoolArgs P{};
  P.k = static_cast<char*>(pool->k);
  P.v = static_cast<char*>(pool->v);
  P.table = pool->block_table;
  P.refs = pool->refs;
  P.n_pages = pool->n_pages;
  P.max_blocks = pool->max_blocks;
  P.n_seqs = pool->n_seqs;
  P.hkv = G.hkv;
  P.chunk = G.chunk;
  P.row_bytes = G.d * (G.kv_bf16 ? 2 : 4);
  *out = P;
  return ZHA_OK;
}

zha_status need_ws(void* d_ws, size_t have, int64_t need) {
  if (d_ws != nullptr && reinterpret_cast<uintptr_t>(d_ws) % 256 == 0 && int64_t(have) >= need) return ZHA_OK;
  return zha_report_error(ZHA_ERR_CAPACITY, "zha_pages: workspace must be 256-byte aligned with zha_pages_workspace_bytes");
}

constexpr int64_t kMaxItemRows = int64_t(1) << 24;

zha_status words_ok(const int32_t* a, const int32_t* b, const int64_t* c, const int32_t* status) {
  if (zha_may_lie(a) && zha_may_lie(b) && zha_may_lie(c) && zha_may_lie(status)) return ZHA_OK;
  return zha_report_error(ZHA_ERR_INVALID, "zha_pages: a list, output or status at no multiple of its type's size");
}

zha_status items_ok(const PoolArgs& P, int32_t n_items, const void* a, const void* b, const char* what) {
  if (n_items < 0 || n_items > 65535 || int64_t(n_items) * P.hkv > kMaxItemRows)
    return zha_report_error(ZHA_ERR_INVALID, what);
  if (n_items > 0 && (a == nullptr || b == nullptr)) return zha_report_error(ZHA_ERR_INVALID, what);
  return ZHA_OK;
}

template <typename... K, typename... A>
zha_status launch_page_kernel(const char* name, const char* who, void (*kernel)(K...), int64_t grid, cudaStream_t s,
                              A&&... args) {
  TraceScope ts(name, 0, s);
  zha_count_launch();
  const cudaError_t e = launch_pdl(kernel, dim3(unsigned(grid)), dim3(kPageThreads), 0, s, args...);
  return e == cudaSuccess ? ZHA_OK : zha_report_cuda(e, who);
}

// One cluster, of one CTA per 4096 counts or 32 rows: a power of two, up to the `most`
// that the device can hold. The kernels take any number.
constexpr int book_ctas(int64_t n_pages, int64_t rows, int most) {
  const int64_t by_pages = (n_pages + 4095) / 4096, by_rows = (rows + 31) / 32;
  int ctas = 1;
  while (ctas < (by_pages > by_rows ? by_pages : by_rows) && ctas < most) ctas *= 2;
  return ctas;
}
static_assert(book_ctas(1, 0, 16) == 1 && book_ctas(4097, 0, 16) == 2 && book_ctas(1, 160, 16) == 8 &&
                  book_ctas(65536, 0, 16) == 16 && book_ctas(int64_t(1) << 30, 1 << 24, 16) == kMostCtas &&
                  book_ctas(65536, 0, 8) == 8 && book_ctas(int64_t(1) << 30, 1 << 24, 8) == 8,
              "no more CTAs than fit, and none without work");

template <typename... K, typename... A>
zha_status launch_book(const char* name, const char* who, void (*kernel)(K...), const PoolArgs& P, int64_t rows,
                       cudaStream_t s, A&&... args) {
  int most = 0;
  cudaError_t e = widest_cluster(reinterpret_cast<const void*>(kernel), kBookThreads, &most);
  if (e != cudaSuccess) return zha_report_cuda(e, who);
  const int ctas = book_ctas(P.n_pages, rows, most);
  TraceScope ts(name, 0, s);
  zha_count_launch();
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(ctas));
  cfg.blockDim = dim3(kBookThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(ctas);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kernel, static_cast<K>(args)...);
  return e == cudaSuccess ? ZHA_OK : zha_report_cuda(e, who);
}

template <bool kFork>
zha_status run_items(const PoolArgs& P, const int32_t* src, const int32_t* dst, const int64_t* tokens, int32_t n_items,
                     void* d_ws, size_t ws_bytes, cudaStream_t s, const char* who) {
  const int64_t rows = int64_t(n_items) * P.hkv;
  const PageWs W = page_ws(d_ws, P.n_pages, rows);
  zha_status st = need_ws(d_ws, ws_bytes, W.bytes);
  if (st != ZHA_OK) return st;
  const int64_t page_bytes = int64_t(P.chunk) * P.row_bytes;
  const bool copy_here = page_bytes <= kCopyPage && rows * page_bytes <= kCopyHere;
  st = launch_book("pages_items_kernel", who, pages_items_kernel<kFork>, P, rows, s, P, W, src, dst, tokens, n_items,
                   copy_here);
  if (st != ZHA_OK || !kFork || copy_here) return st;
  return launch_page_kernel("pages_copy_kernel", who, pages_copy_kernel, rows, s, P, W, src, tokens);
}

}  // namespace

}  // namespace zha

using zha::PoolArgs;

extern "C" {

size_t zha_pages_workspace_bytes(const zha_config* cfg, const zha_page_pool* pool, int32_t n_items) {
  PoolArgs P;
  if (zha::pool_args(cfg, pool, "zha_pages_workspace_bytes", &P) != ZHA_OK || n_items < 0 || n_items > 65535 ||
      int64_t(n_items) * P.hkv > zha::kMaxItemRows)
    return 0;
  return size_t(zha::page_ws(nullptr, P.n_pages, int64_t(n_items) * P.hkv).bytes);
}

zha_status zha_pages_extend(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_seqs,
                            const int64_t* d_n_tokens, int32_t n_items, void* d_ws, size_t ws_bytes, int32_t* d_status,
                            void* stream) {
  PoolArgs P;
  zha_status st = zha::pool_args(cfg, pool, "zha_pages_extend", &P);
  if (st != ZHA_OK) return st;
  if ((st = zha::items_ok(P, n_items, d_seqs, d_n_tokens,
                          "zha_pages_extend: n_items out of range, or seqs or n_tokens NULL")) != ZHA_OK || n_items == 0)
    return st;
  if ((st = zha::words_ok(d_seqs, nullptr, d_n_tokens, d_status)) != ZHA_OK) return st;
  P.status = d_status;
  return zha::run_items<false>(P, nullptr, d_seqs, d_n_tokens, n_items, d_ws, ws_bytes,
                               static_cast<cudaStream_t>(stream), "zha_pages_extend");
}

zha_status zha_pages_fork(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_src, const int32_t* d_dst,
                          const int64_t* d_n_tokens, int32_t n_items, void* d_ws, size_t ws_bytes, int32_t* d_status,
                          void* stream) {
  PoolArgs P;
  zha_status st = zha::pool_args(cfg, pool, "zha_pages_fork", &P);
  if (st != ZHA_OK) return st;
  if ((st = zha::items_ok(P, n_items, d_dst, d_n_tokens,
                          "zha_pages_fork: n_items out of range, or dst or n_tokens NULL")) != ZHA_OK || n_items == 0)
    return st;
  if (d_src == nullptr) return zha_report_error(ZHA_ERR_INVALID, "zha_pages_fork: src is NULL");
  if ((st = zha::words_ok(d_src, d_dst, d_n_tokens, d_status)) != ZHA_OK) return st;
  P.status = d_status;
  return zha::run_items<true>(P, d_src, d_dst, d_n_tokens, n_items, d_ws, ws_bytes, static_cast<cudaStream_t>(stream),
                              "zha_pages_fork");
}

zha_status zha_pages_free(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_seqs,
                          const int64_t* d_keep, int32_t n_items, int32_t* d_status, void* stream) {
  PoolArgs P;
  zha_status st = zha::pool_args(cfg, pool, "zha_pages_free", &P);
  if (st != ZHA_OK) return st;
  if ((st = zha::items_ok(P, n_items, d_seqs, d_seqs,
                          "zha_pages_free: n_items out of range, or seqs NULL")) != ZHA_OK || n_items == 0)
    return st;
  if ((st = zha::words_ok(d_seqs, nullptr, d_keep, d_status)) != ZHA_OK) return st;
  P.status = d_status;
  return zha::launch_page_kernel("pages_free_kernel", "zha_pages_free", zha::pages_free_kernel,
                                 int64_t(n_items) * P.hkv, static_cast<cudaStream_t>(stream), P, d_seqs, d_keep);
}

zha_status zha_pages_compact(const zha_config* cfg, const zha_page_pool* pool, int32_t* d_page_map, int32_t* d_n_live,
                             void* d_ws, size_t ws_bytes, int32_t* d_status, void* stream) {
  PoolArgs P;
  const char* who = "zha_pages_compact";
  zha_status st = zha::pool_args(cfg, pool, who, &P);
  if (st != ZHA_OK) return st;
  if ((st = zha::words_ok(d_page_map, d_n_live, nullptr, d_status)) != ZHA_OK) return st;
  P.status = d_status;
  const zha::PageWs W = zha::page_ws(d_ws, P.n_pages, 0);
  if ((st = zha::need_ws(d_ws, ws_bytes, W.bytes)) != ZHA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  const cudaError_t e = zha::device_sm_count(&sms);
  if (e != cudaSuccess) return zha_report_cuda(e, who);
  const bool move_here = P.n_pages * P.chunk * P.row_bytes <= 2 * zha::kCopyHere;
  st = zha::launch_book("pages_plan_kernel", who, zha::pages_plan_kernel, P, 0, s, P, W, d_page_map, d_n_live, move_here);
  if (st != ZHA_OK || move_here) return st;
  return zha::launch_page_kernel("pages_move_kernel", who, zha::pages_move_kernel, int64_t(sms) * 8, s, P, W,
                                 d_page_map, d_n_live);
}

}  // extern "C"
