// zha_pages.cu -- page bookkeeping of a paged cache on the device: extend, fork,
// free and compact. Semantics are in include/zha.h.
//
// The free pages are those with reference count 0, and the r-th page a call needs
// (items, then KV heads, then blocks in order) is the r-th lowest free one. Both
// ranks are prefix sums, so that no atomic's order shows in a result. Three launches:
//   count  blocks of 2048 counts: how many are free (in use, for compact);
//          one block per (item, KV head): is it valid, how many pages does it need
//   list   each block's prefix over the blocks before it turns its free pages into
//          list[rank]; one more block turns the needs into offsets
//   fill   entries, counts and the rows to copy, with every rank known
// Bound: the launches for small pools; the copied rows (HBM) for compact.
#include <cstdio>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kPageThreads = 256;
constexpr int kSegment = 2048;            // reference counts per block
constexpr int kPerThread = kSegment / kPageThreads;

struct PoolArgs {
  char* k;
  char* v;
  int32_t* table;
  int32_t* refs;
  int64_t n_pages, max_blocks;
  int32_t n_seqs, hkv, chunk, row_bytes;
  int32_t* status;
};

// Workspace, int32: scal[8] (total free or live, total need, moves), seg[n_seg],
// need[items * hkv], offs[items * hkv], list[n_pages], code[n_pages] (compact).
struct PageWs {
  int32_t *scal, *seg, *need, *offs, *list, *code;
  int64_t bytes;
};

PageWs page_ws(void* base, int64_t n_pages, int64_t rows) {
  const int64_t n_seg = (n_pages + kSegment - 1) / kSegment;
  int32_t* p = static_cast<int32_t*>(base);
  PageWs w{};
  int64_t at = 0;
  auto take = [&](int64_t n) { int32_t* q = base == nullptr ? nullptr : p + at; at += round_up(n, 64); return q; };
  w.scal = take(8);
  w.seg = take(n_seg);
  w.need = take(rows);
  w.offs = take(rows);
  w.list = take(n_pages);
  w.code = take(n_pages);
  w.bytes = at * 4;
  return w;
}

enum { kFree = 0, kNeed = 1, kMoves = 2 };

__device__ __forceinline__ void flag(const PoolArgs& P, int bit) {
  if (P.status != nullptr) atomicOr(P.status, bit);
}

// Sum over the block; every thread gets it.
__device__ int block_sum(int v, int* s_red) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if (threadIdx.x % 32 == 0) s_red[threadIdx.x / 32] = v;
  __syncthreads();
  int t = 0;
#pragma unroll
  for (int w = 0; w < kPageThreads / 32; ++w) t += s_red[w];
  return t;
}

// Exclusive prefix of v over the block's threads, and the sum of all.
template <typename I>
__device__ I block_prefix(I v, I* s_red, I* sum = nullptr) {
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
  I base = 0, all = 0;
  for (int w = 0; w < kPageThreads / 32; ++w) {
    if (w < warp) base += s_red[w];
    all += s_red[w];
  }
  if (sum != nullptr) *sum = all;
  return base + x - v;
}

__device__ __forceinline__ bool counted(int32_t refs, bool live) { return live ? refs > 0 : refs == 0; }

__device__ void count_segment(const PoolArgs& P, const PageWs& W, bool live, int* s_red) {
  const int64_t base = int64_t(blockIdx.x) * kSegment;
  int n = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    const int64_t p = base + i * kPageThreads + threadIdx.x;
    if (p < P.n_pages) n += counted(P.refs[p], live);
  }
  n = block_sum(n, s_red);
  if (threadIdx.x == 0) W.seg[blockIdx.x] = n;
}

// ---- count -----------------------------------------------------------------
__global__ void __launch_bounds__(kPageThreads) pages_count_live_kernel(PoolArgs P, PageWs W) {
  __shared__ int s_red[kPageThreads / 32];
  pdl_trigger();
  pdl_wait();
  count_segment(P, W, true, s_red);
}

// Whether `seq` stands in list[0, n).
__device__ bool listed(const int32_t* list, int n, int32_t seq, int* s_red) {
  int hit = 0;
  for (int j = threadIdx.x; j < n; j += kPageThreads) hit |= list[j] == seq;
  return block_sum(hit, s_red) != 0;
}

// kFork: src, dst, tokens; else seqs = dst.
template <bool kFork>
__global__ void __launch_bounds__(kPageThreads)
    pages_count_kernel(PoolArgs P, PageWs W, int n_seg, const int32_t* src, const int32_t* dst, const int64_t* tokens,
                       int n_items) {
  __shared__ int s_red[kPageThreads / 32];
  pdl_trigger();
  pdl_wait();
  if (int(blockIdx.x) < n_seg) {
    count_segment(P, W, false, s_red);
    return;
  }
  const int idx = blockIdx.x - n_seg, item = idx / P.hkv, g = idx % P.hkv;
  const int32_t d = dst[item];
  const int64_t n = tokens[item];
  int bad = 0;
  if (d < 0 || d >= P.n_seqs || listed(dst, item, d, s_red)) bad = ZHA_DEV_BAD_SEQUENCE;
  int32_t s = d;
  if (kFork) {
    s = src[item];
    if (s < 0 || s >= P.n_seqs || listed(dst, n_items, s, s_red)) bad = ZHA_DEV_BAD_SEQUENCE;
  }
  if (bad == 0 && (n < 0 || n > P.max_blocks * P.chunk)) bad = ZHA_DEV_BAD_LENGTH;
  int need = 0;
  if (bad == 0) {
    const int64_t blocks = (n + P.chunk - 1) / P.chunk;
    const int32_t* row = P.table + (int64_t(s) * P.hkv + g) * P.max_blocks;
    int miss = 0, wrong = 0;
    for (int64_t b = threadIdx.x; b < blocks; b += kPageThreads) {
      const int32_t e = row[b];
      miss += e < 0;
      wrong |= e >= P.n_pages || (e >= 0 && P.refs[e] <= 0);
    }
    miss = block_sum(miss, s_red);
    wrong = block_sum(wrong, s_red);
    if (kFork) {
      int full = 0;
      const int32_t* to = P.table + (int64_t(d) * P.hkv + g) * P.max_blocks;
      for (int64_t b = threadIdx.x; b < P.max_blocks; b += kPageThreads) full |= to[b] >= 0;
      if (block_sum(full, s_red)) bad = ZHA_DEV_BAD_SEQUENCE;
      else if (wrong || miss) bad = ZHA_DEV_BAD_PAGE;
      need = n % P.chunk != 0;
    } else {
      if (wrong) bad = ZHA_DEV_BAD_PAGE;
      need = miss;
    }
  }
  if (threadIdx.x == 0) {
    W.need[idx] = bad ? -1 : need;
    if (bad) flag(P, bad);
  }
}

// ---- list ------------------------------------------------------------------
// Exclusive prefix of this block's segment over the segments' counts, and (all
// segments) the total.
__device__ int segment_base(const PageWs& W, int n_seg, int* total, int* s_red) {
  int below = 0, all = 0;
  for (int i = threadIdx.x; i < n_seg; i += kPageThreads) {
    const int v = W.seg[i];
    all += v;
    if (i < int(blockIdx.x)) below += v;
  }
  *total = block_sum(all, s_red);
  return block_sum(below, s_red);
}

// Calls f(page, counted, exclusive rank) for the block's pages in order.
template <typename F>
__device__ void rank_segment(const PoolArgs& P, bool live, int base, int* s_red, F f) {
  const int64_t p0 = int64_t(blockIdx.x) * kSegment + int64_t(threadIdx.x) * kPerThread;
  int n = 0;
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < kPerThread; ++i)
    if (p0 + i < P.n_pages && counted(P.refs[p0 + i], live)) { bits |= 1u << i; ++n; }
  int rank = base + block_prefix(n, s_red);
#pragma unroll
  for (int i = 0; i < kPerThread; ++i) {
    if (p0 + i >= P.n_pages) break;
    const bool c = (bits >> i) & 1u;
    f(p0 + i, c, rank);
    rank += c;
  }
}

__global__ void __launch_bounds__(kPageThreads) pages_list_kernel(PoolArgs P, PageWs W, int n_seg, int n_items) {
  __shared__ int s_red[kPageThreads / 32];
  pdl_trigger();
  pdl_wait();
  if (int(blockIdx.x) < n_seg) {
    int total;
    const int base = segment_base(W, n_seg, &total, s_red);
    rank_segment(P, false, base, s_red, [&](int64_t p, bool c, int rank) {
      if (c) W.list[rank] = int32_t(p);
    });
    if (blockIdx.x == 0 && threadIdx.x == 0) W.scal[kFree] = total;
    return;
  }
  // Offsets of the (item, head) needs. One refused head refuses the item: its
  // offset is then -1 and it needs nothing.
  // Sums may pass 31 bits where no pool could serve them: they are kept in 64
  // and stored cut to 31, which is above every count of free pages.
  __shared__ int64_t s_red64[kPageThreads / 32];
  constexpr int64_t kMost = 0x7fffffff;
  int64_t carry = 0;
  const int64_t rows = int64_t(n_items) * P.hkv;
  for (int64_t r0 = 0; r0 < rows; r0 += kPageThreads) {
    const int64_t r = r0 + threadIdx.x;
    int64_t v = 0, sum;
    bool ok = false;
    if (r < rows) {
      ok = true;
      const int64_t i0 = r / P.hkv * P.hkv;
      for (int g = 0; g < P.hkv; ++g) ok = ok && W.need[i0 + g] >= 0;
      v = ok ? W.need[r] : 0;
    }
    const int64_t pre = block_prefix(v, s_red64, &sum);
    if (r < rows) W.offs[r] = ok ? int32_t(min64(carry + pre, kMost)) : -1;
    carry += sum;
  }
  if (threadIdx.x == 0) W.scal[kNeed] = int32_t(min64(carry, kMost));
}

// ---- fill ------------------------------------------------------------------
__device__ __forceinline__ void copy_bytes(char* to, const char* from, int64_t n) {
  const uint4* f = reinterpret_cast<const uint4*>(from);
  uint4* t = reinterpret_cast<uint4*>(to);
  for (int64_t i = threadIdx.x; i < n / 16; i += kPageThreads) t[i] = f[i];
}

template <bool kFork>
__global__ void __launch_bounds__(kPageThreads)
    pages_fill_kernel(PoolArgs P, PageWs W, const int32_t* src, const int32_t* dst, const int64_t* tokens) {
  __shared__ int s_red[kPageThreads / 32];
  pdl_trigger();
  pdl_wait();
  if (W.scal[kNeed] > W.scal[kFree]) {
    if (blockIdx.x == 0 && threadIdx.x == 0) flag(P, ZHA_DEV_NO_PAGES);
    return;
  }
  const int idx = blockIdx.x, item = idx / P.hkv, g = idx % P.hkv;
  int at = W.offs[idx];
  if (at < 0) return;
  const int64_t n = tokens[item];
  int32_t* row = P.table + (int64_t(dst[item]) * P.hkv + g) * P.max_blocks;
  if (!kFork) {
    const int64_t blocks = (n + P.chunk - 1) / P.chunk;
    for (int64_t b0 = 0; b0 < blocks; b0 += kPageThreads) {
      const int64_t b = b0 + threadIdx.x;
      const int miss = b < blocks && row[b] < 0;
      int sum;
      const int pre = block_prefix(miss, s_red, &sum);
      if (miss) {
        const int32_t page = W.list[at + pre];
        row[b] = page;
        P.refs[page] = 1;
      }
      at += sum;
    }
    return;
  }
  const int64_t full = n / P.chunk, rest = n % P.chunk;
  const int32_t* from = P.table + (int64_t(src[item]) * P.hkv + g) * P.max_blocks;
  const int32_t page = rest ? W.list[at] : -1;
  for (int64_t b = threadIdx.x; b < P.max_blocks; b += kPageThreads) {
    int32_t e = b == full ? page : -1;
    if (b < full) {
      e = from[b];
      atomicAdd(&P.refs[e], 1);
    }
    row[b] = e;
  }
  if (rest) {
    if (threadIdx.x == 0) P.refs[page] = 1;
    const int64_t f = int64_t(from[full]) * P.chunk * P.row_bytes, t = int64_t(page) * P.chunk * P.row_bytes;
    copy_bytes(P.k + t, P.k + f, rest * P.row_bytes);
    copy_bytes(P.v + t, P.v + f, rest * P.row_bytes);
  }
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
__global__ void __launch_bounds__(kPageThreads) pages_moves_kernel(PoolArgs P, PageWs W, int n_seg) {
  __shared__ int s_red[kPageThreads / 32];
  pdl_trigger();
  pdl_wait();
  int n;
  const int base = segment_base(W, n_seg, &n, s_red);
  rank_segment(P, true, base, s_red, [&](int64_t p, bool live, int rank) {
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
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    W.scal[kFree] = n;
    if (n == 0) W.scal[kMoves] = 0;
  }
}

__global__ void __launch_bounds__(kPageThreads)
    pages_move_kernel(PoolArgs P, PageWs W, int32_t* page_map, int32_t* n_live) {
  pdl_trigger();
  pdl_wait();
  const int moves = W.scal[kMoves];
  const int64_t page_bytes = int64_t(P.chunk) * P.row_bytes;
  auto place = [&](int32_t code) { return code < -1 ? W.list[moves - 1 - (-2 - code)] : code; };
  for (int k = blockIdx.x; k < moves; k += gridDim.x) {
    const int32_t to = W.list[k], from = W.list[P.n_pages - 1 - (moves - 1 - k)];
    copy_bytes(P.k + to * page_bytes, P.k + from * page_bytes, page_bytes);
    copy_bytes(P.v + to * page_bytes, P.v + from * page_bytes, page_bytes);
    if (threadIdx.x == 0) {
      P.refs[to] = P.refs[from];
      P.refs[from] = 0;
    }
  }
  const int64_t cells = int64_t(P.n_seqs) * P.hkv * P.max_blocks, step = int64_t(gridDim.x) * kPageThreads;
  const int64_t id = int64_t(blockIdx.x) * kPageThreads + threadIdx.x;
  for (int64_t i = id; i < cells; i += step) {
    const int32_t e = P.table[i];
    if (e < 0 || e >= P.n_pages) continue;
    const int32_t to = place(W.code[e]);
    if (to < 0) flag(P, ZHA_DEV_BAD_PAGE);
    if (to != e) P.table[i] = to;
  }
  if (page_map != nullptr)
    for (int64_t p = id; p < P.n_pages; p += step) page_map[p] = place(W.code[p]);
  if (n_live != nullptr && id == 0) *n_live = W.scal[kFree];
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

int segments(const PoolArgs& P) { return int((P.n_pages + kSegment - 1) / kSegment); }

zha_status need_ws(void* d_ws, size_t have, int64_t need) {
  if (d_ws != nullptr && reinterpret_cast<uintptr_t>(d_ws) % 256 == 0 && int64_t(have) >= need) return ZHA_OK;
  return zha_report_error(ZHA_ERR_CAPACITY, "zha_pages: workspace must be 256-byte aligned with zha_pages_workspace_bytes");
}

constexpr int64_t kMaxItemRows = int64_t(1) << 24;

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

// extend and fork: count, list, fill.
template <bool kFork>
zha_status run_items(const PoolArgs& P, const int32_t* src, const int32_t* dst, const int64_t* tokens, int32_t n_items,
                     void* d_ws, size_t ws_bytes, cudaStream_t s, const char* who) {
  const int64_t rows = int64_t(n_items) * P.hkv;
  const PageWs W = page_ws(d_ws, P.n_pages, rows);
  zha_status st = need_ws(d_ws, ws_bytes, W.bytes);
  if (st != ZHA_OK) return st;
  const int n_seg = segments(P);
  if ((st = launch_page_kernel("pages_count_kernel", who, pages_count_kernel<kFork>, n_seg + rows, s, P, W, n_seg, src,
                               dst, tokens, n_items)) != ZHA_OK)
    return st;
  if ((st = launch_page_kernel("pages_list_kernel", who, pages_list_kernel, n_seg + 1, s, P, W, n_seg, n_items)) !=
      ZHA_OK)
    return st;
  return launch_page_kernel("pages_fill_kernel", who, pages_fill_kernel<kFork>, rows, s, P, W, src, dst, tokens);
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
  if ((st = zha::items_ok(P, n_items, d_seqs, d_n_tokens, "zha_pages_extend: n_items out of range, or seqs or n_tokens NULL")) != ZHA_OK || n_items == 0)
    return st;
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
  if ((st = zha::items_ok(P, n_items, d_dst, d_n_tokens, "zha_pages_fork: n_items out of range, or dst or n_tokens NULL")) != ZHA_OK || n_items == 0)
    return st;
  if (d_src == nullptr) return zha_report_error(ZHA_ERR_INVALID, "zha_pages_fork: src is NULL");
  P.status = d_status;
  return zha::run_items<true>(P, d_src, d_dst, d_n_tokens, n_items, d_ws, ws_bytes, static_cast<cudaStream_t>(stream),
                              "zha_pages_fork");
}

zha_status zha_pages_free(const zha_config* cfg, const zha_page_pool* pool, const int32_t* d_seqs,
                          const int64_t* d_keep, int32_t n_items, int32_t* d_status, void* stream) {
  PoolArgs P;
  zha_status st = zha::pool_args(cfg, pool, "zha_pages_free", &P);
  if (st != ZHA_OK) return st;
  if ((st = zha::items_ok(P, n_items, d_seqs, d_seqs, "zha_pages_free: n_items out of range, or seqs NULL")) != ZHA_OK || n_items == 0)
    return st;
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
  P.status = d_status;
  const zha::PageWs W = zha::page_ws(d_ws, P.n_pages, 0);
  if ((st = zha::need_ws(d_ws, ws_bytes, W.bytes)) != ZHA_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  const cudaError_t e = zha::device_sm_count(&sms);
  if (e != cudaSuccess) return zha_report_cuda(e, who);
  const int n_seg = zha::segments(P);
  if ((st = zha::launch_page_kernel("pages_count_live_kernel", who, zha::pages_count_live_kernel, n_seg, s, P, W)) != ZHA_OK)
    return st;
  if ((st = zha::launch_page_kernel("pages_moves_kernel", who, zha::pages_moves_kernel, n_seg, s, P, W, n_seg)) != ZHA_OK)
    return st;
  return zha::launch_page_kernel("pages_move_kernel", who, zha::pages_move_kernel, int64_t(sms) * 8, s, P, W,
                                 d_page_map, d_n_live);
}

}  // extern "C"
