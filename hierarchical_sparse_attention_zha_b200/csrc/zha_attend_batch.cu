// zha_attend_batch.cu -- dense attention of one query token per sequence over a
// batch of (paged) caches. Semantics are in include/zha.h.
//
// Mathematics. o = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m), x_j = q.k_j
// log2(e) / sqrt(d): any m gives the same quotient, and states (m, l, o) of two
// parts of the keys join as m = max, l = sum l_i 2^(m_i - m), o alike.
//
// Split. A unit is (sequence, KV head, block of up to 8 of its query heads);
// its keys are cut into tiles of 64. All units' tiles, one behind the other,
// are dealt out evenly to the CTAs (CTA c has tiles [c T / n, (c + 1) T / n)),
// from the counts in device memory, so that ragged lengths cost nothing.
// A unit that lies in one CTA is finished there; the pieces of the others go to the
// workspace (piece of CTA c in unit u at slot c + u, so that no two meet) and a
// second kernel joins them in a fixed order.
#include <cmath>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kTile = 64;               // keys per tile
constexpr int kWarps = 4;               // a tile's keys are split over the warps
constexpr int kThreads = kWarps * 32;
constexpr int kHeads = 8;               // query heads per unit
constexpr int kMinTiles = 2;            // no CTA takes less, unless there is less
constexpr int kMaxCtas = 148 * 4;

struct BatchLayout {
  int64_t units, slots, bytes, slots_off;
  int32_t hb;                           // head blocks per KV head
};

// Workspace: int64 prefix[n_seqs + 1] (tiles of one unit of the sequences
// before s), int32 CTA count; then slots [m, l, 0, 0, o[d]] of 8 heads a piece.
inline BatchLayout batch_layout(const Geom& G, int32_t n_seqs) {
  BatchLayout b{};
  b.hb = (G.group + kHeads - 1) / kHeads;
  b.units = int64_t(n_seqs) * G.hkv * b.hb;
  b.slots = kMaxCtas + b.units;
  b.slots_off = round_up((int64_t(n_seqs) + 2) * 8, 256);
  b.bytes = b.slots_off + round_up(b.slots * kHeads * (G.d + 4) * 4, 256);
  return b;
}

struct BatchArgs {
  const void* Q;
  KvView kv;
  const int64_t* n_tokens;
  int64_t max_tokens;
  void* O;
  float* lse;
  int64_t* prefix;
  float* slots;
  int32_t* status;
  int32_t n_seqs, hkv, hq, group, hb, chunk;
  float scale_log2;                     // log2(e) / sqrt(d)
};

__device__ __forceinline__ int64_t clamped(const BatchArgs& A, int s) {
  return max64(0, min64(A.n_tokens[s], A.max_tokens));
}
__device__ __forceinline__ int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }

template <typename T>
__device__ __forceinline__ float load_q(const T* p) { return float(*p); }

__device__ __forceinline__ void store_o(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_o(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename Kv, typename Qt, int D>
__global__ void __launch_bounds__(kThreads) attend_batch_kernel(const BatchArgs A) {
  constexpr int EPL = D / 32;
  __shared__ int64_t s_scan[kThreads];
  __shared__ int64_t s_at[3];                        // sequence, its first tile, total
  __shared__ float s_m[kWarps][kHeads], s_l[kWarps][kHeads];
  __shared__ float s_o[kWarps][kHeads][D];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  pdl_trigger();
  pdl_wait();

  // Tiles of all sequences and where this CTA's begin. Thread i scans a run of
  // ceil(S / 128) sequences.
  const int run = (A.n_seqs + kThreads - 1) / kThreads;
  const int s0 = min(A.n_seqs, tid * run), s1 = min(A.n_seqs, s0 + run);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) mine += tiles_of(clamped(A, s));
  s_scan[tid] = mine;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int i = 0; i < kThreads; ++i) {
    if (i < tid) before += s_scan[i];
    all += s_scan[i];
  }
  const int64_t per = int64_t(A.hkv) * A.hb;         // units of a sequence
  const int64_t T = all * per;
  const int64_t n_cta = max64(1, min64(gridDim.x, (T + kMinTiles - 1) / kMinTiles));
  const int64_t c = blockIdx.x;
  const int64_t t0 = c < n_cta ? c * T / n_cta : T, t1 = c < n_cta ? (c + 1) * T / n_cta : T;
  {
    int64_t at = before;
    for (int s = s0; s < s1; ++s) {
      const int64_t n = A.n_tokens[s], tl = tiles_of(clamped(A, s));
      if (t0 >= at * per && t0 < (at + tl) * per) { s_at[0] = s; s_at[1] = at; }
      if (c == 0) {
        A.prefix[s] = at;
        if ((n < 0 || n > A.max_tokens) && A.status != nullptr) atomicOr(A.status, ZHA_DEV_BAD_LENGTH);
      }
      at += tl;
    }
    if (c == 0 && tid == 0) { A.prefix[A.n_seqs] = all; A.prefix[A.n_seqs + 1] = n_cta; }
  }
  __syncthreads();
  if (t0 >= t1) return;
  int s = int(s_at[0]);
  int64_t seq_tile = s_at[1];

  int64_t t = t0;
  while (t < t1) {
    const int64_t n = clamped(A, s), tl = tiles_of(n);
    if (tl == 0 || t >= (seq_tile + tl) * per) { seq_tile += tl; ++s; continue; }
    const int64_t local = t - seq_tile * per;
    const int ub = int(local / tl);
    const int64_t first = seq_tile * per + int64_t(ub) * tl;      // the unit's first tile
    const int64_t stop = min64(t1, first + tl);
    const int g = ub / A.hb, h0 = (ub % A.hb) * kHeads, heads = min(kHeads, A.group - h0);
    const int64_t qrow = int64_t(s) * A.hq + int64_t(g) * A.group + h0;

    float q[kHeads][EPL], o[kHeads][EPL], m[kHeads], l[kHeads];
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      m[h] = -INFINITY; l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        o[h][e] = 0.f;
        q[h][e] = h < heads ? load_q(static_cast<const Qt*>(A.Q) + (qrow + h) * D + lane * EPL + e) * A.scale_log2 : 0.f;
      }
    }
    for (int64_t tile = t - first; tile < stop - first; ++tile) {
      for (int i = 0; i < kTile / kWarps; ++i) {
        const int64_t tok = tile * kTile + i * kWarps + warp;
        if (tok >= n) break;
        const int32_t row = kv_batch_row(A.kv, A.hkv, s, g, tok, A.chunk);
        if (row < 0) {
          if (lane == 0 && A.status != nullptr) atomicOr(A.status, ZHA_DEV_BAD_PAGE);
          continue;
        }
        float k[EPL], v[EPL];
        load_slice<EPL>(static_cast<const Kv*>(A.kv.k) + int64_t(row) * D, lane * EPL, k);
        load_slice<EPL>(static_cast<const Kv*>(A.kv.v) + int64_t(row) * D, lane * EPL, v);
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          float x = 0.f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) x = fmaf(q[h][e], k[e], x);
          x = warp_sum(x);
          const float mn = fmaxf(m[h], x), at = mn == -INFINITY ? 0.f : mn, a = exp2f(m[h] - at), p = exp2f(x - at);
          m[h] = mn;
          l[h] = l[h] * a + p;
#pragma unroll
          for (int e = 0; e < EPL; ++e) o[h][e] = fmaf(p, v[e], o[h][e] * a);
        }
      }
    }
    // The warps' states joined, in warp order.
    __syncthreads();
#pragma unroll
    for (int h = 0; h < kHeads; ++h) {
      if (lane == 0) { s_m[warp][h] = m[h]; s_l[warp][h] = l[h]; }
#pragma unroll
      for (int e = 0; e < EPL; ++e) s_o[warp][h][lane * EPL + e] = o[h][e];
    }
    __syncthreads();
    const bool whole = t == first && stop == first + tl;
    const int64_t unit = int64_t(s) * per + ub;
    for (int i = tid; i < heads * D; i += kThreads) {
      const int h = i / D, e = i % D;
      float M = -INFINITY;
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
      float L = 0.f, acc = 0.f;
      for (int w = 0; w < kWarps; ++w) {
        const float f = s_l[w][h] > 0.f || isnan(s_l[w][h]) ? exp2f(s_m[w][h] - M) : 0.f;
        L += s_l[w][h] * f;
        acc += s_o[w][h][e] * f;
      }
      if (whole) {
        store_o(static_cast<Qt*>(A.O) + (qrow + h) * D + e, L == 0.f ? 0.f : acc / L);
        if (e == 0 && A.lse != nullptr) A.lse[qrow + h] = L == 0.f ? -INFINITY : 0.69314718056f * (M + log2f(L));
      } else {
        float* slot = A.slots + ((c + unit) * kHeads + h) * (D + 4);
        slot[4 + e] = acc;
        if (e == 0) { slot[0] = M; slot[1] = L; }
      }
    }
    t = stop;
  }
}

// One warp per (sequence, query head): nothing to do for a unit that one CTA
// finished; zeros for one without tiles; else its pieces joined in CTA order.
template <typename Qt, int D>
__global__ void __launch_bounds__(kThreads) attend_batch_join_kernel(const BatchArgs A) {
  constexpr int EPL = D / 32;
  const int lane = threadIdx.x % 32;
  const int64_t row = int64_t(blockIdx.x) * kWarps + threadIdx.x / 32;
  pdl_trigger();
  pdl_wait();
  if (row >= int64_t(A.n_seqs) * A.hq) return;
  const int s = int(row / A.hq), qh = int(row % A.hq), g = qh / A.group, hh = qh % A.group;
  const int64_t per = int64_t(A.hkv) * A.hb, ub = int64_t(g) * A.hb + hh / kHeads;
  const int64_t seq_tile = A.prefix[s], tl = A.prefix[s + 1] - seq_tile;
  const int64_t T = A.prefix[A.n_seqs] * per, n_cta = A.prefix[A.n_seqs + 1];
  float acc[EPL] = {}, M = -INFINITY, L = 0.f;
  if (tl > 0) {
    const int64_t lo = seq_tile * per + ub * tl, hi = lo + tl;
    const int64_t c0 = ((lo + 1) * n_cta - 1) / T, c1 = (hi * n_cta - 1) / T;
    if (c0 == c1) return;
    for (int64_t c = c0; c <= c1; ++c) {
      const float* slot = A.slots + ((c + s * per + ub) * kHeads + hh % kHeads) * (D + 4);
      const float m = slot[0], l = slot[1];
      if (l == 0.f) continue;
      const float mn = fmaxf(M, m), a = L == 0.f ? 0.f : exp2f(M - mn), b = exp2f(m - mn);
      M = mn;
      L = L * a + l * b;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = acc[e] * a + slot[4 + lane * EPL + e] * b;
    }
  }
#pragma unroll
  for (int e = 0; e < EPL; ++e)
    store_o(static_cast<Qt*>(A.O) + row * D + lane * EPL + e, L == 0.f ? 0.f : acc[e] / L);
  if (lane == 0 && A.lse != nullptr) A.lse[row] = L == 0.f ? -INFINITY : 0.69314718056f * (M + log2f(L));
}

template <typename Kv, typename Qt, int D>
cudaError_t launch_batch(const BatchArgs& A, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t most = int64_t(A.n_seqs) * A.hkv * A.hb * ((A.max_tokens + kTile - 1) / kTile);
  const int64_t ctas = max64(1, min64(min64(int64_t(sms) * 4, kMaxCtas), (most + kMinTiles - 1) / kMinTiles));
  {
    TraceScope ts("attend_batch_kernel", 0, s);
    zha_count_launch();
    e = launch_pdl(attend_batch_kernel<Kv, Qt, D>, dim3(unsigned(ctas)), dim3(kThreads), 0, s, A);
    if (e != cudaSuccess) return e;
  }
  TraceScope ts("attend_batch_join_kernel", 0, s);
  zha_count_launch();
  const int64_t rows = int64_t(A.n_seqs) * A.hq;
  return launch_pdl(attend_batch_join_kernel<Qt, D>, dim3(unsigned((rows + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                    s, A);
}

template <typename Kv, typename Qt>
cudaError_t launch_batch_d(const BatchArgs& A, int d, cudaStream_t s) {
  return d == 128 ? launch_batch<Kv, Qt, 128>(A, s) : launch_batch<Kv, Qt, 64>(A, s);
}

// Units beyond this are refused: slots and grids stay far below 2^31.
constexpr int64_t kMaxUnits = int64_t(1) << 22;

bool units_ok(const Geom& G, int32_t n_seqs) {
  const int64_t hb = (G.group + kHeads - 1) / kHeads;
  return int64_t(G.hkv) * hb <= kMaxUnits / n_seqs;
}

}  // namespace

}  // namespace zha

extern "C" {

size_t zha_attend_batch_workspace_bytes(const zha_config* cfg, int32_t n_seqs, int64_t max_tokens) {
  zha::Geom G;
  if (zha_geometry(cfg, &G) != ZHA_OK || n_seqs < 1 || n_seqs > 65535 || max_tokens < 0 || !zha::units_ok(G, n_seqs))
    return 0;
  return size_t(zha::batch_layout(G, n_seqs).bytes);
}

zha_status zha_attend_batch_kv(const zha_config* cfg, const void* d_Q, int32_t q_dtype, const zha_kv_cache* kv,
                               int32_t n_seqs, const int64_t* d_n_tokens, int64_t max_tokens, void* d_O, float* d_lse,
                               void* d_ws, size_t ws_bytes, int32_t* d_status, void* stream) {
  const char* who = "zha_attend_batch_kv";
  auto aligned16 = [](const void* p) { return p != nullptr && reinterpret_cast<uintptr_t>(p) % 16 == 0; };
  zha::Geom G;
  zha_status st = zha_geometry(cfg, &G);
  if (st != ZHA_OK) return st;
  zha::BatchArgs A{};
  if ((st = zha_batch_view(G, kv, n_seqs, max_tokens, who, &A.kv)) != ZHA_OK) return st;
  if (!aligned16(d_Q) || !aligned16(d_O))
    return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: Q and O must be non-NULL 16-byte aligned device pointers");
  if (q_dtype != ZHA_F32 && q_dtype != ZHA_BF16)
    return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: unknown q_dtype");
  if (d_n_tokens == nullptr) return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: n_tokens is NULL");
  if (!zha::units_ok(G, n_seqs))
    return zha_report_error(ZHA_ERR_UNSUPPORTED, "zha_attend_batch_kv: more than 2^22 (sequence, KV head, 8-query block) units");
  const zha::BatchLayout lay = zha::batch_layout(G, n_seqs);
  if (d_ws == nullptr || reinterpret_cast<uintptr_t>(d_ws) % 256 != 0 || int64_t(ws_bytes) < lay.bytes)
    return zha_report_error(ZHA_ERR_CAPACITY,
                            "zha_attend_batch_kv: workspace must be 256-byte aligned with zha_attend_batch_workspace_bytes");
  A.Q = d_Q;
  A.n_tokens = d_n_tokens;
  A.max_tokens = max_tokens;
  A.O = d_O;
  A.lse = d_lse;
  A.prefix = static_cast<int64_t*>(d_ws);
  A.slots = reinterpret_cast<float*>(static_cast<char*>(d_ws) + lay.slots_off);
  A.status = d_status;
  A.n_seqs = n_seqs;
  A.hkv = G.hkv;
  A.hq = G.hq;
  A.group = G.group;
  A.hb = lay.hb;
  A.chunk = G.chunk;
  A.scale_log2 = float(1.4426950408889634 / std::sqrt(double(G.d)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using bf = __nv_bfloat16;
  const cudaError_t e = G.kv_bf16 ? (q_dtype == ZHA_F32 ? zha::launch_batch_d<bf, float>(A, G.d, s)
                                                        : zha::launch_batch_d<bf, bf>(A, G.d, s))
                                  : (q_dtype == ZHA_F32 ? zha::launch_batch_d<float, float>(A, G.d, s)
                                                        : zha::launch_batch_d<float, bf>(A, G.d, s));
  return e == cudaSuccess ? ZHA_OK : zha_report_cuda(e, who);
}

}  // extern "C"
