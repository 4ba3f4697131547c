// zha_rope.cu -- rotary positions: the frequency table of a rotation, the turn of
// strided rows (and back, its gradient), and the turn fused with the write of a
// batch's new tokens into its caches. Semantics are in include/zha.h.
//
// Mathematics. Pair (a, b) at position m becomes A (a cos - b sin, a sin + b cos)
// with phi = m * theta_i. An fp32 product m * theta_i would be off by m * 2^-24
// radians, which at a million tokens is 0.06. Here theta_i / (2 pi) is a 64-bit
// fraction of a turn, the product with m wraps modulo one turn by itself
// (unsigned arithmetic, also for negative m), and what is left is exact to
// m * 2^-54 turns (the table's own rounding). The nearest quarter turn comes off as two
// bits, so the sine and cosine see an argument of at most an eighth of a turn,
// rounded at 2^-28 turns: there their Taylor series to x^9 and x^10 are off by less
// than 2^-28.
//
// A row is read in pieces of 8 elements, two a lane: the two that hold the elements of
// 8 pairs, so that a lane turns what it has read. (Half layout with a split inside a
// piece: two adjacent pieces, and the pairs' other elements through shared memory.) A
// block makes the cosines and sines of its tokens once, while its first rows are on
// their way.
//
// Bound: HBM, each row read once and written once; the launch for few tokens. Measured
// (the copy rate is 6.55 TB/s): 32K tokens x 32 bf16 rows of 128 in 89 us (6.0 TB/s, 92%);
// 16K tokens of 32 query, 8 key and 8 value rows into pages in 78 us (5.2 TB/s, 79%); 4
// tokens in 3 us on the device. Turning by a lane's own piece with the other elements
// from another lane took 98 and 86 us (twice the conversions); 4 rows in flight a lane
// instead of 2, which costs occupancy, 86 and 99. A split inside a piece (37 pairs): 136
// us for the 32K rows, 191 with the other elements read again.
#include <cmath>
#include <type_traits>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeWarps = kRopeThreads / 32;
constexpr int kRopeTokens = 32;          // a block, at most
// Rows a block. In one run each, inputs partly in L2: 96: 16K tokens 81 us, 32K rows 84; 192: 76, 85; 384:
// 76, 89. 200K tokens of 4 rows: 130, 125, 125.
constexpr int kRopeTarget = 192;

struct RopeTable {
  int32_t pairs;               // 0: nothing is turned
  int32_t half;                // pair i = (i, i + pairs) instead of (2i, 2i + 1)
  float amplitude;
  uint64_t turn[64];
};

// One kind of rows of a token: source and destination with their strides.
struct RowSet {
  const void* src;
  void* dst;
  int64_t src_token, src_head, dst_token, dst_head;
  int32_t heads;
};

__device__ __forceinline__ float2 cos_sin_of(uint64_t turn, int64_t pos, float amplitude, bool back) {
  const uint32_t u = uint32_t((turn * uint64_t(pos) + 0x80000000ull) >> 32);   // turns * 2^32
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const float x = float(int32_t(u - (quarter << 30))) * 0x1p-31f;                // half turns, |x| <= 1/4
  const float z = x * 3.14159265359f, y = z * z;
  const float s = fmaf(z * y, fmaf(y, fmaf(y, fmaf(y, 1.f / 362880, -1.f / 5040), 1.f / 120), -1.f / 6), z);
  const float c = fmaf(y, fmaf(y, fmaf(y, fmaf(y, fmaf(y, -1.f / 3628800, 1.f / 40320), -1.f / 720), 1.f / 24), -0.5f), 1.f);
  float co = (quarter & 1u) ? s : c, si = (quarter & 1u) ? c : s;
  if (quarter == 1u || quarter == 2u) co = -co;
  if (quarter == 2u || quarter == 3u) si = -si;
  if (back) si = -si;
  return make_float2(co * amplitude, si * amplitude);
}

// Pieces of 8 elements as they lie in memory.
template <typename T>
struct Piece;
template <>
struct Piece<float> {
  uint32_t w[8];
  __device__ void load(const float* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p), b = *reinterpret_cast<const uint4*>(p + 4);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
  __device__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  }
};
template <>
struct Piece<__nv_bfloat16> {
  uint32_t w[4];
  __device__ void load(const __nv_bfloat16* p) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
  }
  __device__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
__device__ __forceinline__ void store_8(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_8(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 x;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = x;
}

// Where the other element of a pair is: beside it, in the lane's other piece, elsewhere.
enum { kOwn = 0, kPair = 1, kAcross = 2 };
int mode_of(const RopeTable& R) { return !R.half ? kOwn : R.pairs % 8 == 0 ? kPair : kAcross; }

// Where a token's cosine and sine of pair p lie: so that the lanes of a row, which
// take two pairs of their 8 at a time, read adjacent 16 bytes.
template <int MODE>
__device__ __forceinline__ int turn_slot(int p) {
  return MODE == kAcross ? p + p / 16 : ((p % 8 / 2) * 8 + p / 8) * 2 + p % 2;
}
constexpr int kTurns = 64 + 4;           // places of a token's turns

// For kAcross a warp's rows pass through shared memory, element e at e + e / 16, so that
// the lanes, 16 elements apart, and the rows meet no bank twice.
constexpr int row_floats(int d) { return d + d / 16; }
template <int D, int MODE>
struct RowBuffer {
  float x[MODE == kAcross ? kRopeWarps : 1][MODE == kAcross ? 512 / D * row_floats(D) : 1];
};

// What a lane does with its two pieces (from elements a0 and b0 on) of every row.
template <int D, int MODE>
struct Lane {
  int unit, a0, b0;
  bool on;
  __device__ Lane(int P, int lane) : unit(lane % (D / 16)) {
    const bool pair = MODE == kPair && unit < P / 8;          // the others copy the pieces behind the pairs
    a0 = pair ? unit * 8 : unit * 16;
    b0 = pair ? a0 + P : a0 + 8;
    on = MODE == kPair ? pair : MODE == kOwn ? unit * 8 < P : a0 < 2 * P;
  }

  // The pieces a and b of a row, turned. For kAcross `row` is the row in shared memory.
  __device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float2* cs, const float* row, int P) const {
    const float4* two = reinterpret_cast<const float4*>(cs);
    if constexpr (MODE == kPair) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 t = two[j * 8 + unit];
        const float a0 = a[2 * j], a1 = a[2 * j + 1], b0 = b[2 * j], b1 = b[2 * j + 1];
        a[2 * j] = a0 * t.x - b0 * t.y;
        b[2 * j] = a0 * t.y + b0 * t.x;
        a[2 * j + 1] = a1 * t.z - b1 * t.w;
        b[2 * j + 1] = a1 * t.w + b1 * t.z;
      }
    } else if constexpr (MODE == kOwn) {
      const int left = P - unit * 8;                          // pairs of the lane's 8 that turn
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 t = two[j * 8 + unit];
        float* v = j < 2 ? a + 4 * j : b + 4 * (j - 2);
        const float v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3];
        if (2 * j < left) {
          v[0] = v0 * t.x - v1 * t.y;
          v[1] = v0 * t.y + v1 * t.x;
        }
        if (2 * j + 1 < left) {
          v[2] = v2 * t.z - v3 * t.w;
          v[3] = v2 * t.w + v3 * t.z;
        }
      }
    } else {
      // Element a0 + i's place is 17 unit + i; that of an element `by` further on 17 unit
      // + (i + by) + floor((i + by) / 16), with the same step for all lanes.
      const float* mine = row + unit * 17;
      const float2* turns = cs + unit * 17;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int up = i + P, down = i - P;
        if (a0 + i >= 2 * P) break;
        const bool first = a0 + i < P;
        float& v = i < 8 ? a[i & 7] : b[i & 7];
        const int down_at = down + (down >> 4);
        const float2 t = turns[first ? i : down_at];
        const float w = mine[first ? up + (up >> 4) : down_at];
        v = v * t.x + w * (first ? -t.y : t.y);
      }
    }
  }
};

// The shape of a block's work. Its warps read `slots` rows at a time (with the blocks
// in y); a lane keeps its row's number, and goes from token to token: every
// `abreast`-th, where that many tokens' rows fit in the slots.
struct RowPlan {
  int tokens, rows, abreast;
};

// One kind of row of one token.
template <typename Src>
struct Row {
  const Src* at;
  int64_t token;                                             // stride
};

// Calls store(row, element, values, to) with the pieces of all rows of `have` tokens.
// where(row) gives the place of the first token's row, and target(token, row) the
// destination `to`, asked for a batch at a time; rows from `plain` on are not turned.
// ready() runs while the first batch is on its way, and ends with the block in step.
template <int D, int MODE, typename Src, typename Where, typename Ready, typename Target, typename Store>
__device__ __forceinline__ void turn_rows(const RowPlan& plan, int have, const float2 (*cs)[kTurns],
                                          RowBuffer<D, MODE>& rows_in, int P, int plain, Where where, Ready ready,
                                          Target target, Store store) {
  constexpr int kPer = 512 / D;                               // rows a warp reads at a time
  constexpr int kRows = 2;                                    // a lane has in flight
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const Lane<D, MODE> mine(P, lane);
  const int slots = kRopeWarps * kPer * int(gridDim.y);
  const int slot = (int(blockIdx.y) * kRopeWarps + warp) * kPer + lane / (D / 16);
  const int t_first = plan.abreast > 1 ? slot / plan.rows : 0;
  const bool idle = t_first >= plan.abreast;
  bool begun = false;
  for (int pass = 0; pass < plan.rows; pass += slots) {
    const int r = slot - t_first * plan.rows + pass;
    const bool there = r < plan.rows && !idle, turned = mine.on && r < plain;
    const Row<Src> row = where(there ? r : 0);
    for (int t0 = 0; t0 < have; t0 += plan.abreast * kRows) {
      Piece<Src> x[kRows], y[kRows];
      int64_t to[kRows];
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int t = t0 + t_first + k * plan.abreast;
        if (there && t < have) {
          x[k].load(row.at + t * row.token + mine.a0);
          y[k].load(row.at + t * row.token + mine.b0);
        }
      }
      if (!begun) ready();
      begun = true;
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int t = t0 + t_first + k * plan.abreast;
        to[k] = there && t < have ? target(t, r) : 0;
      }
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        if (t0 + k * plan.abreast >= have) break;
        const int t = t0 + t_first + k * plan.abreast;
        const bool here = there && t < have;
        float a[8], b[8];
        x[k].get(a);
        y[k].get(b);
        float* through = rows_in.x[MODE == kAcross ? warp : 0];
        if constexpr (MODE == kAcross) {
          through += lane / (D / 16) * row_floats(D);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            through[mine.unit * 17 + i] = a[i];
            through[mine.unit * 17 + 8 + i] = b[i];
          }
          __syncwarp();
        }
        if (here && turned) mine.turn(a, b, cs[t], through, P);
        if constexpr (MODE == kAcross) __syncwarp();         // read before the next row is put there
        if (here) {
          store(r, mine.a0, a, to[k]);
          store(r, mine.b0, b, to[k]);
        }
      }
    }
  }
}

// Cosines and sines of `have` tokens from t0 on.
template <int MODE>
__device__ __forceinline__ void fill_turns(const RopeTable& R, float2 (*cs)[kTurns], const int64_t* pos, int have,
                                           bool back) {
  for (int i = threadIdx.x; i < have * 64; i += kRopeThreads)
    if (i % 64 < R.pairs) cs[i / 64][turn_slot<MODE>(i % 64)] = cos_sin_of(R.turn[i % 64], pos[i / 64], R.amplitude, back);
}

// Blocks in x take `plan.tokens` tokens each, blocks in y share out their rows.
template <typename Src, typename Dst, int D, int MODE>
__global__ void __launch_bounds__(kRopeThreads, sizeof(Src) == 2 ? 4 : 3)
    rope_apply_kernel(const __grid_constant__ RopeTable R, RowSet X, const int64_t* pos, int64_t n_tokens, RowPlan plan,
                      int back) {
  __shared__ __align__(16) float2 cs[kRopeTokens][kTurns];
  __shared__ RowBuffer<D, MODE> rows_in;
  pdl_trigger();
  pdl_wait();
  for (int64_t t0 = int64_t(blockIdx.x) * plan.tokens; t0 < n_tokens; t0 += int64_t(gridDim.x) * plan.tokens) {
    const int have = int(min64(plan.tokens, n_tokens - t0));
    const Src* src = static_cast<const Src*>(X.src) + t0 * X.src_token;
    Dst* dst = static_cast<Dst*>(X.dst) + t0 * X.dst_token;
    turn_rows<D, MODE, Src>(
        plan, have, cs, rows_in, R.pairs, X.heads, [&](int r) { return Row<Src>{src + r * X.src_head, X.src_token}; },
        [&] {
          __syncthreads();
          fill_turns<MODE>(R, cs, pos + t0, have, back != 0);
          __syncthreads();
        },
        [&](int t, int r) { return t * X.dst_token + r * X.dst_head; },
        [&](int, int e, const float (&v)[8], int64_t to) { store_8(dst + to + e, v); });
  }
}

template <typename Src, typename Kv, typename Qo, int D, int MODE>
__global__ void __launch_bounds__(kRopeThreads, sizeof(Src) == 2 ? 4 : 3)
    rope_append_kernel(const __grid_constant__ RopeTable R, RowSet Q, RowSet K, RowSet V, KvView kv, int n_seqs,
                       const int32_t* seq, const int64_t* index, const int64_t* pos, int64_t n_new, RowPlan plan, int chunk,
                       int32_t* status) {
  __shared__ __align__(16) float2 cs[kRopeTokens][kTurns];
  __shared__ RowBuffer<D, MODE> rows_in;
  // Of each token, for its first KV head (-1: nothing is written): the table's entry
  // and the place in the page; in a contiguous cache the row.
  __shared__ int64_t s_at[kRopeTokens];
  __shared__ int32_t s_in[kRopeTokens];
  pdl_trigger();
  pdl_wait();
  const int hq = Q.heads, hkv = K.heads;
  const int64_t limit = kv.table == nullptr ? kv.ld : kv.max_blocks * chunk;
  for (int64_t t0 = int64_t(blockIdx.x) * plan.tokens; t0 < n_new; t0 += int64_t(gridDim.x) * plan.tokens) {
    const int have = int(min64(plan.tokens, n_new - t0));
    const Src* q = static_cast<const Src*>(Q.src) + t0 * Q.src_token;
    const Src* k = static_cast<const Src*>(K.src) + t0 * K.src_token;
    const Src* v = static_cast<const Src*>(V.src) + t0 * V.src_token;
    turn_rows<D, MODE, Src>(
        plan, have, cs, rows_in, R.pairs, R.pairs > 0 ? hq + hkv : 0,
        [&](int r) {
          return r < hq         ? Row<Src>{q + r * Q.src_head, Q.src_token}
                 : r < hq + hkv ? Row<Src>{k + (r - hq) * K.src_head, K.src_token}
                                : Row<Src>{v + (r - hq - hkv) * V.src_head, V.src_token};
        },
        [&] {
          __syncthreads();
          if (threadIdx.x < have) {
            const int t = threadIdx.x;
            const int32_t s = seq[t0 + t];
            const int64_t at = index[t0 + t];
            const bool fits = s < n_seqs && at >= 0 && at < limit;
            if (s >= 0 && !fits && status != nullptr && blockIdx.y == 0) atomicOr(status, ZHA_DEV_BAD_SEQUENCE);
            const int block = kv.table == nullptr || !fits ? 0 : int(at >> 32 ? at / chunk : uint32_t(at) / uint32_t(chunk));
            const int64_t head = int64_t(s) * hkv;
            s_at[t] = s < 0 || !fits ? -1 : kv.table == nullptr ? head * kv.ld + at : head * kv.max_blocks + block;
            s_in[t] = int(at - int64_t(block) * chunk);
          }
          fill_turns<MODE>(R, cs, (pos != nullptr ? pos : index) + t0, have, false);
          __syncthreads();
        },
        // the row in q_out or in the cache, -1: none
        [&](int t, int r) -> int64_t {
          const int64_t at = s_at[t];
          if (at < 0) return -1;
          if (r < hq) return (t0 + t) * hq + r;
          const int g = r < hq + hkv ? r - hq : r - hq - hkv;
          if (kv.table == nullptr) return at + g * kv.ld;
          const int32_t page = kv.table[at + g * kv.max_blocks];
          if (page >= 0 && page < kv.ld) return int64_t(page) * chunk + s_in[t];
          if (status != nullptr) atomicOr(status, ZHA_DEV_BAD_PAGE);
          return -1;
        },
        [&](int r, int e, const float (&x)[8], int64_t to) {
          if (to < 0) return;
          if (r < hq) store_8(static_cast<Qo*>(Q.dst) + to * D + e, x);
          else store_8(static_cast<Kv*>(r < hq + hkv ? K.dst : V.dst) + to * D + e, x);
        });
  }
}

RopeTable table_of(const zha_rope* r) {
  RopeTable t{};
  if (r == nullptr) return t;
  t.pairs = r->pairs;
  t.half = r->layout == ZHA_ROPE_HALF;
  t.amplitude = r->amplitude;
  for (int i = 0; i < 64; ++i) t.turn[i] = r->turn[i];
  return t;
}

// Tokens a block: enough for kRopeTarget rows of 128 elements (the turns and the
// block's start are paid once), but none idle while another has two.
// Few tokens have their rows spread over blocks in y.
struct RopeGrid {
  dim3 grid;
  RowPlan plan;
};
RopeGrid rope_grid(int64_t n, int64_t rows, int d, int sms) {
  RopeGrid g;
  const int64_t target = int64_t(kRopeTarget) * 128 / d, at_once = kRopeWarps * (512 / d);
  int64_t tokens = min64(kRopeTokens, round_up((target + rows - 1) / rows, 2));
  tokens = max64(1, min64(tokens, n / (int64_t(sms) * 2)));
  const int64_t x = (n + tokens - 1) / tokens;
  const int64_t y = max64(1, min64((tokens * rows + at_once - 1) / at_once, int64_t(sms) * 8 / x));
  g.grid = dim3(unsigned(min64(x, 1 << 20)), unsigned(min64(y, 65535)));
  g.plan.tokens = int(tokens);
  g.plan.rows = int(rows);
  g.plan.abreast = int(max64(1, min64(tokens, at_once * g.grid.y / rows)));
  return g;
}

bool rope_ok(const zha_rope* r) {
  return r->pairs >= 1 && (r->head_dim == 64 || r->head_dim == 128) && r->pairs <= r->head_dim / 2 &&
         (r->layout == ZHA_ROPE_INTERLEAVED || r->layout == ZHA_ROPE_HALF);
}

bool dtype_ok(int32_t t) { return t == ZHA_F32 || t == ZHA_BF16; }

// Rows addressable in 16-byte pieces.
bool rows_ok(const zha_rows* r, int32_t dtype) {
  const int64_t per = dtype == ZHA_F32 ? 4 : 8;
  auto in_range = [](int64_t v) { return v >= -(int64_t(1) << 40) && v <= (int64_t(1) << 40); };
  return r != nullptr && r->data != nullptr && reinterpret_cast<uintptr_t>(r->data) % 16 == 0 &&
         r->token_stride % per == 0 && r->head_stride % per == 0 && in_range(r->token_stride) &&
         in_range(r->head_stride);
}

// Whether no two rows overlap, judged by strides in sizes: the smaller stride
// spans a row, the larger one all rows of the other kind. (Interleaved layouts
// that avoid each other some other way are refused.)
bool rows_apart(const zha_rows* r, int64_t tokens, int64_t heads, int64_t d) {
  const int64_t t = r->token_stride < 0 ? -r->token_stride : r->token_stride;
  const int64_t h = r->head_stride < 0 ? -r->head_stride : r->head_stride;
  if (tokens == 1) return heads == 1 || h >= d;
  if (heads == 1) return t >= d;
  return h <= t ? h >= d && (t - d) / h >= heads - 1 : t >= d && (h - d) / t >= tokens - 1;
}

template <typename Src, typename Dst, int D, int MODE>
cudaError_t launch_apply(const RopeTable& R, const RowSet& X, const int64_t* pos, int64_t n, int back, const RopeGrid& g,
                         cudaStream_t s) {
  TraceScope ts("rope_apply_kernel", 0, s);
  zha_count_launch();
  return launch_pdl(rope_apply_kernel<Src, Dst, D, MODE>, g.grid, dim3(kRopeThreads), 0, s, R, X, pos, n, g.plan, back);
}

template <typename Src, typename Kv, typename Qo, int D, int MODE>
cudaError_t launch_append(const RopeTable& R, const RowSet& Q, const RowSet& K, const RowSet& V, const KvView& kv,
                          int n_seqs, const int32_t* seq, const int64_t* index, const int64_t* pos, int64_t n, int chunk,
                          int32_t* status, const RopeGrid& g, cudaStream_t s) {
  TraceScope ts("rope_append_kernel", 0, s);
  zha_count_launch();
  return launch_pdl(rope_append_kernel<Src, Kv, Qo, D, MODE>, g.grid, dim3(kRopeThreads), 0, s, R, Q, K, V, kv, n_seqs, seq,
                    index, pos, n, g.plan, chunk, status);
}

// f(head dimension, mode) with both as types.
template <typename F>
cudaError_t with_shape(int d, int mode, F f) {
  using std::integral_constant;
  auto by_mode = [&](auto dim) {
    switch (mode) {
      case kOwn: return f(dim, integral_constant<int, kOwn>());
      case kPair: return f(dim, integral_constant<int, kPair>());
      default: return f(dim, integral_constant<int, kAcross>());
    }
  };
  return d == 128 ? by_mode(integral_constant<int, 128>()) : by_mode(integral_constant<int, 64>());
}
template <typename F>
cudaError_t with_type(int32_t dtype, F f) {
  return dtype == ZHA_F32 ? f(float()) : f(__nv_bfloat16());
}

}  // namespace

}  // namespace zha

using zha::RowSet;

static zha_status rope_fail(zha_status s, const char* msg) { return zha_report_error(s, msg); }

extern "C" {

zha_status zha_rope_init(const zha_rope_spec* c, zha_rope* out) {
  if (c == nullptr || out == nullptr) return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: spec or out is NULL");
  if (c->head_dim != 64 && c->head_dim != 128)
    return rope_fail(ZHA_ERR_UNSUPPORTED, "zha_rope_init: head_dim must be 64 or 128");
  if (c->pairs < 1 || c->pairs > c->head_dim / 2)
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: pairs outside [1, head_dim / 2]");
  if (c->layout != ZHA_ROPE_INTERLEAVED && c->layout != ZHA_ROPE_HALF)
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: unknown layout");
  if (c->scaling < ZHA_ROPE_PLAIN || c->scaling > ZHA_ROPE_BANDS)
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: unknown scaling");
  if (c->reserved != 0) return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: reserved must be 0");
  if (!(c->base > 1.0) || !std::isfinite(c->base))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: base must be finite and > 1");
  const int D = c->freq_dim == 0 ? 2 * c->pairs : c->freq_dim;
  if (D < 2) return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: freq_dim must be 0 or >= 2");
  const double f = c->scaling == ZHA_ROPE_PLAIN ? 1.0 : c->factor;
  if (!(f >= 1.0) || !std::isfinite(f))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: factor must be finite and >= 1");
  const bool banded = c->scaling == ZHA_ROPE_YARN || c->scaling == ZHA_ROPE_BANDS;
  if (banded && !(c->original_tokens > 0 && std::isfinite(c->original_tokens) && c->low > 0 && c->high > c->low &&
                  std::isfinite(c->high)))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: need original_tokens > 0 and 0 < low < high");
  if (!(c->amplitude >= 0.0) || !std::isfinite(float(c->amplitude)) || (c->amplitude > 0.0 && float(c->amplitude) == 0.f))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: amplitude must be >= 0 and in the range of float32");
  const double two_pi = 6.283185307179586476925286766559;
  double base = c->base;
  if (c->scaling == ZHA_ROPE_NTK && D > 2) base *= std::pow(f, double(D) / (D - 2));
  double lo = 0.0, hi = 0.0;
  if (c->scaling == ZHA_ROPE_YARN) {
    auto where = [&](double turns) {
      return D * std::log(c->original_tokens / (two_pi * turns)) / (2.0 * std::log(c->base));
    };
    lo = std::fmax(0.0, std::floor(where(c->high)));
    hi = std::fmin(double(D - 1), std::ceil(where(c->low)));
  }
  zha_rope r{};
  r.head_dim = c->head_dim;
  r.pairs = c->pairs;
  r.layout = c->layout;
  r.amplitude = float(c->amplitude > 0.0                  ? c->amplitude
                      : c->scaling == ZHA_ROPE_YARN ? 0.1 * std::log(f) + 1.0
                                                    : 1.0);
  for (int i = 0; i < c->pairs; ++i) {
    double theta = std::pow(base, -2.0 * i / D);
    if (c->scaling == ZHA_ROPE_LINEAR || (c->scaling == ZHA_ROPE_NTK && D == 2)) {
      theta /= f;
    } else if (c->scaling == ZHA_ROPE_YARN) {
      const double w = std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 0.001)));
      theta = theta * (1.0 - w) + theta / f * w;
    } else if (c->scaling == ZHA_ROPE_BANDS) {
      const double n = c->original_tokens * theta / two_pi;
      const double w = std::fmin(1.0, std::fmax(0.0, (n - c->low) / (c->high - c->low)));
      theta = w * theta + (1.0 - w) * theta / f;
    }
    r.turn[i] = uint64_t(std::ldexp(theta / two_pi, 64));      // theta <= 1: below 2^62
  }
  *out = r;
  return ZHA_OK;
}

zha_status zha_rope_apply(const zha_rope* rope, const zha_rows* x, int32_t x_dtype, const int64_t* d_pos,
                          int64_t n_tokens, int32_t n_heads, int32_t inverse, const zha_rows* y, int32_t y_dtype,
                          void* stream) {
  if (rope == nullptr || !zha::rope_ok(rope))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_apply: rope is NULL or was not filled by zha_rope_init");
  if (!zha::dtype_ok(x_dtype) || !zha::dtype_ok(y_dtype))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_apply: unknown element type");
  if (n_tokens < 0 || n_tokens > (int64_t(1) << 40) || n_heads < 1 || n_heads > 65536)
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_apply: n_tokens or n_heads out of range");
  if (n_tokens == 0) return ZHA_OK;
  if (!zha::rows_ok(x, x_dtype) || !zha::rows_ok(y, y_dtype) || d_pos == nullptr)
    return rope_fail(ZHA_ERR_INVALID,
                     "zha_rope_apply: rows and positions must be non-NULL, rows 16-byte aligned with strides of "
                     "whole 16-byte pieces");
  if (!zha_may_lie(d_pos))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_apply: positions at no multiple of 8 bytes");
  if (x->data == y->data &&
      (x_dtype != y_dtype || x->token_stride != y->token_stride || x->head_stride != y->head_stride))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_apply: in place, both sides need one type and one set of strides");
  if (!zha::rows_apart(y, n_tokens, n_heads, rope->head_dim))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_apply: rows of y overlap one another");
  const zha::RopeTable R = zha::table_of(rope);
  RowSet X{x->data, const_cast<void*>(y->data), x->token_stride, x->head_stride, y->token_stride, y->head_stride,
           n_heads};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int d = rope->head_dim, back = inverse != 0;
  int sms = 0;
  cudaError_t e = zha::device_sm_count(&sms);
  if (e != cudaSuccess) return zha_report_cuda(e, "zha_rope_apply");
  const zha::RopeGrid g = zha::rope_grid(n_tokens, n_heads, d, sms);
  e = zha::with_shape(d, zha::mode_of(R), [&](auto dim, auto mode) {
    return zha::with_type(x_dtype, [&](auto src) {
      return zha::with_type(y_dtype, [&](auto dst) {
        return zha::launch_apply<decltype(src), decltype(dst), dim.value, mode.value>(R, X, d_pos, n_tokens, back, g, s);
      });
    });
  });
  return e == cudaSuccess ? ZHA_OK : zha_report_cuda(e, "zha_rope_apply");
}

zha_status zha_rope_append_kv(const zha_config* cfg, const zha_rope* rope, const zha_rows* q, const zha_rows* k,
                              const zha_rows* v, int32_t src_dtype, int64_t n_new, const zha_kv_cache* kv,
                              int32_t n_seqs, const int32_t* d_seq, const int64_t* d_index, const int64_t* d_pos,
                              void* d_q_out, int32_t q_dtype, int32_t* d_status, void* stream) {
  const char* who = "zha_rope_append_kv";
  zha::Geom G;
  zha_status st = zha_geometry(cfg, &G);
  if (st != ZHA_OK) return st;
  zha::KvView view{};
  if ((st = zha_batch_view(G, kv, n_seqs, 0, who, &view)) != ZHA_OK) return st;
  if (rope != nullptr && (!zha::rope_ok(rope) || rope->head_dim != G.d))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_append_kv: rope was not filled by zha_rope_init for this head_dim");
  if (!zha::dtype_ok(src_dtype) || !zha::dtype_ok(q_dtype))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_append_kv: unknown element type");
  if (n_new < 0 || n_new > (int64_t(1) << 40) || G.hq > 65536)
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_append_kv: n_new or n_q_heads out of range");
  if (n_new == 0) return ZHA_OK;
  if (!zha::rows_ok(k, src_dtype) || !zha::rows_ok(v, src_dtype) || (q != nullptr && !zha::rows_ok(q, src_dtype)))
    return rope_fail(ZHA_ERR_INVALID,
                     "zha_rope_append_kv: rows must be non-NULL and 16-byte aligned with strides of whole 16-byte "
                     "pieces");
  if (q != nullptr && (d_q_out == nullptr || reinterpret_cast<uintptr_t>(d_q_out) % 16 != 0))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_append_kv: q_out must be a non-NULL 16-byte aligned device pointer");
  if (d_seq == nullptr || d_index == nullptr)
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_append_kv: seq and index must be non-NULL");
  if (!zha_may_lie(d_seq) || !zha_may_lie(d_index) || !zha_may_lie(d_pos) || !zha_may_lie(d_status))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_append_kv: seq, index, positions or status at no multiple of its type's size");
  const zha::RopeTable R = zha::table_of(rope);
  RowSet Q{}, K{}, V{};
  if (q != nullptr) Q = RowSet{q->data, d_q_out, q->token_stride, q->head_stride, int64_t(G.hq) * G.d, G.d, G.hq};
  K = RowSet{k->data, const_cast<void*>(kv->k), k->token_stride, k->head_stride, 0, 0, G.hkv};
  V = RowSet{v->data, const_cast<void*>(kv->v), v->token_stride, v->head_stride, 0, 0, G.hkv};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int sms = 0;
  cudaError_t e = zha::device_sm_count(&sms);
  if (e != cudaSuccess) return zha_report_cuda(e, who);
  const zha::RopeGrid g = zha::rope_grid(n_new, int64_t(Q.heads) + 2 * G.hkv, G.d, sms);
  e = zha::with_shape(G.d, zha::mode_of(R), [&](auto dim, auto mode) {
    return zha::with_type(src_dtype, [&](auto src) {
      return zha::with_type(G.kv_bf16 ? ZHA_BF16 : ZHA_F32, [&](auto cache) {
        return zha::with_type(q_dtype, [&](auto out) {
          return zha::launch_append<decltype(src), decltype(cache), decltype(out), dim.value, mode.value>(
              R, Q, K, V, view, n_seqs, d_seq, d_index, d_pos, n_new, G.chunk, d_status, g, s);
        });
      });
    });
  });
  return e == cudaSuccess ? ZHA_OK : zha_report_cuda(e, who);
}

}  // extern "C"
