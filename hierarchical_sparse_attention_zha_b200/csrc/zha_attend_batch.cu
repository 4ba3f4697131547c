// zha_attend_batch.cu -- dense attention of one query token per sequence over a
// batch of (paged) caches. Semantics are in include/zha.h.
//
// Mathematics. o = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m), x_j = q.k_j
// log2(e) / sqrt(d): any m gives the same quotient, and states (m, l, o) of two
// parts of the keys join as m = max, l = sum l_i 2^(m_i - m), o alike.
//
// Split. A unit is (sequence, KV head, block of its query heads); its keys are cut
// into tiles of 4 KB of K and 4 KB of V. All units' tiles, one behind the other, are
// dealt out evenly to the warps from the counts in device memory, so that ragged
// lengths cost nothing. SMs do not read equally fast (240K tokens: their shares took 58
// to 78 us), so a long call deals 11/12 of the tiles to the CTAs that the GPU holds at
// a time, and the rest to half as many more, which the SMs that are done first take.
// A warp keeps its own ring of tiles in flight (cp.async), across the borders of units,
// and waits for no other until its tiles are done. What then becomes of a unit's state:
//   - all of its tiles in one warp: the warp writes the result;
//   - it ends before the warp's last tile, having begun in an earlier warp: an end
//     piece in the workspace, at the warp's number;
//   - it reaches the warp's last tile: the CTA joins the states of its warps in that
//     unit, and writes the result or, with more of the unit elsewhere, a group piece, at
//     the number of the group's first warp.
// A second kernel finds a unit's pieces from the tile counts alone and joins them in a
// fixed order.
//
// Products. Up to 8 query heads a KV head the call is bound by the cache it reads and, when
// it runs for long, by the power that the products take: the warps' own matrix
// instructions (16 x 8 x 16 bf16, 16 x 8 x 8 tf32) take their operands from the warp's
// registers and tile without a hand-over. With 9 to 16 heads it is bound by the issue of these
// instructions, which is this choice's limit and not the hardware's (keys as the M of a tcgen05
// instruction would take them); beyond 16 the cache is read once per 16 heads. Keys
// and elements of V are their 16 rows, heads their 8 columns, so that no row is padding:
// S^T = K Q^T, O^T = V^T P^T. With up to 4 heads the columns hold two terms of the
// fp32 operand side by side.
//   bf16 cache: keys and values enter exactly. fp32 queries and weights are three
//   bf16 terms cut off one after the other (8 + 8 + 8 bits: exact); with bf16
//   queries, which are exact, weights are two terms (2^-16, below the output's 2^-8).
//   fp32 cache: every operand is two tf32 terms (cut, then rounded: 2^-22), and of
//   weight times value the product of the two second terms (2^-11 of the weight, 2^-10
//   of the value) is left out where it would take an instruction of its own.
// Measured (held for half a second; the copy rate is 6.55 TB/s): 1M bf16 tokens of 4 KV
// heads with 8 fp32 query heads each in 321 to 347 us by GPU (6.2 to 6.57 TB/s); 8
// sequences up to 32K of 8 KV heads, 4 bf16 query heads each, in 98 to 102 us (91 to 94%);
// 160 ragged ones up to 3001 in 90 us (80%). A call starts to read after 3 us, and the
// join takes 3 to 4 us, whatever the length. One bulk copy per row instead of 16 cp.async
// of 16 bytes: 495 us for the 1M tokens, 17 cycles of an SM each.
#include <cmath>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;              // tiles in a warp's ring
constexpr int kTileBytes = 4096;        // of K, and of V
constexpr int kMaxSms = 148;
constexpr int kMaxCtas = kMaxSms * 3;   // two a SM at a time, and half as many later
constexpr int kMaxWarps = kMaxCtas * kWarps;
// The second deal pays from some tiles a warp on (8 x 32K tokens, 4 heads a unit: 100
// us with it, 106 without; 160 ragged sequences 92, 95), but not where the products, not
// the reads, take the time (12 heads: 143 with it, 135 without). An eighth to as many
// CTAs as in the first: 105 and 95; a sixteenth to half as many 102 and 93.
constexpr int kTwoTiers = 24;
// What a unit's start and end cost, in tiles: the deal counts them, so that a warp with
// many short units has fewer tiles (238 sequences up to 255 tokens of 8 KV heads, with their
// caches partly in L2: 33.7 us, 53.5 without; 1 37.2, 5 34.7; from HBM 40).
constexpr int kUnitCost = 2;
constexpr int kMinTiles = 2;            // no warp takes less, unless there is less
// Up to so many tiles a unit, and no more units than CTAs at a time, a CTA takes a
// whole unit and no second kernel is needed (64 sequences of 500 tokens and 4 heads:
// 12.1 us, split 16.9; 4 of 256 8.5, 11.2; but 4 of 1000 19.0, split 13.1).
constexpr int kSingleTiles = 32;
constexpr int kJoinThreads = 256;
// Up to so many units, each in many pieces, a CTA joins one head, else one unit (60K
// tokens in 4 units: 31.1 us, 36.9 by units).
constexpr int kWideUnits = 148;
// A unit's warps otherwise, two heads each (160 ragged sequences of 4 heads a unit: 89.3
// us, 91.7 with 4 heads each).
__host__ __device__ constexpr int join_warps_of(int hu, int group) { return ((group < hu ? group : hu) + 1) / 2; }

// Heads a unit: the fewest columns that take the group (8 x 32K tokens of 4 heads: 102.5
// us with 4 columns and two terms side by side, 104.4 with 8; of 12 heads 142.9 with
// 16, 184.0 with two units of 8, which read the cache twice).
inline int head_cols(int group) { return group > 8 ? 16 : group > 4 ? 8 : 4; }

struct BatchLayout {
  int64_t slots, bytes, slots_off;
  int32_t hb, hu;                       // head blocks per KV head, heads per block
};

// Workspace: int64 prefix[n_seqs + 1] (tiles of one unit of the sequences before s);
// then the group pieces and the end pieces, [m, l, -, -, o[d]] for each of a unit's
// heads.
inline BatchLayout batch_layout(const Geom& G, int32_t n_seqs) {
  BatchLayout b{};
  b.hu = head_cols(G.group);
  b.hb = (G.group + b.hu - 1) / b.hu;
  b.slots = 2 * kMaxWarps;
  b.slots_off = round_up((int64_t(n_seqs) + 1) * 8, 256);
  b.bytes = b.slots_off + round_up(b.slots * b.hu * (G.d + 4) * 4, 256);
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
  int32_t n_seqs, hkv, hq, group, hb, chunk, single, wide;
  int32_t first_ctas, ctas;             // of the first deal, of both
  uint32_t div_mul, div_shift;          // t / chunk = t * div_mul >> div_shift for t < 2^31
  float scale_log2;                     // log2(e) / sqrt(d)
};

// ---- small pieces -----------------------------------------------------------
__device__ __forceinline__ void store_o(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_o(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  uint2 x;
  __nv_bfloat162 lo = __floats2bfloat162_rn(a, b), hi = __floats2bfloat162_rn(c, d);
  x.x = *reinterpret_cast<uint32_t*>(&lo);
  x.y = *reinterpret_cast<uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(p) = x;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes into shared memory, or 16 zeros.
__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t to, const void* from, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The next bf16 term of a pair of values: the upper halves cut off and taken away.
// (Of an infinite value the next term is NaN.)
__device__ __forceinline__ uint32_t cut_bf16(float& a, float& b) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  a = a - __uint_as_float(ua & 0xffff0000u);
  b = b - __uint_as_float(ub & 0xffff0000u);
  return __byte_perm(ua, ub, 0x7632);
}
// The two tf32 terms of a value: 11 bits cut off, the rest rounded to 11.
__device__ __forceinline__ void split_tf32(float x, uint32_t& one, uint32_t& two) {
  one = __float_as_uint(x) & 0xffffe000u;
  two = (__float_as_uint(x - __uint_as_float(one)) + 0x1000u) & 0xffffe000u;
}

// Of a weight in [0, 1], which rounding cannot take out of range: both rounded (2^-23).
__device__ __forceinline__ void split_weight(float x, uint32_t& one, uint32_t& two) {
  one = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  two = (__float_as_uint(x - __uint_as_float(one)) + 0x1000u) & 0xffffe000u;
}

// An 8 x 8 matrix of 16-bit values turned over its diagonal: lane (g, t) gives row g,
// columns 2 t and 2 t + 1, and gets column g, rows 2 t and 2 t + 1.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// ---- tiles ------------------------------------------------------------------
// Shared memory keeps a row's 16-byte pieces at piece ^ swizzle(row), so that the
// reads below meet no bank twice: a K read takes four adjacent pieces of two rows per 8
// lanes; a V read takes one piece of 8 rows (bf16), or two of every second row (fp32).
template <typename Kv, int D>
struct Tile {
  static constexpr int kRow = D * int(sizeof(Kv));
  static constexpr int kKeys = kTileBytes / kRow;         // bf16: 16 or 32; fp32: 8 or 16
  static constexpr int kPieces = kRow / 16;               // 8, 16 or 32
  __device__ static int at_k(int row, int piece) { return row * kRow + ((piece ^ ((row & 1) << 2)) << 4); }
  __device__ static int at_v(int row, int piece) { return row * kRow + ((piece ^ (row & 7)) << 4); }
};

// A place in the row of tiles: unit (s, ub) of sequence s with n tokens has the
// tiles [first, end), behind kUnitCost places that stand for its start and end.
struct Place {
  int64_t first, end, n;
  int s, ub;
};

__device__ __forceinline__ int64_t clamped(const BatchArgs& A, int s) {
  return max64(0, min64(A.n_tokens[s], A.max_tokens));
}
template <int KEYS>
__device__ __forceinline__ int64_t tiles_of(int64_t n) { return (n + KEYS - 1) / KEYS; }
// A unit's places in the row.
template <int KEYS>
__device__ __forceinline__ int64_t places_of(int64_t n) { return n == 0 ? 0 : kUnitCost + (n + KEYS - 1) / KEYS; }

// (The hardware has no integer division: 32-bit ones take a fifth of the 64-bit ones.)
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// n tiles dealt to w warps: the first r get q + 1.
struct Even {
  int64_t q, r;
  __device__ Even(int64_t n, int64_t w) : q(quotient(n, w)), r(n - q * w) {}
  __device__ int64_t start(int64_t w) const { return w * q + min64(w, r); }
  __device__ int64_t owner(int64_t t) const {
    const int64_t more = r * (q + 1);
    return t < more ? quotient(t, q + 1) : r + quotient(t - more, q);
  }
};

// All tiles dealt to the warps of both tiers.
struct Deal {
  int64_t total, n1, w1, w2;
  Even one, two;
  __device__ static int64_t first_tiles(const BatchArgs& A, int64_t n) {
    return A.ctas > A.first_ctas && n >= int64_t(kTwoTiers) * kWarps * A.first_ctas ? n - n / 12 : n;
  }
  __device__ static int64_t first_warps(const BatchArgs& A, int64_t n) {
    return max64(1, min64(int64_t(A.first_ctas) * kWarps, (n + kMinTiles - 1) / kMinTiles));
  }
  __device__ Deal(const BatchArgs& A, int64_t n)
      : total(n), n1(first_tiles(A, n)), w1(first_warps(A, n)), w2(max64(1, int64_t(A.ctas - A.first_ctas) * kWarps)),
        one(n1, w1), two(n - n1, w2) {}
  __device__ int64_t start(int64_t w) const {
    return w <= w1 ? one.start(w) : n1 == total ? total : n1 + two.start(min64(w - w1, w2));
  }
  __device__ int64_t owner(int64_t t) const { return t < n1 ? one.owner(t) : w1 + two.owner(t - n1); }
};

// To the next unit that has tiles; the caller knows that there is one.
template <int KEYS>
__device__ __forceinline__ void next_unit(const BatchArgs& A, Place& p) {
  if (++p.ub == A.hkv * A.hb) {
    p.ub = 0;
    do p.n = clamped(A, ++p.s); while (p.n == 0);
  }
  p.first = p.end + kUnitCost;
  p.end = p.first + tiles_of<KEYS>(p.n);
}

// What a lane (g, t) = (lane / 4, lane % 4) has of the columns: 2 t and 2 t + 1 of a
// product, g of an operand. Column c of tile q is head c % HU + 8 q, and (HU 4) term
// c / HU of the pair of terms that an instruction takes.
template <int HU>
struct Columns {
  static constexpr int kTiles = HU == 16 ? 2 : 1;
  static constexpr int kTerms = HU == 4 ? 2 : 1;             // terms side by side
  __device__ static int head(int q, int t, int e) { return HU == 4 ? 2 * (t & 1) + e : 8 * q + 2 * t + e; }
};

// Queries as operands: [step][tile][instruction][2]. The order of a head's elements
// within a step is that of the K reads: lane t's piece of 16 bytes serves two steps.
template <typename Kv, typename Qt, int D, int HU>
struct Queries {
  static constexpr bool kBf = sizeof(Kv) == 2;
  static constexpr int kSteps = kBf ? D / 16 : D / 8;
  static constexpr int kTerms = kBf ? (sizeof(Qt) == 2 ? 1 : 3) : 2;
  static constexpr int kTiles = Columns<HU>::kTiles, kSide = Columns<HU>::kTerms;
  static constexpr int kOps = (kTerms + kSide - 1) / kSide;
  uint32_t b[kSteps][kTiles][kOps][2];

  // Operand register i of step st from the terms of its value (a pair of values).
  __device__ __forceinline__ void put(int st, int q, int i, const uint32_t (&term)[kTerms], int side) {
#pragma unroll
    for (int k = 0; k < kOps; ++k) {
      if constexpr (kSide == 1) {
        b[st][q][k][i] = term[k];
      } else {
        const uint32_t first = term[2 * k], second = 2 * k + 1 < kTerms ? term[min(2 * k + 1, kTerms - 1)] : 0u;
        b[st][q][k][i] = side ? second : first;
      }
    }
  }

  __device__ void load(const Qt* queries, int heads, int lane) {
    const int g = lane / 4, t = lane % 4, side = HU == 4 ? g / 4 : 0;
#pragma unroll
    for (int q = 0; q < kTiles; ++q) {
      const int h = HU == 4 ? g % 4 : g + 8 * q;
      const Qt* row = queries + h * D;
#pragma unroll
      for (int j = 0; j < kSteps / 2; ++j) {
        if constexpr (kBf) {
          float v[8] = {};
          if (h < heads) {
            if constexpr (sizeof(Qt) == 2) {
              load_slice<8>(row, 32 * j + 8 * t, v);
            } else {
              float x[4], y[4];
              load_slice<4>(row, 32 * j + 8 * t, x);
              load_slice<4>(row, 32 * j + 8 * t + 4, y);
#pragma unroll
              for (int i = 0; i < 4; ++i) { v[i] = x[i]; v[4 + i] = y[i]; }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t term[kTerms];
#pragma unroll
            for (int k = 0; k < kTerms; ++k) term[k] = cut_bf16(v[2 * i], v[2 * i + 1]);
            put(2 * j + i / 2, q, i % 2, term, side);
          }
        } else {
          float v[4] = {};
          if (h < heads) load_slice<4>(row, 16 * j + 4 * t, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t term[kTerms];
            split_tf32(v[i], term[0], term[1]);
            put(2 * j + i / 2, q, i % 2, term, side);
          }
        }
      }
    }
  }

  // s[q][block][e]: key 8 * block + g, column 2 t + e.
  template <int NB>
  __device__ void scores(const char* tile, int lane, float (&s)[kTiles][NB][2]) const {
    const int g = lane / 4, t = lane % 4;
    if constexpr (kBf) {
#pragma unroll
      for (int mb = 0; mb < NB / 2; ++mb) {                  // 16 keys
        float c[kTiles][kOps][4] = {};
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 x = *reinterpret_cast<const uint4*>(tile + Tile<Kv, D>::at_k(16 * mb + g, 4 * j + t));
          const uint4 y = *reinterpret_cast<const uint4*>(tile + Tile<Kv, D>::at_k(16 * mb + 8 + g, 4 * j + t));
#pragma unroll
          for (int q = 0; q < kTiles; ++q)
#pragma unroll
            for (int k = 0; k < kOps; ++k) {
              mma_bf16(c[q][k], x.x, y.x, x.y, y.y, b[2 * j][q][k][0], b[2 * j][q][k][1]);
              mma_bf16(c[q][k], x.z, y.z, x.w, y.w, b[2 * j + 1][q][k][0], b[2 * j + 1][q][k][1]);
            }
        }
#pragma unroll
        for (int q = 0; q < kTiles; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = c[q][kOps - 1][i];
#pragma unroll
            for (int k = kOps - 2; k >= 0; --k) v += c[q][k][i];
            s[q][2 * mb + i / 2][i % 2] = v;
          }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NB; ++n) {                         // 8 keys: rows g first terms, rows g + 8 second terms
        float c[kTiles][kOps][4] = {};
#pragma unroll
        for (int j = 0; j < D / 16; ++j) {
          const float4 x = *reinterpret_cast<const float4*>(tile + Tile<Kv, D>::at_k(8 * n + g, 4 * j + t));
          uint32_t one[4], two[4];
          split_tf32(x.x, one[0], two[0]);
          split_tf32(x.y, one[1], two[1]);
          split_tf32(x.z, one[2], two[2]);
          split_tf32(x.w, one[3], two[3]);
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int q = 0; q < kTiles; ++q)
#pragma unroll
              for (int k = 0; k < kOps; ++k)
                mma_tf32(c[q][k], one[2 * u], two[2 * u], one[2 * u + 1], two[2 * u + 1], b[2 * j + u][q][k][0],
                         b[2 * j + u][q][k][1]);
        }
#pragma unroll
        for (int q = 0; q < kTiles; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float low = c[q][0][2 + e];
#pragma unroll
            for (int k = 1; k < kOps; ++k) low += c[q][k][e] + c[q][k][2 + e];
            s[q][n][e] = c[q][0][e] + low;
          }
      }
    }
    if constexpr (kSide == 2) {                              // the two terms' parts
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) s[0][n][e] += __shfl_xor_sync(0xffffffffu, s[0][n][e], 2);
    }
  }
};

// o[q][tile of 16 elements] += V^T * weights; p as the scores. The matrix instructions
// cut their sums off instead of rounding them, which over a long cache adds up (1M
// keys: 9e-6 of the largest output): they sum a tile's keys alone, from zero, and o is
// summed by rounded additions (1e-6).
template <typename Kv, int D, int HU, int TERMS, int NB>
__device__ __forceinline__ void add_values(uint32_t tile_at, const char* tile, int lane,
                                           float (&p)[Columns<HU>::kTiles][NB][2],
                                           float (&o)[Columns<HU>::kTiles][D / 16][4]) {
  constexpr int kTiles = Columns<HU>::kTiles, kSide = Columns<HU>::kTerms, kOps = (TERMS + kSide - 1) / kSide;
  const int g = lane / 4, t = lane % 4;
  const bool second = kSide == 2 && t >= 2;
  if constexpr (sizeof(Kv) == 2) {
#pragma unroll
    for (int mb = 0; mb < NB / 2; ++mb) {
      uint32_t w[kTiles][kOps][2];
#pragma unroll
      for (int q = 0; q < kTiles; ++q)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float* v = p[q][2 * mb + i];
          uint32_t term[TERMS];
#pragma unroll
          for (int k = 0; k < TERMS; ++k) term[k] = cut_bf16(v[0], v[1]);
#pragma unroll
          for (int k = 0; k < kOps; ++k) {
            uint32_t x = term[kSide * k];
            if constexpr (kSide == 2)
              if (second) x = 2 * k + 1 < TERMS ? term[min(2 * k + 1, TERMS - 1)] : 0u;
            w[q][k][i] = transposed(x);
          }
        }
      const int row = 16 * mb + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
      for (int d0 = 0; d0 < D / 16; d0 += 4) {               // 64 elements: every term in turn on 4 tiles of o
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                       : "=r"(v[i][0]), "=r"(v[i][1]), "=r"(v[i][2]), "=r"(v[i][3])
                       : "r"(tile_at + Tile<Kv, D>::at_v(row, 2 * (d0 + i) + ((lane >> 3) & 1)))
                       : "memory");
#pragma unroll
        for (int q = 0; q < kTiles; ++q) {
          float c[4][4] = {};
#pragma unroll
          for (int k = kOps - 1; k >= 0; --k)
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_bf16(c[i], v[i][0], v[i][1], v[i][2], v[i][3], w[q][k][0], w[q][k][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[q][d0 + i][j] += c[i][j];
        }
      }
    }
  } else {
    // Within 8 keys, the step's elements t and t + 4 are the keys 2 t and 2 t + 1.
    // Rows g and g + 8 of tile 4 j + i are the elements 64 j + 4 g + i and 32 more.
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      uint32_t w[kTiles][kOps][2];
#pragma unroll
      for (int q = 0; q < kTiles; ++q) {
        uint32_t one[2], two[2];
        split_weight(p[q][n][0], one[0], two[0]);
        split_weight(p[q][n][1], one[1], two[1]);
#pragma unroll
        for (int k = 0; k < kOps; ++k) {
          const uint32_t x = (kSide == 2 ? second : k == 1) ? two[0] : one[0];
          const uint32_t y = (kSide == 2 ? second : k == 1) ? two[1] : one[1];
          const uint32_t lo = transposed(__byte_perm(x, y, 0x5410)), hi = transposed(__byte_perm(x, y, 0x7632));
          w[q][k][0] = __byte_perm(lo, hi, 0x5410);
          w[q][k][1] = __byte_perm(lo, hi, 0x7632);
        }
      }
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        const float4 a = *reinterpret_cast<const float4*>(tile + Tile<Kv, D>::at_v(8 * n + 2 * t, 16 * j + g));
        const float4 b = *reinterpret_cast<const float4*>(tile + Tile<Kv, D>::at_v(8 * n + 2 * t, 16 * j + 8 + g));
        const float4 c = *reinterpret_cast<const float4*>(tile + Tile<Kv, D>::at_v(8 * n + 2 * t + 1, 16 * j + g));
        const float4 d = *reinterpret_cast<const float4*>(tile + Tile<Kv, D>::at_v(8 * n + 2 * t + 1, 16 * j + 8 + g));
        const float v[4][4] = {{a.x, b.x, c.x, d.x}, {a.y, b.y, c.y, d.y}, {a.z, b.z, c.z, d.z}, {a.w, b.w, c.w, d.w}};
        uint32_t one[4][4], two[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) split_tf32(v[i][r], one[i][r], two[i][r]);
#pragma unroll
        for (int q = 0; q < kTiles; ++q) {
          float e[4][4] = {};
#pragma unroll
          for (int i = 0; i < 4; ++i) mma_tf32(e[i], two[i][0], two[i][1], two[i][2], two[i][3], w[q][0][0], w[q][0][1]);
#pragma unroll
          for (int k = kOps - 1; k >= 0; --k)
#pragma unroll
            for (int i = 0; i < 4; ++i) mma_tf32(e[i], one[i][0], one[i][1], one[i][2], one[i][3], w[q][k][0], w[q][k][1]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) o[q][4 * j + i][r] += e[i][r];
        }
      }
    }
  }
}

// The element of the head in row g + 8 r of o's tile.
template <typename Kv>
__device__ __forceinline__ int element_of(int tile, int r, int g) {
  return sizeof(Kv) == 2 ? 16 * tile + 8 * r + g : 64 * (tile / 4) + 32 * r + 4 * g + tile % 4;
}

// Column e of o's tiles times f, lane g's elements of a head's row.
template <typename Kv, int D, typename Dst>
__device__ __forceinline__ void put_row(Dst* row, int g, int e, float f, const float (&o)[D / 16][4]) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int r = 0; r < 2; ++r) store_o(row + element_of<Kv>(i, r, g), o[i][2 * r + e] * f);
}

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }
__device__ __forceinline__ bool not_finite(__nv_bfloat16 x) { return not_finite(__bfloat162float(x)); }

// A score of -inf is a weight of 0 where finite operands passed the range of fp32, but an
// infinite operand must show in its head: those scores become NaN. Which of its products
// cancel depends on the terms (0 * inf is NaN, one term alone keeps -inf), so what decides
// is the key's row and the head's query themselves. Called where a tile has a score of -inf
// only. Asking for that takes 3% with fp32 caches and more than 8 heads (8 x 32K tokens, 12
// heads: 164.5 us, 160.1 without), up to 1% elsewhere; a flag for the unit and one check behind
// its tiles took more registers (166 to 168).
template <typename Kv, typename Qt, int D, int HU, int NB>
__device__ void mark_infinite(const char* tile, uint32_t mask, const Qt* queries, int heads, int lane,
                              float (&p)[Columns<HU>::kTiles][NB][2]) {
  uint32_t keys = 0, cols = 0;
#pragma unroll 1
  for (int r = 0; r < 8 * NB; ++r) {
    bool bad = false;
    const Kv* row = reinterpret_cast<const Kv*>(tile + r * Tile<Kv, D>::kRow);
#pragma unroll 1
    for (int i = lane; i < D; i += 32) bad |= not_finite(row[i]);
    if (__any_sync(0xffffffffu, bad)) keys |= 1u << r;
  }
#pragma unroll 1
  for (int h = 0; h < heads; ++h) {
    bool bad = false;
#pragma unroll 1
    for (int i = lane; i < D; i += 32) bad |= not_finite(queries[h * D + i]);
    if (__any_sync(0xffffffffu, bad)) cols |= 1u << h;
  }
#pragma unroll
  for (int c = 0; c < Columns<HU>::kTiles; ++c)
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (((mask >> (8 * n + lane / 4)) & 1u) &&
            (((keys >> (8 * n + lane / 4)) | (cols >> Columns<HU>::head(c, lane % 4, e))) & 1u))
          p[c][n][e] = __int_as_float(0x7fc00000);
}

struct BatchSmem {
  uint32_t mask[kWarps][kStages];                            // keys of a tile that are there
  int64_t scan[kWarps], at[kWarps][2];                       // where a warp's tiles begin: sequence, its first tile
  int64_t unit[kWarps];                                      // the unit of a warp's open state, -1: none
  int32_t starts[kWarps], ends[kWarps];                      // the warp has its first, its last tile
  float m[kWarps][16], l[kWarps][16];
};
constexpr size_t kRingBytes = size_t(kWarps) * kStages * 2 * kTileBytes;
constexpr size_t kBatchSmem = kRingBytes + sizeof(BatchSmem);

template <typename Kv, typename Qt, int D, int HU>
__global__ void __launch_bounds__(kThreads, 2) attend_batch_kernel(const BatchArgs A) {
  using T = Tile<Kv, D>;
  constexpr int KEYS = T::kKeys, NB = KEYS / 8, NQ = Columns<HU>::kTiles;
  constexpr int TERMS = sizeof(Kv) == 4 || sizeof(Qt) == 2 ? 2 : 3;
  extern __shared__ __align__(128) char smem[];
  BatchSmem& J = *reinterpret_cast<BatchSmem*>(smem + kRingBytes);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, g = lane / 4, t4 = lane % 4;
  char* ring = smem + warp * kStages * 2 * kTileBytes;
  const uint32_t ring_at = uint32_t(__cvta_generic_to_shared(ring));
  pdl_trigger();
  pdl_wait();

  const int per = A.hkv * A.hb;                              // units of a sequence
  int64_t t0, t1;
  Place cur;
  if (A.single) {                                            // one unit a CTA
    cur.s = blockIdx.x / per;
    cur.ub = blockIdx.x - cur.s * per;
    const int64_t n = A.n_tokens[cur.s];
    if (tid == 0 && cur.ub == 0 && (n < 0 || n > A.max_tokens) && A.status != nullptr)
      atomicOr(A.status, ZHA_DEV_BAD_LENGTH);
    cur.n = clamped(A, cur.s);
    cur.first = 0;
    cur.end = tiles_of<KEYS>(cur.n);
    if (cur.n == 0) {
      const int h0 = (cur.ub % A.hb) * HU, heads = min(HU, A.group - h0);
      const int64_t qrow = int64_t(cur.s) * A.hq + int64_t(cur.ub / A.hb) * A.group + h0;
      for (int i = tid; i < heads * D; i += kThreads) store_o(static_cast<Qt*>(A.O) + qrow * D + i, 0.f);
      if (tid < heads && A.lse != nullptr) A.lse[qrow + tid] = -INFINITY;
      return;
    }
    const int n_w = int(min64(kWarps, cur.end));
    const int tiles = int(cur.end), each = tiles / n_w, more = tiles - each * n_w;     // at most kSingleTiles
    t0 = min(tiles, warp * each + min(warp, more));
    t1 = min(tiles, (warp + 1) * each + min(warp + 1, more));
  } else {
    // Tiles of all sequences and where this CTA's warps begin. Thread i scans a run of
    // ceil(S / threads) sequences.
    const int run = (A.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(A.n_seqs, tid * run), s1 = min(A.n_seqs, s0 + run);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += places_of<KEYS>(clamped(A, s));
    int64_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += x;
    }
    if (lane == 31) J.scan[warp] = upto;
    __syncthreads();
    int64_t at = upto - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += J.scan[w];
      all += J.scan[w];
    }
    const int64_t total = all * per;
    const Deal deal(A, total);
    const int64_t w0 = int64_t(blockIdx.x) * kWarps;
    int64_t starts[kWarps];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) starts[w] = deal.start(w0 + w);
    for (int s = s0; s < s1; ++s) {
      const int64_t n = A.n_tokens[s], tl = places_of<KEYS>(clamped(A, s));
#pragma unroll
      for (int w = 0; w < kWarps; ++w)
        if (starts[w] >= at * per && starts[w] < (at + tl) * per) { J.at[w][0] = s; J.at[w][1] = at; }
      if (blockIdx.x == 0) {
        A.prefix[s] = at;
        if ((n < 0 || n > A.max_tokens) && A.status != nullptr) atomicOr(A.status, ZHA_DEV_BAD_LENGTH);
      }
      at += tl;
    }
    if (blockIdx.x == 0 && tid == 0) A.prefix[A.n_seqs] = all;
    __syncthreads();
    t0 = deal.start(w0 + warp);
    t1 = deal.start(w0 + warp + 1);
    if (starts[0] >= total) return;
    if (t0 < t1) {
      cur.s = int(J.at[warp][0]);
      cur.n = clamped(A, cur.s);
      const int64_t tl = places_of<KEYS>(cur.n), base = J.at[warp][1] * per;
      cur.ub = int(quotient(t0 - base, tl));
      cur.end = base + (cur.ub + 1) * tl;
      cur.first = cur.end - tl + kUnitCost;
    }
  }

  // The ring. `row` is the cache row of the next tile's key `lane`, looked up one
  // tile ahead of its copy; -1: absent.
  Place ahead = cur;
  int64_t next = t0;
  int32_t row = -1;
  int64_t head = t0 < t1 ? int64_t(cur.s) * A.hkv + cur.ub / A.hb : 0;
  auto look_up = [&] {
    row = -1;
    if (next >= t1) return;
    while (next >= ahead.end) {
      next_unit<KEYS>(A, ahead);
      head = int64_t(ahead.s) * A.hkv + ahead.ub / A.hb;
    }
    next = max64(next, ahead.first);
    if (next >= t1) return;
    const int64_t tok = (next - ahead.first) * KEYS + lane;
    if (lane < KEYS && tok < ahead.n) {
      const uint32_t t = uint32_t(tok);
      if (A.kv.table == nullptr) {
        row = int32_t(head) * int32_t(A.kv.ld) + int32_t(t);
      } else {
        const uint32_t block = uint32_t(uint64_t(t) * A.div_mul >> A.div_shift);
        const int32_t page = A.kv.table[head * A.kv.max_blocks + block];
        if (page >= 0 && page < A.kv.ld) row = page * A.chunk + int32_t(t - block * A.chunk);
        else if (A.status != nullptr) atomicOr(A.status, ZHA_DEV_BAD_PAGE);
      }
    }
  };
  auto issue = [&](int stage) {
    if (next < t1) {
      const uint32_t mask = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) J.mask[warp][stage] = mask;
      const uint32_t to = ring_at + stage * 2 * kTileBytes;
      const int piece = lane % T::kPieces, key0 = lane / T::kPieces;
      constexpr int kStep = 32 / T::kPieces;                 // keys of a round of 32 pieces
      const int32_t first = __shfl_sync(0xffffffffu, row, 0);
      if (__all_sync(0xffffffffu, lane >= KEYS || (row == first + lane && first >= 0))) {
        // rows one behind the other: one address
        const int64_t off = int64_t(first) * T::kRow + lane * 16;
        const char* k = static_cast<const char*>(A.kv.k) + off;
        const char* v = static_cast<const char*>(A.kv.v) + off;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          copy16(to + T::at_k(i * kStep + key0, piece), k + i * 512);
          copy16(to + kTileBytes + T::at_v(i * kStep + key0, piece), v + i * 512);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int key = i * kStep + key0;
          const int32_t r = __shfl_sync(0xffffffffu, row, key);
          const int64_t off = int64_t(max(r, 0)) * T::kRow + piece * 16;
          copy16(to + T::at_k(key, piece), static_cast<const char*>(A.kv.k) + off, r >= 0);
          copy16(to + kTileBytes + T::at_v(key, piece), static_cast<const char*>(A.kv.v) + off, r >= 0);
        }
      }
      ++next;
      look_up();
    }
    copy_commit();
  };
  look_up();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  int64_t at = t0 < t1 ? max64(t0, cur.first) : t1;
  int stage = 0;
  float m[NQ][2], l[NQ][2], o[NQ][D / 16][4];
  const bool mine = HU != 4 || t4 < 2;                       // of two lanes with the same heads
  if (lane == 0) J.unit[warp] = -1;
  while (at < t1) {
    const int h0 = (cur.ub % A.hb) * HU, heads = min(HU, A.group - h0);
    const int64_t qrow = int64_t(cur.s) * A.hq + int64_t(cur.ub / A.hb) * A.group + h0;
    Queries<Kv, Qt, D, HU> q;
    q.load(static_cast<const Qt*>(A.Q) + qrow * D, heads, lane);
#pragma unroll
    for (int c = 0; c < NQ; ++c) {
      m[c][0] = m[c][1] = -INFINITY;
      l[c][0] = l[c][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) o[c][i][0] = o[c][i][1] = o[c][i][2] = o[c][i][3] = 0.f;
    }

    const int64_t stop = min64(t1, cur.end);
    for (; at < stop; ++at) {
      __syncwarp();                                          // the stage that is refilled has been read by all lanes
      issue(stage == 0 ? kStages - 1 : stage - 1);
      copy_wait<kStages - 1>();
      __syncwarp();
      const char* tile = ring + stage * 2 * kTileBytes;
      const uint32_t mask = J.mask[warp][stage];
      float p[NQ][NB][2];
      q.scores(tile, lane, p);
      float low = 0.f;
#pragma unroll
      for (int c = 0; c < NQ; ++c)
#pragma unroll
        for (int n = 0; n < NB; ++n) low = fminf(low, fminf(p[c][n][0], p[c][n][1]));
      if (mask != (KEYS == 32 ? ~0u : (1u << (KEYS % 32)) - 1)) {
#pragma unroll
        for (int c = 0; c < NQ; ++c)
#pragma unroll
          for (int n = 0; n < NB; ++n)
            if (!((mask >> (8 * n + g)) & 1u)) p[c][n][0] = p[c][n][1] = -INFINITY;
      }
      float top[NQ][2];
      bool higher = low == -INFINITY;
#pragma unroll
      for (int c = 0; c < NQ; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = -INFINITY;
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            p[c][n][e] *= A.scale_log2;
            x = fmaxf(x, p[c][n][e]);
          }
#pragma unroll
          for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
          top[c][e] = x;
          higher |= x > m[c][e];
        }
      if (__any_sync(0xffffffffu, higher)) {
        if (__any_sync(0xffffffffu, low == -INFINITY))
          mark_infinite<Kv, Qt, D, HU, NB>(tile, mask, static_cast<const Qt*>(A.Q) + qrow * D, heads, lane, p);
#pragma unroll
        for (int c = 0; c < NQ; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float mn = fmaxf(m[c][e], top[c][e]), a = mn == -INFINITY ? 1.f : ex2(m[c][e] - mn);
            m[c][e] = mn;
            l[c][e] *= a;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) { o[c][i][e] *= a; o[c][i][2 + e] *= a; }
          }
      }
#pragma unroll
      for (int c = 0; c < NQ; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float base = m[c][e] == -INFINITY ? 0.f : m[c][e];
#pragma unroll
          for (int n = 0; n < NB; ++n) {
            p[c][n][e] = ex2(p[c][n][e] - base);
            l[c][e] += p[c][n][e];
          }
        }
      add_values<Kv, D, HU, TERMS, NB>(ring_at + stage * 2 * kTileBytes + kTileBytes, tile + kTileBytes, lane, p, o);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

#pragma unroll
    for (int c = 0; c < NQ; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[c][e] += __shfl_xor_sync(0xffffffffu, l[c][e], w);
        if constexpr (HU == 4) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            o[c][i][e] += __shfl_xor_sync(0xffffffffu, o[c][i][e], 2);
            o[c][i][2 + e] += __shfl_xor_sync(0xffffffffu, o[c][i][2 + e], 2);
          }
        }
      }
    const bool starts = cur.first >= t0, ends = cur.end <= t1;
    if (starts && ends) {
#pragma unroll
      for (int c = 0; c < NQ; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int h = Columns<HU>::head(c, t4, e);
          if (h < heads && mine) {
            const int64_t out = qrow + h;
            const float L = l[c][e];
            put_row<Kv, D>(static_cast<Qt*>(A.O) + out * D, g, e, L == 0.f ? 0.f : 1.f / L, o[c]);
            if (g == 0 && A.lse != nullptr) A.lse[out] = L == 0.f ? -INFINITY : 0.69314718056f * (m[c][e] + log2f(L));
          }
        }
    } else if (cur.end < t1) {
      float* piece = A.slots + (kMaxWarps + int64_t(blockIdx.x) * kWarps + warp) * HU * (D + 4);
#pragma unroll
      for (int c = 0; c < NQ; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          if (mine) {
            float* slot = piece + Columns<HU>::head(c, t4, e) * (D + 4);
            put_row<Kv, D>(slot + 4, g, e, 1.f, o[c]);
            if (g == 0) { slot[0] = m[c][e]; slot[1] = l[c][e]; }
          }
    } else if (lane == 0) {
      J.unit[warp] = int64_t(cur.s) * per + cur.ub;
      J.starts[warp] = starts;
      J.ends[warp] = ends;
    }
    if (at < t1) {
      next_unit<KEYS>(A, cur);
      at = max64(at, cur.first);
    }
  }

  // The open states, joined where neighbouring warps have the same unit. The rings
  // are done with.
  copy_wait<0>();
  __syncthreads();
  float* states = reinterpret_cast<float*>(smem);            // [warp][HU][D]
  if (J.unit[warp] >= 0) {
#pragma unroll
    for (int c = 0; c < NQ; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (mine) {
          const int h = Columns<HU>::head(c, t4, e);
          put_row<Kv, D>(states + (warp * HU + h) * D, g, e, 1.f, o[c]);
          if (g == 0) { J.m[warp][h] = m[c][e]; J.l[warp][h] = l[c][e]; }
        }
  }
  __syncthreads();
  for (int a = 0, b; a < kWarps; a = b) {
    const int64_t unit = J.unit[a];
    for (b = a + 1; b < kWarps && J.unit[b] == unit; ++b) {}
    if (unit < 0) continue;
    const bool whole = J.starts[a] && J.ends[b - 1];
    const int64_t s = unit / per;
    const int ub = int(unit - s * per), h0 = (ub % A.hb) * HU, heads = min(HU, A.group - h0);
    const int64_t qrow = s * A.hq + int64_t(ub / A.hb) * A.group + h0;
    for (int i = tid * 4; i < heads * D; i += kThreads * 4) {
      const int h = i / D, e = i % D;
      float M = -INFINITY, L = 0.f, acc[4] = {};
      for (int w = a; w < b; ++w) M = fmaxf(M, J.m[w][h]);
      for (int w = a; w < b; ++w) {
        const float lw = J.l[w][h], f = lw != 0.f ? ex2(J.m[w][h] - M) : 0.f;
        const float4 x = *reinterpret_cast<const float4*>(states + (w * HU + h) * D + e);
        L += lw * f;
        acc[0] += x.x * f; acc[1] += x.y * f; acc[2] += x.z * f; acc[3] += x.w * f;
      }
      if (whole) {
        const float f = L == 0.f ? 0.f : 1.f / L;
        store4(static_cast<Qt*>(A.O) + (qrow + h) * D + e, acc[0] * f, acc[1] * f, acc[2] * f, acc[3] * f);
        if (e == 0 && A.lse != nullptr) A.lse[qrow + h] = L == 0.f ? -INFINITY : 0.69314718056f * (M + log2f(L));
      } else {
        float* slot = A.slots + ((int64_t(blockIdx.x) * kWarps + a) * HU + h) * (D + 4);
        store4(slot + 4 + e, acc[0], acc[1], acc[2], acc[3]);
        if (e == 0) { slot[0] = M; slot[1] = L; }
      }
    }
  }
}

// A unit's pieces joined: nothing to do for a finished unit; zeros for one without
// tiles. Grid (units, heads): one CTA a head, its pieces dealt to the warps (few
// units, many pieces each). Otherwise one warp for two heads of a unit.
template <typename Qt, int D, int HU>
__global__ void __launch_bounds__(kJoinThreads) attend_batch_join_kernel(const BatchArgs A) {
  constexpr int EPL = D / 32, kJoinWarps = kJoinThreads / 32;
  __shared__ float s_o[kJoinWarps][D], s_m[kJoinWarps], s_l[kJoinWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool wide = A.wide != 0;
  const int split = wide ? kJoinWarps : 1, part = wide ? warp : 0;
  pdl_trigger();
  pdl_wait();
  const int per = A.hkv * A.hb, join_warps = join_warps_of(HU, A.group);
  const int in_cta = kJoinWarps / join_warps, unit = wide ? blockIdx.x : blockIdx.x * in_cta + warp / join_warps;
  const int s = unit / per, ub = unit - s * per;
  if (s >= A.n_seqs || (!wide && warp >= in_cta * join_warps)) return;
  const int heads = min(HU, A.group - (ub % A.hb) * HU);
  const int64_t row0 = int64_t(s) * A.hq + int64_t(ub / A.hb) * A.group + (ub % A.hb) * HU;
  const int64_t seq_tile = A.prefix[s], tl = A.prefix[s + 1] - seq_tile;
  const int64_t total = A.prefix[A.n_seqs] * per;
  int w0 = 0, w1 = 0, groups = 0, n = 0;
  if (tl > 0) {
    // Warps w0..w1 have the unit; the last one's state is an end piece unless the unit
    // ends with that warp's tiles.
    const Deal deal(A, total);
    const int64_t hi = seq_tile * per + (ub + 1) * tl, lo = hi - tl + kUnitCost;
    w0 = int(deal.owner(lo));
    w1 = int(deal.owner(hi - 1));
    const bool apart = hi != deal.start(w1 + 1);
    groups = w1 - apart < w0 ? 0 : (w1 - apart) / kWarps - w0 / kWarps + 1;
    n = groups + apart;
    if (w0 == w1 || n == 1) return;
  }
  const int h0 = wide ? blockIdx.y : warp % join_warps * 2, h1 = wide ? h0 + 1 : h0 + 2;
  for (int h = h0; h < min(heads, h1); ++h) {
    // Pieces in rounds of 8, all of a round's loads before its arithmetic.
    float M = -INFINITY, L = 0.f, acc[EPL] = {};
    for (int i0 = part; i0 < n; i0 += 8 * split) {
      float2 ml[8];
      float x[8][EPL];
      float top = M;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * split;
        ml[k] = make_float2(0.f, 0.f);
        if (i < n) {
          const int64_t at = i < groups ? max(w0, (w0 / kWarps + i) * kWarps) : kMaxWarps + w1;
          const float* p = A.slots + (at * HU + h) * (D + 4);
          ml[k] = *reinterpret_cast<const float2*>(p);
          load_slice<EPL>(p + 4, lane * EPL, x[k]);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (ml[k].y != 0.f) top = fmaxf(top, ml[k].x);
      const float keep = L != 0.f ? ex2(M - top) : 0.f;
      M = top;
      L *= keep;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] *= keep;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (ml[k].y != 0.f) {
          const float f = ex2(ml[k].x - top);
          L += ml[k].y * f;
#pragma unroll
          for (int e = 0; e < EPL; ++e) acc[e] = fmaf(x[k][e], f, acc[e]);
        }
    }
    if (wide) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) s_o[warp][lane * EPL + e] = acc[e];
      if (lane == 0) { s_m[warp] = M; s_l[warp] = L; }
      __syncthreads();
      if (warp != 0) return;
      M = -INFINITY;
      L = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
#pragma unroll
      for (int k = 0; k < kJoinWarps; ++k) M = fmaxf(M, s_m[k]);
#pragma unroll
      for (int k = 0; k < kJoinWarps; ++k) {
        const float f = s_l[k] != 0.f ? ex2(s_m[k] - M) : 0.f;
        L += s_l[k] * f;
#pragma unroll
        for (int e = 0; e < EPL; ++e) acc[e] += s_o[k][lane * EPL + e] * f;
      }
    }
    const float f = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] *= f;
    if constexpr (EPL == 4) store4(static_cast<Qt*>(A.O) + (row0 + h) * D + lane * 4, acc[0], acc[1], acc[2], acc[3]);
    else
#pragma unroll
      for (int e = 0; e < EPL; ++e) store_o(static_cast<Qt*>(A.O) + (row0 + h) * D + lane * EPL + e, acc[e]);
    if (lane == 0 && A.lse != nullptr) A.lse[row0 + h] = L == 0.f ? -INFINITY : 0.69314718056f * (M + log2f(L));
    if (wide) return;
  }
}

template <typename Kv, typename Qt, int D, int HU>
cudaError_t launch_batch(BatchArgs A, cudaStream_t s) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  auto kernel = attend_batch_kernel<Kv, Qt, D, HU>;
  e = ensure_dynamic_smem(kernel, kBatchSmem);
  if (e != cudaSuccess) return e;
  const int64_t units = int64_t(A.n_seqs) * A.hkv * A.hb;
  const int64_t tiles = (A.max_tokens + Tile<Kv, D>::kKeys - 1) / Tile<Kv, D>::kKeys;
  A.single = tiles <= kSingleTiles && units <= int64_t(sms) * 2;
  sms = sms < kMaxSms ? sms : kMaxSms;
  const int64_t most = units * (tiles + kUnitCost);
  A.first_ctas = int32_t(max64(1, min64(sms * 2, (most + kWarps * kMinTiles - 1) / (kWarps * kMinTiles))));
  A.ctas = HU < 16 && most >= int64_t(kTwoTiers) * kWarps * sms * 2 ? sms * 3 : A.first_ctas;
  const int64_t ctas = A.single ? units : A.ctas;
  {
    TraceScope ts("attend_batch_kernel", 0, s);
    zha_count_launch();
    e = launch_pdl(kernel, dim3(unsigned(ctas)), dim3(kThreads), kBatchSmem, s, A);
    if (e != cudaSuccess) return e;
  }
  if (A.single) return cudaSuccess;
  TraceScope ts("attend_batch_join_kernel", 0, s);
  zha_count_launch();
  A.wide = units <= kWideUnits;
  const int64_t in_cta = kJoinThreads / 32 / join_warps_of(HU, A.group);
  const dim3 grid = A.wide ? dim3(unsigned(units), unsigned(min64(HU, A.group)))
                           : dim3(unsigned((units + in_cta - 1) / in_cta));
  return launch_pdl(attend_batch_join_kernel<Qt, D, HU>, grid, dim3(kJoinThreads), 0, s, A);
}

template <typename Kv, typename Qt>
cudaError_t launch_batch_d(const BatchArgs& A, int d, cudaStream_t s) {
  switch (head_cols(A.group)) {
    case 4: return d == 128 ? launch_batch<Kv, Qt, 128, 4>(A, s) : launch_batch<Kv, Qt, 64, 4>(A, s);
    case 8: return d == 128 ? launch_batch<Kv, Qt, 128, 8>(A, s) : launch_batch<Kv, Qt, 64, 8>(A, s);
    default: return d == 128 ? launch_batch<Kv, Qt, 128, 16>(A, s) : launch_batch<Kv, Qt, 64, 16>(A, s);
  }
}

// Units beyond this are refused: slots and grids stay far below 2^31.
constexpr int64_t kMaxUnits = int64_t(1) << 22;

bool units_ok(const Geom& G, int32_t n_seqs) {
  const int64_t hb = (G.group + head_cols(G.group) - 1) / head_cols(G.group);
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
    return zha_report_error(ZHA_ERR_INVALID,
                            "zha_attend_batch_kv: Q and O must be non-NULL 16-byte aligned device pointers");
  if (q_dtype != ZHA_F32 && q_dtype != ZHA_BF16)
    return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: unknown q_dtype");
  if (d_n_tokens == nullptr) return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: n_tokens is NULL");
  if (!zha_may_lie(d_n_tokens) || !zha_may_lie(d_lse) || !zha_may_lie(d_status))
    return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: n_tokens, lse or status at no multiple of its type's size");
  const uintptr_t q0 = reinterpret_cast<uintptr_t>(d_Q), o0 = reinterpret_cast<uintptr_t>(d_O);
  if (q0 != o0 && (q0 < o0 ? o0 - q0 : q0 - o0) < uint64_t(n_seqs) * G.hq * G.d * (q_dtype == ZHA_F32 ? 4 : 2))
    return zha_report_error(ZHA_ERR_INVALID, "zha_attend_batch_kv: O overlaps Q without being Q");
  if (!zha::units_ok(G, n_seqs))
    return zha_report_error(ZHA_ERR_UNSUPPORTED,
                            "zha_attend_batch_kv: more than 2^22 (sequence, KV head, query block) units");
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
  A.div_shift = 31;
  while ((1 << (A.div_shift - 31)) < G.chunk) ++A.div_shift;
  A.div_mul = uint32_t(((uint64_t(1) << A.div_shift) + G.chunk - 1) / G.chunk);
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
