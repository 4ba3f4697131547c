// zha_attend_batch.cu -- dense attention of one query token per sequence over a
// batch of (paged) caches. Semantics are in include/zha.h.
//
// Mathematics. o = sum_j p_j v_j / sum_j p_j with p_j = 2^(x_j - m), x_j = q.k_j
// log2(e) / sqrt(d): any m gives the same quotient, and states (m, l, o) of two
// parts of the keys join as m = max, l = sum l_i 2^(m_i - m), o alike.
//
// Split. A unit is (sequence, KV head, block of its query heads); its keys are cut
// into tiles of 4 KB of K and 4 KB of V. All units' tiles, one behind the other, are
// dealt out evenly to the warps (warp w has tiles [w T / n, (w + 1) T / n)), from the
// counts in device memory, so that ragged lengths cost nothing. A warp keeps its own
// ring of tiles in flight (cp.async), across the borders of units, and waits for no
// other until its tiles are done. What then becomes of a unit's state:
//   - all of its tiles in one warp: the warp writes the result;
//   - it ends before the warp's last tile, having begun in an earlier warp: an end
//     piece in the workspace, at the warp's number;
//   - it reaches the warp's last tile: the CTA joins the states of its warps in that
//     unit, and writes the result or, with more of the unit elsewhere, a group piece, at
//     the number of the group's first warp.
// A second kernel finds a unit's pieces from the tile counts alone and joins them in a
// fixed order.
//
// Products. A unit has at most 16 query rows, an eighth of a tcgen05 tile, and
// the call is bound by the cache it reads: the warps' own matrix instructions
// (16 x 8 x 16 bf16, 16 x 8 x 8 tf32) take their operands from the warp's registers and
// tile without a hand-over. Their 16 rows hold 8 heads twice, as the first and the
// following terms of the fp32 operand, or 16 heads.
//   bf16 cache: keys and values enter exactly. fp32 queries and weights are three
//   bf16 terms cut off one after the other (8 + 8 + 8 bits: exact); with bf16
//   queries, which are exact, weights are two terms (2^-16, below the output's 2^-8).
//   fp32 cache: every operand is two tf32 terms (2^-23), and the product of the
//   two second terms (2^-24) is left out where 16 heads fill the rows.
#include <cmath>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 3;              // tiles in a warp's ring
constexpr int kTileBytes = 4096;        // of K, and of V
constexpr int kMaxCtas = 148 * 2;
constexpr int kMaxWarps = kMaxCtas * kWarps;
constexpr int kMinTiles = 2;            // no warp takes less, unless there is less
constexpr int kSingleTiles = 32;
constexpr int kJoinThreads = 256;
constexpr int kWideUnits = 148;        // up to so many units a CTA joins one head

inline int head_rows(int group) { return group > 8 ? 16 : 8; }

struct BatchLayout {
  int64_t units, slots, bytes, slots_off;
  int32_t hb, hu;                       // head blocks per KV head, heads per block
};

// Workspace: int64 prefix[n_seqs + 1] (tiles of one unit of the sequences
// before s), int64 warp count; then the group pieces and the end pieces, [m, l, 0, 0,
// o[d]] for each of the unit's heads.
inline BatchLayout batch_layout(const Geom& G, int32_t n_seqs) {
  BatchLayout b{};
  b.hu = head_rows(G.group);
  b.hb = (G.group + b.hu - 1) / b.hu;
  b.units = int64_t(n_seqs) * G.hkv * b.hb;
  b.slots = 2 * kMaxWarps;
  b.slots_off = round_up((int64_t(n_seqs) + 2) * 8, 256);
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
  int32_t n_seqs, hkv, hq, group, hb, chunk, single;
  float scale_log2;                     // log2(e) / sqrt(d)
};

// ---- small pieces -----------------------------------------------------------
__device__ __forceinline__ void store_o(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_o(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 16 bytes into shared memory, or 16 zeros.
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
// (An infinite value has one term.)
__device__ __forceinline__ uint32_t cut_bf16(float& a, float& b) {
  const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
  a = a - __uint_as_float(ua & 0xffff0000u);
  b = b - __uint_as_float(ub & 0xffff0000u);
  return __byte_perm(ua, ub, 0x7632);
}
// The next tf32 term of a value, rounded and taken away.
__device__ __forceinline__ uint32_t cut_tf32(float& a) {
  uint32_t t;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(t) : "f"(a));
  a -= __uint_as_float(t);
  return t;
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
// tiles [first, end).
struct Place {
  int64_t first, end, n;
  int s, ub;
};

__device__ __forceinline__ int64_t clamped(const BatchArgs& A, int s) {
  return max64(0, min64(A.n_tokens[s], A.max_tokens));
}
template <int KEYS>
__device__ __forceinline__ int64_t tiles_of(int64_t n) { return (n + KEYS - 1) / KEYS; }

// To the next unit that has tiles; the caller knows that there is one.
template <int KEYS>
__device__ __forceinline__ void next_unit(const BatchArgs& A, Place& p) {
  if (++p.ub == A.hkv * A.hb) {
    p.ub = 0;
    do p.n = clamped(A, ++p.s); while (p.n == 0);
  }
  p.first = p.end;
  p.end += tiles_of<KEYS>(p.n);
}

// A warp's query rows as matrix operands. Lane (g, t) = (lane / 4, lane % 4)
// has rows g and g + 8; the order of the head's elements within a step is that of the K
// reads: lane t's piece of 16 bytes serves two steps.
template <typename Kv, typename Qt, int D, int HU>
struct Queries;

template <typename Qt, int D, int HU>
struct Queries<__nv_bfloat16, Qt, D, HU> {
  static constexpr bool kExact = sizeof(Qt) == 2;          // one term
  static constexpr int kSteps = D / 16;
  static constexpr int kMore = kExact ? 0 : HU == 16 ? 4 : 1;
  uint32_t a[kSteps][HU == 16 ? 4 : kExact ? 2 : 4];       // first terms of rows g, g + 8 (HU 8: rows g; second terms)
  uint32_t b[kSteps][kMore == 0 ? 1 : kMore * (HU == 16 ? 1 : 2)];   // HU 16: second, third terms; HU 8: third

  __device__ void load(const Qt* q, int heads, int lane) {
    const int g = lane / 4, t = lane % 4;
#pragma unroll
    for (int r = 0; r < HU / 8; ++r) {
      const int h = g + 8 * r;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) {
        float v[8] = {};
        if (h < heads) {
          if constexpr (kExact) {
            load_slice<8>(q + h * D, 32 * j + 8 * t, v);
          } else {
            float x[4], y[4];
            load_slice<4>(q + h * D, 32 * j + 8 * t, x);
            load_slice<4>(q + h * D, 32 * j + 8 * t + 4, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) { v[i] = x[i]; v[4 + i] = y[i]; }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {                        // step 2j + i / 2, first or second half of its elements
          const int st = 2 * j + i / 2, hi = i % 2;
          const uint32_t one = cut_bf16(v[2 * i], v[2 * i + 1]);
          if constexpr (kExact) {
            a[st][HU == 16 ? r + 2 * hi : hi] = one;
          } else {
            const uint32_t two = cut_bf16(v[2 * i], v[2 * i + 1]), three = cut_bf16(v[2 * i], v[2 * i + 1]);
            if constexpr (HU == 16) {
              a[st][r + 2 * hi] = one;
              b[st][r + 2 * hi] = two;
              c[st][r + 2 * hi] = three;
            } else {
              a[st][2 * hi] = one;
              a[st][2 * hi + 1] = two;
              b[st][hi] = three;
            }
          }
        }
      }
    }
  }
  uint32_t c[kSteps][kMore == 4 ? 4 : 1];

  // s[n tile][2 r + e]: row g + 8 r, key 8 * tile + 2 t + e.
  template <int NT>
  __device__ void scores(const char* tile, int lane, float (&s)[NT][4]) const {
    const int g = lane / 4, t = lane % 4;
    float low[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = low[n][i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint4 k = *reinterpret_cast<const uint4*>(tile + Tile<__nv_bfloat16, D>::at_k(8 * n + g, 4 * j + t));
        const uint32_t kb[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int st = 2 * j + u;
          if constexpr (HU == 16) {
            mma_bf16(s[n], a[st][0], a[st][1], a[st][2], a[st][3], kb[2 * u], kb[2 * u + 1]);
            if constexpr (!kExact) {
              mma_bf16(low[n], b[st][0], b[st][1], b[st][2], b[st][3], kb[2 * u], kb[2 * u + 1]);
              mma_bf16(low[n], c[st][0], c[st][1], c[st][2], c[st][3], kb[2 * u], kb[2 * u + 1]);
            }
          } else if constexpr (kExact) {
            mma_bf16(s[n], a[st][0], 0u, a[st][1], 0u, kb[2 * u], kb[2 * u + 1]);
          } else {
            mma_bf16(s[n], a[st][0], a[st][1], a[st][2], a[st][3], kb[2 * u], kb[2 * u + 1]);
            mma_bf16(low[n], 0u, b[st][0], 0u, b[st][1], kb[2 * u], kb[2 * u + 1]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (HU == 16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[n][i] += low[n][i];
      } else {
        s[n][0] += s[n][2] + low[n][2];
        s[n][1] += s[n][3] + low[n][3];
      }
    }
  }
};

template <typename Qt, int D, int HU>
struct Queries<float, Qt, D, HU> {
  static constexpr int kSteps = D / 8;
  uint32_t a[kSteps][4];                                     // HU 8: rows g first terms, rows g + 8 second terms
  uint32_t b[HU == 16 ? kSteps : 1][4];                      // HU 16: second terms

  __device__ void load(const Qt* q, int heads, int lane) {
    const int g = lane / 4, t = lane % 4;
#pragma unroll
    for (int r = 0; r < HU / 8; ++r) {
      const int h = g + 8 * r;
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        float v[4] = {};
        if (h < heads) load_slice<4>(q + h * D, 16 * j + 4 * t, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int st = 2 * j + i / 2, hi = i % 2;
          const uint32_t one = cut_tf32(v[i]), two = cut_tf32(v[i]);
          a[st][2 * hi + r] = one;
          if constexpr (HU == 16) b[st][2 * hi + r] = two;
          else a[st][2 * hi + 1] = two;
        }
      }
    }
  }

  template <int NT>
  __device__ void scores(const char* tile, int lane, float (&s)[NT][4]) const {
    const int g = lane / 4, t = lane % 4;
    float low[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] = low[n][i] = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float4 k = *reinterpret_cast<const float4*>(tile + Tile<float, D>::at_k(8 * n + g, 4 * j + t));
        float kr[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int st = 2 * j + u;
          const uint32_t h0 = cut_tf32(kr[2 * u]), h1 = cut_tf32(kr[2 * u + 1]);
          const uint32_t l0 = cut_tf32(kr[2 * u]), l1 = cut_tf32(kr[2 * u + 1]);
          mma_tf32(s[n], a[st][0], a[st][1], a[st][2], a[st][3], h0, h1);
          mma_tf32(low[n], a[st][0], a[st][1], a[st][2], a[st][3], l0, l1);
          if constexpr (HU == 16) mma_tf32(low[n], b[st][0], b[st][1], b[st][2], b[st][3], h0, h1);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i) s[n][i] += low[n][i];
      if constexpr (HU == 8) {
        s[n][0] += s[n][2];
        s[n][1] += s[n][3];
      }
    }
  }
};

// o[n tile] += weights * V. p[n tile][2 r + e] as the scores.
template <int D, int HU, int TERMS, int NT>
__device__ __forceinline__ void add_values(const __nv_bfloat16*, uint32_t tile, const char*, int lane, float (&p)[NT][4],
                                           float (&o)[D / 8][4]) {
#pragma unroll
  for (int kb = 0; kb < NT / 2; ++kb) {
    uint32_t w[TERMS][4];                                    // [term][element half * 2 + row]: a0..a3 of 16 rows
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int r = 0; r < HU / 8; ++r)
#pragma unroll
        for (int k = 0; k < TERMS; ++k) w[k][2 * half + r] = cut_bf16(p[2 * kb + half][2 * r], p[2 * kb + half][2 * r + 1]);
    const int row = kb * 16 + (lane & 15);
#pragma unroll
    for (int n0 = 0; n0 < D / 16; n0 += 4) {                 // 64 elements: every term in turn on 8 tiles of o
      uint32_t v[8][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[2 * i][0]), "=r"(v[2 * i][1]), "=r"(v[2 * i + 1][0]), "=r"(v[2 * i + 1][1])
                     : "r"(tile + Tile<__nv_bfloat16, D>::at_v(row, 2 * (n0 + i) + (lane >> 4)))
                     : "memory");
      if constexpr (HU == 16) {
#pragma unroll
        for (int k = TERMS - 1; k >= 0; --k)
#pragma unroll
          for (int i = 0; i < 8; ++i) mma_bf16(o[2 * n0 + i], w[k][0], w[k][1], w[k][2], w[k][3], v[i][0], v[i][1]);
      } else {
        if constexpr (TERMS == 3) {
#pragma unroll
          for (int i = 0; i < 8; ++i) mma_bf16(o[2 * n0 + i], 0u, w[2][0], 0u, w[2][2], v[i][0], v[i][1]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) mma_bf16(o[2 * n0 + i], w[0][0], w[1][0], w[0][2], w[1][2], v[i][0], v[i][1]);
      }
    }
  }
}

// fp32: within a tile of 8 keys, the step's elements t and t + 4 are the keys 2 t and
// 2 t + 1, which is how the scores lie.
template <int D, int HU, int TERMS, int NT>
__device__ __forceinline__ void add_values(const float*, uint32_t, const char* tile, int lane, float (&p)[NT][4],
                                           float (&o)[D / 8][4]) {
  const int g = lane / 4, t = lane % 4;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    uint32_t w[2][4];
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int r = 0; r < HU / 8; ++r) {
        w[0][2 * e + r] = cut_tf32(p[n][2 * r + e]);
        w[1][2 * e + r] = cut_tf32(p[n][2 * r + e]);
      }
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const float4 x = *reinterpret_cast<const float4*>(tile + Tile<float, D>::at_v(8 * n + 2 * t, 8 * j + g));
      const float4 y = *reinterpret_cast<const float4*>(tile + Tile<float, D>::at_v(8 * n + 2 * t + 1, 8 * j + g));
      float vx[4] = {x.x, x.y, x.z, x.w}, vy[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t h0 = cut_tf32(vx[i]), h1 = cut_tf32(vy[i]), l0 = cut_tf32(vx[i]), l1 = cut_tf32(vy[i]);
        float(&c)[4] = o[4 * j + i];
        if constexpr (HU == 16) {
          mma_tf32(c, w[0][0], w[0][1], w[0][2], w[0][3], l0, l1);
          mma_tf32(c, w[1][0], w[1][1], w[1][2], w[1][3], h0, h1);
          mma_tf32(c, w[0][0], w[0][1], w[0][2], w[0][3], h0, h1);
        } else {
          mma_tf32(c, w[0][0], w[1][0], w[0][2], w[1][2], l0, l1);
          mma_tf32(c, w[0][0], w[1][0], w[0][2], w[1][2], h0, h1);
        }
      }
    }
  }
}

__device__ __forceinline__ void put2(float* p, float a, float b) { *reinterpret_cast<float2*>(p) = make_float2(a, b); }
__device__ __forceinline__ void put2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// Row r of o times f, lane t4's part of it. Column 2 t4 + e of o's tile i is the head's
// element 8 i + 2 t4 + e (bf16 V) or 32 (i / 4) + 4 (2 t4 + e) + i % 4 (fp32 V).
template <typename Kv, int D, typename Dst>
__device__ __forceinline__ void put_row(Dst* row, int t4, int r, float f, const float (&o)[D / 8][4]) {
#pragma unroll
  for (int i = 0; i < D / 8; i += sizeof(Kv) == 2 ? 1 : 2) {
    if constexpr (sizeof(Kv) == 2) {
      put2(row + 8 * i + 2 * t4, o[i][2 * r] * f, o[i][2 * r + 1] * f);
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e)
        put2(row + 32 * (i / 4) + 4 * (2 * t4 + e) + i % 4, o[i][2 * r + e] * f, o[i + 1][2 * r + e] * f);
    }
  }
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
  constexpr int KEYS = T::kKeys, NT = KEYS / 8, NH = HU / 8;
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
    t0 = warp < n_w ? warp * cur.end / n_w : cur.end;
    t1 = warp < n_w ? (warp + 1) * cur.end / n_w : cur.end;
  } else {
    // Tiles of all sequences and where this CTA's warps begin. Thread i scans a run of
    // ceil(S / threads) sequences.
    const int run = (A.n_seqs + kThreads - 1) / kThreads;
    const int s0 = min(A.n_seqs, tid * run), s1 = min(A.n_seqs, s0 + run);
    int64_t mine = 0;
    for (int s = s0; s < s1; ++s) mine += tiles_of<KEYS>(clamped(A, s));
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
    const int64_t n_w = max64(1, min64(int64_t(gridDim.x) * kWarps, (total + kMinTiles - 1) / kMinTiles));
    const int64_t w0 = int64_t(blockIdx.x) * kWarps;
    for (int s = s0; s < s1; ++s) {
      const int64_t n = A.n_tokens[s], tl = tiles_of<KEYS>(clamped(A, s));
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int64_t t = w0 + w < n_w ? (w0 + w) * total / n_w : total;
        if (t >= at * per && t < (at + tl) * per) { J.at[w][0] = s; J.at[w][1] = at; }
      }
      if (blockIdx.x == 0) {
        A.prefix[s] = at;
        if ((n < 0 || n > A.max_tokens) && A.status != nullptr) atomicOr(A.status, ZHA_DEV_BAD_LENGTH);
      }
      at += tl;
    }
    if (blockIdx.x == 0 && tid == 0) { A.prefix[A.n_seqs] = all; A.prefix[A.n_seqs + 1] = n_w; }
    __syncthreads();
    if (w0 >= n_w || total == 0) return;
    const int64_t w = w0 + warp;
    t0 = w < n_w ? w * total / n_w : total;
    t1 = w < n_w ? (w + 1) * total / n_w : total;
    if (t0 < t1) {
      cur.s = int(J.at[warp][0]);
      cur.n = clamped(A, cur.s);
      const int64_t tl = tiles_of<KEYS>(cur.n), base = J.at[warp][1] * per;
      cur.ub = int((t0 - base) / tl);
      cur.first = base + cur.ub * tl;
      cur.end = cur.first + tl;
    }
  }

  // The ring. `row` is the cache row of the next tile's key `lane`, looked up one
  // tile ahead of its copy; -1: absent.
  Place ahead = cur;
  int64_t next = t0;
  int32_t row = -1;
  auto look_up = [&] {
    row = -1;
    if (next >= t1) return;
    while (next >= ahead.end) next_unit<KEYS>(A, ahead);
    const int64_t tok = (next - ahead.first) * KEYS + lane;
    if (lane < KEYS && tok < ahead.n) {
      row = kv_batch_row(A.kv, A.hkv, ahead.s, ahead.ub / A.hb, tok, A.chunk);
      if (row < 0 && A.status != nullptr) atomicOr(A.status, ZHA_DEV_BAD_PAGE);
    }
  };
  auto issue = [&](int stage) {
    if (next < t1) {
      const uint32_t mask = __ballot_sync(0xffffffffu, row >= 0);
      if (lane == 0) J.mask[warp][stage] = mask;
      const uint32_t to = ring_at + stage * 2 * kTileBytes;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int key = (i * 32 + lane) / T::kPieces, piece = lane % T::kPieces;
        const int32_t r = __shfl_sync(0xffffffffu, row, key);
        const int64_t off = int64_t(max(r, 0)) * T::kRow + piece * 16;
        copy16(to + T::at_k(key, piece), static_cast<const char*>(A.kv.k) + off, r >= 0);
        copy16(to + kTileBytes + T::at_v(key, piece), static_cast<const char*>(A.kv.v) + off, r >= 0);
      }
      ++next;
      look_up();
    }
    copy_commit();
  };
  look_up();
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i) issue(i);

  int64_t at = t0;
  int stage = 0;
  float m[NH], l[NH], o[D / 8][4];
  if (lane == 0) J.unit[warp] = -1;
  while (at < t1) {
    const int h0 = (cur.ub % A.hb) * HU, heads = min(HU, A.group - h0);
    const int64_t qrow = int64_t(cur.s) * A.hq + int64_t(cur.ub / A.hb) * A.group + h0;
    Queries<Kv, Qt, D, HU> q;
    q.load(static_cast<const Qt*>(A.Q) + qrow * D, heads, lane);
#pragma unroll
    for (int r = 0; r < NH; ++r) { m[r] = -INFINITY; l[r] = 0.f; }
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

    const int64_t stop = min64(t1, cur.end);
    for (; at < stop; ++at) {
      __syncwarp();                                          // the stage that is refilled has been read by all lanes
      issue(stage == 0 ? kStages - 1 : stage - 1);
      copy_wait<kStages - 1>();
      __syncwarp();
      const char* tile = ring + stage * 2 * kTileBytes;
      const uint32_t mask = J.mask[warp][stage];
      float p[NT][4];
      q.scores(tile, lane, p);
      float top[NH];
#pragma unroll
      for (int r = 0; r < NH; ++r) {
        top[r] = -INFINITY;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = p[n][2 * r + e];
            x = (mask >> (8 * n + 2 * t4 + e)) & 1u ? x * A.scale_log2 : -INFINITY;
            top[r] = fmaxf(top[r], x);
          }
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      }
      bool higher = false;
#pragma unroll
      for (int r = 0; r < NH; ++r) higher |= top[r] > m[r];
      if (__any_sync(0xffffffffu, higher)) {
#pragma unroll
        for (int r = 0; r < NH; ++r) {
          const float mn = fmaxf(m[r], top[r]), a = mn == -INFINITY ? 1.f : ex2(m[r] - mn);
          m[r] = mn;
          l[r] *= a;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[i][2 * r] *= a;
            o[i][2 * r + 1] *= a;
            if constexpr (HU == 8) { o[i][2] *= a; o[i][3] *= a; }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NH; ++r) {
        const float base = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = p[n][2 * r + e];
            x = ex2(x - base);
            l[r] += x;
          }
      }
      add_values<D, HU, TERMS, NT>(static_cast<const Kv*>(nullptr), ring_at + stage * 2 * kTileBytes + kTileBytes,
                                   tile + kTileBytes, lane, p, o);
      stage = stage == kStages - 1 ? 0 : stage + 1;
    }

#pragma unroll
    for (int r = 0; r < NH; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    }
    if constexpr (HU == 8) {
#pragma unroll
      for (int i = 0; i < D / 8; ++i) { o[i][0] += o[i][2]; o[i][1] += o[i][3]; }
    }
    const bool starts = cur.first >= t0, ends = cur.end <= t1;
    if (starts && ends) {
#pragma unroll
      for (int r = 0; r < NH; ++r)
        if (g + 8 * r < heads) {
          const int64_t out = qrow + g + 8 * r;
          const float f = l[r] == 0.f ? 0.f : 1.f / l[r];
          put_row<Kv, D>(static_cast<Qt*>(A.O) + out * D, t4, r, f, o);
          if (t4 == 0 && A.lse != nullptr) A.lse[out] = l[r] == 0.f ? -INFINITY : 0.69314718056f * (m[r] + log2f(l[r]));
        }
    } else if (cur.end < t1) {
      float* piece = A.slots + (kMaxWarps + int64_t(blockIdx.x) * kWarps + warp) * HU * (D + 4);
#pragma unroll
      for (int r = 0; r < NH; ++r) {
        float* slot = piece + (g + 8 * r) * (D + 4);
        put_row<Kv, D>(slot + 4, t4, r, 1.f, o);
        if (t4 == 0) { slot[0] = m[r]; slot[1] = l[r]; }
      }
    } else if (lane == 0) {
      J.unit[warp] = int64_t(cur.s) * per + cur.ub;
      J.starts[warp] = starts;
      J.ends[warp] = ends;
    }
    if (at < t1) next_unit<KEYS>(A, cur);
  }

  // The open states, joined where neighbouring warps have the same unit. The rings
  // are done with.
  copy_wait<0>();
  __syncthreads();
  float* states = reinterpret_cast<float*>(smem);            // [warp][HU][D]
  if (J.unit[warp] >= 0) {
#pragma unroll
    for (int r = 0; r < NH; ++r) {
      put_row<Kv, D>(states + (warp * HU + g + 8 * r) * D, t4, r, 1.f, o);
      if (t4 == 0) { J.m[warp][g + 8 * r] = m[r]; J.l[warp][g + 8 * r] = l[r]; }
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
    for (int i = tid; i < heads * D; i += kThreads) {
      const int h = i / D, e = i % D;
      float M = -INFINITY, L = 0.f, acc = 0.f;
      for (int w = a; w < b; ++w) M = fmaxf(M, J.m[w][h]);
      for (int w = a; w < b; ++w) {
        const float lw = J.l[w][h], f = lw != 0.f ? ex2(J.m[w][h] - M) : 0.f;
        L += lw * f;
        acc += states[(w * HU + h) * D + e] * f;
      }
      if (whole) {
        store_o(static_cast<Qt*>(A.O) + (qrow + h) * D + e, L == 0.f ? 0.f : acc / L);
        if (e == 0 && A.lse != nullptr) A.lse[qrow + h] = L == 0.f ? -INFINITY : 0.69314718056f * (M + log2f(L));
      } else {
        float* slot = A.slots + ((int64_t(blockIdx.x) * kWarps + a) * HU + h) * (D + 4);
        slot[4 + e] = acc;
        if (e == 0) { slot[0] = M; slot[1] = L; }
      }
    }
  }
}

// a / b for quotients below 2^31 and a below 2^53: a quotient in 64-bit floats, then
// put right (the hardware has no 64-bit integer division).
__device__ __forceinline__ int quotient(int64_t a, int64_t b) {
  int64_t q = int64_t(double(a) / double(b));
  const int64_t r = a - q * b;
  if (r < 0) --q;
  if (r >= b) ++q;
  return int(q);
}

// A unit's pieces joined: nothing to do for a finished unit; zeros for one without
// tiles. Grid (units, heads): one CTA a head, its pieces dealt to the warps (few
// units, many pieces each). Grid (units, 1): one warp a head.
template <typename Qt, int D, int HU>
__global__ void __launch_bounds__(kJoinThreads) attend_batch_join_kernel(const BatchArgs A) {
  constexpr int EPL = D / 32, kJoinWarps = kJoinThreads / 32;
  __shared__ float s_o[kJoinWarps][D], s_l[kJoinWarps];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const bool wide = gridDim.y > 1;
  const int split = wide ? kJoinWarps : 1, part = wide ? warp : 0;
  pdl_trigger();
  pdl_wait();
  const int per = A.hkv * A.hb, s = blockIdx.x / per, ub = blockIdx.x - s * per;
  const int heads = min(HU, A.group - (ub % A.hb) * HU);
  const int64_t row0 = int64_t(s) * A.hq + int64_t(ub / A.hb) * A.group + (ub % A.hb) * HU;
  const int64_t seq_tile = A.prefix[s], tl = A.prefix[s + 1] - seq_tile;
  const int64_t total = A.prefix[A.n_seqs] * per, n_w = A.prefix[A.n_seqs + 1];
  int w0 = 0, w1 = 0, groups = 0, n = 0;
  if (tl > 0) {
    // Warps w0..w1 have the unit; the last one's state is an end piece unless the unit
    // ends with that warp's tiles.
    const int64_t lo = seq_tile * per + ub * tl, hi = lo + tl;
    w0 = quotient((lo + 1) * n_w - 1, total);
    w1 = quotient(hi * n_w - 1, total);
    const bool apart = hi != quotient((w1 + 1) * total, n_w);
    groups = w1 - apart < w0 ? 0 : (w1 - apart) / kWarps - w0 / kWarps + 1;
    n = groups + apart;
    if (w0 == w1 || n == 1) return;
  }
  for (int h = wide ? blockIdx.y : warp; h < heads; h += kJoinWarps) {
    auto slot = [&](int i) {
      const int64_t at = i < groups ? max(w0, (w0 / kWarps + i) * kWarps) : kMaxWarps + w1;
      return const_cast<const float*>(A.slots) + (at * HU + h) * (D + 4);
    };
    float M = -INFINITY, L = 0.f, acc[EPL] = {};
#pragma unroll 4
    for (int i = lane; i < n; i += 32) {
      const float2 ml = __ldg(reinterpret_cast<const float2*>(slot(i)));
      if (ml.y != 0.f) M = fmaxf(M, ml.x);
    }
    M = warp_max(M);
#pragma unroll 8
    for (int i = part; i < n; i += split) {
      const float* p = slot(i);
      const float2 ml = __ldg(reinterpret_cast<const float2*>(p));
      float x[EPL];
      load_slice<EPL>(p + 4, lane * EPL, x);
      const float f = ml.y != 0.f ? ex2(ml.x - M) : 0.f;
      L += ml.y * f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) acc[e] = f == 0.f ? acc[e] : fmaf(x[e], f, acc[e]);
    }
    if (wide) {
#pragma unroll
      for (int e = 0; e < EPL; ++e) s_o[warp][lane * EPL + e] = acc[e];
      if (lane == 0) s_l[warp] = L;
      __syncthreads();
      if (warp != 0) return;
      L = 0.f;
#pragma unroll
      for (int k = 0; k < kJoinWarps; ++k) L += s_l[k];
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        acc[e] = 0.f;
#pragma unroll
        for (int k = 0; k < kJoinWarps; ++k) acc[e] += s_o[k][lane * EPL + e];
      }
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e)
      store_o(static_cast<Qt*>(A.O) + (row0 + h) * D + lane * EPL + e, L == 0.f ? 0.f : acc[e] / L);
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
  const int64_t ctas = A.single ? units : max64(1, min64(min64(int64_t(sms) * 2, kMaxCtas), (units * tiles + kWarps * kMinTiles - 1) / (kWarps * kMinTiles)));
  {
    TraceScope ts("attend_batch_kernel", 0, s);
    zha_count_launch();
    e = launch_pdl(kernel, dim3(unsigned(ctas)), dim3(kThreads), kBatchSmem, s, A);
    if (e != cudaSuccess) return e;
  }
  if (A.single) return cudaSuccess;
  TraceScope ts("attend_batch_join_kernel", 0, s);
  zha_count_launch();
  return launch_pdl(attend_batch_join_kernel<Qt, D, HU>, dim3(unsigned(units), unsigned(units <= kWideUnits ? min64(HU, A.group) : 1)), dim3(kJoinThreads), 0, s, A);
}

template <typename Kv, typename Qt>
cudaError_t launch_batch_d(const BatchArgs& A, int d, cudaStream_t s) {
  if (head_rows(A.group) == 16) return d == 128 ? launch_batch<Kv, Qt, 128, 16>(A, s) : launch_batch<Kv, Qt, 64, 16>(A, s);
  return d == 128 ? launch_batch<Kv, Qt, 128, 8>(A, s) : launch_batch<Kv, Qt, 64, 8>(A, s);
}

// Units beyond this are refused: slots and grids stay far below 2^31.
constexpr int64_t kMaxUnits = int64_t(1) << 22;

bool units_ok(const Geom& G, int32_t n_seqs) {
  const int64_t hb = (G.group + head_rows(G.group) - 1) / head_rows(G.group);
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
    return zha_report_error(ZHA_ERR_UNSUPPORTED, "zha_attend_batch_kv: more than 2^22 (sequence, KV head, query block) units");
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
