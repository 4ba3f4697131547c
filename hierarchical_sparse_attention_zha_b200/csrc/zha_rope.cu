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
// rounded at 2^-28 turns.
//
// Bound: HBM, each row read once and written once.
#include <cmath>

#include "zha_host.cuh"
#include "zha_internal.cuh"

namespace zha {

namespace {

constexpr int kRopeThreads = 128;

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
  float s, c;
  sincospif(x, &s, &c);
  float co = (quarter & 1u) ? s : c, si = (quarter & 1u) ? c : s;
  if (quarter == 1u || quarter == 2u) co = -co;
  if (quarter == 2u || quarter == 3u) si = -si;
  if (back) si = -si;
  return make_float2(co * amplitude, si * amplitude);
}

template <int N>
__device__ __forceinline__ void load_n(const float* p, float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(p + i);
    v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
  }
}
__device__ __forceinline__ void load_n(const __nv_bfloat16* p, float (&v)[8]) { load_slice<8>(p, 0, v); }

__device__ __forceinline__ void store_n(float* p, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store_n(__nv_bfloat16* p, const float (&v)[8]) {
  uint4 x;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&x);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = x;
}
__device__ __forceinline__ float load_1(const float* p) { return *p; }
__device__ __forceinline__ float load_1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Work units of a row. Every unit owns all the elements it reads, so a row may
// be turned in place.
//   interleaved:               d/8 units of 8 elements (4 pairs)
//   half, pairs % 8 == 0:      pairs/8 units of 8 pairs, then (d - 2 pairs)/8 of
//                              8 elements that stay
//   half, other pair counts:   pairs units of one pair, then d - 2 pairs single
//                              elements (rows are not 16-byte addressable at i + pairs)
__host__ __device__ inline int row_units(const RopeTable& R, int d) {
  if (!R.half || R.pairs == 0) return d / 8;
  return R.pairs % 8 == 0 ? d / 8 - R.pairs / 8 : d - R.pairs;
}

template <typename Src, typename Dst>
__device__ __forceinline__ void turn_unit(const Src* x, Dst* y, int u, int P, bool half, bool turned,
                                          const float2* cs) {
  if (!turned || !half) {
    float v[8];
    load_n(x + u * 8, v);
    if (turned) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (u * 4 + i < P) {
          const float2 t = cs[u * 4 + i];
          const float a = v[2 * i], b = v[2 * i + 1];
          v[2 * i] = a * t.x - b * t.y;
          v[2 * i + 1] = a * t.y + b * t.x;
        }
      }
    }
    store_n(y + u * 8, v);
    return;
  }
  if (P % 8 == 0) {
    if (u < P / 8) {
      float a[8], b[8];
      load_n(x + u * 8, a);
      load_n(x + P + u * 8, b);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 t = cs[u * 8 + i];
        const float p = a[i], q = b[i];
        a[i] = p * t.x - q * t.y;
        b[i] = p * t.y + q * t.x;
      }
      store_n(y + u * 8, a);
      store_n(y + P + u * 8, b);
    } else {
      float v[8];
      load_n(x + P + u * 8, v);
      store_n(y + P + u * 8, v);
    }
    return;
  }
  if (u < P) {
    const float2 t = cs[u];
    const float a = load_1(x + u), b = load_1(x + P + u);
    store_1(y + u, a * t.x - b * t.y);
    store_1(y + P + u, a * t.y + b * t.x);
  } else {
    store_1(y + P + u, load_1(x + P + u));
  }
}

// Units of a row that is only copied: d/8.
template <typename Src, typename Dst>
__device__ __forceinline__ void turn_row_unit(const void* src, int64_t so, void* dst, int64_t d_o, int u,
                                              const RopeTable& R, bool turned, const float2* cs) {
  turn_unit(static_cast<const Src*>(src) + so, static_cast<Dst*>(dst) + d_o, u, R.pairs, R.half != 0, turned, cs);
}

template <typename Src, typename Dst>
__global__ void __launch_bounds__(kRopeThreads) rope_apply_kernel(const __grid_constant__ RopeTable R, RowSet X,
                                                                  const int64_t* pos, int64_t n_tokens, int d,
                                                                  int back) {
  __shared__ float2 cs[64];
  pdl_trigger();
  pdl_wait();
  const int units = row_units(R, d), total = X.heads * units;
  for (int64_t t = blockIdx.x; t < n_tokens; t += gridDim.x) {
    if (threadIdx.x < R.pairs) cs[threadIdx.x] = cos_sin_of(R.turn[threadIdx.x], pos[t], R.amplitude, back != 0);
    __syncthreads();
    for (int i = threadIdx.x + blockIdx.y * kRopeThreads; i < total; i += kRopeThreads * gridDim.y) {
      const int h = i / units, u = i - h * units;
      turn_row_unit<Src, Dst>(X.src, t * X.src_token + h * X.src_head, X.dst, t * X.dst_token + h * X.dst_head, u,
                              R, true, cs);
    }
    __syncthreads();
  }
}

template <typename Src, typename Kv, typename Qo>
__global__ void __launch_bounds__(kRopeThreads)
    rope_append_kernel(const __grid_constant__ RopeTable R, RowSet Q, RowSet K, RowSet V, KvView kv, int n_seqs,
                       const int32_t* seq, const int64_t* index, const int64_t* pos, int64_t n_new, int d, int chunk,
                       int32_t* status) {
  __shared__ float2 cs[64];
  pdl_trigger();
  pdl_wait();
  const int hkv = K.heads;
  const int units = row_units(R, d), vunits = d / 8;
  const int nq = Q.heads * units, nk = hkv * units, total = nq + nk + hkv * vunits;
  const int64_t limit = kv.table == nullptr ? kv.ld : kv.max_blocks * chunk;
  for (int64_t t = blockIdx.x; t < n_new; t += gridDim.x) {
    const int32_t s = seq[t];
    if (s < 0) continue;                              // the whole block agrees
    const int64_t at = index[t];
    if (s >= n_seqs || at < 0 || at >= limit) {
      if (threadIdx.x == 0 && blockIdx.y == 0 && status != nullptr) atomicOr(status, ZHA_DEV_BAD_SEQUENCE);
      continue;
    }
    if (threadIdx.x < R.pairs)
      cs[threadIdx.x] = cos_sin_of(R.turn[threadIdx.x], pos != nullptr ? pos[t] : at, R.amplitude, false);
    __syncthreads();
    for (int i = threadIdx.x + blockIdx.y * kRopeThreads; i < total; i += kRopeThreads * gridDim.y) {
      if (i < nq) {
        const int h = i / units, u = i - h * units;
        turn_row_unit<Src, Qo>(Q.src, t * Q.src_token + h * Q.src_head, Q.dst, t * Q.dst_token + int64_t(h) * d, u, R,
                               R.pairs > 0, cs);
        continue;
      }
      const bool key = i < nq + nk;
      const int j = key ? i - nq : i - nq - nk, per = key ? units : vunits;
      const int g = j / per, u = j - g * per;
      const int32_t row = kv_batch_row(kv, hkv, s, g, at, chunk);
      if (row < 0) {
        if (status != nullptr) atomicOr(status, ZHA_DEV_BAD_PAGE);
        continue;
      }
      const RowSet& S = key ? K : V;
      turn_row_unit<Src, Kv>(S.src, t * S.src_token + g * S.src_head, S.dst, int64_t(row) * d, u, R,
                             key && R.pairs > 0, cs);
    }
    __syncthreads();
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

// One block per token; few tokens with many units are spread over blocks in y.
dim3 rope_grid(int64_t tokens, int64_t units) {
  const int64_t x = tokens < (1 << 20) ? tokens : (1 << 20);
  int64_t y = (units + kRopeThreads - 1) / kRopeThreads;
  if (x * y > 148 * 16) y = (148 * 16 + x - 1) / x;
  return dim3(unsigned(x), unsigned(y < 1 ? 1 : y > 65535 ? 65535 : y));
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

template <typename Src, typename Dst>
cudaError_t launch_apply(const RopeTable& R, const RowSet& X, const int64_t* pos, int64_t n, int d, int back,
                         cudaStream_t s) {
  TraceScope ts("rope_apply_kernel", 0, s);
  zha_count_launch();
  return launch_pdl(rope_apply_kernel<Src, Dst>, rope_grid(n, int64_t(X.heads) * row_units(R, d)),
                    dim3(kRopeThreads), 0, s, R, X, pos, n, d, back);
}

template <typename Src, typename Kv, typename Qo>
cudaError_t launch_append(const RopeTable& R, const RowSet& Q, const RowSet& K, const RowSet& V, const KvView& kv,
                          int n_seqs, const int32_t* seq, const int64_t* index, const int64_t* pos, int64_t n,
                          int d, int chunk, int32_t* status, cudaStream_t s) {
  TraceScope ts("rope_append_kernel", 0, s);
  zha_count_launch();
  const int64_t units = int64_t(Q.heads + K.heads) * row_units(R, d) + int64_t(V.heads) * (d / 8);
  return launch_pdl(rope_append_kernel<Src, Kv, Qo>, rope_grid(n, units), dim3(kRopeThreads), 0, s, R, Q, K, V, kv,
                    n_seqs, seq, index, pos, n, d, chunk, status);
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
  if (!(c->amplitude >= 0.0) || !std::isfinite(c->amplitude))
    return rope_fail(ZHA_ERR_INVALID, "zha_rope_init: amplitude must be finite and >= 0");
  const double two_pi = 6.283185307179586476925286766559;
  double base = c->base;
  if (c->scaling == ZHA_ROPE_NTK && D > 2) base *= std::pow(f, double(D) / (D - 2));
  double lo = 0.0, hi = 0.0;
  if (c->scaling == ZHA_ROPE_YARN) {
    auto where = [&](double turns) {
      return D * std::log(c->original_tokens / (two_pi * turns)) / (2.0 * std::log(c->base));
    };
    lo = std::fmax(0.0, std::floor(where(c->high)));
    hi = std::fmin(double(c->pairs - 1), std::ceil(where(c->low)));
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
  using bf = __nv_bfloat16;
  cudaError_t e =
      x_dtype == ZHA_F32
          ? (y_dtype == ZHA_F32 ? zha::launch_apply<float, float>(R, X, d_pos, n_tokens, d, back, s)
                                : zha::launch_apply<float, bf>(R, X, d_pos, n_tokens, d, back, s))
          : (y_dtype == ZHA_F32 ? zha::launch_apply<bf, float>(R, X, d_pos, n_tokens, d, back, s)
                                : zha::launch_apply<bf, bf>(R, X, d_pos, n_tokens, d, back, s));
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
  const zha::RopeTable R = zha::table_of(rope);
  RowSet Q{}, K{}, V{};
  if (q != nullptr) Q = RowSet{q->data, d_q_out, q->token_stride, q->head_stride, int64_t(G.hq) * G.d, G.d, G.hq};
  K = RowSet{k->data, const_cast<void*>(kv->k), k->token_stride, k->head_stride, 0, 0, G.hkv};
  V = RowSet{v->data, const_cast<void*>(kv->v), v->token_stride, v->head_stride, 0, 0, G.hkv};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  using bf = __nv_bfloat16;
  auto go = [&](auto launch) {
    return launch(R, Q, K, V, view, n_seqs, d_seq, d_index, d_pos, n_new, G.d, G.chunk, d_status, s);
  };
  const int which = (src_dtype == ZHA_BF16 ? 4 : 0) + (G.kv_bf16 ? 2 : 0) + (q_dtype == ZHA_BF16 ? 1 : 0);
  cudaError_t e = cudaSuccess;
  switch (which) {
    case 0: e = go(zha::launch_append<float, float, float>); break;
    case 1: e = go(zha::launch_append<float, float, bf>); break;
    case 2: e = go(zha::launch_append<float, bf, float>); break;
    case 3: e = go(zha::launch_append<float, bf, bf>); break;
    case 4: e = go(zha::launch_append<bf, float, float>); break;
    case 5: e = go(zha::launch_append<bf, float, bf>); break;
    case 6: e = go(zha::launch_append<bf, bf, float>); break;
    default: e = go(zha::launch_append<bf, bf, bf>); break;
  }
  return e == cudaSuccess ? ZHA_OK : zha_report_cuda(e, who);
}

}  // extern "C"
