// What the forward and the backward row passes share: which columns a thread
// owns, the ring of rows in shared memory, and the statistics of a row.
//
// A block holds K rows at a time and a thread the same columns of each: NV
// times eight, in pieces of P neighbours that lie P * blockDim apart, so that a
// warp's access is contiguous.  P is eight bfloat16 elements where stream and
// branch are bfloat16, four where the stream is float32 (a bfloat16 branch then
// moves 8 bytes at a time), if the row length and every row's address allow it;
// else two (bfloat16 stream), else a single element.
// Rows that come in are copied ahead of their use into a ring of `depth` rows
// (RING): every thread copies and reads its own columns only, so a ring needs
// no barrier, and keeps some 100 KB in flight on an SM, which loads into
// registers could not.  Without RING (pieces below 4 bytes, and long rows: see
// the launch code) rows are read from global memory where they are used.
#pragma once
#include "row_io.cuh"
#include "spade_internal.cuh"

namespace spade {
namespace rowpass {

using namespace rowio;

enum { kNone = SPADE_NORM_NONE, kRms = SPADE_NORM_RMS, kLayer = SPADE_NORM_LAYER };

// FULL: the threads' columns are exactly the row's.
template <int P_, bool FULL_, bool RING_, int NV_>
struct Layout {
  static constexpr int P = P_, NV = NV_;
  static constexpr bool FULL = FULL_, RING = RING_;
};
template <class L>
__device__ __forceinline__ int column(int i, int e) {
  constexpr int P = L::P;
  return ((i * (8 / P) + e / P) * (int)blockDim.x + (int)threadIdx.x) * P + e % P;
}

template <class L>
__device__ __forceinline__ bool inside(int column, int dim) {
  return L::FULL || column < dim;
}

// A thread's eight elements, as pairs.
struct Eight {
  float2 p[4];

  __device__ __forceinline__ float* f() { return &p[0].x; }
  __device__ __forceinline__ const float* f() const { return &p[0].x; }
  __device__ __forceinline__ void fill(float v) {
#pragma unroll
    for (int q = 0; q < 4; ++q) p[q] = both(v);
  }
};

template <class L, typename T>
__device__ __forceinline__ void load8(Eight& v, const T* row, int i, int dim) {
  constexpr int P = L::P;
#pragma unroll
  for (int e = 0; e < 8; e += P) {
    const int c = column<L>(i, e);
    if (inside<L>(c, dim)) {
      load_piece<T, P>(v.f() + e, row + c);
    } else {
#pragma unroll
      for (int q = 0; q < P; ++q) v.f()[e + q] = 0.f;
    }
  }
}
template <class L, typename T>
__device__ __forceinline__ void store8(T* row, const Eight& v, int i, int dim) {
  constexpr int P = L::P;
#pragma unroll
  for (int e = 0; e < 8; e += P) {
    const int c = column<L>(i, e);
    if (inside<L>(c, dim)) store_piece<P>(row + c, v.f() + e);
  }
}
// A parameter row in either type; absent ones read as `none`.
template <class L>
__device__ __forceinline__ void load_param(Eight& v, const void* p, long long off, bool is_bf16, float none, int i,
                                           int dim) {
  if (!p) v.fill(none);
  else if (is_bf16) load8<L>(v, static_cast<const bf16*>(p) + off, i, dim);
  else load8<L>(v, static_cast<const float*>(p) + off, i, dim);
}
// v in the columns of pair q that the row has, 0 in the others.
template <class L>
__device__ __forceinline__ float2 present(float2 v, int i, int q, int dim) {
  if (L::FULL) return v;
  if (L::P > 1) return column<L>(i, 2 * q) < dim ? v : both(0.f);
  return make_float2(column<L>(i, 2 * q) < dim ? v.x : 0.f, column<L>(i, 2 * q + 1) < dim ? v.y : 0.f);
}

// A row operand: the next row to copy (RING) or to read, and the operand's
// place in a slot of the ring.
template <typename T, class L>
struct Stream {
  static constexpr int P = L::P, NV = L::NV;
  const T* p;
  uint32_t at;       // bytes into a slot

  __device__ __forceinline__ void seek(const void* base, long long stride, long long r) {
    p = static_cast<const T*>(base) + r * stride;
  }
  __device__ __forceinline__ void fetch(uint32_t slot, int dim) const {
    if constexpr (L::RING) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; e += P) {
          const int c = column<L>(i, e);
          if (inside<L>(c, dim)) copy_async<P * (int)sizeof(T)>(slot + at + c * (int)sizeof(T), p + c);
        }
    }
  }
  // Columns past the row's end read as zero.
  __device__ __forceinline__ void clear(unsigned char* slot, int dim) const {
    if constexpr (!L::FULL) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = column<L>(i, e);
          if (!inside<L>(c, dim)) reinterpret_cast<T*>(slot + at)[c] = T(0.f);
        }
    }
  }
  // The row in a slot, or `ahead` elements past the next one in memory.
  __device__ __forceinline__ void get(Eight& v, const unsigned char* slot, long long ahead, int i, int dim) const {
    if constexpr (L::RING) {
      const T* row = reinterpret_cast<const T*>(slot + at);
#pragma unroll
      for (int e = 0; e < 8; e += P) load_piece<T, P>(v.f() + e, row + column<L>(i, e));
    } else {
      load8<L>(v, p + ahead, i, dim);
    }
  }
};

// The bytes an operand takes in a slot.
__host__ __device__ inline uint32_t slot_bytes(int threads, int nv, int elem) { return (uint32_t)(threads * nv * 8 * elem); }

// Scratch of the sums of N values at once, and the columns that each warp owns
// (0 past the last warp) with the reciprocal.
template <int N>
struct Shared {
  Scratch<N> sums;
  float count[32], inv_count[32];
};
template <class L, int N>
__device__ __forceinline__ void count_columns(Shared<N>& sh, int dim) {
  float c[1] = {0.f};
#pragma unroll
  for (int i = 0; i < L::NV; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) c[0] += inside<L>(column<L>(i, e), dim) ? 1.f : 0.f;
  const float s = warp_sum_spread<1>(c);
  for (int i = threadIdx.x; i < 2 * N * 33; i += blockDim.x) (&sh.sums.v[0][0])[i] = make_float2(0.f, 0.f);
  if (threadIdx.x < 32) sh.count[threadIdx.x] = sh.inv_count[threadIdx.x] = 0.f;
  __syncthreads();
  if ((threadIdx.x & 31) == 0 && s > 0.f) {
    sh.count[threadIdx.x >> 5] = s;
    sh.inv_count[threadIdx.x >> 5] = 1.f / s;
  }
  __syncthreads();
}
// The columns of a warp; all own the same in a FULL layout.
template <class L, int N>
__device__ __forceinline__ float count_of(const Shared<N>& sh, int warp) {
  return L::FULL ? 256.f * L::NV : sh.count[warp];
}
template <class L, int N>
__device__ __forceinline__ float inv_count_of(const Shared<N>& sh, int warp) {
  return L::FULL ? 1.f / (256.f * L::NV) : sh.inv_count[warp];
}

// Mean (0 for the rms norm) and reciprocal deviation of K rows held in
// registers.  The layer norm's second moment is taken about each warp's own
// mean and the warps' moments are merged (Chan, Golub and LeVeque, 1979), so
// a row far from zero loses nothing and one barrier is enough.
template <class L, int K, int S>
__device__ __forceinline__ void row_stats(const Eight (&v)[K][L::NV], int kind, float eps, float inv_dim, int dim,
                                          Shared<S>& sh, int& half, int nwarps, float (&mean)[K], float (&rstd)[K]) {
  constexpr int NV = L::NV;
  float s[K];
  if (kind == kRms) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 t = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) t = fma(v[k][i].p[q], v[k][i].p[q], t);
      s[k] = sum_of(t);
    }
    block_sum(s, sh.sums, half, nwarps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      mean[k] = 0.f;
      rstd[k] = rsqrtf(s[k] * inv_dim + eps);
    }
    return;
  }
  constexpr int M = 32 / K, W = (32 + M - 1) / M;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % M;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 t = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) t = add(t, v[k][i].p[q]);
    s[k] = sum_of(t);
  }
  float mu = warp_sum_spread<K>(s) * inv_count_of<L>(sh, warp);      // of the row this lane stands for
  float m[K];
  spread_get<K>(m, mu);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 t = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 off = add(v[k][i].p[q], present<L>(both(-m[k]), i, q, dim));
        t = fma(off, off, t);
      }
    s[k] = sum_of(t);
  }
  float q = warp_sum_spread<K>(s);
  if (nwarps > 1) {
    float2* b = sh.sums.v[half] + (lane / M) * 33;
    if (sub == 0) b[warp] = make_float2(mu, q);
    __syncthreads();
    float2 p[W];
    float total = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      p[j] = b[sub + j * M];                     // warps that are not there: zeros, or (block sums) leftovers
      total += sub + j * M < nwarps ? count_of<L>(sh, sub + j * M) * p[j].x : 0.f;
    }
    mu = spread_sum<K>(total) * inv_dim;
    q = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float off = p[j].x - mu;
      q += sub + j * M < nwarps ? count_of<L>(sh, sub + j * M) * off * off + p[j].y : 0.f;
    }
    q = spread_sum<K>(q);
    half ^= 1;
  }
  spread_get<K>(mean, mu);
  spread_get<K>(rstd, rsqrtf(q * inv_dim + eps));
}

// The statistics of K rows x' and, for the gradient u that reaches their norm,
// mean(u) (0 for the rms norm) and mean(u xhat), with one barrier: the sums
// with u are taken about the warps' means as well and merged alike.
template <class L, int K, int S>
__device__ __forceinline__ void row_stats_bwd(const Eight (&v)[K][L::NV], const Eight (&u)[K][L::NV], int kind, float eps,
                                              float inv_dim, int dim, Shared<S>& sh, int& half, int nwarps,
                                              float (&mean)[K], float (&rstd)[K], float (&mu0)[K], float (&mu1)[K]) {
  constexpr int NV = L::NV;
  float s[2 * K];
  if (kind == kRms) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float2 t0 = both(0.f), t1 = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          t0 = fma(v[k][i].p[q], v[k][i].p[q], t0);
          t1 = fma(u[k][i].p[q], v[k][i].p[q], t1);
        }
      s[k] = sum_of(t0);
      s[K + k] = sum_of(t1);
    }
    block_sum(s, sh.sums, half, nwarps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      mean[k] = mu0[k] = 0.f;
      rstd[k] = rsqrtf(s[k] * inv_dim + eps);
      mu1[k] = s[K + k] * inv_dim * rstd[k];
    }
    return;
  }
  // values of a warp: first the sums of x' and u, then the second moment and
  // the sum of u (x' - its mean); lanes below 16 stand for x', the others for u
  constexpr int N = 2 * K, M = 32 / N, W = (32 + M - 1) / M;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % M;
  const bool is_x = lane < 16;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 t0 = both(0.f), t1 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        t0 = add(t0, v[k][i].p[q]);
        t1 = add(t1, u[k][i].p[q]);
      }
    s[k] = sum_of(t0);
    s[K + k] = sum_of(t1);
  }
  float first = warp_sum_spread<N>(s);
  first *= is_x ? inv_count_of<L>(sh, warp) : 1.f;
  float m[K];
#pragma unroll
  for (int k = 0; k < K; ++k) m[k] = __shfl_sync(0xffffffffu, first, k * M);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    float2 t0 = both(0.f), t1 = both(0.f);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 off = add(v[k][i].p[q], present<L>(both(-m[k]), i, q, dim));
        t0 = fma(off, off, t0);
        t1 = fma(u[k][i].p[q], off, t1);
      }
    s[k] = sum_of(t0);
    s[K + k] = sum_of(t1);
  }
  float second = warp_sum_spread<N>(s);
  if (nwarps > 1) {
    float2* b = sh.sums.v[half] + (lane / M) * 33;
    if (sub == 0) b[warp] = make_float2(first, second);
    __syncthreads();
    const float2* bx = sh.sums.v[half] + ((lane & 15) / M) * 33;     // x' of the row this lane stands for
    float2 p[W];
    float total = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      p[j] = b[sub + j * M];
      total += sub + j * M < nwarps ? (is_x ? count_of<L>(sh, sub + j * M) : 1.f) * p[j].x : 0.f;
    }
    first = spread_sum<N>(total) * (is_x ? inv_dim : 1.f);
    const float mx = __shfl_sync(0xffffffffu, first, lane & 15);
    second = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) {
      const float off = bx[sub + j * M].x - mx;
      second += sub + j * M < nwarps ? off * (is_x ? count_of<L>(sh, sub + j * M) * off : p[j].x) + p[j].y : 0.f;
    }
    second = spread_sum<N>(second);
    half ^= 1;
  }
  if (is_x) second = rsqrtf(second * inv_dim + eps);
  float a[N], b2[N];
  spread_get<N>(a, first);
  spread_get<N>(b2, second);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    mean[k] = a[k];
    rstd[k] = b2[k];
    mu0[k] = a[K + k] * inv_dim;
    mu1[k] = b2[K + k] * inv_dim * b2[k];
  }
}

// ----------------------------------------------------------------- launch --
// The widest piece, in elements, that every row of every operand allows.
inline int piece_of(const RowArgs& a) {
  const int ex = a.x_bf16 ? 2 : 4, eb = a.branch_bf16 ? 2 : 4, ep = a.param_bf16 ? 2 : 4;
  const struct { const void* p; long long stride; int size; } ops[] = {
      {a.x, a.x_stride, ex}, {a.x_out, a.x_out_stride, ex}, {a.dx_out, a.dx_out_stride, ex}, {a.dx, a.dx_stride, ex},
      {a.y, a.y_stride, eb}, {a.h, a.h_stride, eb}, {a.dh, a.dh_stride, eb}, {a.dy, a.dy_stride, eb},
      {a.gate, a.gate_stride, ep}, {a.scale, a.scale_stride, ep}, {a.shift, a.shift_stride, ep}, {a.weight, 0, ep},
      {a.bias, 0, ep}, {a.post_weight, 0, ep}, {a.dgate, a.dim, 4}, {a.dscale, a.dim, 4}, {a.dshift, a.dim, 4}};
  for (int p = ex == 2 && eb == 2 ? 8 : 4; p > 1; p >>= 1) {
    bool ok = a.dim % p == 0;
    for (const auto& o : ops) {
      const int need = p * o.size < 16 ? p * o.size : 16;
      ok = ok && (!o.p || (reinterpret_cast<uintptr_t>(o.p) % need == 0 && o.stride % p == 0));
    }
    if (ok) return p;
  }
  return 1;
}

constexpr int kSmemSm = 227 * 1024;     // shared memory of an SM that blocks can use
constexpr int kDepthMax = 14;           // rows of a ring: wait_async_upto covers depth - K

inline int row_threads(int dim, int nv) {
  const int t = (dim + 8 * nv - 1) / (8 * nv);
  return (t + 31) / 32 * 32;
}

// Blocks of an SM in a backward pass, by registers: 96 a thread, 128 where a
// thread holds more than eight columns.
inline int bwd_blocks(int dim) {
  if (dim > 5120) return 1;
  const int b = 640 / row_threads(dim, 1);
  return b < 1 ? 1 : (b > 16 ? 16 : b);
}

}  // namespace rowpass
}  // namespace spade
