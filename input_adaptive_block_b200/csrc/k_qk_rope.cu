// Norm and several-axis rotation of Q and K, one pass over both
// (spade_qk_norm_rope, spade_qk_norm_rope_bwd).
//
// Pair i of a head rotates by pos[axis_i] * freq_i.  The angle is formed in
// turns, position times turns-per-unit in float64, its nearest integer is
// taken off there and the rest (at most half a turn, rounded once to float32)
// goes to sincospif: positions anywhere in int32 keep an angle good to
// float32.  A token's angles are computed once and serve every head of Q and
// of K.
//
// Forward:  n = x * rstd * w (rms over the token's heads * d values, over
//           each head's d, or no norm), out = rotation of n.
// Backward: u = dout rotated back, dw = sum of u * x * rstd over the rows (and
//           heads, for the per-head norm), dx = rstd (w u - x rstd^2 mean(w u x)).
//
// `lanes` threads share a head (d / 16 rounded up to a power of two), each
// owning eight pairs: the same pairs of every head it meets, so their sines
// and cosines stay in its registers for the whole token.  A block takes kTok
// tokens at a time and loads all of them before it uses the first, which keeps
// enough bytes in flight; their sums share one barrier.  Bound by memory.
#include "row_io.cuh"
#include "spade_internal.cuh"

namespace spade {
namespace {

using namespace rowio;

constexpr int kTok = 2;     // tokens a block holds at once

// A thread's eight pairs of one head: first elements in a, second in b.
template <typename T>
struct Unit {
  Raw8<T> lo, hi;
};

// Pairs of a thread: eight neighbours (VEC), or every lanes-th pair.
template <bool VEC>
__device__ __forceinline__ int pair_of(int j, int e, int lanes) {
  return VEC ? j * 8 + e : e * lanes + j;
}

// Element offset of pair p's first and second element in a head.
__device__ __forceinline__ int first_of(int p, bool half) { return half ? p : 2 * p; }
__device__ __forceinline__ int second_of(int p, bool half, int d) { return half ? p + (d >> 1) : 2 * p + 1; }

// The sixteen elements in head order of a VEC unit: [8j, 8j+8) and d/2 later
// (halves), or [16j, 16j+16) (neighbouring pairs).
template <typename T>
__device__ __forceinline__ void load_unit(Unit<T>& u, const T* head, int j, bool half, int d) {
  const T* p = head + (half ? 8 * j : 16 * j);
  load_raw(u.lo, p);
  load_raw(u.hi, p + (half ? (d >> 1) : 8));
}
template <typename T>
__device__ __forceinline__ void split_unit(float (&a)[8], float (&b)[8], const Unit<T>& u, bool half) {
  float lo[8], hi[8];
  unpack(lo, u.lo);
  unpack(hi, u.hi);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = half ? lo[e] : (e < 4 ? lo[2 * e] : hi[2 * e - 8]);
    b[e] = half ? hi[e] : (e < 4 ? lo[2 * e + 1] : hi[2 * e - 7]);
  }
}
template <typename T>
__device__ __forceinline__ void store_unit(T* head, const float (&a)[8], const float (&b)[8], int j, bool half, int d) {
  float lo[8], hi[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int i = e >> 1;
    lo[e] = half ? a[e] : (e & 1 ? b[i] : a[i]);
    hi[e] = half ? b[e] : (e & 1 ? b[4 + i] : a[4 + i]);
  }
  T* p = head + (half ? 8 * j : 16 * j);
  store_vec(p, lo);
  store_vec(p + (half ? (d >> 1) : 8), hi);
}

// One thread's share of one head, as pair elements in float32; absent pairs
// and heads are zero.
template <bool VEC, typename T>
struct Share {
  Unit<T> u;                 // VEC
  float a[VEC ? 1 : 8], b[VEC ? 1 : 8];

  __device__ __forceinline__ void load(const T* head, bool in, int j, int lanes, bool half, int d) {
    if (VEC) {
      if (in) load_unit(u, head, j, half, d);
      else {
        clear_raw(u.lo);
        clear_raw(u.hi);
      }
    } else {
#pragma unroll
      for (int e = 0; e < (VEC ? 1 : 8); ++e) {
        const int p = pair_of<false>(j, e, lanes);
        const bool ok = in && p < (d >> 1);
        a[e] = ok ? to_float(head[first_of(p, half)]) : 0.f;
        b[e] = ok ? to_float(head[second_of(p, half, d)]) : 0.f;
      }
    }
  }
  __device__ __forceinline__ void get(float (&oa)[8], float (&ob)[8], bool half) const {
    if (VEC) {
      split_unit(oa, ob, u, half);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        oa[e] = a[VEC ? 0 : e];
        ob[e] = b[VEC ? 0 : e];
      }
    }
  }
};
template <bool VEC, typename T>
__device__ __forceinline__ void store_share(T* head, const float (&a)[8], const float (&b)[8], int j, int lanes,
                                            bool half, int d) {
  if (VEC) {
    store_unit(head, a, b, j, half, d);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int p = pair_of<false>(j, e, lanes);
      if (p < (d >> 1)) {
        store_one(head + first_of(p, half), a[e]);
        store_one(head + second_of(p, half, d), b[e]);
      }
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void load_weight(float (&a)[8], float (&b)[8], const void* w, bool bf16, int off, bool in,
                                            int j, int lanes, bool half, int d) {
  if (!w || !in) {
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = b[e] = 1.f;
  } else if (bf16) {
    Share<VEC, __nv_bfloat16> s;
    s.load(static_cast<const __nv_bfloat16*>(w) + off, true, j, lanes, half, d);
    s.get(a, b, half);
  } else {
    Share<VEC, float> s;
    s.load(static_cast<const float*>(w) + off, true, j, lanes, half, d);
    s.get(a, b, half);
  }
}

// Cosine and sine of every pair of the block's next tokens.
__device__ __forceinline__ void angles(const QkArgs& a, long long r0, int n, float2* cs) {
  const int half_d = a.d >> 1;
  for (int i = threadIdx.x; i < n * half_d; i += blockDim.x) {
    const int k = i / half_d, p = i - k * half_d;
    const long long r = r0 + k;
    float2 v = make_float2(1.f, 0.f);
    if (p < a.pairs && r < a.video_rows) {
      int pos;
      if (a.positions) {
        pos = a.positions[r * 3 + a.axis[p]];
      } else {
        const int tok = a.tok0 + (int)r;
        const int row = tok / a.W;
        pos = a.axis[p] == 2 ? tok - row * a.W : (a.axis[p] == 1 ? row % a.H : row / a.H);
      }
      const double t = (double)pos * a.turn[p];
      sincospif(2.f * (float)(t - rint(t)), &v.y, &v.x);
    }
    cs[i] = v;
  }
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- forward --
template <typename T, bool VEC, int UPT>
__global__ void __launch_bounds__(UPT == 1 ? 512 : 1024, 1) qk_fwd_kernel(const __grid_constant__ QkArgs a) {
  extern __shared__ float2 cs[];         // [2][kTok][d / 2]
  __shared__ SumScratch<2 * kTok> sums;
  const int lanes = a.lanes, j = threadIdx.x & (lanes - 1), head0 = threadIdx.x / lanes;
  const int hstep = blockDim.x / lanes, nwarps = blockDim.x >> 5, d = a.d;
  const bool half = a.half, own = VEC ? 16 * j < d : true;
  int sh = 0, buf = 0;
  for (long long r0 = (long long)blockIdx.x * kTok; r0 < a.rows; r0 += (long long)gridDim.x * kTok) {
    const int n = (int)min((long long)kTok, a.rows - r0);
    Share<VEC, T> x[kTok][2][UPT];
#pragma unroll
    for (int k = 0; k < kTok; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          const int h = head0 + i * hstep;
          const bool in = k < n && own && h < a.heads[t];
          x[k][t][i].load(static_cast<const T*>(a.x[t]) + (r0 + k) * a.x_stride[t] + (long long)h * d, in, j, lanes,
                          half, d);
        }
    float2* c = cs + buf * (kTok * (d >> 1));
    angles(a, r0, n, c);
    float s[2 * kTok];
    float rs[kTok][2][UPT];
    if (a.norm != SPADE_QK_NORM_NONE) {
#pragma unroll
      for (int k = 0; k < kTok; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          s[2 * k + t] = 0.f;
#pragma unroll
          for (int i = 0; i < UPT; ++i) {
            float u[8], v[8], q = 0.f;
            x[k][t][i].get(u, v, half);
#pragma unroll
            for (int e = 0; e < 8; ++e) q += u[e] * u[e] + v[e] * v[e];
            s[2 * k + t] += q;
            rs[k][t][i] = q;
          }
        }
    }
    if (a.norm == SPADE_QK_NORM_TOKEN && nwarps > 1) {
      block_sum(s, sums, sh, nwarps);      // its barrier also covers the angles
    } else {
      if (a.norm == SPADE_QK_NORM_TOKEN) block_sum(s, sums, sh, nwarps);
      __syncthreads();
    }
#pragma unroll
    for (int k = 0; k < kTok; ++k)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          if (a.norm == SPADE_QK_NORM_TOKEN)
            rs[k][t][i] = rsqrtf(s[2 * k + t] / (float)(a.heads[t] * d) + a.eps);
          else if (a.norm == SPADE_QK_NORM_HEAD)
            rs[k][t][i] = rsqrtf(lanes_sum(rs[k][t][i], lanes) / (float)d + a.eps);
          else
            rs[k][t][i] = 1.f;
        }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int h = head0 + i * hstep;
        const bool in = own && h < a.heads[t];
        float wa[8], wb[8];
        load_weight<VEC>(wa, wb, a.weight[t], a.weight_bf16, a.norm == SPADE_QK_NORM_TOKEN ? h * d : 0, in, j, lanes,
                         half, d);
#pragma unroll
        for (int k = 0; k < kTok; ++k) {
          if (!in || k >= n) continue;
          float u[8], v[8];
          x[k][t][i].get(u, v, half);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int p = pair_of<VEC>(j, e, lanes);
            const float2 r = p < (d >> 1) ? c[k * (d >> 1) + p] : make_float2(1.f, 0.f);
            const float p0 = u[e] * (rs[k][t][i] * wa[e]), p1 = v[e] * (rs[k][t][i] * wb[e]);
            u[e] = p0 * r.x - p1 * r.y;
            v[e] = p0 * r.y + p1 * r.x;
          }
          store_share<VEC>(static_cast<T*>(a.out[t]) + (r0 + k) * a.out_stride[t] + (long long)h * d, u, v, j, lanes,
                           half, d);
        }
      }
    buf ^= 1;
  }
}

// --------------------------------------------------------------- backward --
template <typename T, bool VEC, int UPT>
__global__ void __launch_bounds__(UPT == 1 ? 512 : 1024, 1) qk_bwd_kernel(const __grid_constant__ QkArgs a) {
  extern __shared__ float2 cs[];         // [2][d / 2]
  __shared__ SumScratch<4> sums;
  const int lanes = a.lanes, j = threadIdx.x & (lanes - 1), head0 = threadIdx.x / lanes;
  const int hstep = blockDim.x / lanes, nwarps = blockDim.x >> 5, d = a.d;
  const bool half = a.half, own = VEC ? 16 * j < d : true;
  const bool normed = a.norm != SPADE_QK_NORM_NONE, token = a.norm == SPADE_QK_NORM_TOKEN;
  int sh = 0, buf = 0;
  float dw[2][UPT][2][8];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int i = 0; i < UPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[t][i][0][e] = dw[t][i][1][e] = 0.f;
  for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
    Share<VEC, T> x[2][UPT], g[2][UPT];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int h = head0 + i * hstep;
        const bool in = own && h < a.heads[t];
        g[t][i].load(static_cast<const T*>(a.dout[t]) + r * a.dout_stride[t] + (long long)h * d, in, j, lanes, half, d);
        if (normed)
          x[t][i].load(static_cast<const T*>(a.x[t]) + r * a.x_stride[t] + (long long)h * d, in, j, lanes, half, d);
      }
    float2* c = cs + buf * (d >> 1);
    angles(a, r, 1, c);
    __syncthreads();
    float ua[2][UPT][8], ub[2][UPT][8];
    float s[4] = {0.f, 0.f, 0.f, 0.f};       // per tensor: sum of x^2, sum of w u x
    float hs[2][UPT][2];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int h = head0 + i * hstep;
        const bool in = own && h < a.heads[t];
        float xa[8], xb[8], wa[8], wb[8];
        g[t][i].get(ua[t][i], ub[t][i], half);
        if (normed) x[t][i].get(xa, xb, half);
        load_weight<VEC>(wa, wb, normed ? a.weight[t] : nullptr, a.weight_bf16, token ? h * d : 0, in, j, lanes, half,
                         d);
        float q0 = 0.f, q1 = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int p = pair_of<VEC>(j, e, lanes);
          const float2 r2 = p < (d >> 1) ? c[p] : make_float2(1.f, 0.f);
          const float p0 = ua[t][i][e], p1 = ub[t][i][e];
          ua[t][i][e] = p0 * r2.x + p1 * r2.y;
          ub[t][i][e] = p1 * r2.x - p0 * r2.y;
          if (normed) {
            q0 += xa[e] * xa[e] + xb[e] * xb[e];
            q1 += (ua[t][i][e] * wa[e]) * xa[e] + (ub[t][i][e] * wb[e]) * xb[e];
          }
        }
        s[2 * t] += q0;
        s[2 * t + 1] += q1;
        hs[t][i][0] = q0;
        hs[t][i][1] = q1;
      }
    if (token) block_sum(s, sums, sh, nwarps);
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int h = head0 + i * hstep;
        const bool in = own && h < a.heads[t];
        if (normed) {      // absent heads hold zeros, and stay out of dw whatever eps makes of them
          float q0 = s[2 * t], q1 = s[2 * t + 1];
          float inv = 1.f / (float)(token ? a.heads[t] * d : d);
          if (!token) {
            q0 = lanes_sum(hs[t][i][0], lanes);
            q1 = lanes_sum(hs[t][i][1], lanes);
          }
          const float rs = rsqrtf(q0 * inv + a.eps);
          const float k = rs * rs * q1 * inv;
          float xa[8], xb[8], wa[8], wb[8];
          x[t][i].get(xa, xb, half);
          load_weight<VEC>(wa, wb, a.weight[t], a.weight_bf16, token ? h * d : 0, in, j, lanes, half, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (in) {
              dw[t][i][0][e] += ua[t][i][e] * (xa[e] * rs);
              dw[t][i][1][e] += ub[t][i][e] * (xb[e] * rs);
            }
            ua[t][i][e] = rs * (ua[t][i][e] * wa[e] - xa[e] * k);
            ub[t][i][e] = rs * (ub[t][i][e] * wb[e] - xb[e] * k);
          }
        }
        if (in)
          store_share<VEC>(static_cast<T*>(a.out[t]) + r * a.out_stride[t] + (long long)h * d, ua[t][i], ub[t][i], j,
                           lanes, half, d);
      }
    buf ^= 1;
  }
  if (!normed || !a.part) return;
  // this block's weight sums: [heads * d] of Q then of K, or (per-head norm)
  // [d] of each, its heads added in head order
  float* part = a.part + (long long)blockIdx.x * (token ? (a.heads[0] + a.heads[1]) * d : 2 * d);
  if (token) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        const int h = head0 + i * hstep;
        if (own && h < a.heads[t]) {
          float* o = part + (t ? a.heads[0] * d : 0) + h * d;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int p = pair_of<VEC>(j, e, lanes);
            if (p < (d >> 1)) {
              o[first_of(p, half)] = dw[t][i][0][e];
              o[second_of(p, half, d)] = dw[t][i][1][e];
            }
          }
        }
      }
    return;
  }
  __shared__ float heads_part[32][256];
  for (int t = 0; t < 2; ++t) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < UPT; ++i) v += dw[t][i][k][e];
        // the heads of one warp, then the warps through shared memory
        for (int o = lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int p = pair_of<VEC>(j, e, lanes);
        if ((int)(threadIdx.x & 31) < lanes && p < (d >> 1))
          heads_part[threadIdx.x >> 5][k ? second_of(p, half, d) : first_of(p, half)] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      float v = 0.f;
      for (int w = 0; w < nwarps; ++w) v += heads_part[w][i];
      part[t * d + i] = v;
    }
    __syncthreads();
  }
}

// Adds the blocks' weight sums in a fixed order, in float64.
__global__ void __launch_bounds__(1024) qk_reduce_kernel(const float* part, int blocks, int wq, int wk, float* dq,
                                                         float* dk) {
  __shared__ double sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = wq + wk;
  const int col = blockIdx.x * 32 + lane;
  double s = 0.0;
  if (col < width)
    for (int b = warp; b < blocks; b += 32) s += (double)part[(long long)b * width + col];
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < width) {
    for (int v = 1; v < 32; ++v) s += sh[v][lane];
    float* o = col < wq ? dq : dk;
    if (o) o[col < wq ? col : col - wq] = (float)s;
  }
}

// ----------------------------------------------------------------- launch --
int most_heads(const QkArgs& a) { return a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1]; }

// A thread takes one head's share of a token, or two where a block of 512
// threads would not cover the heads.
int units_per_thread(const QkArgs& a) { return most_heads(a) * a.lanes <= 512 ? 1 : 2; }
int block_threads(const QkArgs& a) {
  const int upt = units_per_thread(a);
  const int t = (most_heads(a) * a.lanes + upt - 1) / upt;
  return (t + 31) / 32 * 32;
}

int bwd_grid(const QkArgs& a) {
  const int t = block_threads(a);
  const long long resident = (long long)num_sms() * (t > 512 ? 1 : (t > 256 ? 2 : (t > 128 ? 4 : 8)));
  return (int)(a.rows < resident ? a.rows : resident);
}

template <typename T, bool VEC>
cudaError_t run_fwd(const QkArgs& a, cudaStream_t s) {
  const int upt = units_per_thread(a), threads = block_threads(a);
  const long long tiles = (a.rows + kTok - 1) / kTok;
  const long long resident = (long long)num_sms() * (threads > 512 ? 1 : (1024 / threads > 16 ? 16 : 1024 / threads));
  const int grid = (int)(tiles < resident ? tiles : resident);
  const size_t smem = 2 * kTok * (a.d / 2) * sizeof(float2);
  if (upt == 1) qk_fwd_kernel<T, VEC, 1><<<grid, threads, smem, s>>>(a);
  else qk_fwd_kernel<T, VEC, 2><<<grid, threads, smem, s>>>(a);
  return cudaGetLastError();
}

template <typename T, bool VEC>
cudaError_t run_bwd(const QkArgs& a, cudaStream_t s) {
  const int upt = units_per_thread(a), threads = block_threads(a);
  const size_t smem = 2 * (a.d / 2) * sizeof(float2);
  const int grid = bwd_grid(a);
  if (upt == 1) qk_bwd_kernel<T, VEC, 1><<<grid, threads, smem, s>>>(a);
  else qk_bwd_kernel<T, VEC, 2><<<grid, threads, smem, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.part) return e;
  const bool token = a.norm == SPADE_QK_NORM_TOKEN;
  const int wq = token ? a.heads[0] * a.d : a.d, wk = token ? a.heads[1] * a.d : a.d;
  qk_reduce_kernel<<<(wq + wk + 31) / 32, 1024, 0, s>>>(a.part, grid, wq, wk, a.dweight[0], a.dweight[1]);
  return cudaGetLastError();
}

}  // namespace

size_t qk_bwd_floats(const QkArgs& a) {
  if (a.norm == SPADE_QK_NORM_NONE) return 0;
  return (size_t)bwd_grid(a) * (a.norm == SPADE_QK_NORM_TOKEN ? (a.heads[0] + a.heads[1]) * a.d : 2 * a.d);
}

cudaError_t launch_qk_fwd(const QkArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) return a.vec ? run_fwd<__nv_bfloat16, true>(a, s) : run_fwd<__nv_bfloat16, false>(a, s);
  return a.vec ? run_fwd<float, true>(a, s) : run_fwd<float, false>(a, s);
}

cudaError_t launch_qk_bwd(const QkArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) return a.vec ? run_bwd<__nv_bfloat16, true>(a, s) : run_bwd<__nv_bfloat16, false>(a, s);
  return a.vec ? run_bwd<float, true>(a, s) : run_bwd<float, false>(a, s);
}

}  // namespace spade
