// Gradients of the row passes (spade_norm_modulate_bwd,
// spade_gate_residual_bwd, spade_gate_residual_norm_bwd).  With A_g = sum of
// dh and B_g = sum of dh * xhat over the rows of group g, C_g = sum of
// dx' * yhat:
//   dshift = A, dscale = w B + b A, dw = sum_g (1 + scale_g) B_g,
//   db = sum_g (1 + scale_g) A_g, dgate = r pw C, dpw = r sum_g gate_g C_g,
// so three column sums serve every parameter, and
//   u = dh (1 + scale) w,  dx = dx' + rstd (u - mean(u) - xhat mean(u xhat))
// (the mean(u) term for the layer norm only), dy likewise through P.
//
// A block works on units, runs of rows of one modulation group: the column
// sums stay in registers until the unit ends, then go to the workspace, and a
// second small launch adds them in a fixed order, in float64: no atomics, the
// same result on every run.  Rows are walked K at a time, read again from the
// ring where a later step needs them, which costs fewer registers than keeping
// them.
//
// The sums of a unit, and of a block's units where it has several of one
// launch, run in float32, over some 2 rows / SMs additions at most; from there
// on in float64.
//
// With x' and h bound by memory: 75600 rows of 5120 (bfloat16) take 760 to 863 us
// on different cards, 5.4 to 6.1 TB/s of the 6.55 that a copy reaches (steps on
// one card: 2571 with one row to a block, 1680 with the ring, 1010 paired, 880
// with the moments merged without divisions, 819 without a spill).  h alone moves
// fewer bytes for the same statistics and waits: for shared memory, which dh is
// read from twice, and at barriers, with a quarter of an SM's warps at work and
// 56 % of the issue slots used.  32760 rows of 1536 in 21 groups, float32 stream,
// 106 to 109 us, 4.7 TB/s; bfloat16 stream 102 us, 3.0 TB/s; 75600 rows of 5120,
// bfloat16, 578 us, 4.0 TB/s.  Copying whole rows in bulk, one thread for all,
// was slower (930 us: its state takes registers or calls), and so were chunks
// that take turns (800).
//
// Rows above 8192 columns, and narrow pieces above 5120, spill 0.2 to 1.1 KB with
// a norm: 723 us for x' and h of 8192 x 16384, three times their bytes (16384 x
// 8192: 295 us, 1.2 times).  32760 rows of 1540 bfloat16 (h alone) in pieces of
// two 145 us, of 1537 in single elements 244, where 1536 take 46 of bytes.
#pragma once
#include "row_pass.cuh"

namespace spade {
namespace {

using namespace rowpass;

// A unit is chunk c of group g: rows [g R + R c / C, g R + R (c + 1) / C) of a
// group of R rows cut into C chunks.
struct Run {
  long long group, first;
  int rows;

  __device__ __forceinline__ Run(const RowArgs& a, long long u) {
    if (a.chunks == 1) {
      group = u;
      first = u * a.rows_per_group;
      rows = (int)a.rows_per_group;
    } else {
      const long long c = u % a.chunks;
      group = u / a.chunks;
      const long long from = a.rows_per_group * c / a.chunks, to = a.rows_per_group * (c + 1) / a.chunks;
      first = group * a.rows_per_group + from;
      rows = (int)(to - from);
    }
  }
};

// With C > 1 a unit's sums A, B, C go to `part` [unit][3][dim] and
// row_reduce_kernel makes every parameter gradient of them.  With C = 1 a unit
// is a whole group: its modulation gradients are final and written here, and
// the weights' sums are added up over the block's units in `part`
// [block][3][dim].
// POST: the branch has a norm (0 no, 1 yes, 2 as the call says).
template <typename XT, typename BT, class L, int K, bool RES, bool NORM, int POST>
__global__ void __launch_bounds__(L::NV == 1 ? 640 : 512, 1)
    row_bwd_kernel(const __grid_constant__ RowArgs a, int depth, bool weights) {
  constexpr int NV = L::NV;
  constexpr bool RING = L::RING;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Shared<2 * K> sh;
  const int dim = a.dim, nwarps = blockDim.x >> 5;
  const bool post = RES && (POST == 2 ? a.post_norm != kNone : POST == 1), grad = a.dx_out != nullptr;
  const uint32_t xb = slot_bytes(blockDim.x, NV, sizeof(XT)), bb = slot_bytes(blockDim.x, NV, sizeof(BT));
  Stream<XT, L> sg, sx;
  Stream<BT, L> sy, sd;
  sg.at = 0;
  sy.at = xb;
  sx.at = xb + (RES ? bb : 0);
  sd.at = sx.at + xb;
  const uint32_t slot = NORM ? sd.at + bb : sx.at, ring_bytes = depth * slot;
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const long long units = a.groups * a.chunks;
  auto seek = [&](long long r) {
    sg.seek(a.dx_out, a.dx_out_stride, r);
    if (RES) sy.seek(a.y, a.y_stride, r);
    if (NORM) {
      sx.seek(a.x, a.x_stride, r);
      sd.seek(a.dh, a.dh_stride, r);
    }
  };
  auto advance = [&](int n) {
    sg.p += n * a.dx_out_stride;
    if (RES) sy.p += n * a.y_stride;
    if (NORM) {
      sx.p += n * a.x_stride;
      sd.p += n * a.dh_stride;
    }
  };

  long long fu = blockIdx.x;     // the unit of the next row to copy, and its rows to copy
  int to_copy = 0;
  uint32_t fs = 0, us = 0;       // slot of the next row to copy, of the next to use
  if (RING && fu < units) {
    const Run f(a, fu);
    seek(f.first);
    to_copy = f.rows;
  }
  auto fetch = [&]() {
    if (to_copy > 0) {
      const uint32_t to = ring_at + fs;
      if (grad) sg.fetch(to, dim);
      if (RES) sy.fetch(to, dim);
      if (NORM) {
        sx.fetch(to, dim);
        sd.fetch(to, dim);
      }
      advance(1);
      if (--to_copy == 0) {
        fu += gridDim.x;
        if (fu < units) {
          const Run f(a, fu);
          seek(f.first);
          to_copy = f.rows;
        }
      }
    }
    commit_async();
    fs = fs + slot == ring_bytes ? 0 : fs + slot;
  };
  if (RING) {
    for (int d = 0; d < depth; ++d) {
      unsigned char* p = ring + d * slot;
      if (grad) sg.clear(p, dim);
      if (RES) sy.clear(p, dim);
      if (NORM) {
        sx.clear(p, dim);
        sd.clear(p, dim);
      }
      fetch();
    }
  }
  count_columns<L>(sh, dim);
  int half = 0;
  bool first = true;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const Run run(a, u);
    const long long g = run.group;
    if (!RING) seek(run.first);
    XT* dxo = NORM ? static_cast<XT*>(a.dx) + run.first * a.dx_stride : nullptr;
    BT* dyo = RES ? static_cast<BT*>(a.dy) + run.first * a.dy_stride : nullptr;
    Eight gate[NV], times[NV];     // r gate pw, and (1 + s) w
    Eight A[NV], B[NV], C[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Eight t;
      if (RES) {
        load_param<L>(gate[i], a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
        load_param<L>(t, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          gate[i].p[q] = present<L>(mul(gate[i].p[q], mul(both(a.residual_scale), t.p[q])), i, q, dim);
      }
      if (NORM) {
        load_param<L>(times[i], a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
        load_param<L>(t, a.weight, 0, a.param_bf16, 1.f, i, dim);
#pragma unroll
        for (int q = 0; q < 4; ++q) times[i].p[q] = mul(add(both(1.f), times[i].p[q]), t.p[q]);
      }
      A[i].fill(0.f);
      B[i].fill(0.f);
      C[i].fill(0.f);
    }
    for (int left = run.rows; left > 0;) {
      // K rows at once; where fewer are left, the first stands in for the others,
      // which are neither added up nor written
      const int n = left < K ? left : K;
      auto at_row = [&](int k) { return k < n ? k : 0; };
      if (RING) wait_async_upto(depth - K);
      const unsigned char* at[K];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const uint32_t s = us + at_row(k) * slot;
        at[k] = ring + (s >= ring_bytes ? s - ring_bytes : s);
      }
      Eight v[K][NV];                  // x', then the gradient that reaches P (0 past the row's end)
      float ym[K], ys[K];
      auto get_yhat = [&](Eight& y, int k, int i) {
        sy.get(y, at[k], at_row(k) * a.y_stride, i, dim);
        if (post) {
#pragma unroll
          for (int q = 0; q < 4; ++q) y.p[q] = mul(add(y.p[q], both(-ym[k])), both(ys[k]));
        }
      };
      if (post) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) sy.get(v[k][i], at[k], at_row(k) * a.y_stride, i, dim);
        row_stats<L, K>(v, a.post_norm, a.post_eps, a.inv_dim, dim, sh, half, nwarps, ym, ys);
      }
      float xm[K], xs[K], m0[K], m1[K];
      if (NORM) {
        Eight w[K][NV];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            sx.get(v[k][i], at[k], at_row(k) * a.x_stride, i, dim);
            if (RES) {
              Eight y;
              get_yhat(y, k, i);
#pragma unroll
              for (int q = 0; q < 4; ++q) v[k][i].p[q] = fma(gate[i].p[q], y.p[q], v[k][i].p[q]);
            }
            sd.get(w[k][i], at[k], at_row(k) * a.dh_stride, i, dim);
#pragma unroll
            for (int q = 0; q < 4; ++q) w[k][i].p[q] = mul(w[k][i].p[q], times[i].p[q]);
          }
        row_stats_bwd<L, K>(v, w, a.norm, a.eps, a.inv_dim, dim, sh, half, nwarps, xm, xs, m0, m1);
      }
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (k >= n) break;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          Eight gr;
          if (grad) sg.get(gr, at[k], at_row(k) * a.dx_out_stride, i, dim);
          else gr.fill(0.f);
          if (NORM) {
            Eight dh;
            sd.get(dh, at[k], at_row(k) * a.dh_stride, i, dim);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float2 xh = mul(add(v[k][i].p[q], both(-xm[k])), both(xs[k]));
              A[i].p[q] = add(A[i].p[q], dh.p[q]);
              B[i].p[q] = fma(dh.p[q], xh, B[i].p[q]);
              const float2 u = fma(dh.p[q], times[i].p[q], both(-m0[k]));
              gr.p[q] = fma(both(xs[k]), fma(xh, both(-m1[k]), u), gr.p[q]);
            }
            store8<L>(dxo + k * a.dx_stride, gr, i, dim);
          }
          if (RES) {
            Eight y;
            get_yhat(y, k, i);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              C[i].p[q] = fma(gr.p[q], y.p[q], C[i].p[q]);
              v[k][i].p[q] = mul(gr.p[q], gate[i].p[q]);
            }
            if (!post) store8<L>(dyo + k * a.dy_stride, v[k][i], i, dim);
          }
        }
      }
      if (post) {
        float t[2 * K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          float2 t0 = both(0.f), t1 = both(0.f);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            Eight y;
            get_yhat(y, k, i);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              t0 = add(t0, v[k][i].p[q]);
              t1 = fma(v[k][i].p[q], y.p[q], t1);
            }
          }
          t[k] = sum_of(t0);
          t[K + k] = sum_of(t1);
        }
        block_sum(t, sh.sums, half, nwarps);
#pragma unroll
        for (int k = 0; k < K; ++k) {
          if (k >= n) break;
          const float p0 = a.post_norm == kLayer ? t[k] * a.inv_dim : 0.f, p1 = t[K + k] * a.inv_dim;
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            Eight y;
            get_yhat(y, k, i);
#pragma unroll
            for (int q = 0; q < 4; ++q)
              y.p[q] = mul(both(ys[k]), fma(y.p[q], both(-p1), add(v[k][i].p[q], both(-p0))));
            store8<L>(dyo + k * a.dy_stride, y, i, dim);
          }
        }
      }
      if (RING) {
        #pragma unroll
        for (int k = 0; k < K; ++k)
          if (k < n) fetch();
        us = us + n * slot >= ring_bytes ? us + n * slot - ring_bytes : us + n * slot;
      } else {
        advance(n);
      }
      if (NORM) dxo += n * a.dx_stride;
      if (RES) dyo += n * a.dy_stride;
      left -= n;
    }
    if (a.chunks > 1) {
      if (!a.part) continue;     // no gradient of a parameter is wanted
      float* p = a.part + u * 3 * dim;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (NORM) {
          store8<L>(p, A[i], i, dim);
          store8<L>(p + dim, B[i], i, dim);
        }
        if (RES) store8<L>(p + 2 * (long long)dim, C[i], i, dim);
      }
      continue;
    }
    float* p = a.part + (long long)blockIdx.x * 3 * dim;
    auto add_up = [&](float* to, const Eight& t, int i) {       // columns of this thread alone
      Eight s;
      if (first) s.fill(0.f);
      else load8<L>(s, to, i, dim);
#pragma unroll
      for (int q = 0; q < 4; ++q) s.p[q] = add(s.p[q], t.p[q]);
      store8<L>(to, s, i, dim);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Eight t, w, b;
      if (NORM) {
        load_param<L>(w, a.weight, 0, a.param_bf16, 1.f, i, dim);
        load_param<L>(b, a.bias, 0, a.param_bf16, 0.f, i, dim);
        if (a.dshift) store8<L>(a.dshift + g * dim, A[i], i, dim);
        if (a.dscale) {
#pragma unroll
          for (int q = 0; q < 4; ++q) t.p[q] = fma(w.p[q], B[i].p[q], mul(b.p[q], A[i].p[q]));
          store8<L>(a.dscale + g * dim, t, i, dim);
        }
        if (weights) {
          load_param<L>(b, a.scale, g * a.scale_stride, a.param_bf16, 0.f, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q) t.p[q] = mul(add(both(1.f), b.p[q]), A[i].p[q]);
          add_up(p, t, i);
#pragma unroll
          for (int q = 0; q < 4; ++q) t.p[q] = mul(add(both(1.f), b.p[q]), B[i].p[q]);
          add_up(p + dim, t, i);
        }
      }
      if (RES) {
        load_param<L>(w, a.post_weight, 0, a.param_bf16, 1.f, i, dim);
        if (a.dgate) {
#pragma unroll
          for (int q = 0; q < 4; ++q) t.p[q] = mul(mul(both(a.residual_scale), w.p[q]), C[i].p[q]);
          store8<L>(a.dgate + g * dim, t, i, dim);
        }
        if (weights) {
          load_param<L>(b, a.gate, g * a.gate_stride, a.param_bf16, 1.f, i, dim);
#pragma unroll
          for (int q = 0; q < 4; ++q) t.p[q] = mul(mul(both(a.residual_scale), b.p[q]), C[i].p[q]);
          add_up(p + 2 * (long long)dim, t, i);
        }
      }
    }
    first = false;
  }
  if (RING) wait_async<0>();
}

// ----------------------------------------------------------------- launch --
template <typename XT, typename BT, class L, bool RES, bool NORM, int POST>
cudaError_t run(const RowArgs& a, int grid, bool weights, cudaStream_t s) {
  constexpr int K = L::NV == 1 && POST != 1 ? 2 : 1;
  const int threads = row_threads(a.dim, L::NV);
  const size_t slot = slot_bytes(threads, L::NV, sizeof(XT)) * (NORM ? 2 : 1) +
                      slot_bytes(threads, L::NV, sizeof(BT)) * ((RES ? 1 : 0) + (NORM ? 1 : 0));
  int depth = 0;
  size_t smem = 0;
  if (L::RING) {
    const size_t room = kSmemSm / bwd_blocks(a.dim) - 1024 - sizeof(Shared<2 * K>);
    const long long rows = (a.rows + grid - 1) / grid;
    depth = (int)(room / slot < kDepthMax ? room / slot : kDepthMax);
    if (rows < depth) depth = (int)(rows > K ? rows : K);
    if (depth < K) return cudaErrorInvalidConfiguration;
    smem = depth * slot;
  }
  const auto kernel = row_bwd_kernel<XT, BT, L, K, RES, NORM, POST>;
  if (smem > 32 * 1024) {        // one value for all launches: callers on other threads may be between theirs and this
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSmemSm - 1024 - (int)sizeof(Shared<2 * K>));
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, threads, smem, s>>>(a, depth, weights);
  return cudaGetLastError();
}

template <typename XT, typename BT, class L>
cudaError_t by_op(const RowArgs& a, int grid, bool weights, cudaStream_t s) {
  if (a.dy && a.dh)
    return a.post_norm == kNone ? run<XT, BT, L, true, true, 0>(a, grid, weights, s)
                                : run<XT, BT, L, true, true, 1>(a, grid, weights, s);
  if (a.dy) return run<XT, BT, L, true, false, 2>(a, grid, weights, s);
  return run<XT, BT, L, false, true, 0>(a, grid, weights, s);
}

// The widest pieces have kernels for every length; rows above 8192 elements,
// and rows above 5120 in narrower pieces, are read where they are used.
template <typename XT, typename BT>
cudaError_t by_width(const RowArgs& a, int grid, bool weights, cudaStream_t s) {
  constexpr int P = sizeof(XT) == 2 ? 8 : 4;
  const int p = piece_of(a);
  const bool wide = p == P;
  if (a.dim <= 5120) {
    const bool full = a.dim % 256 == 0;
    if (wide) return full ? by_op<XT, BT, Layout<P, true, true, 1>>(a, grid, weights, s) : by_op<XT, BT, Layout<P, false, true, 1>>(a, grid, weights, s);
    if constexpr (sizeof(XT) == 2) {
      if (p > 1) return by_op<XT, BT, Layout<2, false, true, 1>>(a, grid, weights, s);
    }
    return by_op<XT, BT, Layout<1, false, sizeof(BT) == 4, 1>>(a, grid, weights, s);
  }
  if (a.dim <= 8192 && wide)
    return a.dim % 512 == 0 ? by_op<XT, BT, Layout<P, true, true, 2>>(a, grid, weights, s) : by_op<XT, BT, Layout<P, false, true, 2>>(a, grid, weights, s);
  return wide ? by_op<XT, BT, Layout<P, false, false, 4>>(a, grid, weights, s) : by_op<XT, BT, Layout<1, false, false, 4>>(a, grid, weights, s);
}

}  // namespace

template <typename XT, typename BT>
cudaError_t row_bwd(const RowArgs& a, int grid, bool weights, cudaStream_t s) {
  return by_width<XT, BT>(a, grid, weights, s);
}

}  // namespace spade
