// Norm and several-axis rotation of Q and K, one pass over both
// (spade_qk_norm_rope, spade_qk_norm_rope_bwd).
//
// Pair i of a head rotates by pos[axis_i] * freq_i.  The angle is formed in
// turns, position times turns-per-unit in float64, its nearest integer is
// taken off there and the rest (at most half a turn, rounded once to float32)
// goes to sincospif: positions anywhere in int32 keep an angle good to
// float32.  A token's angles are computed once, ahead of its data, and serve
// every head of Q and of K.
//
// Forward:  n = x * rstd * w (rms over the token's heads * d values, over
//           each head's d, or no norm), out = rotation of n.
// Backward: u = dout rotated back, dw = sum of u * x * rstd over the rows (and
//           heads, for the per-head norm), dx = rstd (w u - x rstd^2 mean(w u x)).
//
// `lanes` threads (d / 16 rounded up to a power of two) share a head, sixteen
// channels each: a unit.  The units of Q and K are numbered through; a thread
// has UPT of them, the same of every token, and the same eight pairs in each,
// so weights and the sums of their gradient stay in its registers and a
// token's sines and cosines are read once for all its units.  Channels are
// owned in pieces of P that alternate between the lanes, so that a warp's
// access is contiguous.  Tokens are copied ahead into a ring in shared memory,
// by the thread that uses them (no barrier); a block takes K tokens at a time,
// whose sums share one barrier.
//
// Forward, bound by memory: 506 to 547 us on different cards for 75600 tokens
// of 2 x 40 heads of 128 channels (bfloat16, norm over the token), 5.7 to 6.1
// TB/s of the 6.55 that a copy reaches, at 14 instructions an element and 61 %
// of the issue slots; float32 967 us, 6.4 TB/s.  Steps, on one card: 1314 us
// with loads where they are needed, the ring (709), paired float32 arithmetic
// (586), no checks where heads and threads divide evenly and no divisions (520),
// angles of four tokens at once (509).
//
// Backward, bound by waits: 139 to 143 us for 32760 tokens of 2 x 12 heads
// (bfloat16), 4.3 TB/s, with a quarter of an SM's warps at work, one token to a
// barrier and 56 % of the issue slots used (150 us before warps of one tensor
// summed for it alone and addresses took one multiply-add).  With two units a
// thread (513 to 1024 units) a token is read from the ring and turned twice:
// 1237 us for 75600 tokens of 2 x 40 heads, 3.8 TB/s.
//
// Registers are capped by what the blocks of an SM leave a thread.  The kernels
// of 16-byte pieces with one or two units spill nothing or up to 16 bytes; with
// narrower pieces 0 to 232 bytes.  Those of four units have 64 registers, spill
// 0.9 to 2.2 KB and read every token twice, when it is needed: 2567 us forward
// and 3657 backward for 32760 tokens of 2 x 40 heads of 160 channels, ten times
// their bytes.  Narrow pieces cost as their accesses do (32760 tokens
// of 2 x 12 heads, forward): 145 us in pieces of two, 301 in single elements.
// Few heads leave threads of a warp without a unit: 114 us for 75600 tokens of
// 2 x 2 heads, five times their bytes.
#include <algorithm>

#include "row_io.cuh"
#include "spade_internal.cuh"

namespace spade {
namespace {

using namespace rowio;

constexpr int kDepthMax = 14;
constexpr int kAhead = 4;        // tokens whose angles are made at once, spread over the block

// FULL: heads of 16 * lanes channels, and a unit for every thread and place.
template <int P_, bool HALF_, bool FULL_, bool RING_, int UPT_>
struct Layout {
  static constexpr int P = P_, UPT = UPT_;
  static constexpr bool HALF = HALF_, FULL = FULL_, RING = RING_;
};

// Channel of a thread's element e (0..15).  Interleaved: pairs (2m, 2m + 1)
// are neighbours in a piece (P = 1: two single accesses).  Halves: elements
// m and m + 8 are half a head apart.
template <class L>
__device__ __forceinline__ int channel(int j, int lanes, int e, int d) {
  constexpr int O = !L::HALF && L::P == 1 ? 2 : L::P;
  constexpr bool HALF = L::HALF;
  if (HALF) return ((e & 7) / O * lanes + j) * O + (e & 7) % O + (e >= 8 ? d >> 1 : 0);
  return (e / O * lanes + j) * O + e % O;
}
template <class L>
__device__ __forceinline__ bool owned(int j, int lanes, int e, int d) {
  if (L::FULL) return true;
  return L::HALF ? channel<L>(j, lanes, e & 7, d) < (d >> 1) : channel<L>(j, lanes, e, d) < d;
}
// Where the cosine of pair p lies, its sine two floats on: as entry m of lane
// j, two entries to a 16-byte word (cos, cos, sin, sin), so that a thread reads
// its eight as four words, without bank conflicts, ready for paired arithmetic.
template <class L>
__device__ __forceinline__ int angle_slot(int p, int lanes) {
  constexpr int O = !L::HALF && L::P == 1 ? 2 : L::P;
  constexpr bool HALF = L::HALF;
  const int c = HALF ? p : 2 * p, piece = c / O;
  const int e = piece / lanes * O + c % O, j = piece & (lanes - 1), m = HALF ? e : e >> 1;
  return ((m >> 1) * lanes + j) * 4 + (m & 1);
}

// A thread's unit: its sixteen elements in global memory and in the ring, and
// as eight rotated pairs (a, b), two and two together.
struct Unit {
  float2 a[4], b[4];
};
template <class L>
__device__ __forceinline__ void pairs_of(Unit& u, const float (&v)[16]) {
  constexpr bool HALF = L::HALF;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    u.a[q] = HALF ? make_float2(v[2 * q], v[2 * q + 1]) : make_float2(v[4 * q], v[4 * q + 2]);
    u.b[q] = HALF ? make_float2(v[2 * q + 8], v[2 * q + 9]) : make_float2(v[4 * q + 1], v[4 * q + 3]);
  }
}
template <class L>
__device__ __forceinline__ void elements_of(float (&v)[16], const Unit& u) {
  constexpr bool HALF = L::HALF;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    v[HALF ? 2 * q : 4 * q] = u.a[q].x;
    v[HALF ? 2 * q + 1 : 4 * q + 2] = u.a[q].y;
    v[HALF ? 2 * q + 8 : 4 * q + 1] = u.b[q].x;
    v[HALF ? 2 * q + 9 : 4 * q + 3] = u.b[q].y;
  }
}
template <typename T, class L>
__device__ __forceinline__ void load16(Unit& u, const T* head, bool in, int j, int lanes, int d) {
  constexpr int P = L::P;
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; e += P) {
    if (in && owned<L>(j, lanes, e, d)) {
      load_piece<T, P>(v + e, head + channel<L>(j, lanes, e, d));
    } else {
#pragma unroll
      for (int q = 0; q < P; ++q) v[e + q] = 0.f;
    }
  }
  pairs_of<L>(u, v);
}
template <typename T, class L>
__device__ __forceinline__ void store16(T* head, const Unit& u, int j, int lanes, int d) {
  constexpr int P = L::P;
  float v[16];
  elements_of<L>(v, u);
#pragma unroll
  for (int e = 0; e < 16; e += P)
    if (owned<L>(j, lanes, e, d)) store_piece<P>(head + channel<L>(j, lanes, e, d), v + e);
}
// The ring keeps a unit's pieces [16 / P][threads][P].
template <typename T, class L>
__device__ __forceinline__ void fetch16(uint32_t to, const T* head, int j, int lanes, int d) {
  constexpr int P = L::P;
#pragma unroll
  for (int e = 0; e < 16; e += P)
    if (owned<L>(j, lanes, e, d))
      copy_async<P * (int)sizeof(T)>(to + (e / P * blockDim.x + threadIdx.x) * P * (int)sizeof(T),
                                     head + channel<L>(j, lanes, e, d));
}
template <typename T, class L>
__device__ __forceinline__ void ring16(Unit& u, const unsigned char* at) {
  constexpr int P = L::P;
  const T* p = reinterpret_cast<const T*>(at);
  float v[16];
#pragma unroll
  for (int e = 0; e < 16; e += P) load_piece<T, P>(v + e, p + (e / P * blockDim.x + threadIdx.x) * P);
  pairs_of<L>(u, v);
}
// What is not copied reads as zero.
template <typename T, class L>
__device__ __forceinline__ void clear16(unsigned char* at, bool in, int j, int lanes, int d) {
  constexpr int P = L::P;
#pragma unroll
  for (int e = 0; e < 16; ++e)
    if (!in || !owned<L>(j, lanes, e, d))
      reinterpret_cast<T*>(at)[(e / P * blockDim.x + threadIdx.x) * P + e % P] = T(0.f);
}

struct Turns {
  double turn[SPADE_ROPE_MAX_PAIRS];
  int axis[SPADE_ROPE_MAX_PAIRS];
};

// n / divisor for n below 2^31 (Granlund and Montgomery, 1994).
__device__ __forceinline__ unsigned divide(unsigned n, const QkArgs::Divisor& by) {
  return (unsigned)(((unsigned long long)n * by.mul) >> by.shift);
}

// Cosine and sine of every pair of the block's next kAhead tokens.
template <class L>
__device__ __forceinline__ void angles(const QkArgs& a, const Turns& tu, long long r0, long long r1, float* cs) {
  const int half_d = a.d >> 1;
  for (int i = threadIdx.x; i < kAhead * half_d; i += blockDim.x) {
    int k = 0, p = i;
#pragma unroll
    for (int m = 1; m < kAhead; ++m)
      if (p >= half_d) {
        p -= half_d;
        ++k;
      }
    const long long r = r0 + k;
    float c = 1.f, s = 0.f;
    if (p < a.pairs && r < a.video_rows && r < r1) {
      const int axis = tu.axis[p];
      int pos;
      if (a.positions) {
        pos = a.positions[r * 3 + axis];
      } else {
        const unsigned tok = (unsigned)a.tok0 + (unsigned)r, row = divide(tok, a.W), t = divide(row, a.H);
        pos = axis == 2 ? tok - row * a.W.by : (axis == 1 ? row - t * a.H.by : t);
      }
      const double t = (double)pos * tu.turn[p];
      sincospif(2.f * (float)(t - rint(t)), &s, &c);
    }
    float* o = cs + k * 16 * a.lanes + angle_slot<L>(p, a.lanes);
    o[0] = c;
    o[2] = s;
  }
}
struct Angles {
  float2 c[4], s[4];
};
__device__ __forceinline__ void get_angles(Angles& t, const float* cs, int j, int lanes) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 f = *reinterpret_cast<const float4*>(cs + (q * lanes + j) * 4);
    t.c[q] = make_float2(f.x, f.y);
    t.s[q] = make_float2(f.z, f.w);
  }
}
// (a, b) -> (a c - b s, a s + b c), or back.
__device__ __forceinline__ void turn(Unit& u, const Angles& t, bool back) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 minus = make_float2(-t.s[q].x, -t.s[q].y), a = u.a[q], b = u.b[q];
    u.a[q] = fma(b, back ? t.s[q] : minus, mul(a, t.c[q]));
    u.b[q] = fma(a, back ? minus : t.s[q], mul(b, t.c[q]));
  }
}

// What forward and backward share: the units of this thread and its ring.
template <typename T, class L>
struct Units {
  static constexpr int UPT = L::UPT;
  int j, lanes, d;
  int head[UPT];
  float inv[UPT];                // 1 / the values that a norm of the unit runs over
  bool k_side[UPT], in[UPT];
  uint32_t slot;

  __device__ __forceinline__ Units(const QkArgs& a, int ops) {
    lanes = a.lanes;
    d = a.d;
    j = threadIdx.x & (lanes - 1);
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      const int h = ((int)threadIdx.x + i * (int)blockDim.x) / lanes;
      k_side[i] = h >= a.heads[0];
      head[i] = h - (k_side[i] ? a.heads[0] : 0);
      inv[i] = a.inv_count[k_side[i]];
      in[i] = L::FULL || h < a.heads[0] + a.heads[1];
    }
    slot = (uint32_t)(ops * UPT * 16 * sizeof(T)) * blockDim.x;
  }
  // Unit i's head of row r, and the way to its next row.
  template <typename V>
  __device__ __forceinline__ V* at(V* const (&base)[2], const long long (&stride)[2], long long r, int i) const {
    return (k_side[i] ? base[1] + r * stride[1] : base[0] + r * stride[0]) + head[i] * d;
  }
  __device__ __forceinline__ long long step(const long long (&stride)[2], int i) const {
    return k_side[i] ? stride[1] : stride[0];
  }
  __device__ __forceinline__ uint32_t place(int op, int i) const {
    return (uint32_t)((op * UPT + i) * 16 * sizeof(T)) * blockDim.x;
  }
  __device__ __forceinline__ void clear(unsigned char* ring, int depth, int ops) const {
    for (int s = 0; s < depth; ++s)
      for (int o = 0; o < ops; ++o)
#pragma unroll
        for (int i = 0; i < UPT; ++i) clear16<T, L>(ring + s * slot + place(o, i), in[i], j, lanes, d);
  }
  __device__ __forceinline__ void weights(Unit& w, const QkArgs& a, int i) const {
    const void* p = a.weight[k_side[i]];
    const int off = a.norm == SPADE_QK_NORM_TOKEN ? head[i] * d : 0;
    if (!p || !in[i]) {
#pragma unroll
      for (int q = 0; q < 4; ++q) w.a[q] = w.b[q] = both(1.f);
    } else if (a.weight_bf16) {
      load16<bf16, L>(w, static_cast<const bf16*>(p) + off, true, j, lanes, d);
    } else {
      load16<float, L>(w, static_cast<const float*>(p) + off, true, j, lanes, d);
    }
  }
};

// Two sums over the units of this thread's tensor, where every warp's units are
// of one tensor: the warps from `first` to `last`.
template <int M>
__device__ __forceinline__ void side_sum(float (&v)[2], Scratch<M>& sh, int& half, int first, int last) {
  const int lane = threadIdx.x & 31, sub = lane & 15;
  float s = warp_sum_spread<2>(v);
  float* b = reinterpret_cast<float*>(sh.v[half]) + (lane >> 4) * 33;
  if (sub == 0) b[threadIdx.x >> 5] = s;
  __syncthreads();
  s = first + sub < last ? b[first + sub] : 0.f;      // 512 threads of one unit: 16 warps at most
  s = spread_sum<2>(s);
  half ^= 1;
  spread_get<2>(v, s);
}

__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ void read_turns(Turns& tu, const QkArgs& a, float* cs, int n) {
  for (int i = threadIdx.x; i < a.pairs; i += blockDim.x) {
    tu.turn[i] = a.turn[i];
    tu.axis[i] = a.axis[i];
  }
  for (int i = threadIdx.x; i < n; i += blockDim.x) cs[i] = i & 2 ? 0.f : 1.f;    // pairs that heads lack
  __syncthreads();
}

// ---------------------------------------------------------------- forward --
// Fits in 96 registers: bfloat16 words from the ring.  What a thread holds of
// float32 tokens, or of tokens it loads itself, does not.
template <typename T, class L>
constexpr bool lean() {
  return sizeof(T) == 2 && L::RING;
}
template <typename T, class L, int K>
__global__ void __maxnreg__(L::UPT == 4 ? 64 : (lean<T, L>() ? 96 : 128)) qk_fwd_kernel(const __grid_constant__ QkArgs a, int depth) {
  constexpr int UPT = L::UPT;
  constexpr bool RING = L::RING;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Turns tu;
  __shared__ Scratch<K> sums;
  __shared__ __align__(16) float cs[2][kAhead * 2 * SPADE_ROPE_MAX_PAIRS];
  const Units<T, L> un(a, 1);
  const int lanes = un.lanes, j = un.j, d = un.d, nwarps = blockDim.x >> 5;
  const long long r0 = a.rows * blockIdx.x / gridDim.x, r1 = a.rows * (blockIdx.x + 1) / gridDim.x;
  const T* const xs[2] = {static_cast<const T*>(a.x[0]), static_cast<const T*>(a.x[1])};
  T* const outs[2] = {static_cast<T*>(a.out[0]), static_cast<T*>(a.out[1])};
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  const T* from[UPT];            // the next token to copy and the next to write
  T* to[UPT];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    from[i] = un.at(xs, a.x_stride, r0, i);
    to[i] = un.at(outs, a.out_stride, r0, i);
  }
  long long fr = r0;             // the next token to copy, its slot, and the slot of the next one to use
  int fs = 0, us = 0;
  auto fetch = [&]() {
    if (fr < r1) {
#pragma unroll
      for (int i = 0; i < UPT; ++i)
        if constexpr (RING)
          if (un.in[i]) {
            fetch16<T, L>(ring_at + fs * un.slot + un.place(0, i), from[i], j, lanes, d);
            from[i] += un.step(a.x_stride, i);
          }
    }
    commit_async();
    ++fr;
    fs = fs + 1 == depth ? 0 : fs + 1;
  };
  if (RING) {
    un.clear(ring, depth, 1);
    for (int s = 0; s < depth; ++s) fetch();
  }
  Unit w[UPT];
  const bool normed = a.norm != SPADE_QK_NORM_NONE, token = a.norm == SPADE_QK_NORM_TOKEN;
  if (normed) {
#pragma unroll
    for (int i = 0; i < UPT; ++i) un.weights(w[i], a, i);
  }
  read_turns(tu, a, cs[0], 4 * kAhead * SPADE_ROPE_MAX_PAIRS);
  angles<L>(a, tu, r0, r1, cs[0]);
  int half = 0, buf = 0, ago = 0;      // which angles, and how many of their tokens are done
  auto get = [&](Unit& v, const unsigned char* at, long long r, int i) {
    if constexpr (RING) ring16<T, L>(v, at + un.place(0, i));
    else load16<T, L>(v, un.at(xs, a.x_stride, r, i), un.in[i], j, lanes, d);
  };
  for (long long r = r0; r < r1; r += K) {
    const int n = r1 - r < K ? (int)(r1 - r) : K;
    // UPT, unknown to the compiler: a branch on it, never taken, keeps a later
    // unit's loads, and so their registers, behind the unit before
    int opaque = UPT;
    asm volatile("" : "+r"(opaque));
    if (RING) wait_async_upto(depth - K);
    const unsigned char* at[K];
#pragma unroll
    for (int k = 0; k < K; ++k) at[k] = ring + (us + k >= depth ? us + k - depth : us + k) * un.slot;
    float s[2 * K], rs[K][UPT];
    if (normed) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        s[k] = s[K + k] = 0.f;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          float q = 0.f;
          if (k < n) {
            Unit v;
            float2 q2 = both(0.f);
            get(v, at[k], r + k, i);
#pragma unroll
            for (int p = 0; p < 4; ++p) q2 = fma(v.b[p], v.b[p], fma(v.a[p], v.a[p], q2));
            q = sum_of(q2);
          }
          if (un.k_side[i]) s[K + k] += q;
          else s[k] += q;
          rs[k][i] = q;
        }
      }
    }
    if (token && nwarps > 1) {
      block_sum(s, sums, half, nwarps);          // its barrier also covers the angles
    } else {
      __syncthreads();
      if (token) block_sum(s, sums, half, nwarps);
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (token) rs[k][i] = rsqrtf((un.k_side[i] ? s[K + k] : s[k]) * un.inv[i] + a.eps);
        else if (normed) rs[k][i] = rsqrtf(lanes_sum(rs[k][i], lanes) * un.inv[i] + a.eps);
      }
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (k >= n) break;
      Angles t;
      get_angles(t, cs[buf] + (ago + k) * 16 * lanes, j, lanes);
#pragma unroll
      for (int i = 0; i < UPT; ++i) {
        if (i >= opaque) break;
        if (!un.in[i]) continue;
        Unit v;
        get(v, at[k], r + k, i);
        if (normed) {
          const float2 f = both(rs[k][i]);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            v.a[p] = mul(v.a[p], mul(f, w[i].a[p]));
            v.b[p] = mul(v.b[p], mul(f, w[i].b[p]));
          }
        }
        turn(v, t, false);
        store16<T, L>(to[i], v, j, lanes, d);
        to[i] += un.step(a.out_stride, i);
      }
    }
    if (RING) {
      for (int k = 0; k < n; ++k) fetch();
      us = us + n >= depth ? us + n - depth : us + n;
    }
    ago += K;
    if (ago == kAhead) {         // the next ones, where those before these were: last read before this barrier
      ago = 0;
      buf ^= 1;
      if (r + K < r1) angles<L>(a, tu, r + K, r1, cs[buf]);
    }
  }
  if (RING) wait_async<0>();
}

// --------------------------------------------------------------- backward --
template <typename T, class L, int K>
__global__ void __maxnreg__(L::UPT == 1 ? 96 : (L::UPT == 2 ? 128 : 64)) qk_bwd_kernel(const __grid_constant__ QkArgs a, int depth) {
  constexpr int UPT = L::UPT;
  constexpr bool ONE_SIDE = UPT == 1 && L::FULL && K == 1;       // a warp's units are of Q or of K alone
  constexpr bool KEEP = UPT == 1;          // tokens stay in registers between the two passes over them
  constexpr bool RING = L::RING;
  extern __shared__ __align__(16) unsigned char ring[];
  __shared__ Turns tu;
  __shared__ Scratch<2 * K> sums;
  __shared__ __align__(16) float cs[2][kAhead * 2 * SPADE_ROPE_MAX_PAIRS];
  const bool normed = a.norm != SPADE_QK_NORM_NONE, token = a.norm == SPADE_QK_NORM_TOKEN;
  const int ops = normed ? 2 : 1;
  const Units<T, L> un(a, ops);
  const int lanes = un.lanes, j = un.j, d = un.d, nwarps = blockDim.x >> 5;
  const long long r0 = a.rows * blockIdx.x / gridDim.x, r1 = a.rows * (blockIdx.x + 1) / gridDim.x;
  const T* const gs[2] = {static_cast<const T*>(a.dout[0]), static_cast<const T*>(a.dout[1])};
  const T* const xs[2] = {static_cast<const T*>(a.x[0]), static_cast<const T*>(a.x[1])};
  T* const outs[2] = {static_cast<T*>(a.out[0]), static_cast<T*>(a.out[1])};
  const uint32_t ring_at = (uint32_t)__cvta_generic_to_shared(ring);
  // with one unit: its place in row 0 and the bytes to the next row (rows and
  // strides below 2^32: one multiply-add makes an address)
  const unsigned char *g0 = nullptr, *x0 = nullptr;
  unsigned char* o0 = nullptr;
  uint32_t g_step = 0, x_step = 0, o_step = 0;
  if constexpr (KEEP) {
    const int t = un.k_side[0];
    g0 = reinterpret_cast<const unsigned char*>(un.at(gs, a.dout_stride, 0, 0));
    x0 = reinterpret_cast<const unsigned char*>(un.at(xs, a.x_stride, 0, 0));
    o0 = reinterpret_cast<unsigned char*>(un.at(outs, a.out_stride, 0, 0));
    g_step = (uint32_t)(a.dout_stride[t] * sizeof(T));
    x_step = (uint32_t)(a.x_stride[t] * sizeof(T));
    o_step = (uint32_t)(a.out_stride[t] * sizeof(T));
  }
  auto row = [](const unsigned char* p, uint32_t step, long long r) {
    return reinterpret_cast<const T*>(p + (unsigned long long)(uint32_t)r * step);
  };
  long long fr = r0;
  int fs = 0, us = 0;
  auto fetch = [&]() {
    if (fr < r1) {
#pragma unroll
      for (int i = 0; i < UPT; ++i)
        if constexpr (RING)
          if (un.in[i]) {
            const uint32_t slot = ring_at + fs * un.slot;
            if constexpr (KEEP) {
              fetch16<T, L>(slot + un.place(0, i), row(g0, g_step, fr), j, lanes, d);
              if (normed) fetch16<T, L>(slot + un.place(1, i), row(x0, x_step, fr), j, lanes, d);
            } else {
              fetch16<T, L>(slot + un.place(0, i), un.at(gs, a.dout_stride, fr, i), j, lanes, d);
              if (normed) fetch16<T, L>(slot + un.place(1, i), un.at(xs, a.x_stride, fr, i), j, lanes, d);
            }
          }
    }
    commit_async();
    ++fr;
    fs = fs + 1 == depth ? 0 : fs + 1;
  };
  if (RING) {
    un.clear(ring, depth, ops);
    for (int s = 0; s < depth; ++s) fetch();
  }
  Unit w[UPT], dw[UPT];
#pragma unroll
  for (int i = 0; i < UPT; ++i) {
    if (normed) un.weights(w[i], a, i);
#pragma unroll
    for (int p = 0; p < 4; ++p) dw[i].a[p] = dw[i].b[p] = both(0.f);
  }
  read_turns(tu, a, cs[0], 4 * kAhead * SPADE_ROPE_MAX_PAIRS);
  angles<L>(a, tu, r0, r1, cs[0]);
  const int q_warps = a.heads[0] * lanes / 32;
  const int side_first = un.k_side[0] ? q_warps : 0, side_last = un.k_side[0] ? nwarps : q_warps;
  int half = 0, buf = 0, ago = 0;      // which angles, and how many of their tokens are done
  auto get_g = [&](Unit& v, const unsigned char* at, long long r, int i, const Angles& t) {
    if constexpr (RING) ring16<T, L>(v, at + un.place(0, i));
    else load16<T, L>(v, un.at(gs, a.dout_stride, r, i), un.in[i], j, lanes, d);
    turn(v, t, true);
  };
  auto get_x = [&](Unit& v, const unsigned char* at, long long r, int i) {
    if constexpr (RING) ring16<T, L>(v, at + un.place(1, i));
    else load16<T, L>(v, un.at(xs, a.x_stride, r, i), un.in[i], j, lanes, d);
  };
  auto next = [&](int n) {       // n tokens are used: copy as many, ahead
    if (RING) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k < n) fetch();
      us = us + n >= depth ? us + n - depth : us + n;
    }
  };
  for (long long r = r0; r < r1; r += K) {
    const int n = r1 - r < K ? (int)(r1 - r) : K;
    if (RING) wait_async_upto(depth - K);
    if (ago == 0) __syncthreads();               // the angles are there
    const unsigned char* at[K];
#pragma unroll
    for (int k = 0; k < K; ++k) at[k] = ring + (us + k >= depth ? us + k - depth : us + k) * un.slot;
    // per token and tensor: sum of x^2, sum of w u x; then 1 / deviation and rstd^2 mean(w u x)
    float s[4 * K], rs[K][UPT], cf[K][UPT];
    Unit xk[KEEP ? K : 1], uk[KEEP ? K : 1];
    if (normed || KEEP) {
#pragma unroll
      for (int i = 0; i < 4 * K; ++i) s[i] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        Angles t;
        get_angles(t, cs[buf] + (ago + k) * 16 * lanes, j, lanes);
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          float q0 = 0.f, q1 = 0.f;
          if (k < n) {
            Unit x, u;
            get_g(u, at[k], r + k, i, t);
            if (normed) {
              float2 s0 = both(0.f), s1 = both(0.f);
              get_x(x, at[k], r + k, i);
#pragma unroll
              for (int p = 0; p < 4; ++p) {
                s0 = fma(x.b[p], x.b[p], fma(x.a[p], x.a[p], s0));
                s1 = fma(mul(u.b[p], w[i].b[p]), x.b[p], fma(mul(u.a[p], w[i].a[p]), x.a[p], s1));
              }
              q0 = sum_of(s0);
              q1 = sum_of(s1);
            }
            if constexpr (KEEP) {
              xk[k] = x;
              uk[k] = u;
            }
          }
          if (un.k_side[i]) {
            s[K + k] += q0;
            s[3 * K + k] += q1;
          } else {
            s[k] += q0;
            s[2 * K + k] += q1;
          }
          rs[k][i] = q0;
          cf[k][i] = q1;
        }
      }
      if (KEEP) next(n);
      if (ONE_SIDE) {
        if (token && nwarps > 1) {
          float both_sums[2] = {rs[0][0], cf[0][0]};
          side_sum(both_sums, sums, half, side_first, side_last);
          s[0] = s[K] = both_sums[0];
          s[2 * K] = s[3 * K] = both_sums[1];
        } else if (token) {
          block_sum(s, sums, half, nwarps);
        }
      } else if (token) {
        block_sum(s, sums, half, nwarps);
      }
      if (normed) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < UPT; ++i) {
            const bool ks = un.k_side[i];
            const float q0 = token ? (ks ? s[K + k] : s[k]) : lanes_sum(rs[k][i], lanes);
            const float q1 = token ? (ks ? s[3 * K + k] : s[2 * K + k]) : lanes_sum(cf[k][i], lanes);
            rs[k][i] = rsqrtf(q0 * un.inv[i] + a.eps);
            cf[k][i] = rs[k][i] * rs[k][i] * q1 * un.inv[i];
          }
      }
    }
    auto finish = [&](int k, int i, Unit& u, const Unit& x) {
      if (normed) {
        const float2 f = both(rs[k][i]), g = both(-cf[k][i]);
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          dw[i].a[p] = fma(u.a[p], mul(x.a[p], f), dw[i].a[p]);
          dw[i].b[p] = fma(u.b[p], mul(x.b[p], f), dw[i].b[p]);
          u.a[p] = mul(f, fma(x.a[p], g, mul(u.a[p], w[i].a[p])));
          u.b[p] = mul(f, fma(x.b[p], g, mul(u.b[p], w[i].b[p])));
        }
      }
      if constexpr (KEEP) {
        store16<T, L>(const_cast<T*>(row(o0, o_step, r + k)), u, j, lanes, d);
      } else {
        store16<T, L>(un.at(outs, a.out_stride, r + k, i), u, j, lanes, d);
      }
    };
    // absent heads stay out of dw whatever eps makes of their zeros
    if constexpr (KEEP) {
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (k < n && un.in[0]) finish(k, 0, uk[k], xk[k]);
    } else {
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        Angles t;
        get_angles(t, cs[buf] + (ago + k) * 16 * lanes, j, lanes);
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
          if (!un.in[i]) continue;
          Unit u, x;
          get_g(u, at[k], r + k, i, t);
          if (normed) get_x(x, at[k], r + k, i);
          finish(k, i, u, x);
        }
      }
      next(n);
    }
    ago += K;
    if (ago == kAhead) {         // the next ones, where those before these were: last read before this barrier
      ago = 0;
      buf ^= 1;
      if (r + K < r1) angles<L>(a, tu, r + K, r1, cs[buf]);
    }
  }
  if (RING) wait_async<0>();
  if (!normed || !a.part) return;
  // this block's weight sums: [heads * d] of Q then of K, or (per-head norm)
  // [d] of each, its heads added in a fixed order
  float* part = a.part + (long long)blockIdx.x * (token ? (a.heads[0] + a.heads[1]) * d : 2 * d);
  if (token) {
#pragma unroll
    for (int i = 0; i < UPT; ++i)
      if (un.in[i]) {
        float* o = part + ((un.k_side[i] ? a.heads[0] : 0) + un.head[i]) * d;
        float v[16];
        elements_of<L>(v, dw[i]);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          if (owned<L>(j, lanes, e, d)) o[channel<L>(j, lanes, e, d)] = v[e];
      }
    return;
  }
  float* by_warp = reinterpret_cast<float*>(ring);       // [warps][d]
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
    float sum[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) sum[e] = 0.f;
#pragma unroll
    for (int i = 0; i < UPT; ++i) {
      float v[16];
      elements_of<L>(v, dw[i]);
#pragma unroll
      for (int e = 0; e < 16; ++e) sum[e] += un.k_side[i] == (t == 1) ? v[e] : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float v = sum[e];
      // the heads of one warp, then the warps through shared memory
      for (int o = lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if ((int)(threadIdx.x & 31) < lanes && owned<L>(j, lanes, e, d))
        by_warp[(threadIdx.x >> 5) * d + channel<L>(j, lanes, e, d)] = v;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
      float v = 0.f;
      for (int wp = 0; wp < nwarps; ++wp) v += by_warp[wp * d + i];
      part[t * d + i] = v;
    }
  }
}

// Adds the blocks' weight sums in a fixed order, in float64.
__global__ void __launch_bounds__(1024) qk_reduce_kernel(const float* __restrict__ part, int blocks, int wq, int wk, float* dq,
                                                         float* dk) {
  __shared__ double sh[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, width = wq + wk;
  const int col = blockIdx.x * 32 + lane;
  cudaGridDependencySynchronize();
  double s = 0.0;
  for (int b = warp; b < blocks && col < width; b += 32 * 8) {      // a round of loads in flight together
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = b + 32 * i < blocks ? part[(long long)(b + 32 * i) * width + col] : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += (double)v[i];
  }
  sh[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && col < width) {
#pragma unroll 8
    for (int v = 1; v < 32; ++v) s += sh[v][lane];
    float* o = col < wq ? dq : dk;
    if (o) o[col < wq ? col : col - wq] = (float)s;
  }
}

// ----------------------------------------------------------------- launch --
// Two units a thread, or four where 512 threads of two would not cover them;
// backward one where 512 threads of one do, so that a token's inputs stay in
// registers.
int units_per_thread(const QkArgs& a, bool back, int size) {
  const int units = (a.heads[0] + a.heads[1]) * a.lanes;
  bool narrow = a.rows < 1LL << 32;          // addresses by a 32-bit row and step
  for (int t = 0; t < 2; ++t)
    for (long long st : {a.x_stride[t], a.dout_stride[t], a.out_stride[t]}) narrow = narrow && st * size < 1LL << 32;
  return back && units <= 512 && narrow ? 1 : (units <= 1024 ? 2 : 4);
}
int block_threads(const QkArgs& a, int upt) {
  return (((a.heads[0] + a.heads[1]) * a.lanes + upt - 1) / upt + 31) / 32 * 32;
}

constexpr int kSmemSm = 227 * 1024;
constexpr int kStatic = sizeof(Turns) + sizeof(Scratch<4>) + 4 * kAhead * SPADE_ROPE_MAX_PAIRS * sizeof(float) + 1024 + 64;

// Blocks of an SM: by registers (`sm_threads` threads in all), and so
// that `least` tokens a block fit in shared memory.
int blocks_of(int threads, int sm_threads, size_t slot, int least) {
  int b = sm_threads / threads;
  const int fit = (int)(kSmemSm / (slot * least + kStatic));
  b = b < fit ? b : fit;
  return b < 1 ? 1 : (b > 8 ? 8 : b);
}
int grid_of(const QkArgs& a, int blocks, int k) {
  const long long resident = (long long)num_sms() * blocks, most = (a.rows + k - 1) / k;
  return (int)(most < resident ? most : resident);
}

template <typename K>
cudaError_t launch(K kernel, const QkArgs& a, int grid, int threads, int blocks, int k, size_t slot, bool ring,
                   size_t least, cudaStream_t s) {
  int depth = 0;
  size_t smem = 0;
  if (ring) {
    const size_t room = kSmemSm / blocks - kStatic;
    const long long rows = (a.rows + grid - 1) / grid;
    depth = (int)(room / slot < kDepthMax ? room / slot : kDepthMax);
    if (rows < depth) depth = (int)(rows > k ? rows : k);
    if (depth < k) return cudaErrorInvalidConfiguration;
    smem = depth * slot;
  }
  if (smem < least) smem = least;
  if (smem > 32 * 1024) {        // one value for all launches: callers on other threads may be between theirs and this
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemSm - kStatic);
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, threads, smem, s>>>(a, depth);
  return cudaGetLastError();
}

template <typename T, class L>
cudaError_t run_fwd(const QkArgs& a, cudaStream_t s) {
  constexpr int K = 2;
  const int threads = block_threads(a, L::UPT);
  const size_t slot = (size_t)threads * L::UPT * 16 * sizeof(T);
  const int blocks = blocks_of(threads, lean<T, L>() ? 640 : 512, L::RING ? slot : 0, K);
  return launch(qk_fwd_kernel<T, L, K>, a, grid_of(a, blocks, K), threads, blocks, K, slot, L::RING, 0, s);
}

// Threads of an SM in the backward pass, by registers (96 or 128 a thread: five or four warps in each quarter of an SM).
constexpr int bwd_sm_threads(int upt) { return upt == 1 ? 640 : 512; }
// Blocks of an SM in the backward pass at most, whatever units a thread has.
int bwd_blocks(const QkArgs& a) {
  int most = 1;
  for (int upt : {1, 2, 4})
    if (block_threads(a, upt) <= (upt == 4 ? 1024 : 512))
      most = std::max(most, blocks_of(block_threads(a, upt), bwd_sm_threads(upt), 0, 0));
  return most;
}

template <typename T, class L>
cudaError_t run_bwd(const QkArgs& a, cudaStream_t s) {
  constexpr int K = sizeof(T) == 2 && L::UPT > 1 ? 2 : 1;
  const int threads = block_threads(a, L::UPT);
  const size_t slot = (size_t)threads * L::UPT * 16 * sizeof(T) * (a.norm != SPADE_QK_NORM_NONE ? 2 : 1);
  const size_t least = a.norm == SPADE_QK_NORM_HEAD ? (size_t)(threads / 32) * a.d * sizeof(float) : 0;
  const int blocks = blocks_of(threads, bwd_sm_threads(L::UPT), L::RING ? slot : 0, K == 1 ? 3 : K), grid = grid_of(a, blocks, K);
  cudaError_t e = launch(qk_bwd_kernel<T, L, K>, a, grid, threads, blocks, K, slot, L::RING, least, s);
  if (e != cudaSuccess || !a.part) return e;
  const bool token = a.norm == SPADE_QK_NORM_TOKEN;
  const int wq = token ? a.heads[0] * a.d : a.d, wk = token ? a.heads[1] * a.d : a.d;
  return launch_behind(qk_reduce_kernel, (wq + wk + 31) / 32, 1024, s, a.part, grid, wq, wk, a.dweight[0], a.dweight[1]);
}

// Threads of four units read tokens where they are used: two tokens of so
// many channels need not fit in shared memory.
template <typename T, int P, bool HALF, bool RING, bool WIDE>
cudaError_t by_shape(const QkArgs& a, bool back, cudaStream_t s) {
  const int upt = units_per_thread(a, back, sizeof(T));
  if (upt == 4) {
    using L = Layout<P, HALF, false, false, 4>;
    return back ? run_bwd<T, L>(a, s) : run_fwd<T, L>(a, s);
  }
  if constexpr (WIDE) {
    if (a.d == 16 * a.lanes && (a.heads[0] + a.heads[1]) * a.lanes == upt * block_threads(a, upt)) {
      if (upt == 1 && a.heads[0] * a.lanes % 32 == 0) return run_bwd<T, Layout<P, HALF, true, RING, 1>>(a, s);
      if (upt == 1) return run_bwd<T, Layout<P, HALF, false, RING, 1>>(a, s);
      using L = Layout<P, HALF, true, RING, 2>;
      return back ? run_bwd<T, L>(a, s) : run_fwd<T, L>(a, s);
    }
  }
  if (upt == 1) return run_bwd<T, Layout<P, HALF, false, RING, 1>>(a, s);
  using L = Layout<P, HALF, false, RING, 2>;
  return back ? run_bwd<T, L>(a, s) : run_fwd<T, L>(a, s);
}
template <typename T, int P, bool RING, bool WIDE>
cudaError_t by_style(const QkArgs& a, bool back, cudaStream_t s) {
  return a.half ? by_shape<T, P, true, RING, WIDE>(a, back, s) : by_shape<T, P, false, RING, WIDE>(a, back, s);
}

// The widest piece, in channels, that heads (halves of heads) and every row
// allow: 16 bytes, 4 bytes, or a single channel.
int piece_of(const QkArgs& a, int size) {
  for (int p = 16 / size; p > 1; p = p > 2 ? 2 : 1) {
    bool ok = a.d % (a.half ? 2 * p : p) == 0;
    for (int t = 0; t < 2; ++t) {
      const struct { const void* p; long long stride; int size; } ops[] = {
          {a.x[t], a.x_stride[t], size}, {a.dout[t], a.dout_stride[t], size}, {a.out[t], a.out_stride[t], size},
          {a.weight[t], 0, a.weight_bf16 ? 2 : 4}};
      for (const auto& o : ops) {
        const int need = p * o.size < 16 ? p * o.size : 16;
        ok = ok && (!o.p || (reinterpret_cast<uintptr_t>(o.p) % need == 0 && o.stride % p == 0));
      }
    }
    if (ok) return p;
  }
  return 1;
}

cudaError_t run(const QkArgs& a, bool is_bf16, bool back, cudaStream_t s) {
  const int p = piece_of(a, is_bf16 ? 2 : 4);
  if (is_bf16) {
    if (p == 8) return by_style<bf16, 8, true, true>(a, back, s);
    return p == 2 ? by_style<bf16, 2, true, false>(a, back, s) : by_style<bf16, 1, false, false>(a, back, s);
  }
  return p == 4 ? by_style<float, 4, true, true>(a, back, s) : by_style<float, 1, true, false>(a, back, s);
}

}  // namespace

size_t qk_bwd_floats(const QkArgs& a) {
  if (a.norm == SPADE_QK_NORM_NONE) return 0;
  return (size_t)grid_of(a, bwd_blocks(a), 1) * (a.norm == SPADE_QK_NORM_TOKEN ? (a.heads[0] + a.heads[1]) * a.d : 2 * a.d);
}

cudaError_t launch_qk_fwd(const QkArgs& a, bool is_bf16, cudaStream_t s) { return run(a, is_bf16, false, s); }
cudaError_t launch_qk_bwd(const QkArgs& a, bool is_bf16, cudaStream_t s) { return run(a, is_bf16, true, s); }

}  // namespace spade
