// Row access and reductions shared by the row passes around the attention
// (k_qk_rope.cu, row_pass.cuh): loads, stores and asynchronous
// copies of eight float32 or bfloat16 elements in pieces of P, and sums over
// warps and blocks in float32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

namespace spade {
namespace rowio {

using bf16 = __nv_bfloat16;

template <int BYTES>
struct Word;
template <> struct Word<2> { using type = unsigned short; };
template <> struct Word<4> { using type = unsigned int; };
template <> struct Word<8> { using type = uint2; };
template <> struct Word<16> { using type = uint4; };
struct alignas(16) Word32 { uint4 a, b; };
template <> struct Word<32> { using type = Word32; };

// Arithmetic on pairs: one instruction for two float32 operations.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float sum_of(float2 a) { return a.x + a.y; }

// P neighbouring elements as one access.  bfloat16 is the upper half of a
// float32: the low element of a word shifts up, the high one is masked.
template <int P>
__device__ __forceinline__ void widen(float* v, const uint32_t* w, bf16) {
  if (P == 1) {
    v[0] = __uint_as_float(w[0] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}
template <int P>
__device__ __forceinline__ void widen(float* v, const uint32_t* w, float) {
#pragma unroll
  for (int i = 0; i < P; ++i) v[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void words_of(uint32_t* w, unsigned short u) { w[0] = u; }
__device__ __forceinline__ void words_of(uint32_t* w, unsigned int u) { w[0] = u; }
__device__ __forceinline__ void words_of(uint32_t* w, uint2 u) { w[0] = u.x; w[1] = u.y; }
__device__ __forceinline__ void words_of(uint32_t* w, uint4 u) { w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w; }
__device__ __forceinline__ void words_of(uint32_t* w, const Word32& u) { words_of(w, u.a); words_of(w + 4, u.b); }
__device__ __forceinline__ void from_words(unsigned short& u, const uint32_t* w) { u = (unsigned short)w[0]; }
__device__ __forceinline__ void from_words(unsigned int& u, const uint32_t* w) { u = w[0]; }
__device__ __forceinline__ void from_words(uint2& u, const uint32_t* w) { u = make_uint2(w[0], w[1]); }
__device__ __forceinline__ void from_words(uint4& u, const uint32_t* w) { u = make_uint4(w[0], w[1], w[2], w[3]); }
__device__ __forceinline__ void from_words(Word32& u, const uint32_t* w) { from_words(u.a, w); from_words(u.b, w + 4); }

template <typename T, int P>
__device__ __forceinline__ void load_piece(float* v, const T* p) {
  using W = typename Word<P * (int)sizeof(T)>::type;
  uint32_t w[8];
  words_of(w, *reinterpret_cast<const W*>(p));
  widen<P>(v, w, T());
}
template <int P>
__device__ __forceinline__ void store_piece(bf16* p, const float* v) {      // rounds to nearest even
  uint32_t w[4];
  if (P == 1) {
    w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
  } else {
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  typename Word<P * 2>::type u;
  from_words(u, w);
  *reinterpret_cast<typename Word<P * 2>::type*>(p) = u;
}
template <int P>
__device__ __forceinline__ void store_piece(float* p, const float* v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < P; ++i) w[i] = __float_as_uint(v[i]);
  typename Word<P * 4>::type u;
  from_words(u, w);
  *reinterpret_cast<typename Word<P * 4>::type*>(p) = u;
}

// Asynchronous copy of 4, 8 or 16 bytes to shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  static_assert(BYTES == 4 || BYTES == 8 || BYTES == 16, "no such copy");
  if (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else if (BYTES == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Waits until at most `left` of this thread's groups are in flight (waits for
// more than asked where `left` is above the cases).
__device__ __forceinline__ void wait_async_upto(int left) {
  switch (left) {
    case 0: wait_async<0>(); break;
    case 1: wait_async<1>(); break;
    case 2: wait_async<2>(); break;
    case 3: wait_async<3>(); break;
    case 4: wait_async<4>(); break;
    case 5: wait_async<5>(); break;
    case 6: wait_async<6>(); break;
    case 7: wait_async<7>(); break;
    case 8: wait_async<8>(); break;
    case 9: wait_async<9>(); break;
    case 10: wait_async<10>(); break;
    case 11: wait_async<11>(); break;
    default: wait_async<12>(); break;
  }
}

// Sums N values (a power of two, up to 32) over the warp at once: halves of
// the values change places until every lane carries one, so N - 1 + 5 -
// log2(N) shuffles do for all of them.  Lane l gets the sum of value
// l / (32 / N).
template <int N>
__device__ __forceinline__ float warp_sum_spread(const float (&in)[N]) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = in[i];
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int n = N; n > 1; n >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float give = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
    o >>= 1;
  }
  float s = v[0];
#pragma unroll
  for (; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// Adds up the 32 / N lanes that share a value.
template <int N>
__device__ __forceinline__ float spread_sum(float s) {
#pragma unroll
  for (int o = 16 / N; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}
// Every lane gets all N values.
template <int N>
__device__ __forceinline__ void spread_get(float (&v)[N], float s) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, s, i * (32 / N));
}

// Scratch of block-wide sums of up to M float2 values, in two halves.  Calls
// on one scratch alternate its halves, whatever they sum, so one barrier a
// call is enough: a half is written again only after the next call's barrier,
// which every thread reaches after its reads of this one.
template <int M>
struct Scratch {
  float2 v[2][M * 33];
};

// Sums of N values over the block, the same in every thread.  One barrier,
// none in one-warp blocks.
template <int N, int M>
__device__ __forceinline__ void block_sum(float (&v)[N], Scratch<M>& sh, int& half, int nwarps) {
  static_assert(N <= 2 * M, "scratch too small");
  constexpr int L = 32 / N;
  const int lane = threadIdx.x & 31, sub = lane % L;
  float s = warp_sum_spread<N>(v);
  if (nwarps > 1) {
    float* b = reinterpret_cast<float*>(sh.v[half]) + (lane / L) * 33;
    if (sub == 0) b[threadIdx.x >> 5] = s;
    __syncthreads();
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 32; w += L) s += w + sub < nwarps ? b[w + sub] : 0.f;
    s = spread_sum<N>(s);
    half ^= 1;
  }
  spread_get<N>(v, s);
}

// Launches a kernel that follows another in its stream and waits for it with
// cudaGridDependencySynchronize(): its launch is prepared while the other runs.
template <typename... P, typename... A>
cudaError_t launch_behind(void (*kernel)(P...), int grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

}  // namespace rowio
}  // namespace spade
