// adamw.cu — one AdamW step over many tensors in one launch, with optimiser states in 32 bits
// or in 8, and the global norm of the gradients for its clip.
//
// Per value, with g the gradient times grad_scale:
//   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
//   p = p - lr decay p - lr (m / (1 - beta1^step)) / (sqrt(v / (1 - beta2^step)) + eps)
// Everything is computed in fp32; a bf16 parameter or copy is rounded once, to nearest.
//
// 8-bit states: a block of 256 values holds m and sqrt(v) as E4M3 codes with one fp32 scale
// each (largest magnitude / 448), the codes of the library's row quantizer. sqrt(v) and not v:
// the codes span 2^17.8, which is then 2^35 in v, and the step divides by sqrt(v). A code of
// sqrt(v) is never zero where v is not: a second moment that vanished next to a first moment
// that did not would turn the next step into m / eps. The step itself uses m and v before
// they are rounded.
//
// Bound by memory: 30 bytes a value (fp32 parameter, bf16 copy, fp32 gradient and states), 16
// with 8-bit states and bf16 gradients. A thread takes 8 consecutive values, so every access
// is 16 bytes or more a lane with up to 8 loads in flight a thread, and a warp takes one state
// block, so its scale is one warp-wide maximum. The tensors' pointers travel as a kernel
// parameter: no table in device memory, nothing for a captured graph to keep alive. A block
// takes one chunk of 2048 values and ends: walking over chunks in resident blocks lets the SMs
// drift apart and read and write all over the tensors (50M parameters, 32 bits, with the
// norm: 291 us, a block a chunk 251). The step walks the values from the last to the first: what
// the norm's pass (first to last) read last is still in the L2 cache.
//
// Measured with the norm: 50M values, 32 bits, fp32 gradients 253 us (214 the step alone, 7.05
// TB/s of its bytes, a part of them from the L2 cache; a plain copy draws 6.79); 315M, 8 bits,
// bf16 gradients 899 us (6.3 TB/s in the norm and in the step).
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <vector>

#include "../../include/pb.h"
#include "kernels.h"
#include "ptx.cuh"

namespace pb {
pb_status record_error(pb_status s, const char* message);

namespace {

constexpr int THREADS = 256;
constexpr int PER_THREAD = 8;
constexpr int CHUNK = THREADS * PER_THREAD;  // values of one tensor a block takes at a time
static_assert(PB_ADAMW_BLOCK == 32 * PER_THREAD, "one warp takes one state block");
constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Least = 0x1p-9f;  // the least positive value

struct Tensor {
  void* param;
  __nv_bfloat16* copy;
  const void* grad;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  int64_t first_chunk;
  float decay;
};

// As many tensors as fit the 32,764 bytes of kernel parameters, or few for a quicker launch.
constexpr int kFew = 32, kMany = 384;
template <int CAP>
struct Table {
  Tensor t[CAP];
  int count;
  int64_t chunks;
};
static_assert(sizeof(Table<kMany>) + 128 <= 32764, "kernel parameters");

struct Step {
  float lr, beta1, beta2, eps;
  float one_minus_beta1, one_minus_beta2;  // rounded from double: 1 - beta2 loses bits in fp32
  float log_beta1, log_beta2;
  float correction1, correction2;          // 1 / (1 - beta^step)
  const float* d_lr;
  const int32_t* d_step;
  const float* d_grad_scale;
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 u = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  __stcs(reinterpret_cast<uint4*>(p),
         make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7])));
}
// Eight values two at a time (packed fp32 instructions).
__device__ __forceinline__ void mul8(float (&y)[8], const float (&x)[8], float a) {
  const uint64_t aa = f2(a, a);
#pragma unroll
  for (int e = 0; e < 8; e += 2) f2_split(f2_mul(f2(x[e], x[e + 1]), aa), y[e], y[e + 1]);
}
// y = a y + b x
__device__ __forceinline__ void blend8(float (&y)[8], float a, float b, const float (&x)[8]) {
  const uint64_t aa = f2(a, a), bb = f2(b, b);
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    f2_split(f2_fma(f2(x[e], x[e + 1]), bb, f2_mul(f2(y[e], y[e + 1]), aa)), y[e], y[e + 1]);
}
// y = y + a x
__device__ __forceinline__ void add8(float (&y)[8], float a, const float (&x)[8]) {
  const uint64_t aa = f2(a, a);
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    f2_split(f2_fma(f2(x[e], x[e + 1]), aa, f2(y[e], y[e + 1])), y[e], y[e + 1]);
}
__device__ __forceinline__ void square8(float (&y)[8], const float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint64_t xx = f2(x[e], x[e + 1]);
    f2_split(f2_mul(xx, xx), y[e], y[e + 1]);
  }
}

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// To 2^-23; exact rounding would cost more instructions than all else of a value's step.
__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The last values of a tensor, fewer than 8: element by element, zero behind the end.
template <class T>
__device__ __forceinline__ void load_tail(const T* p, int n, float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = e < n ? as_float(p[e]) : 0.f;
}
template <class T>
__device__ __forceinline__ void store_tail(T* p, int n, const float (&f)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) put(p + e, f[e]);
}
template <class T>
__device__ __forceinline__ void load_any(const T* p, int n, float (&f)[8]) {
  if (n == 8)
    load8(p, f);
  else
    load_tail(p, n, f);
}
template <class T>
__device__ __forceinline__ void store_any(T* p, int n, const float (&f)[8]) {
  if (n == 8)
    store8(p, f);
  else
    store_tail(p, n, f);
}

// Two E4M3 codes, the lower byte first.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes), __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ void load_codes(const uint8_t* p, int n, float scale, float (&f)[8]) {
  uint32_t w[2] = {0, 0};
  if (n == 8) {
    const uint2 u = __ldcs(reinterpret_cast<const uint2*>(p));
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) w[e / 4] |= uint32_t(p[e]) << (8 * (e % 4));
  }
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const float2 x = e4m3x2_to_float2((w[e / 4] >> (8 * (e % 4))) & 0xffffu);
    f[e] = x.x;
    f[e + 1] = x.y;
  }
  mul8(f, f, scale);
}

// Warp-wide: the codes of the block's values and its scale. A block whose largest magnitude is
// below 2^-100 is held as zeros (448 divided by it would overflow). Magnitudes beyond 2^63
// are held as that, where the square of sqrt(v) is in range: an infinite scale would make every
// other value of the block NaN, and m beside a sqrt(v) that is held lower a step of any size.
template <bool SECOND>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int n, float (&f)[8]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[e]));
  // magnitudes compare as their bits
  top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
  top = fminf(top, 0x1p63f);
  const bool zero = top < 7.888609052210118e-31f;
  const float inv = zero ? 0.f : __fdividef(kE4m3Max, top);
  float q[8];
  mul8(q, f, inv);
  if (SECOND && !zero) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (f[e] > 0.f) q[e] = fmaxf(q[e], kE4m3Least);
  }
  const uint2 c = quant8_e4m3(q, 1.f);
  if (n == 8) {
    __stcs(reinterpret_cast<uint2*>(p), c);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = uint8_t((e < 4 ? c.x : c.y) >> (8 * (e % 4)));
  }
  if ((threadIdx.x & 31) == 0) *scale = zero ? 0.f : top * (1.f / kE4m3Max);
}

// The tensor that holds `chunk`: the last one whose first chunk is not behind it.
template <int CAP>
__device__ __forceinline__ int find_tensor(const Table<CAP>& tab, int64_t chunk) {
  int a = 0, b = tab.count;
  while (b - a > 1) {
    const int mid = (a + b) / 2;
    if (tab.t[mid].first_chunk <= chunk)
      a = mid;
    else
      b = mid;
  }
  return a;
}

// Blocks an SM: with 8-bit states a thread has fewer bytes in flight and more to compute, and
// five are quicker (315M with the norm: 957 us with four, 899 with five, 907 with six); with
// 32-bit states four are (50M: 253, 254, 258).
template <int CAP, class P, class G, bool EIGHT>
__global__ void __launch_bounds__(THREADS, EIGHT ? 5 : 4)
    adamw_kernel(const __grid_constant__ Table<CAP> tab, const __grid_constant__ Step st) {
  pdl_wait();
  pdl_trigger();
  const float gs = st.d_grad_scale != nullptr ? *st.d_grad_scale : 1.f;
  if (!(fabsf(gs) <= 3.402823466e38f)) return;  // not finite: the step is left out
  const float lr = st.d_lr != nullptr ? *st.d_lr : st.lr;
  float c1 = st.correction1, c2 = st.correction2;
  if (st.d_step != nullptr) {
    const float k = float(max(*st.d_step, 1));
    c1 = -1.f / expm1f(k * st.log_beta1);
    c2 = -1.f / expm1f(k * st.log_beta2);
  }
  const float root2 = sqrtf(c2);
  const int64_t chunk = tab.chunks - 1 - int64_t(blockIdx.x);
  const Tensor& t = tab.t[find_tensor(tab, chunk)];
  const int64_t at = (chunk - t.first_chunk) * CHUNK + int64_t(threadIdx.x) * PER_THREAD;
  // a warp without values leaves as a whole; with 8-bit states a warp with some stays whole
  if (at - int64_t(threadIdx.x & 31) * PER_THREAD >= t.n) return;
  const int n = int(max(int64_t(0), min(int64_t(PER_THREAD), t.n - at)));
  float g[8], m[8], v[8], p[8];
  load_any(static_cast<const G*>(t.grad) + at, n, g);
  load_any(static_cast<const P*>(t.param) + at, n, p);
  const int64_t block = at / PB_ADAMW_BLOCK;
  if (EIGHT) {
    load_codes(static_cast<const uint8_t*>(t.m) + at, n, t.m_scale[block], m);
    load_codes(static_cast<const uint8_t*>(t.v) + at, n, t.v_scale[block], v);
    square8(v, v);
  } else {
    load_any(static_cast<const float*>(t.m) + at, n, m);
    load_any(static_cast<const float*>(t.v) + at, n, v);
  }
  float r[8], up[8];
  mul8(g, g, gs);
  blend8(m, st.beta1, st.one_minus_beta1, g);
  square8(up, g);
  blend8(v, st.beta2, st.one_minus_beta2, up);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    r[e] = sqrt_approx(v[e]);
    // the denominator is a normal number: eps is one
    up[e] = m[e] * rcp_approx(r[e] * root2 + st.eps);
  }
  add8(p, -lr * t.decay, p);
  add8(p, -lr * c1, up);
  store_any(static_cast<P*>(t.param) + at, n, p);
  if (t.copy != nullptr) store_any(t.copy + at, n, p);
  if (EIGHT) {
    store_codes<false>(static_cast<uint8_t*>(t.m) + at, t.m_scale + block, n, m);
    store_codes<true>(static_cast<uint8_t*>(t.v) + at, t.v_scale + block, n, r);
  } else {
    store_any(static_cast<float*>(t.m) + at, n, m);
    store_any(static_cast<float*>(t.v) + at, n, v);
  }
}

// ------------------------------------------------------------------ gradient norm

constexpr int kNormBlocks = 1024;  // partial sums of one launch

// Sum of squares of the block's chunks. fp32 within a thread (four sums, each of some 9,000 of
// 2^33 gradients on 152 SMs), double between threads and blocks, in a fixed order. A thread has the
// loads of four pieces of 8 gradients in flight.
constexpr int NORM_PIECES = 4;
constexpr int NORM_CHUNK = CHUNK * NORM_PIECES;

__device__ __forceinline__ void add_squares(const uint4& u, float (&s)[4], float) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) s[e] += __uint_as_float(w[e]) * __uint_as_float(w[e]);
}
__device__ __forceinline__ void add_squares(const uint4& u, float (&s)[4], __nv_bfloat16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float lo = __uint_as_float(w[e] << 16), hi = __uint_as_float(w[e] & 0xffff0000u);
    s[e] += lo * lo + hi * hi;
  }
}

template <int CAP, class G>
__global__ void __launch_bounds__(THREADS) square_sum_kernel(
    const __grid_constant__ Table<CAP> tab, double* partials) {
  __shared__ double red[THREADS / 32];
  pdl_wait();
  pdl_trigger();
  constexpr int LOADS = NORM_PIECES * PER_THREAD * int(sizeof(G)) / 16;  // 16 bytes each
  constexpr int VEC = 16 / int(sizeof(G));
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t chunk = blockIdx.x; chunk < tab.chunks; chunk += gridDim.x) {
    const Tensor& t = tab.t[find_tensor(tab, chunk)];
    const int64_t at = (chunk - t.first_chunk) * NORM_CHUNK;
    const G* src = static_cast<const G*>(t.grad) + at;
    const int64_t left = t.n - at;
    if (left >= NORM_CHUNK) {
      // plain loads: the step reads the gradients again
      uint4 u[LOADS];
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        u[i] = reinterpret_cast<const uint4*>(src)[i * THREADS + threadIdx.x];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) add_squares(u[i], s, G{});
    } else {
      for (int i = 0; i < LOADS; ++i) {
        const int64_t a = int64_t(i * THREADS + threadIdx.x) * VEC;
        if (a + VEC <= left) {
          add_squares(*reinterpret_cast<const uint4*>(src + a), s, G{});
        } else {
          for (int e = 0; e < VEC && a + e < left; ++e) {
            const float g = as_float(src[a + e]);
            s[e % 4] += g * g;
          }
        }
      }
    }
  }
  double d = (double(s[0]) + double(s[1])) + (double(s[2]) + double(s[3]));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    d = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) d += red[w];
    partials[blockIdx.x] = d;
  }
}

// out[0] = the norm, out[1] = min(1, max_norm / (norm + 1e-6)), NaN where the norm is not
// finite.
__global__ void __launch_bounds__(THREADS) norm_kernel(const double* partials, int count,
                                                       float max_norm, float* out) {
  __shared__ double red[THREADS];
  pdl_wait();
  pdl_trigger();
  double d = 0.0;
  for (int i = threadIdx.x; i < count; i += THREADS) d += partials[i];
  red[threadIdx.x] = d;
  __syncthreads();
  for (int o = THREADS / 2; o > 0; o >>= 1) {
    if (int(threadIdx.x) < o) red[threadIdx.x] += red[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const float norm = float(sqrt(red[0]));
    const bool finite = fabsf(norm) <= 3.402823466e38f;
    out[0] = norm;
    out[1] = finite ? fminf(1.f, max_norm / (norm + 1e-6f)) : __int_as_float(0x7fc00000);
  }
}

// ------------------------------------------------------------------ arguments

pb_status bad(pb_status s, int i, const char* what) {
  char msg[200];
  snprintf(msg, sizeof msg, "tensors[%d]: %s", i, what);
  return record_error(s, msg);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

pb_status cuda_failed(cudaError_t e, const char* what) {
  char msg[256];
  snprintf(msg, sizeof msg, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
  return record_error(PB_ERR_CUDA, msg);
}

pb_status sm_count(int* sms) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cudaGetDevice");
}

// The next tensors that have values, from `at` on, as a kernel's table.
template <int CAP>
void fill(Table<CAP>& tab, const pb_adamw_tensor* tensors, int count, int& at, int chunk = CHUNK) {
  tab.count = 0;
  tab.chunks = 0;
  for (; at < count && tab.count < CAP; ++at) {
    const pb_adamw_tensor& a = tensors[at];
    if (a.n == 0) continue;
    Tensor& t = tab.t[tab.count++];
    t = Tensor{a.param, static_cast<__nv_bfloat16*>(a.param_copy), a.grad, a.m, a.v, a.m_scale,
               a.v_scale, a.n, tab.chunks, a.weight_decay};
    tab.chunks += (a.n + chunk - 1) / chunk;
  }
}

template <int CAP, class P, class G, bool EIGHT>
cudaError_t launch_adamw(const Table<CAP>& tab, const Step& st, cudaStream_t stream) {
  return launch_dependent(adamw_kernel<CAP, P, G, EIGHT>, dim3(unsigned(tab.chunks), 1, 1),
                          dim3(THREADS, 1, 1), 0, 1, stream, tab, st);
}

template <int CAP>
cudaError_t launch_any(const Table<CAP>& tab, const Step& st, const pb_adamw_args& a,
                       cudaStream_t s) {
  const bool p16 = a.param_dtype == PB_DTYPE_BF16, g16 = a.grad_dtype == PB_DTYPE_BF16;
  using B = __nv_bfloat16;
  if (a.state_bits == 8) {
    if (p16)
      return g16 ? launch_adamw<CAP, B, B, true>(tab, st, s)
                 : launch_adamw<CAP, B, float, true>(tab, st, s);
    return g16 ? launch_adamw<CAP, float, B, true>(tab, st, s)
               : launch_adamw<CAP, float, float, true>(tab, st, s);
  }
  if (p16)
    return g16 ? launch_adamw<CAP, B, B, false>(tab, st, s)
               : launch_adamw<CAP, B, float, false>(tab, st, s);
  return g16 ? launch_adamw<CAP, float, B, false>(tab, st, s)
             : launch_adamw<CAP, float, float, false>(tab, st, s);
}

pb_status check_dtype(int32_t d, const char* what) {
  if (d == PB_DTYPE_BF16 || d == PB_DTYPE_FP32) return PB_OK;
  char msg[120];
  snprintf(msg, sizeof msg, "%s must be PB_DTYPE_FP32 or PB_DTYPE_BF16", what);
  return record_error(PB_ERR_UNSUPPORTED, msg);
}

pb_status check_list(const pb_adamw_tensor* tensors, int32_t count) {
  if (count < 0 || (count > 0 && tensors == nullptr))
    return record_error(PB_ERR_INVALID_ARG, "tensors is NULL or their number negative");
  for (int i = 0; i < count; ++i) {
    if (tensors[i].n < 0 || tensors[i].n > (int64_t(1) << 40))
      return bad(PB_ERR_INVALID_ARG, i, "n must be between 0 and 2^40");
    if (tensors[i].n > 0 && (tensors[i].grad == nullptr || !aligned16(tensors[i].grad)))
      return bad(PB_ERR_INVALID_ARG, i, "grad must be a 16-byte aligned device pointer");
  }
  return PB_OK;
}

// A buffer that the step writes or reads, for the check that no two of them overlap.
struct Span {
  uintptr_t a, b;
  int tensor;
  bool written;
};

}  // namespace
}  // namespace pb

using namespace pb;

extern "C" {

pb_status pb_adamw(const pb_adamw_args* args, int32_t n_tensors, const pb_adamw_tensor* tensors,
                   void* stream) {
  if (args == nullptr) return record_error(PB_ERR_INVALID_ARG, "args is NULL");
  const pb_adamw_args& a = *args;
  pb_status s = check_dtype(a.param_dtype, "param_dtype");
  if (s == PB_OK) s = check_dtype(a.grad_dtype, "grad_dtype");
  if (s != PB_OK) return s;
  if (a.state_bits != 8 && a.state_bits != 32)
    return record_error(PB_ERR_UNSUPPORTED, "state_bits must be 8 or 32");
  if (!(a.beta1 >= 0 && a.beta1 < 1 && a.beta2 >= 0 && a.beta2 < 1))
    return record_error(PB_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!(float(a.eps) >= 1.17549435e-38f && std::isfinite(a.eps)) || !std::isfinite(a.lr))
    return record_error(PB_ERR_INVALID_ARG, "eps must be finite and a normal fp32 number, lr finite");
  if (a.d_step == nullptr && a.step < 1)
    return record_error(PB_ERR_INVALID_ARG, "step counts from 1");
  const void* scalars[3] = {a.d_lr, a.d_step, a.d_grad_scale};
  for (const void* p : scalars)
    if ((reinterpret_cast<uintptr_t>(p) & 3) != 0)
      return record_error(PB_ERR_INVALID_ARG, "d_lr, d_step and d_grad_scale must be 4-byte aligned");
  s = check_list(tensors, n_tensors);
  if (s != PB_OK) return s;
  std::vector<Span> spans;
  try {
    spans.reserve(size_t(n_tensors) * 7 + 3);
  } catch (...) {
    return record_error(PB_ERR_INVALID_ARG, "host allocation for the checks failed");
  }
  const int64_t pe = a.param_dtype == PB_DTYPE_BF16 ? 2 : 4;
  const int64_t ge = a.grad_dtype == PB_DTYPE_BF16 ? 2 : 4;
  for (int i = 0; i < n_tensors; ++i) {
    const pb_adamw_tensor& t = tensors[i];
    if (!std::isfinite(t.weight_decay))
      return bad(PB_ERR_INVALID_ARG, i, "weight_decay must be finite");
    if (t.n == 0) continue;
    const int64_t blocks = (t.n + PB_ADAMW_BLOCK - 1) / PB_ADAMW_BLOCK;
    const void* need[3] = {t.param, t.m, t.v};
    for (const void* p : need)
      if (p == nullptr || !aligned16(p))
        return bad(PB_ERR_INVALID_ARG, i, "param, m and v must be 16-byte aligned device pointers");
    if (!aligned16(t.param_copy))
      return bad(PB_ERR_INVALID_ARG, i, "param_copy must be 16-byte aligned (or NULL)");
    if (t.param_copy != nullptr && a.param_dtype != PB_DTYPE_FP32)
      return bad(PB_ERR_INVALID_ARG, i, "param_copy goes with fp32 parameters");
    const float* scales[2] = {t.m_scale, t.v_scale};
    for (const float* p : scales) {
      if (a.state_bits == 8 && (p == nullptr || (reinterpret_cast<uintptr_t>(p) & 3) != 0))
        return bad(PB_ERR_INVALID_ARG, i, "8-bit states need 4-byte aligned m_scale and v_scale");
      if (a.state_bits == 32 && p != nullptr)
        return bad(PB_ERR_INVALID_ARG, i, "scales go with 8-bit states");
    }
    const int64_t se = a.state_bits == 8 ? 1 : 4;
    auto add = [&](const void* p, int64_t bytes, bool written) {
      if (p == nullptr) return;
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      spans.push_back(Span{at, at + uintptr_t(bytes), i, written});
    };
    add(t.param, t.n * pe, true);
    add(t.param_copy, t.n * 2, true);
    add(t.grad, t.n * ge, false);
    add(t.m, t.n * se, true);
    add(t.v, t.n * se, true);
    if (a.state_bits == 8) {
      add(t.m_scale, blocks * 4, true);
      add(t.v_scale, blocks * 4, true);
    }
  }
  for (const void* p : scalars)
    if (p != nullptr) {
      const uintptr_t at = reinterpret_cast<uintptr_t>(p);
      spans.push_back(Span{at, at + 4, -1, false});
    }
  // No written buffer shares bytes with another one: blocks work on all tensors at once, and
  // a tensor that is listed twice would be stepped twice in no order.
  std::sort(spans.begin(), spans.end(), [](const Span& x, const Span& y) { return x.a < y.a; });
  uintptr_t written_to = 0, any_to = 0;
  for (const Span& x : spans) {
    if (x.a < written_to || (x.written && x.a < any_to))
      return x.tensor < 0 ? record_error(PB_ERR_INVALID_ARG,
                                         "d_lr, d_step or d_grad_scale overlaps a tensor")
                          : bad(PB_ERR_INVALID_ARG, x.tensor,
                                "a buffer that the step writes overlaps another");
    any_to = std::max(any_to, x.b);
    if (x.written) written_to = std::max(written_to, x.b);
  }
  Step st{};
  st.lr = float(a.lr);
  st.beta1 = float(a.beta1);
  st.beta2 = float(a.beta2);
  st.eps = float(a.eps);
  st.one_minus_beta1 = float(1.0 - a.beta1);
  st.one_minus_beta2 = float(1.0 - a.beta2);
  st.log_beta1 = float(std::log(a.beta1));  // -inf for 0: the correction is then 1
  st.log_beta2 = float(std::log(a.beta2));
  if (a.d_step == nullptr) {
    st.correction1 = float(-1.0 / std::expm1(double(a.step) * std::log(a.beta1)));
    st.correction2 = float(-1.0 / std::expm1(double(a.step) * std::log(a.beta2)));
  }
  st.d_lr = a.d_lr;
  st.d_step = a.d_step;
  st.d_grad_scale = a.d_grad_scale;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  int at = 0;
  while (at < n_tensors) {
    cudaError_t e = cudaSuccess;
    if (n_tensors - at <= kFew) {
      Table<kFew> tab;
      fill(tab, tensors, n_tensors, at);
      if (tab.count > 0) e = launch_any(tab, st, a, cs);
    } else {
      Table<kMany> tab;
      fill(tab, tensors, n_tensors, at);
      if (tab.count > 0) e = launch_any(tab, st, a, cs);
    }
    if (e != cudaSuccess) return cuda_failed(e, "adamw launch");
  }
  return PB_OK;
}

pb_status pb_grad_norm_scratch_bytes(int32_t n_tensors, size_t* bytes) {
  if (bytes == nullptr) return record_error(PB_ERR_INVALID_ARG, "bytes is NULL");
  if (n_tensors < 0) return record_error(PB_ERR_INVALID_ARG, "n_tensors must be >= 0");
  const int64_t launches = std::max<int64_t>(1, (int64_t(n_tensors) + kMany - 1) / kMany);
  *bytes = size_t(launches) * kNormBlocks * sizeof(double);
  return PB_OK;
}

pb_status pb_grad_norm(int32_t n_tensors, const pb_adamw_tensor* tensors, int32_t grad_dtype,
                       float max_norm, float* out, void* scratch, size_t scratch_bytes,
                       void* stream) {
  pb_status s = check_dtype(grad_dtype, "grad_dtype");
  if (s == PB_OK) s = check_list(tensors, n_tensors);
  if (s != PB_OK) return s;
  if (!(max_norm > 0.f && std::isfinite(max_norm)))
    return record_error(PB_ERR_INVALID_ARG, "max_norm must be finite and > 0");
  if (out == nullptr || (reinterpret_cast<uintptr_t>(out) & 3) != 0)
    return record_error(PB_ERR_INVALID_ARG, "out must be a 4-byte aligned device pointer");
  size_t need = 0;
  s = pb_grad_norm_scratch_bytes(n_tensors, &need);
  if (s != PB_OK) return s;
  if (scratch == nullptr || (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
    return record_error(PB_ERR_INVALID_ARG, "scratch must be a 256-byte aligned device pointer");
  if (scratch_bytes < need)
    return record_error(PB_ERR_WORKSPACE, "scratch is smaller than pb_grad_norm_scratch_bytes");
  const uintptr_t o = reinterpret_cast<uintptr_t>(out), w = reinterpret_cast<uintptr_t>(scratch);
  if (o < w + need && w < o + 8)
    return record_error(PB_ERR_INVALID_ARG, "out overlaps scratch");
  for (int i = 0; i < n_tensors; ++i) {
    const uintptr_t g = reinterpret_cast<uintptr_t>(tensors[i].grad);
    const uintptr_t end = g + uintptr_t(tensors[i].n) * (grad_dtype == PB_DTYPE_BF16 ? 2 : 4);
    if (tensors[i].n > 0 && ((g < o + 8 && o < end) || (g < w + need && w < end)))
      return bad(PB_ERR_INVALID_ARG, i, "grad overlaps out or scratch");
  }
  int sms = 0;
  s = sm_count(&sms);
  if (s != PB_OK) return s;
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  double* partials = static_cast<double*>(scratch);
  int at = 0, count = 0;
  auto launch = [&](auto& tab) {
    const unsigned grid = unsigned(
        std::min<int64_t>(tab.chunks, std::min<int64_t>(kNormBlocks, int64_t(sms) * 6)));
    using T = std::remove_reference_t<decltype(tab)>;
    constexpr int CAP = int(sizeof(T::t) / sizeof(Tensor));
    const cudaError_t e = launch_dependent(
        grad_dtype == PB_DTYPE_BF16 ? square_sum_kernel<CAP, __nv_bfloat16>
                                    : square_sum_kernel<CAP, float>,
        dim3(grid, 1, 1), dim3(THREADS, 1, 1), 0, 1, cs, tab, partials + count);
    count += int(grid);
    return e;
  };
  while (at < n_tensors) {
    cudaError_t e = cudaSuccess;
    if (n_tensors - at <= kFew) {
      Table<kFew> tab;
      fill(tab, tensors, n_tensors, at, NORM_CHUNK);
      if (tab.count > 0) e = launch(tab);
    } else {
      Table<kMany> tab;
      fill(tab, tensors, n_tensors, at, NORM_CHUNK);
      if (tab.count > 0) e = launch(tab);
    }
    if (e != cudaSuccess) return cuda_failed(e, "gradient norm launch");
  }
  const cudaError_t e = launch_dependent(norm_kernel, dim3(1, 1, 1), dim3(THREADS, 1, 1), 0, 1, cs,
                                         partials, count, max_norm, out);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "gradient norm launch");
}

}  // extern "C"
