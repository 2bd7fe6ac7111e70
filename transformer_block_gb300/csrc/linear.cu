// linear.cu — the linear layer's kernels around its tensor-core GEMM (gemm.cu, kEpiLinear):
// the form for few tokens, the activation's backward pass, and the bias gradient.
//
// Few tokens (a decoding step): y = resid + act(x W + b) for up to 32 rows of x is bound by
// reading W once. A tile of the GEMM would hold 256 rows of A for it and leave most SMs
// without a tile, so here a warp takes 64 output features and a share of K, loads W straight
// into registers, 16 bytes a lane and 4 KB a warp in flight, and multiplies with mma.sync (a
// register operand needs no shared memory, and the product's rate does not matter: 32 rows
// cost an eighth of what the loads leave time for). W takes the instruction's 16-row side and
// x its 8-column side. The sum over k may run in any order as long as both operands keep the
// same one, so lane (g, t) of the fragments takes the eight consecutive k from 8 t on:
//   W stored [N, K]: 16 bytes of row g and of row g + 8 of a tile are its fragments;
//   W stored [K, N]: eight k-rows' 16 bytes at column 8 g hold columns (2 r, 2 r + 1) of
//     8 g as tile r's rows g and g + 8; byte permutes pair two k-rows' halves.
// The eight warps of a CTA take every eighth step of 32 k, the CTAs of a cluster equal parts of
// K; partial sums meet in shared memory, then over the cluster, in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "ptx.cuh"

namespace pb {
namespace {

// ------------------------------------------------------------------ activations
// In fp32 with CUDA's own functions: these kernels wait for memory. Past +-80 every
// derivative equals its limit; holding z there keeps infinity times zero away.
constexpr float kFar = 80.f;
constexpr float kTanhC = 0.7978845608028654f, kTanhA = 0.044715f;

__device__ float act_value(int act, float z) {
  switch (act) {
    case kActGelu:
      return z > kFar ? z : z < -kFar ? -0.f : 0.5f * z * erfcf(-0.70710678118654752f * z);
    case kActGeluTanh: {
      if (fabsf(z) > kFar) return z > 0.f ? z : -0.f;
      return z / (1.f + expf(-2.f * kTanhC * (z + kTanhA * z * z * z)));
    }
    case kActSilu:
      return z < -kFar ? -0.f : z / (1.f + expf(-z));
    case kActRelu:
      return z < 0.f ? 0.f : z;
    default:
      return z;
  }
}

__device__ float act_grad(int act, float zz) {
  const float z = fabsf(zz) > kFar ? copysignf(kFar, zz) : zz;
  switch (act) {
    case kActGelu:
      return 0.5f * erfcf(-0.70710678118654752f * z) +
             z * 0.39894228040143268f * expf(-0.5f * z * z);
    case kActGeluTanh: {
      const float s = 1.f / (1.f + expf(-2.f * kTanhC * (z + kTanhA * z * z * z)));
      return s + z * s * (1.f - s) * 2.f * kTanhC * (1.f + 3.f * kTanhA * z * z);
    }
    case kActSilu: {
      const float s = 1.f / (1.f + expf(-z));
      return s * (1.f + z * (1.f - s));
    }
    case kActRelu:
      return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    default:
      return 1.f;
  }
}

template <bool F16>
__device__ __forceinline__ float to_float(uint16_t x) {
  if (F16) return __half2float(__ushort_as_half(x));
  return __uint_as_float(uint32_t(x) << 16);
}
template <bool F16>
__device__ __forceinline__ uint16_t from_float(float x) {
  if (F16) return __half_as_ushort(__float2half_rn(x));
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// ------------------------------------------------------------------ few tokens

constexpr int FEW_WARPS = 8, FEW_THREADS = 32 * FEW_WARPS;
constexpr int FEW_COLS = 64;      // output features of a CTA
constexpr int FEW_STEP = 32;      // k of one step of a warp
constexpr int FEW_PITCH = 68;     // floats a token's row of partial sums takes: no bank twice

__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 u;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "l"(p));
  return u;
}

// Up to 8 values of 16 bits, the first n of them; zero behind.
__device__ __forceinline__ uint4 ld_part(const uint16_t* p, int n) {
  if (n >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (2 * i < n ? uint32_t(__ldg(p + 2 * i)) : 0u) |
           (2 * i + 1 < n ? uint32_t(__ldg(p + 2 * i + 1)) << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, "
        "%7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// One step's operands of a lane: eight 16-byte pieces of W, one of x for every 8 tokens.
template <int NT>
struct FewStep {
  uint4 w[8];
  uint4 x[NT];
};

template <int NT, bool KN>
__device__ __forceinline__ void few_load(const FewParams& p, int n0, int k0, int g, int t,
                                         FewStep<NT>& s) {
  const uint16_t* b = static_cast<const uint16_t*>(p.b);
  const uint16_t* a = static_cast<const uint16_t*>(p.a);
  const int k = k0 + 8 * t;
  if (n0 + FEW_COLS <= p.N && k0 + FEW_STEP <= p.K) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      s.w[i] = KN ? ld_stream(b + int64_t(k + i) * p.ldb + n0 + 8 * g)
                  : ld_stream(b + int64_t(n0 + 8 * i + g) * p.ldb + k);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (KN) {
        const int n = k + i < p.K ? p.N - (n0 + 8 * g) : 0;
        s.w[i] = n > 0 ? ld_part(b + int64_t(k + i) * p.ldb + n0 + 8 * g, n)
                       : make_uint4(0, 0, 0, 0);
      } else {
        const int row = n0 + 8 * i + g;
        const int n = row < p.N ? p.K - k : 0;
        s.w[i] = n > 0 ? ld_part(b + int64_t(row) * p.ldb + k, n) : make_uint4(0, 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int m = 8 * j + g;
    const int n = m < p.M ? p.K - k : 0;
    s.x[j] = n > 0 ? ld_part(a + int64_t(m) * p.lda + k, n) : make_uint4(0, 0, 0, 0);
  }
}

template <int NT, bool KN, bool F16>
__device__ __forceinline__ void few_multiply(const FewStep<NT>& s, float (&acc)[4][NT][4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {  // k 4 h .. 4 h + 3 of the lane's eight
#pragma unroll
    for (int r = 0; r < 4; ++r) {  // 16 features
      uint32_t a0, a1, a2, a3;
      if (KN) {
        auto word = [&](int row) {
          const uint4& u = s.w[row];
          return r == 0 ? u.x : r == 1 ? u.y : r == 2 ? u.z : u.w;
        };
        const uint32_t w0 = word(4 * h), w1 = word(4 * h + 1), w2 = word(4 * h + 2),
                       w3 = word(4 * h + 3);
        a0 = __byte_perm(w0, w1, 0x5410);
        a1 = __byte_perm(w0, w1, 0x7632);
        a2 = __byte_perm(w2, w3, 0x5410);
        a3 = __byte_perm(w2, w3, 0x7632);
      } else {
        const uint4 &lo = s.w[2 * r], &hi = s.w[2 * r + 1];
        a0 = h ? lo.z : lo.x;
        a1 = h ? hi.z : hi.x;
        a2 = h ? lo.w : lo.y;
        a3 = h ? hi.w : hi.y;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
        mma16816<F16>(acc[r][j], a0, a1, a2, a3, h ? s.x[j].z : s.x[j].x,
                      h ? s.x[j].w : s.x[j].y);
    }
  }
}

// grid: tiles of FEW_COLS features x cluster size; steps: k-steps of one CTA's part of K.
template <int NT, bool KN, bool F16>
__global__ void __launch_bounds__(FEW_THREADS, 2)
    few_kernel(const __grid_constant__ FewParams p, int splits, int steps) {
  extern __shared__ float red[];  // [FEW_WARPS][8 NT][FEW_PITCH]
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  const int g = lane >> 2, t = lane & 3;
  const int rank = int(blockIdx.x) % splits;
  const int n0 = int(blockIdx.x) / splits * FEW_COLS;
  const int total = (p.K + FEW_STEP - 1) / FEW_STEP;
  const int end = min(total, (rank + 1) * steps);
  float acc[4][NT][4];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[r][j][e] = 0.f;
  int k = rank * steps + warp;
  if constexpr (NT <= 2) {  // the next step's loads are in flight during a step's products
    FewStep<NT> now, next;
    if (k < end) few_load<NT, KN>(p, n0, k * FEW_STEP, g, t, now);
    for (; k < end; k += FEW_WARPS) {
      if (k + FEW_WARPS < end)
        few_load<NT, KN>(p, n0, (k + FEW_WARPS) * FEW_STEP, g, t, next);
      few_multiply<NT, KN, F16>(now, acc);
      now = next;
    }
  } else {  // the sums take the registers for that; sixteen warps cover one another's loads
    FewStep<NT> now;
    for (; k < end; k += FEW_WARPS) {
      few_load<NT, KN>(p, n0, k * FEW_STEP, g, t, now);
      few_multiply<NT, KN, F16>(now, acc);
    }
  }
  // partial sums [token][feature] of every warp
  float* mine = red + warp * (8 * NT * FEW_PITCH);
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int m = 8 * j + 2 * t;
      const int f0 = KN ? 8 * g + 2 * r : 16 * r + g, f1 = KN ? f0 + 1 : f0 + 8;
      mine[m * FEW_PITCH + f0] = acc[r][j][0];
      mine[(m + 1) * FEW_PITCH + f0] = acc[r][j][1];
      mine[m * FEW_PITCH + f1] = acc[r][j][2];
      mine[(m + 1) * FEW_PITCH + f1] = acc[r][j][3];
    }
  __syncthreads();
  const int f = int(threadIdx.x) % FEW_COLS, m_first = int(threadIdx.x) / FEW_COLS;
  constexpr int ROWS = FEW_THREADS / FEW_COLS;
  if (splits > 1) {
    // the CTA's sums replace warp 0's; then every CTA of the cluster finishes some tokens
#pragma unroll
    for (int m = m_first; m < 8 * NT; m += ROWS) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < FEW_WARPS; ++w) s += red[(w * 8 * NT + m) * FEW_PITCH + f];
      red[m * FEW_PITCH + f] = s;  // read and written by this thread alone
    }
    cluster_sync();
  }
  const int n = n0 + f;
  const LinearEpi& e = p.epi;
  const uint32_t base = smem_u32(red);
  for (int m = m_first + (splits > 1 ? rank * ROWS : 0); m < p.M;
       m += ROWS * (splits > 1 ? splits : 1)) {
    float z = 0.f;
    if (splits > 1) {
      for (int r = 0; r < splits; ++r)
        z += ld_cluster_f32(mapa_shared(base + uint32_t(m * FEW_PITCH + f) * 4u, uint32_t(r)));
    } else {
#pragma unroll
      for (int w = 0; w < FEW_WARPS; ++w) z += red[(w * 8 * NT + m) * FEW_PITCH + f];
    }
    if (n >= p.N) continue;
    if (e.bias != nullptr) z += to_float<F16>(static_cast<const uint16_t*>(e.bias)[n]);
    if (e.pre != nullptr)
      static_cast<uint16_t*>(e.pre)[int64_t(m) * e.ld_pre + n] = from_float<F16>(z);
    float y;
    if (e.mul != nullptr)
      y = z * act_grad(e.act, to_float<F16>(
                                  static_cast<const uint16_t*>(e.mul)[int64_t(m) * e.ld_mul + n]));
    else
      y = act_value(e.act, z);
    if (e.resid != nullptr) {
      const int64_t at = int64_t(m) * e.ld_resid + n;
      y += e.resid_f32 ? static_cast<const float*>(e.resid)[at]
                       : to_float<F16>(static_cast<const uint16_t*>(e.resid)[at]);
    }
    if (e.y32 != nullptr)
      e.y32[int64_t(m) * e.ldy + n] = y;
    else
      static_cast<uint16_t*>(e.y16)[int64_t(m) * e.ldy + n] = from_float<F16>(y);
  }
  if (splits > 1) cluster_sync();  // no CTA leaves while its sums may still be read
}

template <int NT, bool KN, bool F16>
cudaError_t launch_few(const FewParams& p, cudaStream_t stream) {
  constexpr int SMEM = FEW_WARPS * 8 * NT * FEW_PITCH * 4;
  static PerDeviceInit setup;  // per device: shared-memory opt-in; value: number of SMs
  int sms = 0;
  const cudaError_t err = per_device_init(
      setup,
      [](int dev, int* out) {
        const cudaError_t e = cudaFuncSetAttribute(
            few_kernel<NT, KN, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
        if (e != cudaSuccess) return e;
        return cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
      },
      &sms);
  if (err != cudaSuccess) return err;
  const int tiles = (p.N + FEW_COLS - 1) / FEW_COLS;
  const int total = (p.K + FEW_STEP - 1) / FEW_STEP;
  // CTAs of a cluster that share a tile's K: as many as give the shortest sequence of waves
  // over the two resident CTAs an SM, with a hundredth of a tile's time for each more, and two
  // steps of every warp at least
  const int slots = 2 * sms;
  int splits = 1;
  double best = 1e30;
  for (int s = 1; s <= 8 && (s == 1 || total >= s * 2 * FEW_WARPS); ++s) {
    const double cost = double((int64_t(tiles) * s + slots - 1) / slots) / s + 0.01 * s;
    if (cost < best) {
      best = cost;
      splits = s;
    }
  }
  const int steps = (total + splits - 1) / splits;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = unsigned(splits);
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(tiles) * unsigned(splits), 1, 1);
  cfg.blockDim = dim3(FEW_THREADS, 1, 1);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, few_kernel<NT, KN, F16>, p, splits, steps);
}

template <bool KN, bool F16>
cudaError_t launch_few_rows(const FewParams& p, cudaStream_t stream) {
  if (p.M <= 8) return launch_few<1, KN, F16>(p, stream);
  if (p.M <= 16) return launch_few<2, KN, F16>(p, stream);
  if (p.M <= 24) return launch_few<3, KN, F16>(p, stream);
  return launch_few<4, KN, F16>(p, stream);
}

// ------------------------------------------------------------------ activation backward

template <bool F16>
__global__ void __launch_bounds__(256)
    act_backward_kernel(int act, int64_t rows, int64_t cols, const uint16_t* dy, int64_t ld_dy,
                        const uint16_t* pre, int64_t ld_pre, uint16_t* out, int64_t ld_out) {
  const int64_t c = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * 8;
  if (c >= cols) return;
  const int n = int(min(int64_t(8), cols - c));
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const uint16_t *d = dy + r * ld_dy + c, *z = pre + r * ld_pre + c;
    uint16_t* o = out + r * ld_out + c;
    if (n == 8) {
      const uint4 du = *reinterpret_cast<const uint4*>(d), zu = *reinterpret_cast<const uint4*>(z);
      const uint32_t dw[4] = {du.x, du.y, du.z, du.w}, zw[4] = {zu.x, zu.y, zu.z, zu.w};
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = to_float<F16>(uint16_t(dw[i])) * act_grad(act, to_float<F16>(uint16_t(zw[i])));
        const float b = to_float<F16>(uint16_t(dw[i] >> 16)) *
                        act_grad(act, to_float<F16>(uint16_t(zw[i] >> 16)));
        w[i] = F16 ? pack_f16x2(a, b) : pack_bf16x2(a, b);
      }
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      for (int i = 0; i < n; ++i)
        o[i] = from_float<F16>(to_float<F16>(d[i]) * act_grad(act, to_float<F16>(z[i])));
    }
  }
}

// ------------------------------------------------------------------ sums over the rows

// Block (x, y): columns [256 x, 256 x + 256), the y-th of gridDim.y parts of the rows; 32
// threads across (8 columns each), 8 rows at a time.
template <bool F16>
__global__ void __launch_bounds__(256)
    row_sum_kernel(const uint16_t* m, int64_t rows, int64_t cols, int64_t ld, float* partials) {
  __shared__ float red[8][32][9];
  const int tx = int(threadIdx.x) & 31, ty = int(threadIdx.x) >> 5;
  const int64_t c = int64_t(blockIdx.x) * 256 + tx * 8;
  const int64_t per = (rows + gridDim.y - 1) / gridDim.y;
  const int64_t r0 = int64_t(blockIdx.y) * per, r1 = min(rows, r0 + per);
  const int n = int(max(int64_t(0), min(int64_t(8), cols - c)));
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
  if (n > 0)
    for (int64_t r = r0 + ty; r < r1; r += 8) {
      const uint4 u = ld_part(m + r * ld + c, n);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        s[2 * i] += to_float<F16>(uint16_t(w[i]));
        s[2 * i + 1] += to_float<F16>(uint16_t(w[i] >> 16));
      }
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) red[ty][tx][i] = s[i];
  __syncthreads();
  // thread k of the block: column k
  const int64_t col = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (col < cols) {
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][threadIdx.x / 8][threadIdx.x % 8];
    partials[int64_t(blockIdx.y) * cols + col] = v;
  }
}

__global__ void __launch_bounds__(256)
    row_sum_final_kernel(const float* partials, int parts, int64_t cols, float* out,
                         bool accumulate) {
  const int64_t c = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (c >= cols) return;
  float s = 0.f;
  for (int k = 0; k < parts; ++k) s += partials[int64_t(k) * cols + c];
  out[c] = accumulate ? out[c] + s : s;
}

}  // namespace

cudaError_t launch_linear_few(OpType op, bool b_mn, const FewParams& p, cudaStream_t stream) {
  if (p.M < 1 || p.M > kFewRows || p.N < 1 || p.K < 1) return cudaErrorInvalidValue;
  if (op == kOpF16)
    return b_mn ? launch_few_rows<true, true>(p, stream) : launch_few_rows<false, true>(p, stream);
  return b_mn ? launch_few_rows<true, false>(p, stream) : launch_few_rows<false, false>(p, stream);
}

cudaError_t launch_act_backward(OpType op, int act, int64_t rows, int64_t cols, const void* dy,
                                int64_t ld_dy, const void* pre, int64_t ld_pre, void* out,
                                int64_t ld_out, cudaStream_t stream) {
  if (rows < 1 || cols < 1) return cudaSuccess;
  const dim3 grid(unsigned((cols + 2047) / 2048), unsigned(rows < 65535 ? rows : 65535));
  const auto *d = static_cast<const uint16_t*>(dy), *z = static_cast<const uint16_t*>(pre);
  auto* o = static_cast<uint16_t*>(out);
  if (op == kOpF16)
    act_backward_kernel<true><<<grid, 256, 0, stream>>>(act, rows, cols, d, ld_dy, z, ld_pre, o,
                                                        ld_out);
  else
    act_backward_kernel<false><<<grid, 256, 0, stream>>>(act, rows, cols, d, ld_dy, z, ld_pre, o,
                                                         ld_out);
  return cudaGetLastError();
}

cudaError_t launch_row_sums(OpType op, const void* m, int64_t rows, int64_t cols, int64_t ld,
                            float* partials, float* out, bool accumulate, cudaStream_t stream) {
  if (rows < 1 || cols < 1) return cudaSuccess;
  // 32 rows a part at least, and no more parts than kSumBlocks
  const int64_t want = (rows + 31) / 32;
  const unsigned parts = unsigned(want < kSumBlocks ? want : kSumBlocks);
  const unsigned blocks = unsigned((cols + 255) / 256);
  const auto* src = static_cast<const uint16_t*>(m);
  if (op == kOpF16)
    row_sum_kernel<true><<<dim3(blocks, parts), 256, 0, stream>>>(src, rows, cols, ld, partials);
  else
    row_sum_kernel<false><<<dim3(blocks, parts), 256, 0, stream>>>(src, rows, cols, ld, partials);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  row_sum_final_kernel<<<blocks, 256, 0, stream>>>(partials, int(parts), cols, out, accumulate);
  return cudaGetLastError();
}

}  // namespace pb
