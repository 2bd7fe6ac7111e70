// linear.cu — the linear layer's kernels around its products (linear_gemm.cuh):
// the form for few tokens, the activation's backward pass, and the bias gradient.
//
// Few tokens (a decoding step): y = resid + act(x W + b) for up to 32 rows of x is bound by
// reading W once. A tile of the GEMM would hold 256 rows of A for it and leave most SMs
// without a tile, so here one CTA an SM takes an equal share of all (tile of output features,
// stage of k) steps, whatever tiles it cuts. One thread streams W (and x) through a ring of
// five shared-memory stages of 32 KB of W by TMA without a pause between tiles: four times the
// bytes in flight that the memory's latency asks for. Eight warps take 16 or 32 features each
// and multiply with mma.sync, W on the instruction's 16-row side and x on its 8-column side
// (the product's rate does not matter: 32 rows cost an eighth of the time that the loads
// take). ldmatrix reads both operands from the 128-byte swizzled boxes, transposing W where it
// is stored [K, N]; rows, columns and k outside the matrices arrive as zeros. A stage is 256
// features x 64 k of a [K, N] matrix and 128 x 128 of an [N, K] one, so that memory is read in
// runs of 512 or 256 bytes. Tiles that a CTA has whole are finished by it; of the others it
// leaves partial sums, which a second launch adds up in the CTAs' order.
//
// Measured (in a graph): 24 x 12288 x 12288 53.6 us, of which the products take 52 (5.8 TB/s, 86 %
// of a plain copy's rate); 1 x 8192 x 2048 7.4 us (4.5 TB/s: start and end of one launch are most
// of it).
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

// Values of W that equal shares have to take off the longest one for their second launch. Measured
// on 14 shapes for 1, 8 and 32 rows, equal shares against whole tiles: from 340,000 on they gain
// (10240 x 2048, 376,832: 11.1 against 12.8 us for one row, 15.8 against 21.7 for 32), at 81,920 they
// lose (8192 x 8192: 26.6 against 22.2, 30.3 against 26.2). Between, the row counts differ: 32 rows
// gain from 147,456 on (5120 x 5120: 15.9 against 17.1), 1 and 8 rows lose up to a fifth on two
// waves of tiles (20480 x 1024, 114,688: 10.9 against 9.1) and gain on one (2048 x 2048, 98,304: 4.8
// against 5.7; 1024 x 4096, 229,376: 4.1 against 9.5).
constexpr int64_t kFewMinGain = 3 << 15;
// A wide tile (eight multiplying warps) or a narrow one (four): where narrow tiles give the SMs
// one each at most, whole tiles need no second launch, and fewer SMs than all still draw the
// memory's whole rate.
template <int NT, bool KN, bool NARROW>
struct FewGeo {
  static constexpr int WARPS = NARROW ? 4 : 8;  // multiplying warps; one more is the producer's
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int COLS = few_cols(KN, NARROW);  // output features of a tile
  static constexpr int KS = few_ks(KN, NARROW);      // k of a stage
  static constexpr int RT = COLS / (16 * WARPS);     // 16-feature rows of a warp
  static constexpr int W_BYTES = COLS * KS * 2;
  static constexpr int X_BYTES = 8 * NT * 128;  // a box of 64 k x 8 NT rows of x
  static constexpr int STAGE_BYTES = W_BYTES + KS / 64 * X_BYTES;
  static constexpr int STAGES = NARROW ? 8 : 5;
  // per warp, for the results: [8 NT tokens][16 RT features] floats
  static constexpr int OUT_BYTES = 8 * NT * 16 * RT * 4;
  static constexpr int SMEM = 1024 + STAGES * STAGE_BYTES + WARPS * OUT_BYTES;
  static_assert(SMEM + 1024 <= 227 * 1024, "shared memory");
};

// Up to 8 values of 16 bits, the first n of them; zero behind.
__device__ __forceinline__ uint4 ld_part(const uint16_t* p, int n) {
  if (n >= 8) return __ldcg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = (2 * i < n ? uint32_t(__ldcg(p + 2 * i)) : 0u) |
           (2 * i + 1 < n ? uint32_t(__ldcg(p + 2 * i + 1)) << 16 : 0u);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, "
        "%7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit values; lane 8 i + j gives the address of row j of matrix i.
template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// 16-byte piece j of row r of a box whose rows are 128 bytes, in the 128-byte swizzle.
__device__ __forceinline__ uint32_t swizzled(uint32_t box, int r, int j) {
  return box + uint32_t(r * 128 + ((j ^ (r & 7)) << 4));
}

// The results at (m + i step, n) from their sums z[i], those below M. All that is read is
// loaded before anything is stored (the compiler has to take a store for a write to it).
template <bool F16, int COUNT>
__device__ __forceinline__ void finish_values(const LinearEpi& e, int M, int m, int step, int n,
                                              float bias, float (&z)[COUNT]) {
  float a[COUNT], r[COUNT];
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    const int64_t row = m + i * step;
    const bool live = row < M;
    a[i] = e.mul != nullptr && live
               ? to_float<F16>(static_cast<const uint16_t*>(e.mul)[row * e.ld_mul + n])
               : 0.f;
    r[i] = e.resid == nullptr || !live ? 0.f
           : e.resid_f32 ? static_cast<const float*>(e.resid)[row * e.ld_resid + n]
                         : to_float<F16>(static_cast<const uint16_t*>(e.resid)[row * e.ld_resid + n]);
  }
#pragma unroll
  for (int i = 0; i < COUNT; ++i) {
    const int64_t row = m + i * step;
    if (row >= M) break;
    const float pre = z[i] + bias;
    if (e.pre != nullptr)
      static_cast<uint16_t*>(e.pre)[row * e.ld_pre + n] = from_float<F16>(pre);
    float y = e.mul != nullptr ? pre * act_grad(e.act, a[i]) : act_value(e.act, pre);
    if (e.resid != nullptr) y += r[i];
    if (e.y32 != nullptr)
      e.y32[row * e.ldy + n] = y;
    else
      static_cast<uint16_t*>(e.y16)[row * e.ldy + n] = from_float<F16>(y);
  }
}
template <bool F16>
__device__ __forceinline__ float bias_at(const LinearEpi& e, int n, int N) {
  return e.bias != nullptr && n < N ? to_float<F16>(static_cast<const uint16_t*>(e.bias)[n]) : 0.f;
}

// CTA c does steps [c W, (c + 1) W) of the tiles' steps (`total` stages each) in order.
// partials: [CTA][2 slots][8 NT][COLS]; slot 1 for the tile whose first stage the CTA has.
template <int NT, bool KN, bool F16, bool NARROW>
__global__ void __launch_bounds__(FewGeo<NT, KN, NARROW>::THREADS, 1)
    few_kernel(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
               const __grid_constant__ FewParams p, int total, int64_t all, int64_t W,
               float* partials, int* status, uint64_t limit_ns) {
  using G = FewGeo<NT, KN, NARROW>;
  constexpr int STAGES = G::STAGES, RT = G::RT, KS = G::KS;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * STAGES];
  __shared__ int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + STAGES);
  const int warp = int(threadIdx.x) >> 5, lane = int(threadIdx.x) & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, G::WARPS);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{&abort_flag, status, limit_ns};
  int64_t it = int64_t(blockIdx.x) * W;
  const int64_t it_end = min(all, it + W);
  int tile = int(it / total), k = int(it - int64_t(tile) * total);
  int stage = 0;
  uint32_t phase = 0;

  if (warp == G::WARPS) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      uint32_t last_par[STAGES];
      uint32_t used = 0;
      for (; it < it_end; ++it) {
        if (!mbar_wait(empty0 + 8 * stage, phase ^ 1, wc, 1)) break;
        const uint32_t w = smem_u32(smem + size_t(stage) * G::STAGE_BYTES);
        const uint32_t x = w + G::W_BYTES, bar = full0 + 8 * stage;
        const int n0 = tile * G::COLS, k0 = k * KS;
        mbar_arrive_expect_tx(bar, G::STAGE_BYTES);
        if (KN) {  // boxes of 64 features x KS k
#pragma unroll
          for (int i = 0; i < G::COLS / 64; ++i)
            tma_load_2d(w + i * (G::W_BYTES / (G::COLS / 64)), &tm_w, bar, n0 + 64 * i, k0);
        } else {   // boxes of 64 k x COLS features
#pragma unroll
          for (int i = 0; i < KS / 64; ++i)
            tma_load_2d(w + i * (G::W_BYTES / (KS / 64)), &tm_w, bar, k0 + 64 * i, n0);
        }
#pragma unroll
        for (int i = 0; i < KS / 64; ++i)
          tma_load_2d(x + i * G::X_BYTES, &tm_x, bar, k0 + 64 * i, 0);
        last_par[stage] = phase;
        used |= 1u << stage;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
        if (++k == total) {
          k = 0;
          ++tile;
        }
      }
      // every copy has landed before the CTA leaves
      for (int i = 0; i < STAGES; ++i)
        if (used & (1u << i))
          mbar_wait_drain(full0 + 8 * i, last_par[i],
                          limit_ns > kDrainFloorNs ? limit_ns : kDrainFloorNs);
    }
    __syncwarp();
    return;
  }
  // ---------------------------------------------------------------- products
  const int mi = lane >> 3, mr = lane & 7;  // the matrix and row this lane addresses
  const int g = lane >> 2, t = lane & 3;
  float* out = reinterpret_cast<float*>(smem + STAGES * G::STAGE_BYTES + warp * G::OUT_BYTES);
  while (it < it_end) {
    const int k_first = k;
    const int k_last = int(min(int64_t(total), k + (it_end - it)));
    float acc[RT][NT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[r][j][e] = 0.f;
    for (; k < k_last; ++k) {
      if (!mbar_wait_warp(full0 + 8 * stage, phase, wc, 2)) return;
      const uint32_t w = smem_u32(smem + size_t(stage) * G::STAGE_BYTES);
      // A stage's sums by themselves, then added: the tensor core cuts sums off instead of
      // rounding them, which a chain over all of K would pile up (1.2e-6 of an fp32 result at
      // K = 4096 against 0.2e-6).
      float sum[RT][NT][4];
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) sum[r][j][e] = 0.f;
#pragma unroll
      for (int h = 0; h < KS / 32; ++h) {  // 32 k
        const uint32_t x = w + G::W_BYTES + (h >> 1) * G::X_BYTES;
        uint32_t b[NT][4];  // x: 8 tokens x 32 k
#pragma unroll
        for (int j = 0; j < NT; ++j)
          ldmatrix4<false>(swizzled(x, 8 * j + mr, 4 * (h & 1) + mi), b[j]);
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)  // 16 k
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const int f = 16 * (RT * warp + r);  // first feature
            uint32_t a[4];
            if (KN)  // a box for every 64 features; its rows are k, pieces 8 features
              ldmatrix4<true>(swizzled(w + (f >> 6) * (G::W_BYTES / (G::COLS / 64)),
                                       32 * h + 16 * hh + 8 * (mi >> 1) + mr,
                                       (f & 63) / 8 + (mi & 1)),
                              a);
            else     // a box for every 64 k; its rows are features, pieces 8 k
              ldmatrix4<false>(swizzled(w + (h >> 1) * (G::W_BYTES / (KS / 64)),
                                        f + 8 * (mi & 1) + mr,
                                        4 * (h & 1) + 2 * hh + (mi >> 1)),
                               a);
#pragma unroll
            for (int j = 0; j < NT; ++j)
              mma16816<F16>(sum[r][j], a, b[j][2 * hh], b[j][2 * hh + 1]);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * stage);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[r][j][e] += sum[r][j][e];
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    // the warp's results [token][feature], so that lanes go along the features
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = 8 * j + 2 * t, f = 16 * r + g;
        out[m * (16 * RT) + f] = acc[r][j][0];
        out[(m + 1) * (16 * RT) + f] = acc[r][j][1];
        out[m * (16 * RT) + f + 8] = acc[r][j][2];
        out[(m + 1) * (16 * RT) + f + 8] = acc[r][j][3];
      }
    __syncwarp();
    const bool whole = k_first == 0 && k_last == total;
    const int f = lane % (16 * RT), nf = 16 * RT * warp + f;
    const int n = tile * G::COLS + nf;
    float* part = partials + (size_t(blockIdx.x) * 2 + (k_first == 0 ? 1 : 0)) * (8 * NT * G::COLS);
    constexpr int STEP = 2 / RT;  // tokens the warp's lanes take at a time
    const int m0 = lane / (16 * RT);
    if (!whole) {
#pragma unroll 4
      for (int m = m0; m < p.M; m += STEP) __stcg(part + m * G::COLS + nf, out[m * (16 * RT) + f]);
    } else if (n < p.N) {
      const float bias = bias_at<F16>(p.epi, n, p.N);
      for (int m = m0; m < p.M; m += 4 * STEP) {
        float z[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) z[i] = out[min(m + i * STEP, 8 * NT - 1) * (16 * RT) + f];
        finish_values<F16>(p.epi, p.M, m, STEP, n, bias, z);
      }
    }
    __syncwarp();
    it += k_last - k_first;
    k = 0;
    ++tile;
  }
}

// The tiles that several CTAs share: a thread adds up one value.
template <int NT, bool KN, bool F16, bool NARROW>
__global__ void __launch_bounds__(256)
    few_finish_kernel(const __grid_constant__ FewParams p, int total, int64_t W,
                      const float* partials) {
  using G = FewGeo<NT, KN, NARROW>;
  pdl_wait();  // the products' launch is complete
  pdl_trigger();
  const int n = int(blockIdx.x) * 256 + int(threadIdx.x), m = int(blockIdx.y);
  if (n >= p.N) return;
  const int tile = n / G::COLS;
  const int64_t it0 = int64_t(tile) * total;
  const int first = int(it0 / W), last = int((it0 + total - 1) / W);
  if (first == last) return;
  const float bias = bias_at<F16>(p.epi, n, p.N);
  float z[1] = {0.f};
#pragma unroll 8
  for (int c = first; c <= last; ++c)
    z[0] += __ldcg(partials + (size_t(c) * 2 + (c == first ? 1 : 0)) * (8 * NT * G::COLS) +
                m * G::COLS + n % G::COLS);
  finish_values<F16>(p.epi, p.M, m, 1, n, bias, z);
}

template <int NT, bool KN, bool F16, bool NARROW>
cudaError_t launch_few(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const FewParams& p,
                       float* scratch, int* status, uint64_t limit_ns, cudaStream_t stream) {
  using G = FewGeo<NT, KN, NARROW>;
  static PerDeviceInit setup;  // per device: shared-memory opt-in; value: number of SMs
  int sms = 0;
  const cudaError_t err = per_device_init(
      setup,
      [](int dev, int* out) {
        const cudaError_t e = cudaFuncSetAttribute(
            few_kernel<NT, KN, F16, NARROW>, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
        if (e != cudaSuccess) return e;
        return cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
      },
      &sms);
  if (err != cudaSuccess) return err;
  const int64_t tiles = (p.N + G::COLS - 1) / G::COLS;
  const int total = (p.K + G::KS - 1) / G::KS;
  const int64_t all = tiles * total;
  // whole tiles, or equal shares where these are shorter by what the second launch costs
  int64_t W = (tiles + sms - 1) / sms * total;
  const int64_t even = (all + sms - 1) / sms;
  if (scratch != nullptr && (W - even) * G::KS * G::COLS >= kFewMinGain &&
      kLinearScratchBytes >= size_t(sms) * 2 * 8 * NT * G::COLS * 4)
    W = even;
  const unsigned grid = unsigned((all + W - 1) / W);
  const cudaError_t e = launch_dependent(few_kernel<NT, KN, F16, NARROW>, dim3(grid, 1, 1),
                                         dim3(G::THREADS, 1, 1), G::SMEM, 1, stream, tm_x, tm_w, p,
                                         total, all, W, scratch, status, limit_ns);
  if (e != cudaSuccess || W % total == 0) return e;
  return launch_dependent(few_finish_kernel<NT, KN, F16, NARROW>,
                          dim3(unsigned((p.N + 255) / 256), unsigned(p.M), 1), dim3(256, 1, 1), 0, 1,
                          stream, p, total, W, scratch);
}

template <bool KN, bool F16, bool NARROW>
cudaError_t launch_few_rows(const CUtensorMap& tm_x, const CUtensorMap& tm_w, const FewParams& p,
                            float* s, int* status, uint64_t limit_ns, cudaStream_t stream) {
  switch (few_box_rows(p.M)) {
    case 8: return launch_few<1, KN, F16, NARROW>(tm_x, tm_w, p, s, status, limit_ns, stream);
    case 16: return launch_few<2, KN, F16, NARROW>(tm_x, tm_w, p, s, status, limit_ns, stream);
    case 24: return launch_few<3, KN, F16, NARROW>(tm_x, tm_w, p, s, status, limit_ns, stream);
    default: return launch_few<4, KN, F16, NARROW>(tm_x, tm_w, p, s, status, limit_ns, stream);
  }
}

template <bool F16>
cudaError_t launch_few_any(bool b_mn, bool narrow, const CUtensorMap& tm_x, const CUtensorMap& tm_w,
                           const FewParams& p, float* s, int* status, uint64_t limit_ns,
                           cudaStream_t stream) {
  if (b_mn)
    return narrow ? launch_few_rows<true, F16, true>(tm_x, tm_w, p, s, status, limit_ns, stream)
                  : launch_few_rows<true, F16, false>(tm_x, tm_w, p, s, status, limit_ns, stream);
  return narrow ? launch_few_rows<false, F16, true>(tm_x, tm_w, p, s, status, limit_ns, stream)
                : launch_few_rows<false, F16, false>(tm_x, tm_w, p, s, status, limit_ns, stream);
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

// Cluster: 64 columns; its CTAs: equal parts of the rows; 8 threads across (16 bytes each), 32
// rows at a time, four such loads of a thread in flight. Sums over a CTA's threads, then over
// the cluster in distributed shared memory, in a fixed order.
//
// beside: the launch before on the stream is linear_kernel, of which the sums need
// nothing. Its blocks have all passed their pdl_wait when this one begins, so everything before
// it is complete; it itself is only waited for at the end, so that this launch is not complete
// before it. The sums then fill SMs that its last tiles leave idle (777 x 4104 x 2056 backward:
// 7.1 us in front of it, 1.3 beside). Values are read from the L2 cache, where all that
// is complete has arrived.
constexpr int SUM_COLS = 64;
template <bool F16>
__global__ void __launch_bounds__(256)
    row_sum_kernel(const uint16_t* m, int64_t rows, int64_t cols, int64_t ld, int parts, float* out,
                   bool accumulate, bool beside) {
  __shared__ float red[8][SUM_COLS];
  if (!beside) pdl_wait();
  pdl_trigger();
  const int tx = int(threadIdx.x) & 7, ty = int(threadIdx.x) >> 3;
  const int rank = int(blockIdx.x) % parts;
  const int64_t c0 = int64_t(blockIdx.x) / parts * SUM_COLS, c = c0 + tx * 8;
  const int64_t per = (rows + parts - 1) / parts;
  const int64_t r0 = rank * per, r1 = min(rows, r0 + per);
  const int n = int(max(int64_t(0), min(int64_t(8), cols - c)));
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = 0.f;
  auto add = [&](const uint4& u) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s[2 * i] += to_float<F16>(uint16_t(w[i]));
      s[2 * i + 1] += to_float<F16>(uint16_t(w[i] >> 16));
    }
  };
  if (n > 0) {
    const uint16_t* p = m + c;
    int64_t r = r0 + ty;
    for (; r + 96 < r1; r += 128) {
      uint4 u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) u[i] = ld_part(p + (r + 32 * i) * ld, n);
#pragma unroll
      for (int i = 0; i < 4; ++i) add(u[i]);
    }
    for (; r < r1; r += 32) add(ld_part(p + r * ld, n));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    for (int o = 8; o < 32; o <<= 1) s[i] += __shfl_xor_sync(0xffffffffu, s[i], o);
  if ((threadIdx.x & 31) < 8) {
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.x >> 5][tx * 8 + i] = s[i];
  }
  __syncthreads();
  float v = 0.f;
  if (threadIdx.x < SUM_COLS) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v += red[k][threadIdx.x];
  }
  if (parts > 1) {
    __syncthreads();
    if (threadIdx.x < SUM_COLS) red[0][threadIdx.x] = v;
    __syncthreads();
    cluster_sync();
    if (rank == 0 && threadIdx.x < SUM_COLS) {
      v = 0.f;
      for (int k = 0; k < parts; ++k)
        v += ld_cluster_f32(mapa_shared(smem_u32(&red[0][threadIdx.x]), uint32_t(k)));
    }
    __syncthreads();
    cluster_sync();  // no CTA leaves while its sums may still be read
  }
  if (rank == 0 && threadIdx.x < SUM_COLS && c0 + threadIdx.x < cols)
    out[c0 + threadIdx.x] = accumulate ? __ldcg(out + c0 + threadIdx.x) + v : v;
  if (beside) pdl_wait();
}

}  // namespace

cudaError_t launch_linear_few(OpType op, bool b_mn, bool narrow, const CUtensorMap& tmA,
                              const CUtensorMap& tmB, const FewParams& p, void* scratch,
                              int* status, uint64_t limit_ns, cudaStream_t stream) {
  if (p.M < 1 || p.M > kFewRows || p.N < 1 || p.K < 1) return cudaErrorInvalidValue;
  float* s = static_cast<float*>(scratch);
  return op == kOpF16
             ? launch_few_any<true>(b_mn, narrow, tmA, tmB, p, s, status, limit_ns, stream)
             : launch_few_any<false>(b_mn, narrow, tmA, tmB, p, s, status, limit_ns, stream);
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

cudaError_t launch_row_sums(OpType op, const RowSums& s, bool beside, cudaStream_t stream) {
  if (s.rows < 1 || s.cols < 1) return cudaSuccess;
  // up to eight CTAs share a cluster's rows, 128 rows each at least
  const int parts = s.rows >= 1024 ? 8 : s.rows <= 128 ? 1 : int(s.rows / 128);
  const dim3 grid(unsigned((s.cols + SUM_COLS - 1) / SUM_COLS) * unsigned(parts), 1, 1);
  return launch_dependent(op == kOpF16 ? row_sum_kernel<true> : row_sum_kernel<false>, grid,
                          dim3(256, 1, 1), 0, unsigned(parts), stream,
                          static_cast<const uint16_t*>(s.m), s.rows, s.cols, s.ld, parts, s.out,
                          s.accumulate, beside);
}

}  // namespace pb
