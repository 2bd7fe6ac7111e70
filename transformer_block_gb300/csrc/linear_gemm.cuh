// linear_gemm.cuh — the linear layer's products on CTA pairs: y = resid + act(x W + b), dx = dy
// W^T act'(pre) and dW = x^T dy, for any M, N and K. Part of gemm.cu (inside its namespace): the
// same pair tiles, tcgen05 products, TMA ring and stores, with other epilogues and another
// division of the work.
//
// * One launch may hold two products (the backward pass's dx and dW), so the tiles of one fill
//   the waves of the other (36 tiles of 65 k-blocks and 153 of 13: 33 us; apart 25, split along K
//   and summed, and 22).
// * Tiles that would leave pairs idle are split along K; the parts' sums go to scratch and a
//   second launch over all SMs adds them up in a fixed order and finishes the tiles. Nothing
//   waits inside a launch, whatever else runs on the GPU.
// * fp32 results: the tensor core cuts its sums off instead of rounding them, which leaves 1.0e-6
//   of relative error at K = 1024 and, growing with K, 8.6e-6 at 8192, against 0.3e-6 and 1.1e-6
//   of a chain of fp32 fused multiply-adds. So an accumulator sums 896 k at most, and the
//   epilogue warps add such segments up in registers, rounding, while the products go on in the
//   other accumulator (2048 x 2048 x 8192: 42.8 us in one chain, 43.3 in segments of 1792 k, 44.9
//   of 896). 16-bit results take longer segments: the cut, 1.05e-9 of the sum for each k, stays
//   below 1/64 of half a step (fp16 2^-11: 7,168 k; bf16 2^-8: 57,344 k). In one chain a result lost
//   1.4e-4 of itself at K = 131,072 (fp16) and 5.4e-4 at 524,288 (bf16).
// * Eight epilogue warps, each quarter of the tensor memory's lanes shared by two: four do not
//   hide a pre-activation's loads and GeLU' behind a main loop of K = 2048 (8192 x 8192 x 2048:
//   224 us with four, 176 with eight).
//
// Bound by the tensor rate for many tokens: 8192 x 20480 x 5120 with GeLU and the stored
// pre-activation runs at 1790 to 1885 TFLOP/s in short bursts (94 to 99 % of cuBLAS's measured
// 1904), 1570 to 1630 over seconds, where the power limit holds both down. A single wave costs
// 6.5 us (launch, first loads, epilogue, stores) and 0.27 us a k-block for one pair, near the 0.25
// that an SM takes for its 32 KB of operands from the L2 cache; with all pairs at work and operands
// that come from memory 0.33 to 0.41. Fetching them into the L2 cache ahead of the loads costs that
// path twice (2056 x 4104 for 777 rows: 25 us without, 34 with).

namespace {

constexpr int LIN_EPI = 8;                      // epilogue warps
constexpr int LIN_THREADS = 64 + 32 * LIN_EPI;  // and producer and MMA issuer
constexpr int LIN_STAGES = 6;
constexpr int LIN_STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int LIN_BARS = 2 * LIN_STAGES + 5;
// 1024-byte aligned: the TMA-store buffers (64-byte swizzle), 4 KB an epilogue warp
constexpr size_t LIN_OUT_OFF =
    (size_t(LIN_STAGES) * LIN_STAGE_BYTES + 8 * LIN_BARS + 16 + 1023) / 1024 * 1024;
constexpr size_t LIN_SMEM = 1024 + LIN_OUT_OFF + LIN_EPI * 4096;
static_assert(LIN_SMEM <= 227 * 1024, "shared memory of the linear kernel");

// k-blocks (of 64) that one accumulator sums at most, for each type of result.
constexpr int kLinearSegment = 14, kLinearSegmentF16 = 112, kLinearSegmentBf16 = 896;
// k-blocks (0.28 us each) that a part of a split tile has at least, and that splitting has to
// save at least: partial sums and second launch cost 3 to 15 us. Measured over k for 100 to 500 rows
// on 1024 to 8192 features, split against whole: eight parts even at a saving of 25 (256 x 2048 x
// 2048, saving 28: 13.3 against 14.3 us), four at 22, three at 23 (100 x 6144 x 2560, saving 26:
// 16.4 against 16.9), two only at 40 to 60 (256 x 8192 x 3584, saving 28: 24.0 against 21.6; x 8192,
// saving 64: 38.2 against 40.8).
constexpr int kLinearMinBlocks = 4, kLinearMinGain = 28;

// One product D[M, N] = A B^T and its epilogue.
struct LinearJob {
  CUtensorMap tm_a, tm_b, tm_y, tm_pre;
  LinearEpi epi;
  int M, N, num_m, num_n, num_kb;
  int seg;          // k-blocks of one accumulator
  bool a_mn, b_mn;  // operand stored [K, M] / [K, N]
};

// Units of work of one kind: whole tiles (split 1), or parts of W k-blocks of tiles split along
// K, unit t being part t % split of tile first_tile + t / split, its sums in slot slot0 + t.
struct LinearClass {
  int job, first_tile, units, split, W, slot0;
};

// The units of class 0 go round the pairs; those of class 1, not longer, first to the pairs from
// `late` on, which have one of class 0 less, `catch_up` each, then round all.
struct LinearWork {
  LinearJob job[2];
  LinearClass cls[2];
  int late, catch_up;
  float* partials;
};

struct LinearUnit {
  int job, row0, tn, kb0, kb1;
  int slot;  // of its partial sums, -1: a whole tile
};

struct LinearIter {
  int phase, t;
  __device__ explicit LinearIter(int pair) : phase(0), t(pair) {}
  __device__ bool next(const LinearWork& w, int pair, int pairs, LinearUnit& u) {
    if (phase == 0) {
      if (t < w.cls[0].units) {
        make(w, 0, t, u);
        t += pairs;
        return true;
      }
      phase = 1;
      t = w.catch_up > 0 && pair >= w.late ? 0 : w.catch_up;
    }
    const int behind = pairs - w.late;  // pairs that catch up
    if (phase == 1) {
      const int at = (pair - w.late) + t * behind;
      if (t < w.catch_up && at < w.cls[1].units) {
        make(w, 1, at, u);
        ++t;
        return true;
      }
      phase = 2;
      t = w.catch_up * behind + pair;
    }
    if (t >= w.cls[1].units) return false;
    make(w, 1, t, u);
    t += pairs;
    return true;
  }
  __device__ static void make(const LinearWork& w, int c, int t, LinearUnit& u) {
    const LinearClass& k = w.cls[c];
    const LinearJob& jb = w.job[k.job];
    const int tile = k.split > 1 ? t / k.split : t, part = t - tile * k.split;
    int tm;
    tile_coords(k.first_tile + tile, jb.num_m, jb.num_n, kGroupM, tm, u.tn);
    u.job = k.job;
    u.row0 = tm * PM;
    u.kb0 = part * k.W;
    u.kb1 = k.split > 1 ? min(jb.num_kb, u.kb0 + k.W) : jb.num_kb;
    u.slot = k.split > 1 ? k.slot0 + t : -1;
  }
};

// Beyond |z| = kActFar every activation and derivative here equals its limit in fp32 (GeLU's
// tails end at 13, the tanh form's at 9; SiLU's is 1e-33 there): z is held at that bound, so
// an infinite z meets no infinity times zero. NaN stays NaN.
constexpr float kActFar = 80.f;
__device__ __forceinline__ float act_held(float z) {
  return fabsf(z) > kActFar ? copysignf(kActFar, z) : z;
}
// 1 / (1 + exp(-z)) from the approximate exponential and reciprocal (2^-22 relative).
__device__ __forceinline__ float sigmoid_approx(float z) {
  return rcp_approx(1.f + ex2_approx(-1.4426950408889634f * z));
}
// GeLU's tanh form is z sigmoid(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3).
constexpr float kTanh2C = 1.5957691216057308f, kTanhA = 0.044715f;

// GELU for fp32 and fp16 results. gemm.cu's erf terms have an absolute error of 1.5e-7: 5e-5 of
// GELU's value at z = -3 and 4.7e-4 at -4, a tenth of a bf16 step but all of fp16's half step. Here
// the normal distribution's tail is held relative to its size: for a >= 0
//   Phi(-a) = exp(-a^2 / 2) t P(t),  t = 1 / (1 + a / 4),
// P of degree 8 fitted to Phi(-a) exp(a^2 / 2) / t over a <= 14 (behind it the exponential is 0)
// by least squares with weights moved towards an equal relative error: 5.7e-8 (8.4e-8 with the
// rounded coefficients). In fp32 Phi(-a) is then off by at most (1.25 a^2 + 24) 2^-24 of itself: the
// exponent's three roundings, times a^2 / 2; t's (3 with the reciprocal's two) times at most 3.2,
// the exponential's 4, and the sum's. CUDA's erfc is as exact, but its instructions do not hide
// behind the products (8192 x 8192 x 2048 in fp16: 389 us with it, 232 with this, 230 with the
// short form).
__device__ __forceinline__ void phi_terms(float z0, float z1, uint64_t& q, uint64_t& e) {
  constexpr float kP[9] = {0.09979748f,  0.09851684f,  0.10374665f,  0.03292815f, 0.20175754f,
                           -0.20578194f, 0.29612058f, -0.15280867f, 0.025723346f};
  constexpr float kHalfLog2e = 0.72134752f;
  const uint64_t a = f2(fabsf(z0), fabsf(z1));
  float d0, d1;
  f2_split(f2_fma(a, f2(0.25f, 0.25f), f2(1.f, 1.f)), d0, d1);
  const uint64_t t = f2(rcp_approx(d0), rcp_approx(d1));
  uint64_t p = f2(kP[8], kP[8]);
#pragma unroll
  for (int k = 7; k >= 0; --k) p = f2_fma(p, t, f2(kP[k], kP[k]));
  f2_split(f2_mul(f2_mul(a, a), f2(-kHalfLog2e, -kHalfLog2e)), d0, d1);
  e = f2(ex2_approx(d0), ex2_approx(d1));
  q = f2_mul(f2_mul(p, t), e);
}
__device__ __forceinline__ void gelu_pair_full(float& z0, float& z1) {
  uint64_t q, e;
  phi_terms(z0, z1, q, e);
  float h0, h1;
  f2_split(f2_mul(f2(z0, z1), q), h0, h1);
  z0 = z0 >= 0.f ? z0 - h0 : h0;
  z1 = z1 >= 0.f ? z1 - h1 : h1;
}
__device__ __forceinline__ void gelu_grad_pair_full(float& d0, float& d1, float z0, float z1) {
  constexpr float kRsqrt2pi = 0.39894228040143268f;
  uint64_t q, e;
  phi_terms(z0, z1, q, e);
  float q0, q1, g0, g1;
  f2_split(q, q0, q1);
  f2_split(f2_fma(f2(z0 * kRsqrt2pi, z1 * kRsqrt2pi), e,
                  f2(z0 >= 0.f ? 1.f - q0 : q0, z1 >= 0.f ? 1.f - q1 : q1)),
           g0, g1);
  d0 *= g0;
  d1 *= g1;
}

template <bool FULL, int N>
__device__ __forceinline__ void gelu_apply(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float a = act_held(v[i]), b = act_held(v[i + 1]);
    if (FULL)
      gelu_pair_full(a, b);
    else
      gelu_pair(a, b);
    v[i] = v[i] > kActFar ? v[i] : a;
    v[i + 1] = v[i + 1] > kActFar ? v[i + 1] : b;
  }
}

// full: GELU's relative form, for fp32 and fp16 results.
template <int N>
__device__ __forceinline__ void act_apply(int act, bool full, float (&v)[N]) {
  if (act == kActNone) return;
  if (act == kActGelu) {
    if (full)
      gelu_apply<true>(v);
    else
      gelu_apply<false>(v);
  } else if (act == kActGeluTanh) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = act_held(v[i]);
      const float a = z * sigmoid_approx(kTanh2C * (z + kTanhA * z * z * z));
      v[i] = v[i] > kActFar ? v[i] : a;
    }
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = act_held(v[i]);
      const float a = z * sigmoid_approx(z);
      v[i] = v[i] > kActFar ? v[i] : a;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];
  }
}

// d *= act'(z). FULL: for fp16 results.
template <bool FULL, int N>
__device__ __forceinline__ void act_grad_apply(int act, float (&d)[N], const float (&zs)[N]) {
  if (act == kActGelu) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if (FULL)
        gelu_grad_pair_full(d[i], d[i + 1], act_held(zs[i]), act_held(zs[i + 1]));
      else
        gelu_grad_pair(d[i], d[i + 1], act_held(zs[i]), act_held(zs[i + 1]));
    }
  } else if (act == kActGeluTanh) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = act_held(zs[i]);
      const float s = sigmoid_approx(kTanh2C * (z + kTanhA * z * z * z));
      d[i] *= s + z * s * (1.f - s) * kTanh2C * (1.f + 3.f * kTanhA * z * z);
    }
  } else if (act == kActSilu) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float z = act_held(zs[i]), s = sigmoid_approx(z);
      d[i] *= s * (1.f + z * (1.f - s));
    }
  } else if (act == kActRelu) {
#pragma unroll
    for (int i = 0; i < N; ++i) d[i] = zs[i] > 0.f ? d[i] : zs[i] <= 0.f ? 0.f : zs[i];
  }
}

// 32 values of 16 bits from src (64 bytes, 16-byte aligned) or the first n of them.
template <bool F16>
__device__ __forceinline__ void load_row16(const void* src, int n, float (&v)[32]) {
  const uint16_t* s = static_cast<const uint16_t*>(src);
  uint32_t w[16];
  if (n >= 32) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint4 u = reinterpret_cast<const uint4*>(s)[q];
      w[4 * q] = u.x;
      w[4 * q + 1] = u.y;
      w[4 * q + 2] = u.z;
      w[4 * q + 3] = u.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      w[i] = (2 * i < n ? uint32_t(s[2 * i]) : 0u) |
             (2 * i + 1 < n ? uint32_t(s[2 * i + 1]) << 16 : 0u);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    if (F16) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    } else {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

// Without TMA: fp32 result of a warp's 32 x 32 chunk at y (row stride ld), of which `rows` rows
// and n columns are inside the matrix: through shared memory, so that a store instruction writes
// whole 128-byte rows. stage: the warp's 4 KB (its TMA-store buffers); 16-byte piece q of row r
// sits at piece q ^ (r & 7), so neither the rows' writes nor the reads meet a bank twice.
__device__ __forceinline__ void linear_store_f32(float* y, int64_t ld, int rows, int n,
                                                 bool accumulate, const float (&v)[32],
                                                 uint32_t stage) {
  const int lane = int(threadIdx.x & 31);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                     stage + uint32_t(lane * 128 + ((q ^ (lane & 7)) << 4))),
                 "f"(v[4 * q]), "f"(v[4 * q + 1]), "f"(v[4 * q + 2]), "f"(v[4 * q + 3])
                 : "memory");
  __syncwarp();
  const int r0 = lane >> 3, q = lane & 7;  // this lane's first row and its piece of every fourth
  float* dst = y + r0 * ld + 4 * q;
  const int left = n - 4 * q;  // columns from this lane's first on
#pragma unroll
  for (int it = 0; it < 8; ++it, dst += 4 * ld) {
    const int r = 4 * it + r0;
    float4 o;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(o.x), "=f"(o.y), "=f"(o.z), "=f"(o.w)
                 : "r"(stage + uint32_t(r * 128 + ((q ^ (r & 7)) << 4)))
                 : "memory");
    if (r >= rows) continue;
    if (left >= 4) {
      if (accumulate) {
        const float4 a = *reinterpret_cast<const float4*>(dst);
        o.x += a.x;
        o.y += a.y;
        o.z += a.z;
        o.w += a.w;
      }
      *reinterpret_cast<float4*>(dst) = o;
    } else {
      const float w[3] = {o.x, o.y, o.z};
#pragma unroll
      for (int e = 0; e < 3; ++e)
        if (e < left) dst[e] = accumulate ? dst[e] + w[e] : w[e];
    }
  }
  __syncwarp();  // the buffer may be written again
}

// Warp-wide: the warp's 32 rows of 16 fp32 columns at col0 (lane l holds row row0 + l) to the
// tensor of `tm`, or added to it, by one TMA copy from the buffers of tma_store_rows32 (their rows
// are 64 bytes, too). One launch adds to an element once, so the order of adds does not matter.
__device__ __forceinline__ void tma_store_f32x16(StoreStage& ss, const CUtensorMap* tm, int row0,
                                                 int col0, bool add, const float* v) {
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t buf = ss.base + (ss.n & 1u) * 2048u;
  if (ss.n >= 2) {  // the buffer's previous store (two ago) must have read it
    if (lane == 0) bulk_wait_read_1();
    __syncwarp();
  }
  const uint32_t rb = buf + lane * 64u, sw = (lane >> 1) & 3u;
#pragma unroll
  for (uint32_t j = 0; j < 4; ++j)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(rb + ((j ^ sw) << 4)),
                 "f"(v[4 * j]), "f"(v[4 * j + 1]), "f"(v[4 * j + 2]), "f"(v[4 * j + 3])
                 : "memory");
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add)
      tma_reduce_add_2d(tm, buf, col0, row0);
    else
      tma_store_2d(tm, buf, col0, row0);
    bulk_commit();
  }
  ++ss.n;
}

// fp32 result of a warp's 32 rows x 32 columns, n of them inside the matrix. A TMA store cuts a
// box off at the last column only to 16 bytes: where the columns end inside those, the last
// chunk is stored by its lanes.
__device__ __forceinline__ void linear_store32(StoreStage& ss, const CUtensorMap* tm, float* y,
                                               int64_t ld, int row0, int col0, int M, int n,
                                               bool accumulate, const float (&v)[32]) {
  if (row0 >= M) return;
  if (n >= 32 || n % 4 == 0) {
    tma_store_f32x16(ss, tm, row0, col0, accumulate, v);
    if (n > 16) tma_store_f32x16(ss, tm, row0, col0 + 16, accumulate, v + 16);
    return;
  }
  if (ss.n > 0) {  // the TMA stores read the same shared memory
    if ((threadIdx.x & 31) == 0) bulk_wait_read();
    __syncwarp();
  }
  linear_store_f32(y + int64_t(row0) * ld + col0, ld, M - row0, n, accumulate, v, ss.base);
}

// 16-bit result of a warp's 32 rows x 32 columns, n of them inside the matrix. A TMA store
// cuts a box off at the last column only to 16 bytes: where the columns end inside those, the
// last chunk is stored by its lanes.
template <bool F16>
__device__ __forceinline__ void linear_store16(StoreStage& ss, const CUtensorMap* tm, void* dst,
                                               int64_t ld, int row0, int col0, int M, int n,
                                               const float (&v)[32]) {
  uint32_t w[16];
  pack_words16<F16>(v, w);
  if (n >= 32 || n % 8 == 0) {
    tma_store_rows32(ss, tm, row0, col0, M, w);
    return;
  }
  const int row = row0 + int(threadIdx.x & 31);
  if (row < M) {
    uint16_t* d = static_cast<uint16_t*>(dst) + int64_t(row) * ld + col0;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < n) d[i] = uint16_t(w[i / 2] >> (16 * (i % 2)));
  }
}

// A lane's 32 columns of part of a tile, for linear_finish_kernel: in 16-byte pieces in the
// order [piece of a row][row], so a warp's accesses are whole 512-byte runs.
__device__ __forceinline__ void linear_store_part(float* dst, const float (&v)[32]) {
  float4* d4 = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int q = 0; q < 8; ++q)
    __stcg(d4 + 32 * q, make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]));
}

// fp32 results that are the product and nothing else.
__device__ __forceinline__ bool linear_plain(const LinearEpi& e) {
  return e.y32 != nullptr && e.act == kActNone && e.bias == nullptr && e.mul == nullptr &&
         e.resid == nullptr && e.pre == nullptr;
}

// Warp-wide, lane l holding row `row` = the warp's first row + l of columns [col0, col0 + 32).
template <bool F16>
__device__ __forceinline__ void linear_epilogue32(const LinearEpi& e, const LinearJob& jb, int M,
                                                  int N, int row, int col0, float (&v)[32],
                                                  StoreStage& ss) {
  const int row0 = row - int(threadIdx.x & 31);
  if (row0 >= M) return;
  const bool live = row < M;
  const int n = N - col0;
  if (e.bias != nullptr) {
    float b[32];
    load_row16<F16>(static_cast<const uint16_t*>(e.bias) + col0, n, b);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += b[i];
  }
  if (e.pre != nullptr)
    linear_store16<F16>(ss, &jb.tm_pre, e.pre, e.ld_pre, row0, col0, M, n, v);
  if (e.mul != nullptr) {
    if (live) {
      float z[32];
      load_row16<F16>(static_cast<const uint16_t*>(e.mul) + int64_t(row) * e.ld_mul + col0, n, z);
      act_grad_apply<F16>(e.act, v, z);
    }
  } else {
    act_apply(e.act, F16 || e.y32 != nullptr, v);
  }
  if (e.resid != nullptr && live) {
    if (e.resid_f32) {
      const float* r = static_cast<const float*>(e.resid) + int64_t(row) * e.ld_resid + col0;
      if (n >= 32) {
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 f = reinterpret_cast<const float4*>(r)[q];
          v[4 * q] += f.x;
          v[4 * q + 1] += f.y;
          v[4 * q + 2] += f.z;
          v[4 * q + 3] += f.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i)
          if (i < n) v[i] += r[i];
      }
    } else {
      float r[32];
      load_row16<F16>(static_cast<const uint16_t*>(e.resid) + int64_t(row) * e.ld_resid + col0, n,
                      r);
#pragma unroll
      for (int i = 0; i < 32; ++i) v[i] += r[i];
    }
  }
  if (e.y32 != nullptr) {
    linear_store32(ss, &jb.tm_y, e.y32, e.ldy, row0, col0, M, n, e.accumulate, v);
  } else {
    linear_store16<F16>(ss, &jb.tm_y, e.y16, e.ldy, row0, col0, M, n, v);
  }
}

// The ring of operand stages, as the producer or the MMA issuer goes through it.
struct LinearRing {
  uint32_t smem, full0, empty0, full_pair0;  // full_pair0: the even CTA's barriers
  int stage;
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if (++stage == LIN_STAGES) {
      stage = 0;
      phase ^= 1;
    }
  }
};

// Producer: the unit's k-blocks. The operand layouts are template parameters of this and of
// linear_multiply, chosen for each unit: as run-time flags inside the loops they slow a k-block
// from 0.28 to 0.33 us.
template <bool A_MN, bool B_MN>
__device__ __forceinline__ bool linear_load(const LinearJob& jb, LinearRing& ring,
                                            const LinearUnit& u, int m0, int n0, bool leader,
                                            const WaitCtl& wc, uint32_t (&last_par)[LIN_STAGES],
                                            uint32_t& used) {
  for (int kb = u.kb0; kb < u.kb1; ++kb) {
    if (!mbar_wait(ring.empty0 + 8 * ring.stage, ring.phase ^ 1, wc, 1)) return false;
    const uint32_t sa = ring.smem + uint32_t(ring.stage) * LIN_STAGE_BYTES, sb = sa + A_BYTES;
    const uint32_t bar = ring.full_pair0 + 8 * ring.stage;
    if (leader) mbar_arrive_expect_tx(ring.full0 + 8 * ring.stage, 2u * LIN_STAGE_BYTES);
    // K-major: one box of 128 rows x 64 k; MN-major: two of 64 k-rows x 64 elements of M (or N),
    // 8 KB apart
    if (A_MN) {
      tma_load_2d_pair(sa, &jb.tm_a, bar, m0, kb * BK);
      tma_load_2d_pair(sa + A_BYTES / 2, &jb.tm_a, bar, m0 + 64, kb * BK);
    } else {
      tma_load_2d_pair(sa, &jb.tm_a, bar, kb * BK, m0);
    }
    if (B_MN) {
      tma_load_2d_pair(sb, &jb.tm_b, bar, n0, kb * BK);
      tma_load_2d_pair(sb + B_BYTES / 2, &jb.tm_b, bar, n0 + 64, kb * BK);
    } else {
      tma_load_2d_pair(sb, &jb.tm_b, bar, kb * BK, n0);
    }
    last_par[ring.stage] = ring.phase;
    used |= 1u << ring.stage;
    ring.next();
  }
  return true;
}

// MMA issuer: `blocks` k-blocks into one accumulator, from zero.
template <bool F16, bool A_MN, bool B_MN>
__device__ __forceinline__ bool linear_multiply(LinearRing& ring, int blocks, uint32_t d_tmem,
                                                const WaitCtl& wc) {
  constexpr uint32_t idesc = idesc_f32acc(PM, BN, F16, A_MN, B_MN);
  // descriptor start-address step of one MMA (K = 16): along a swizzled row (K-major) or two
  // 1024-byte atoms on (MN-major), in 16-byte units
  constexpr uint64_t kStepA = A_MN ? 128 : 2, kStepB = B_MN ? 128 : 2;
  for (int kb = 0; kb < blocks; ++kb) {
    if (!mbar_wait(ring.full0 + 8 * ring.stage, ring.phase, wc, 3)) return false;
    tc_fence_after();
    const uint32_t sa = ring.smem + uint32_t(ring.stage) * LIN_STAGE_BYTES, sb = sa + A_BYTES;
    const uint64_t da = A_MN ? sdesc_mnmajor_sw128(sa, A_BYTES / 2) : sdesc_kmajor_sw128(sa);
    const uint64_t db = B_MN ? sdesc_mnmajor_sw128(sb, B_BYTES / 2) : sdesc_kmajor_sw128(sb);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      mma_f16kind_ss_pair(d_tmem, da + kStepA * k, db + kStepB * k, idesc, kb > 0 || k > 0);
    mma_commit_pair(ring.empty0 + 8 * ring.stage, 0x3);
    ring.next();
  }
  return true;
}

// Warps: 0 TMA producer (both CTAs), 1 MMA issuer (even CTA) and tensor-memory owner, 2-9
// epilogue; the pair protocol is gemm_kernel's.
template <bool F16>
__global__ void __launch_bounds__(LIN_THREADS, 1)
    linear_kernel(const __grid_constant__ LinearWork work, int* status, uint64_t limit_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + size_t(LIN_STAGES) * LIN_STAGE_BYTES);
  const uint32_t full0 = smem_u32(bars);                         // [LIN_STAGES]
  const uint32_t empty0 = smem_u32(bars + LIN_STAGES);           // [LIN_STAGES]
  const uint32_t tfull0 = smem_u32(bars + 2 * LIN_STAGES);       // [2] accumulator ready
  const uint32_t tempty0 = smem_u32(bars + 2 * LIN_STAGES + 2);  // [2] accumulator drained
  const uint32_t drain_bar = smem_u32(bars + 2 * LIN_STAGES + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + LIN_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t warp = warp_id(), lane = lane_id();
  const uint32_t rank = cluster_ctarank();
  const bool leader = (rank == 0);
  if (threadIdx.x == 0) {
    for (int s = 0; s < LIN_STAGES; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull0 + 8 * a, 1);
      mbar_init(tempty0 + 8 * a, 2 * LIN_EPI);  // the epilogue warps of both CTAs
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&work.job[work.cls[0].job].tm_a);
    tma_prefetch_desc(&work.job[work.cls[0].job].tm_b);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before any remote arrive
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  const WaitCtl wc{abort_flag, status, limit_ns};
  const uint64_t drain_ns = limit_ns > kDrainFloorNs ? limit_ns : kDrainFloorNs;
  const int pair = int(blockIdx.x) >> 1, pairs = int(gridDim.x) >> 1;

  if (warp == 0) {
    if (lane == 0) {
      // ------------------------------------------------------------ TMA producer
      uint32_t last_par[LIN_STAGES];
      uint32_t used = 0;
      LinearRing ring{smem_u32(smem), full0, empty0, mapa_shared(full0, 0), 0, 0u};
      bool ok = true;
      LinearIter it(pair);
      LinearUnit u;
      while (ok && it.next(work, pair, pairs, u)) {
        const LinearJob& jb = work.job[u.job];
        const int m0 = u.row0 + int(rank) * BM;
        const int n0 = u.tn * BN + int(rank) * (BN / 2);
        if (jb.a_mn)
          ok = linear_load<true, true>(jb, ring, u, m0, n0, leader, wc, last_par, used);
        else if (jb.b_mn)
          ok = linear_load<false, true>(jb, ring, u, m0, n0, leader, wc, last_par, used);
        else
          ok = linear_load<false, false>(jb, ring, u, m0, n0, leader, wc, last_par, used);
      }
      // every copy of the pair lands before either CTA exits: the even CTA's barriers count the
      // odd CTA's bytes too, and the odd CTA is held at the last cluster barrier until then
      if (leader)
        for (int s = 0; s < LIN_STAGES; ++s)
          if (used & (1u << s)) mbar_wait_drain(full0 + 8 * s, last_par[s], drain_ns);
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ------------------------------------------------------------ MMA issuer
      LinearRing ring{smem_u32(smem), full0, empty0, 0u, 0, 0u};
      int acc = 0;
      uint32_t acc_par = 0;
      bool ok = true;
      LinearIter it(pair);
      LinearUnit u;
      while (ok && it.next(work, pair, pairs, u)) {
        const LinearJob& jb = work.job[u.job];
        const int seg = jb.seg;
        // every seg k-blocks of the unit to the other accumulator
        for (int ks = u.kb0; ok && ks < u.kb1; ks += seg) {
          const int ke = min(u.kb1, ks + seg);
          if (!mbar_wait(tempty0 + 8 * acc, acc_par ^ 1, wc, 2)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + uint32_t(acc * BN);
          if (jb.a_mn)
            ok = linear_multiply<F16, true, true>(ring, ke - ks, d_tmem, wc);
          else if (jb.b_mn)
            ok = linear_multiply<F16, false, true>(ring, ke - ks, d_tmem, wc);
          else
            ok = linear_multiply<F16, false, false>(ring, ke - ks, d_tmem, wc);
          if (!ok) break;
          mma_commit_pair(tfull0 + 8 * acc, 0x3);
          acc ^= 1;
          if (acc == 0) acc_par ^= 1;
        }
      }
      // every MMA this thread issued (into both CTAs' tensor memory) finishes before either CTA
      // releases it
      mma_commit_pair(drain_bar, 0x1);
      mbar_wait_drain(drain_bar, 0, drain_ns);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- epilogue warps
    const uint32_t quad = warp & 3;
    const uint32_t lane_base = tmem_base + ((quad * 32u) << 16);
    // the 32-column chunks of this warp
    const int c_first = int(warp - 2) / 4 * (BN / 64), c_last = c_first + BN / 64;
    StoreStage ss{smem_u32(smem + LIN_OUT_OFF) + (warp - 2) * 4096u, 0u};
    int acc = 0;
    uint32_t acc_par = 0;
    auto release = [&]() {  // warp-wide: the accumulator may be written again; on to the other
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(tempty0 + 8 * acc);
        else
          mbar_arrive_remote(mapa_shared(tempty0 + 8 * acc, 0));
      }
      acc ^= 1;
      if (acc == 0) acc_par ^= 1;
    };
    LinearIter it(pair);
    LinearUnit u;
    bool ok = true;
    while (ok && it.next(work, pair, pairs, u)) {
      const LinearJob& jb = work.job[u.job];
      const int M = jb.M, N = jb.N, n0 = u.tn * BN;
      if (!mbar_wait_warp(tfull0 + 8 * acc, acc_par, wc, 4)) break;
      tc_fence_after();
      if (u.kb1 - u.kb0 > jb.seg) {
        // Several segments: a lane keeps the sums of its row's columns in registers. What takes
        // no epilogue (a weight's gradient, a split tile's part) is stored from there, with the
        // accumulator released before (8192 x 8192 x 2048: 231 us where it was held for the
        // stores); else the total goes back to the last segment's accumulator.
        float sum[BN / 64][32];
#pragma unroll
        for (int c = 0; c < BN / 64; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
        for (int ks = u.kb0;;) {
#pragma unroll
          for (int c = 0; c < BN / 32; ++c) {  // sixteen columns at a time: registers
            uint32_t r[16];
            tmem_ld16_wait(lane_base + uint32_t(acc * BN + c_first * 32 + c * 16), r);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum[c / 2][16 * (c % 2) + i] += __uint_as_float(r[i]);
          }
          ks += jb.seg;
          if (ks >= u.kb1) break;
          release();
          if (!mbar_wait_warp(tfull0 + 8 * acc, acc_par, wc, 4)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        if (!ok) break;
        const LinearEpi& e = u.job == 0 ? work.job[0].epi : work.job[1].epi;
        if (u.slot >= 0 || linear_plain(e)) {
          release();
          const int row0 = u.row0 + int(rank) * BM + int(quad * 32);
          float* dst = work.partials + size_t(u.slot < 0 ? 0 : u.slot) * (2 * 128 * BN) +
                       (size_t(rank) * 4 + quad) * (32 * BN) + lane * 4;
#pragma unroll
          for (int c = 0; c < BN / 64; ++c) {
            const int col0 = n0 + (c_first + c) * 32;
            if (col0 >= N || row0 >= M) break;
            if (u.slot < 0)
              linear_store32(ss, &jb.tm_y, e.y32, e.ldy, row0, col0, M, N - col0, e.accumulate,
                             sum[c]);
            else if (row0 + int(lane) < M)
              linear_store_part(dst + (c_first + c) * 1024, sum[c]);
          }
          continue;
        }
#pragma unroll
        for (int c = 0; c < BN / 64; ++c) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(sum[c][i]);
          tmem_st32(lane_base + uint32_t(acc * BN + (c_first + c) * 32), r);
        }
        tmem_st_wait();
      }
      // in registers: read through a job's index inside the loops they cost more than the stores
      const LinearEpi e = u.job == 0 ? work.job[0].epi : work.job[1].epi;
      const int row = u.row0 + int(rank) * BM + int(quad * 32 + lane);
      const uint32_t taddr = lane_base + uint32_t(acc * BN);
      if (u.slot >= 0) {
        float* dst = work.partials + size_t(u.slot) * (2 * 128 * BN) +
                     (size_t(rank) * 4 + quad) * (32 * BN) + lane * 4;
#pragma unroll 1
        for (int c = c_first; c < c_last; ++c) {
          if (n0 + c * 32 >= N) break;
          __syncwarp();
          uint32_t r[32];
          tmem_ld32(taddr + uint32_t(c * 32), r);
          tmem_ld_wait(r);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          if (row < M) linear_store_part(dst + c * 1024, v);
        }
      } else {
#pragma unroll 1
        for (int c = c_first; c < c_last; ++c) {
          const int col0 = n0 + c * 32;
          if (col0 >= N) break;
          __syncwarp();
          uint32_t r[32];
          tmem_ld32(taddr + uint32_t(c * 32), r);
          tmem_ld_wait(r);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
          linear_epilogue32<F16>(e, jb, M, N, row, col0, v, ss);
        }
      }
      release();
    }
    // the warp's TMA stores have read their buffers, and landed, before the CTA ends
    if (ss.n > 0 && lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still arrive on it or MMA into it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// The tiles that were split along K. Block: 32 rows x 32 columns of one.
template <bool F16>
__global__ void __launch_bounds__(256)
    linear_finish_kernel(const __grid_constant__ LinearEpi e, int M, int N, int num_m, int num_n,
                         const LinearClass s, const float* partials) {
  __shared__ float tile[32][36];
  pdl_wait();  // the products' launch is complete
  pdl_trigger();
  const int c = int(blockIdx.x) & 7, slice = int(blockIdx.x >> 3) & 7, ts = int(blockIdx.x >> 6);
  int tm, tn;
  tile_coords(s.first_tile + ts, num_m, num_n, kGroupM, tm, tn);
  const int row0 = tm * PM + slice * 32;
  const int col0 = tn * BN + c * 32;
  if (row0 >= M || col0 >= N) return;
  const int r = int(threadIdx.x) & 31, q = int(threadIdx.x) >> 5;  // row, piece of 4 columns
  const size_t at = size_t(slice) * (32 * BN) + c * 1024 + threadIdx.x * 4;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int k = 0; k < s.split; ++k) {
    const float4 v = __ldcg(reinterpret_cast<const float4*>(
        partials + (size_t(s.slot0) + size_t(ts) * s.split + k) * (2 * 128 * BN) + at));
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  *reinterpret_cast<float4*>(&tile[r][4 * q]) = sum;
  __syncthreads();
  // now a warp has four rows, a lane one column
  const int col = col0 + r;
  if (col >= N) return;
  auto load = [&](const void* p, int64_t i) {
    const uint16_t x = static_cast<const uint16_t*>(p)[i];
    return F16 ? __half2float(__ushort_as_half(x)) : __uint_as_float(uint32_t(x) << 16);
  };
  auto store = [&](void* p, int64_t i, float x) {
    static_cast<uint16_t*>(p)[i] = F16 ? __half_as_ushort(__float2half_rn(x))
                                       : __bfloat16_as_ushort(__float2bfloat16_rn(x));
  };
  const float bias = e.bias != nullptr ? load(e.bias, col) : 0.f;
  float v[4], z[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = row0 + 4 * q + i;
    v[i] = tile[4 * q + i][r] + bias;
    z[i] = e.mul != nullptr && row < M ? load(e.mul, int64_t(row) * e.ld_mul + col) : 0.f;
    if (e.pre != nullptr && row < M) store(e.pre, int64_t(row) * e.ld_pre + col, v[i]);
  }
  if (e.mul != nullptr)
    act_grad_apply<F16>(e.act, v, z);
  else
    act_apply(e.act, F16 || e.y32 != nullptr, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * q + i;
    if (row >= M) break;
    if (e.resid != nullptr)
      v[i] += e.resid_f32 ? static_cast<const float*>(e.resid)[row * e.ld_resid + col]
                          : load(e.resid, row * e.ld_resid + col);
    if (e.y32 != nullptr) {
      float* y = e.y32 + row * e.ldy + col;
      *y = e.accumulate ? *y + v[i] : v[i];
    } else {
      store(e.y16, row * e.ldy + col, v[i]);
    }
  }
}

// Splits `tiles` tiles of num_kb k-blocks from first_tile on over at most `pairs` pairs, into
// parts of `least` k-blocks at least, where that saves kLinearMinGain on each.
LinearClass split_class(int job, int first_tile, int tiles, int num_kb, int pairs, int least,
                        int slot0) {
  LinearClass c{job, first_tile, tiles, 1, num_kb, 0};
  const int most = tiles > 0 ? pairs / tiles : 0;
  if (most < 2) return c;
  int w = (num_kb + most - 1) / most;
  if (w < least) w = least;
  if (w < kLinearMinBlocks) w = kLinearMinBlocks;
  if (w + kLinearMinGain > num_kb) return c;
  const int split = (num_kb + w - 1) / w;
  return LinearClass{job, first_tile, tiles * split, split, w, slot0};
}

template <bool F16>
cudaError_t launch_linear_work(LinearWork& w, int jobs, const RowSums& sums, float* scratch,
                               int* status, uint64_t limit_ns, cudaStream_t stream) {
  static PerDeviceInit setup;  // per device: shared-memory opt-in and co-resident pairs
  int pairs = 0;
  const cudaError_t err = per_device_init(
      setup,
      [](int dev, int* out) {
        cudaError_t e = cudaFuncSetAttribute(linear_kernel<F16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             int(LIN_SMEM));
        int sms = 0;
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return e;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 2;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2 * (sms / 2), 1, 1);
        cfg.blockDim = dim3(LIN_THREADS, 1, 1);
        cfg.dynamicSmemBytes = LIN_SMEM;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, linear_kernel<F16>, &cfg);
        *out = (e == cudaSuccess && n > 0) ? n : 0;
        return e;
      },
      &pairs);
  if (err != cudaSuccess) return err;
  if (pairs <= 0) return cudaErrorLaunchOutOfResources;
  const int slots = scratch == nullptr ? 0 : pairs < kSkMaxClusters ? pairs : kSkMaxClusters;
  int tiles[2] = {0, 0};
  int64_t blocks = 0;
  for (int j = 0; j < jobs; ++j) {
    tiles[j] = w.job[j].num_m * w.job[j].num_n;
    blocks += int64_t(tiles[j]) * w.job[j].num_kb;
  }
  w.partials = scratch;
  w.late = w.catch_up = 0;
  if (jobs == 1) {
    // whole tiles in full waves, then the last wave's, split where that pays
    const int rem = tiles[0] % pairs, kb = w.job[0].num_kb;
    const LinearClass last = split_class(0, tiles[0] - rem, rem, kb, slots, 1, 0);
    if (last.split > 1) {
      w.cls[0] = LinearClass{0, 0, tiles[0] - rem, 1, kb, 0};
      w.cls[1] = last;
    } else {
      w.cls[0] = LinearClass{0, 0, tiles[0], 1, kb, 0};
      w.cls[1] = LinearClass{};
    }
  } else {
    // Both products' tiles together. A tile longer than an even share of all k-blocks is split
    // down to that.
    const int share = int((blocks + pairs - 1) / pairs);
    LinearClass c[2];
    int used = 0;
    for (int j = 0; j < 2; ++j) {
      c[j] = split_class(j, 0, tiles[j], w.job[j].num_kb, slots - used, share, used);
      if (c[j].split > 1) used += c[j].units;
    }
    const bool swap = c[1].W > c[0].W;  // the longer units first
    w.cls[0] = c[swap ? 1 : 0];
    w.cls[1] = c[swap ? 0 : 1];
    const int rest = w.cls[0].units % pairs;
    if (rest > 0) {  // a unit costs about two k-blocks besides its own
      w.late = rest;
      w.catch_up = (w.cls[0].W + 2 + (w.cls[1].W + 2) / 2) / (w.cls[1].W + 2);
    }
  }
  const int64_t units = int64_t(w.cls[0].units) + w.cls[1].units;
  const unsigned grid = 2 * unsigned(units < pairs ? units : pairs);
  // with fewer units than pairs, class 1 continues where class 0 ends
  if (units < pairs) {
    w.late = w.cls[0].units;
    w.catch_up = w.cls[1].units > 0 ? 1 : 0;
  }
  cudaError_t e = launch_dependent(linear_kernel<F16>, dim3(grid, 1, 1), dim3(LIN_THREADS, 1, 1),
                                   LIN_SMEM, 2, stream, w, status, limit_ns);
  if (e == cudaSuccess && sums.m != nullptr)
    e = launch_row_sums(F16 ? kOpF16 : kOpBf16, sums, true, stream);
  for (int k = 0; k < 2 && e == cudaSuccess; ++k) {
    const LinearClass& c = w.cls[k];
    if (c.split < 2) continue;
    const LinearJob& jb = w.job[c.job];
    e = launch_dependent(linear_finish_kernel<F16>, dim3(unsigned(c.units / c.split) * 64, 1, 1),
                         dim3(256, 1, 1), 0, 1, stream, jb.epi, jb.M, jb.N, jb.num_m, jb.num_n, c,
                         static_cast<const float*>(scratch));
  }
  return e;
}

}  // namespace

cudaError_t launch_linear(OpType op, const LinearProduct* products, int count, const RowSums& sums,
                          void* scratch, int* status, uint64_t limit_ns, cudaStream_t stream) {
  if (count < 1 || count > 2) return cudaErrorInvalidValue;
  LinearWork w{};
  for (int j = 0; j < count; ++j) {
    const LinearProduct& p = products[j];
    if (p.M < 1 || p.N < 1 || p.K < 1) return cudaErrorInvalidValue;
    LinearJob& jb = w.job[j];
    jb.tm_a = p.tm_a;
    jb.tm_b = p.tm_b;
    jb.tm_y = p.tm_y;
    jb.tm_pre = p.tm_pre;
    jb.epi = p.epi;
    jb.M = p.M;
    jb.N = p.N;
    jb.num_m = (p.M + PM - 1) / PM;
    jb.num_n = (p.N + BN - 1) / BN;
    jb.num_kb = (p.K + BK - 1) / BK;
    // segments of about one length
    const int longest = p.epi.y32 != nullptr ? kLinearSegment
                        : op == kOpF16       ? kLinearSegmentF16
                                             : kLinearSegmentBf16;
    const int segments = (jb.num_kb + longest - 1) / longest;
    jb.seg = (jb.num_kb + segments - 1) / segments;
    jb.a_mn = p.a_mn;
    jb.b_mn = p.b_mn;
  }
  float* s = static_cast<float*>(scratch);
  return op == kOpF16 ? launch_linear_work<true>(w, count, sums, s, status, limit_ns, stream)
                      : launch_linear_work<false>(w, count, sums, s, status, limit_ns, stream);
}
