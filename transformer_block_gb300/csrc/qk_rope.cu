// qk_rope.cu — the norm of every query and key head and its rotation by the token's
// position, in one pass, and the backward pass of the two.
//
// For a head x of dh values at a token with positions pos[axis]:
//   n = x rstd gamma,  rstd = (mean x^2 + eps)^(-1/2)      (skipped where gamma is NULL)
//   y = R n: each rotated pair (a, b) of n -> (a cos - b sin, a sin + b cos), with the angle
//       pos[axis of the pair] * frequency of the pair; values behind rot_dim pass as they are
// and backward, with d = R^T dy:
//   dgamma = sum over tokens and heads of d x rstd
//   dx = rstd (d gamma - x rstd mean(d gamma x rstd))
//
// The angle only matters modulo a turn. A frequency is held as a 64-bit binary fraction of a
// turn per position (up to frequency 1 off by 2^-56 at most), so position times frequency, wrapped
// to 64 bits, is the angle's place in its turn to 2^-33 up to position 2^23 and to 2^-25 at any
// 32-bit one (negative ones too); a product in fp32 would be off by 0.06 radian at position 10^6.
// The top 32 bits, in radians, go to the fast sine and cosine.
//
// Both passes are bound by memory: 4 bytes a value forward, 6 backward (the norm's backward
// reads x again and recomputes rstd, which costs less than storing it). A head belongs to dh /
// 16 lanes rounded up to a power of two; a lane holds the 16-byte chunk at 8 u of the pairs'
// first half and the chunk as far into their second half, so each access of the lanes of a
// head is one run of 16 bytes a lane, and for pairs half a rotation apart both members sit in
// one lane. A lane group takes one token and walks over its heads: sines and cosines are
// computed once a token and a tensor, and where there are few tokens the heads are split over
// more groups. Three heads ahead of the one at work are on their way by asynchronous copies
// into shared memory that only the lane itself reads back (no barrier): registers would hold
// one. Positions and gammas come by plain loads: the launch before may write them (an update's
// bf16 parameters) while this one, which begins early, already lives.
//
// Measured: forward, 32,760 tokens of 32 + 32 heads of 128, 164 us (6.5 TB/s, 96 % of a plain
// copy); a decoding step of 64 tokens, 32 + 8 heads, 2.2 us in a graph. Backward, 8192 tokens of
// 16 + 16 heads, 36.9 us (5.5 TB/s): bound by the instructions of a value's two sums and turn as
// much as by memory (issue slots 55 % busy).
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "heads.h"
#include "kernels.h"
#include "ptx.cuh"

namespace pb {
namespace {

constexpr uint32_t kRopeMagic = 0x45504F52u;  // "ROPE"
constexpr int THREADS = 256;
constexpr int kMaxDh = 256;
// The norm's backward takes rstd^3, up to eps^(-3/2): in fp32's range with room for the sums.
constexpr float kLeastEpsBackward = 0x1p-80f;
// Blocks of the backward pass that leave a partial sum of dgamma for one tensor.
constexpr int kMaxPartials = 1024;
constexpr size_t kPartialBytes = size_t(2) * kMaxPartials * kMaxDh * sizeof(float);

struct View {
  __nv_bfloat16* p;
  int64_t bs, ss, hs;  // strides of batch, sequence and head, in elements
};

// One of the two tensors (queries or keys) of a launch.
struct Job {
  View x, dy, y;  // dy: backward only; y: the result
  const __nv_bfloat16* gamma;
  int heads;
  // forward: heads of a token that one lane group takes; backward: (token, head) items
  int per_group;
  unsigned blocks, groups;  // forward: groups = tokens * splits
};

struct Params {
  Job job[2];  // blocks [0, job[0].blocks) work on job[0], the rest on job[1]
  const int32_t* pos;
  float* partials;  // backward: [2][kMaxPartials][dh]
  unsigned tokens, S;
  int dh, lanes_log2, rot, axes;
  float eps;
  int section_end[PB_ROPE_MAX_AXES];
  uint64_t turns[kMaxDh / 2];
};

__device__ __forceinline__ void unpack(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// Where lane u of a head's group holds its two chunks of 8 values.
__device__ __forceinline__ void chunk_offsets(const Params& p, int u, int& lo, int& hi) {
  const int ru = p.rot / 16;
  if (u < ru) {
    lo = 8 * u;
    hi = lo + p.rot / 2;
  } else {  // values that are not rotated
    lo = p.rot + 8 * (u - ru);
    hi = lo + (p.dh - p.rot) / 2;
  }
}

// Pair of the lane's sine / cosine i: with halves the pair (lo[i], hi[i]); with adjacent
// members (lo[2i], lo[2i + 1]) for i < 4 and (hi[2i - 8], hi[2i - 7]) behind.
template <bool ADJ>
__device__ __forceinline__ void lane_angles(const Params& p, unsigned token, int s, int u,
                                            float (&c)[8], float (&sn)[8]) {
  if (u >= p.rot / 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.f;
      sn[i] = 0.f;
    }
    return;
  }
  int at[PB_ROPE_MAX_AXES];
#pragma unroll
  for (int a = 0; a < PB_ROPE_MAX_AXES; ++a)
    at[a] = p.pos == nullptr ? s
            : a < p.axes    ? p.pos[int64_t(a) * p.tokens + token]
                            : 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pair = ADJ ? (i < 4 ? 4 * u + i : p.rot / 4 + 4 * u + i - 4) : 8 * u + i;
    int pos = at[0];
#pragma unroll
    for (int a = 1; a < PB_ROPE_MAX_AXES; ++a)
      if (pair >= p.section_end[a - 1]) pos = at[a];
    const uint64_t turn = uint64_t(int64_t(pos)) * p.turns[pair];
    // the place in the turn, in radians: [-pi, pi), where the fast functions are off by
    // 2^-20.5 at most (a bf16 result's half step is 2^-9 of its value)
    const float angle = float(int32_t(turn >> 32)) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    __sincosf(angle, &sn[i], &c[i]);
  }
}

// Values in pairs of neighbours, for packed fp32 instructions: u64 i holds values 2 i, 2 i + 1
// of the lane's sixteen.
__device__ __forceinline__ void unpack2(const uint4& u, uint64_t* v) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    v[e] = f2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack2(const uint64_t* v) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    f2_split(v[e], a, b);
    w[e] = pack_bf16x2(a, b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ float sum2(uint64_t v) {
  float a, b;
  f2_split(v, a, b);
  return a + b;
}
// (a, b) -> (a c + b s, b c - a s) for every pair.
template <bool ADJ>
__device__ __forceinline__ void rotate_back2(uint64_t (&v)[8], const float (&c)[8],
                                             const float (&sn)[8]) {
  if (ADJ) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, b;
      f2_split(v[i], a, b);
      v[i] = f2_fma(v[i], f2(c[i], c[i]), f2_mul(f2(b, a), f2(sn[i], -sn[i])));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t cc = f2(c[2 * i], c[2 * i + 1]), ss = f2(sn[2 * i], sn[2 * i + 1]);
      const uint64_t ns = f2(-sn[2 * i], -sn[2 * i + 1]);
      const uint64_t a = v[i], b = v[i + 4];
      v[i] = f2_fma(a, cc, f2_mul(b, ss));
      v[i + 4] = f2_fma(b, cc, f2_mul(a, ns));
    }
  }
}

template <bool ADJ>
__device__ __forceinline__ void rotate(float* v, const float (&c)[8], const float (&sn)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int ia = ADJ ? (i < 4 ? 2 * i : 8 + 2 * (i - 4)) : i;
    const int ib = ADJ ? ia + 1 : i + 8;
    const float a = v[ia], b = v[ib];
    v[ia] = a * c[i] - b * sn[i];
    v[ib] = a * sn[i] + b * c[i];
  }
}

// The lane's ring of copies: [kRing][pieces][THREADS] 16-byte pieces, kRing - 1 heads ahead.
constexpr int kRing = 4;
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// The oldest head's copies have landed.
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
}
// A lane without values (a head whose chunks are no power of two) has zeros.
__device__ __forceinline__ uint4 ring_read(uint32_t src, bool has_values) {
  uint4 u;
  if (!has_values) return make_uint4(0, 0, 0, 0);
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(src)
               : "memory");
  return u;
}

// LOG2: the logarithm of a head's lanes, 2 and 3 for heads of 64 and 128 values, or -1: p's.
template <int LOG2>
__device__ __forceinline__ float group_sum(float v, int lanes_log2) {
  if (LOG2 >= 0) {
#pragma unroll
    for (int o = (1 << LOG2) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  } else {
    for (int o = (1 << lanes_log2) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// The lane group's place: its token and first head, and whether the lane has values.
struct Place {
  unsigned token;
  int h0, h1, s;
  int64_t b;
  bool live;
};
__device__ __forceinline__ Place place_of(const Params& p, const Job& j, unsigned group, int u) {
  Place w;
  const unsigned split = group / p.tokens;
  w.token = group - split * p.tokens;
  w.b = w.token / p.S;
  w.s = int(w.token - unsigned(w.b) * p.S);
  w.h0 = int(split) * j.per_group;
  w.h1 = min(w.h0 + j.per_group, j.heads);
  w.live = u < p.dh / 16;
  return w;
}

template <bool ADJ, int LOG2>
__global__ void __launch_bounds__(THREADS, 3) qk_forward_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) uint4 ring_mem[kRing * 2 * THREADS];
  pdl_wait();
  pdl_trigger();
  const bool second = blockIdx.x >= p.job[0].blocks;
  const Job& j = p.job[second ? 1 : 0];
  const unsigned block = blockIdx.x - (second ? p.job[0].blocks : 0u);
  const unsigned group = block * (THREADS >> p.lanes_log2) + (threadIdx.x >> p.lanes_log2);
  const int u = int(threadIdx.x) & ((1 << p.lanes_log2) - 1);
  const Place w = place_of(p, j, min(group, j.groups - 1), u);
  const bool live = w.live && group < j.groups;
  int lo, hi;
  chunk_offsets(p, u, lo, hi);
  const __nv_bfloat16* x = j.x.p + w.b * j.x.bs + w.s * j.x.ss;
  __nv_bfloat16* y = j.y.p + w.b * j.y.bs + w.s * j.y.ss;
  const uint32_t ring = smem_u32(ring_mem) + threadIdx.x * 16;
  auto fetch = [&](int h, int slot) {
    if (live && h < w.h1) {
      copy16(ring + (2 * slot) * (THREADS * 16), x + h * j.x.hs + lo);
      copy16(ring + (2 * slot + 1) * (THREADS * 16), x + h * j.x.hs + hi);
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(w.h0 + i, i);
  uint4 g0 = {}, g1 = {};
  if (j.gamma != nullptr && w.live) {
    g0 = *reinterpret_cast<const uint4*>(j.gamma + lo);
    g1 = *reinterpret_cast<const uint4*>(j.gamma + hi);
  }
  float c[8], sn[8];
  lane_angles<ADJ>(p, w.token, w.s, u, c, sn);
  // every group of the block makes the same number of steps, so its lanes meet in the sums
  for (int i = 0; i < j.per_group; ++i) {
    const int h = w.h0 + i, slot = i % kRing;
    fetch(h + kRing - 1, (i + kRing - 1) % kRing);
    copies_wait();
    float v[16];
    unpack(ring_read(ring + (2 * slot) * (THREADS * 16), w.live), v);
    unpack(ring_read(ring + (2 * slot + 1) * (THREADS * 16), w.live), v + 8);
    if (j.gamma != nullptr) {
      float sq = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) sq += v[e] * v[e];
      const float rstd = rsqrtf(group_sum<LOG2>(sq, p.lanes_log2) / float(p.dh) + p.eps);
      float g[16];
      unpack(g0, g);
      unpack(g1, g + 8);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] *= rstd * g[e];
    }
    rotate<ADJ>(v, c, sn);
    if (live && h < w.h1) {
      *reinterpret_cast<uint4*>(y + h * j.y.hs + lo) = pack(v);
      *reinterpret_cast<uint4*>(y + h * j.y.hs + hi) = pack(v + 8);
    }
  }
}

// A lane group's place among the (token, head) items of a tensor, in order.
struct Cursor {
  unsigned token;
  int h, s, b;
  __device__ Cursor(const Params& p, int heads, int64_t item) {
    token = unsigned(item / heads);
    h = int(item - int64_t(token) * heads);
    b = int(token / p.S);
    s = int(token - unsigned(b) * p.S);
  }
  // to the next item; whether that is another token's
  __device__ bool next(const Params& p, int heads) {
    if (++h < heads) return false;
    h = 0;
    ++token;
    if (unsigned(++s) == p.S) {
      s = 0;
      ++b;
    }
    return true;
  }
  __device__ int64_t offset(const View& v) const { return int64_t(b) * v.bs + s * v.ss + h * v.hs; }
};

// The grid is as many blocks as the SMs hold at a time, and every lane group has the same
// number of items one after the other, whatever tokens they begin in: no second wave, and the
// copies run on over the tokens' borders. A group carries its sums of dgamma along; each block
// leaves one partial sum, added in the blocks' order by gamma_sum_kernel, so the result has
// the same bits on every run.
template <bool ADJ, int LOG2>
__global__ void __launch_bounds__(THREADS, 2) qk_backward_kernel(const __grid_constant__ Params p) {
  extern __shared__ __align__(16) uint4 ring_dyn[];  // [kRing][4][THREADS]
  __shared__ float red[THREADS / 32][kMaxDh];
  pdl_wait();
  pdl_trigger();
  const bool second = blockIdx.x >= p.job[0].blocks;
  const Job& j = p.job[second ? 1 : 0];
  const unsigned block = blockIdx.x - (second ? p.job[0].blocks : 0u);
  const unsigned per_block = THREADS >> p.lanes_log2;
  const int u = int(threadIdx.x) & ((1 << p.lanes_log2) - 1);
  int lo, hi;
  chunk_offsets(p, u, lo, hi);
  const bool norm = j.gamma != nullptr, has_values = u < p.dh / 16;
  uint4 g0 = {}, g1 = {};
  if (norm && has_values) {
    g0 = *reinterpret_cast<const uint4*>(j.gamma + lo);
    g1 = *reinterpret_cast<const uint4*>(j.gamma + hi);
  }
  uint64_t dg[8];  // sums of dgamma
#pragma unroll
  for (int e = 0; e < 8; ++e) dg[e] = 0;

  const int64_t items = int64_t(p.tokens) * j.heads;
  const int64_t group = int64_t(block) * per_block + (threadIdx.x >> p.lanes_log2);
  const int64_t item0 = group * j.per_group;
  const int count = has_values && item0 < items ? int(min(items - item0, int64_t(j.per_group))) : 0;
  Cursor at(p, j.heads, min(item0, items - 1)), ahead = at;
  const __nv_bfloat16 *next_dy = j.dy.p + ahead.offset(j.dy),
                      *next_x = norm ? j.x.p + ahead.offset(j.x) : nullptr;
  __nv_bfloat16* dx = j.y.p + at.offset(j.y);
  const uint32_t ring = smem_u32(ring_dyn) + threadIdx.x * 16;
  auto fetch = [&](int i, int slot) {
    if (i < count) {
      const uint32_t to = ring + 4 * slot * (THREADS * 16);
      copy16(to, next_dy + lo);
      copy16(to + THREADS * 16, next_dy + hi);
      if (norm) {
        copy16(to + 2 * (THREADS * 16), next_x + lo);
        copy16(to + 3 * (THREADS * 16), next_x + hi);
      }
      if (ahead.next(p, j.heads)) {
        next_dy = j.dy.p + ahead.offset(j.dy);
        if (norm) next_x = j.x.p + ahead.offset(j.x);
      } else {
        next_dy += j.dy.hs;
        if (norm) next_x += j.x.hs;
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int i = 0; i < kRing - 1; ++i) fetch(i, i);
  float c[8], sn[8];
  lane_angles<ADJ>(p, at.token, at.s, u, c, sn);
  // every group makes the same number of steps, so a head's lanes meet in the sums
  for (int i = 0; i < j.per_group; ++i) {
    const bool mine = i < count;
    fetch(i + kRing - 1, (i + kRing - 1) % kRing);
    copies_wait();
    const uint32_t from = ring + 4 * (i % kRing) * (THREADS * 16);
    // a group behind its last item works on zeros
    uint64_t d[8], v[8];
    unpack2(ring_read(from, mine), d);
    unpack2(ring_read(from + THREADS * 16, mine), d + 4);
    rotate_back2<ADJ>(d, c, sn);
    if (norm) {
      unpack2(ring_read(from + 2 * (THREADS * 16), mine), v);
      unpack2(ring_read(from + 3 * (THREADS * 16), mine), v + 4);
      uint64_t g[8];
      unpack2(g0, g);
      unpack2(g1, g + 4);
      uint64_t sq = 0, dot = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[e] = f2_mul(d[e], g[e]);
        sq = f2_fma(v[e], v[e], sq);
        dot = f2_fma(g[e], v[e], dot);
      }
      const float inv = 1.f / float(p.dh);
      const float rstd = rsqrtf(group_sum<LOG2>(sum2(sq), p.lanes_log2) * inv + p.eps);
      // rstd (d gamma - n mean(d gamma n)), n = v rstd
      const float k = -rstd * rstd * rstd * inv * group_sum<LOG2>(sum2(dot), p.lanes_log2);
      const uint64_t rr = f2(rstd, rstd), kk = f2(k, k);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[e] = f2_fma(d[e], f2_mul(v[e], rr), dg[e]);
        d[e] = f2_fma(g[e], rr, f2_mul(v[e], kk));
      }
    }
    if (mine) {
      *reinterpret_cast<uint4*>(dx + lo) = pack2(d);
      *reinterpret_cast<uint4*>(dx + hi) = pack2(d + 4);
    }
    if (!at.next(p, j.heads)) {
      dx += j.y.hs;
    } else if (i + 1 < count) {
      dx = j.y.p + at.offset(j.y);
      lane_angles<ADJ>(p, at.token, at.s, u, c, sn);
    }
  }
  if (!norm) return;
  // lanes of the same u across the warp's groups, then the warps in order
  float dgf[16];
#pragma unroll
  for (int e = 0; e < 8; ++e) f2_split(dg[e], dgf[2 * e], dgf[2 * e + 1]);
#pragma unroll
  for (int e = 0; e < 16; ++e)
    for (int o = 16; o >= (1 << p.lanes_log2); o >>= 1)
      dgf[e] += __shfl_xor_sync(0xffffffffu, dgf[e], o);
  const int warp = int(threadIdx.x) >> 5;
  if ((threadIdx.x & 31) < (1u << p.lanes_log2) && u < p.dh / 16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      red[warp][lo + e] = dgf[e];
      red[warp][hi + e] = dgf[8 + e];
    }
  }
  __syncthreads();
  if (int(threadIdx.x) < p.dh) {
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < THREADS / 32; ++k) s += red[k][threadIdx.x];
    p.partials[(size_t(second ? 1 : 0) * kMaxPartials + block) * p.dh + threadIdx.x] = s;
  }
}

// out[d] (+)= the sum of the partials in the blocks' order, 32 values of d a block.
struct GammaSum {
  float* out[2];
  unsigned blocks[2];
};
__global__ void __launch_bounds__(1024) gamma_sum_kernel(const float* partials, int dh,
                                                         const GammaSum g, bool accumulate) {
  __shared__ float red[32][33];
  pdl_wait();  // the partial sums' launch is complete
  pdl_trigger();
  const int t = blockIdx.y, col = int(blockIdx.x) * 32 + int(threadIdx.x);
  if (g.out[t] == nullptr) return;
  float s = 0.f;
  if (col < dh)
    for (unsigned b = threadIdx.y; b < g.blocks[t]; b += 32)
      s += partials[(size_t(t) * kMaxPartials + b) * dh + col];
  red[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && col < dh) {
    s = accumulate ? g.out[t][col] : 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) s += red[r][threadIdx.x];
    g.out[t][col] = s;
  }
}

// ------------------------------------------------------------------ arguments

View to_view(const pb_heads* v) {
  if (v == nullptr) return View{};
  return View{static_cast<__nv_bfloat16*>(v->ptr), v->batch_stride, v->seq_stride,
              v->head_stride};
}

pb_status check_common(const pb_rope* rope, int32_t batch, int32_t seq, float eps,
                       const void* gamma_q, const void* gamma_k, const void* positions) {
  if (rope == nullptr || rope->magic != kRopeMagic)
    return record_error(PB_ERR_INVALID_ARG, "rope was not filled by pb_rope_init");
  if (batch < 0 || seq < 0)
    return record_error(PB_ERR_INVALID_ARG, "batch and seq must be >= 0");
  if (int64_t(batch) * seq >= (int64_t(1) << 31))
    return record_error(PB_ERR_UNSUPPORTED, "batch * seq >= 2^31");
  if ((gamma_q != nullptr || gamma_k != nullptr) && !(eps > 0.f && std::isfinite(eps)))
    return record_error(PB_ERR_INVALID_ARG, "eps must be finite and > 0");
  if (!aligned16(gamma_q) || !aligned16(gamma_k))
    return record_error(PB_ERR_INVALID_ARG, "gamma_q and gamma_k must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(positions) & 3) != 0)
    return record_error(PB_ERR_INVALID_ARG, "positions must be 4-byte aligned");
  if (positions == nullptr && rope->axes != 1 && rope->rot_dim > 0)
    return record_error(PB_ERR_INVALID_ARG, "positions may be NULL for one axis only");
  return PB_OK;
}

pb_status fill_params(Params& p, const pb_rope* rope, int batch, int seq, float eps,
                      const int32_t* positions, int* sms) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return cuda_failed(e, "cudaGetDevice");
  p.pos = positions;
  p.tokens = unsigned(batch) * unsigned(seq);
  p.S = unsigned(seq);
  p.dh = rope->head_dim;
  p.lanes_log2 = 0;
  while ((16 << p.lanes_log2) < p.dh) ++p.lanes_log2;
  p.rot = rope->rot_dim;
  p.axes = rope->axes;
  p.eps = eps;
  std::copy(rope->section_end, rope->section_end + PB_ROPE_MAX_AXES, p.section_end);
  std::copy(rope->turns, rope->turns + p.rot / 2, p.turns);
  return PB_OK;
}

template <bool ADJ, int LOG2>
cudaError_t launch_backward(const Params& p, unsigned grid, cudaStream_t st) {
  constexpr int SMEM = kRing * 4 * THREADS * 16;
  static PerDeviceInit setup;  // per device: shared-memory opt-in
  const cudaError_t e = per_device_init(setup, [](int, int*) {
    return cudaFuncSetAttribute(qk_backward_kernel<ADJ, LOG2>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  });
  if (e != cudaSuccess) return e;
  return launch_dependent(qk_backward_kernel<ADJ, LOG2>, dim3(grid, 1, 1), dim3(THREADS, 1, 1), SMEM,
                          1, st, p);
}

template <int LOG2>
cudaError_t launch_backward_any(bool adjacent, const Params& p, unsigned grid, cudaStream_t st) {
  return adjacent ? launch_backward<true, LOG2>(p, grid, st) : launch_backward<false, LOG2>(p, grid, st);
}

template <int LOG2>
cudaError_t launch_forward(bool adjacent, const Params& p, unsigned grid, cudaStream_t st) {
  return launch_dependent(adjacent ? qk_forward_kernel<true, LOG2> : qk_forward_kernel<false, LOG2>,
                          dim3(grid, 1, 1), dim3(THREADS, 1, 1), 0, 1, st, p);
}

// Forward: splits the heads of a token over lane groups until `threads` threads have work.
void set_groups(Job& j, const Params& p, int64_t threads) {
  const int64_t per_head = int64_t(p.tokens) << p.lanes_log2;
  int64_t splits = std::min<int64_t>(j.heads, (threads + per_head - 1) / per_head);
  j.per_group = int((j.heads + splits - 1) / splits);
  splits = (j.heads + j.per_group - 1) / j.per_group;
  j.groups = p.tokens * unsigned(splits);
}

}  // namespace
}  // namespace pb

using namespace pb;

extern "C" {

pb_status pb_rope_init(int32_t head_dim, int32_t rot_dim, int32_t pairing, int32_t axes,
                       const int32_t* sections, int32_t ladder, double theta,
                       const double* inv_freq, pb_rope* out) {
  if (out == nullptr) return record_error(PB_ERR_INVALID_ARG, "out is NULL");
  out->magic = 0;
  if (head_dim < 16 || head_dim > kMaxDh || head_dim % 16 != 0)
    return record_error(PB_ERR_UNSUPPORTED, "head_dim must be a multiple of 16, 16 to 256");
  if (rot_dim < 0 || rot_dim > head_dim)
    return record_error(PB_ERR_INVALID_ARG, "rot_dim must be between 0 and head_dim");
  if (rot_dim % 16 != 0)
    return record_error(PB_ERR_UNSUPPORTED, "rot_dim must be a multiple of 16");
  if (pairing != PB_ROPE_HALVES && pairing != PB_ROPE_ADJACENT)
    return record_error(PB_ERR_INVALID_ARG, "pairing is not a pb_rope_pairing");
  if (ladder != PB_ROPE_SHARED && ladder != PB_ROPE_PER_AXIS)
    return record_error(PB_ERR_INVALID_ARG, "ladder is not a pb_rope_ladder");
  if (axes < 1 || axes > PB_ROPE_MAX_AXES)
    return record_error(PB_ERR_INVALID_ARG, "axes must be 1 to 4");
  const int half = rot_dim / 2;
  if (sections == nullptr && axes != 1)
    return record_error(PB_ERR_INVALID_ARG, "sections may be NULL for one axis only");
  if (inv_freq == nullptr && half > 0 && !(theta > 0 && std::isfinite(theta)))
    return record_error(PB_ERR_INVALID_ARG, "theta must be finite and > 0");
  int64_t sum = 0;
  for (int a = 0; a < axes; ++a) {
    const int n = sections != nullptr ? sections[a] : half;
    if (n < 0 || (sum += n) > half)
      return record_error(PB_ERR_INVALID_ARG, "sections must be >= 0 and add up to rot_dim / 2");
    out->section_end[a] = int32_t(sum);
  }
  if (sum != half)
    return record_error(PB_ERR_INVALID_ARG, "sections must be >= 0 and add up to rot_dim / 2");
  for (int a = axes; a < PB_ROPE_MAX_AXES; ++a) out->section_end[a] = half;
  for (int i = 0, a = 0; i < half; ++i) {
    while (i >= out->section_end[a]) ++a;
    const int first = a == 0 ? 0 : out->section_end[a - 1];
    const double e = ladder == PB_ROPE_SHARED
                         ? double(i) / half
                         : double(i - first) / (out->section_end[a] - first);
    const double f = inv_freq != nullptr ? inv_freq[i] : std::pow(theta, -e);
    if (!std::isfinite(f))
      return record_error(PB_ERR_INVALID_ARG, "every frequency must be finite");
    // turns a position, modulo one, as a 64-bit binary fraction (rounding up to a whole turn
    // wraps to none)
    double turn = f / 6.283185307179586476925286766559;
    turn -= std::floor(turn);
    const double scaled = std::nearbyint(std::ldexp(turn, 64));
    out->turns[i] = scaled >= 18446744073709551616.0 ? 0 : uint64_t(scaled);
  }
  for (int i = half; i < kMaxDh / 2; ++i) out->turns[i] = 0;
  out->head_dim = head_dim;
  out->rot_dim = rot_dim;
  out->pairing = pairing;
  out->axes = axes;
  out->magic = kRopeMagic;
  return PB_OK;
}

pb_status pb_qk_norm_rope(const pb_rope* rope, int32_t batch, int32_t seq, const pb_heads* q,
                          const pb_heads* k, const void* gamma_q, const void* gamma_k, float eps,
                          const int32_t* positions, const pb_heads* q_out,
                          const pb_heads* k_out, void* stream) {
  pb_status s = check_common(rope, batch, seq, eps, gamma_q, gamma_k, positions);
  if (s != PB_OK) return s;
  const pb_heads* in[2] = {q, k};
  const pb_heads* out[2] = {q_out, k_out};
  const void* gamma[2] = {gamma_q, gamma_k};
  static const char* const in_name[2] = {"q", "k"};
  static const char* const out_name[2] = {"q_out", "k_out"};
  if (q == nullptr && k == nullptr)
    return record_error(PB_ERR_INVALID_ARG, "q and k are both NULL");
  if (batch == 0 || seq == 0) return PB_OK;
  const int dh = rope->head_dim;
  for (int t = 0; t < 2; ++t) {
    if ((in[t] == nullptr) != (out[t] == nullptr))
      return bad(PB_ERR_INVALID_ARG, "%s: input and result must both be given or both NULL",
                 in_name[t]);
    if (in[t] == nullptr) continue;
    s = check_view(in[t], in_name[t], batch, seq, dh, false);
    if (s == PB_OK) s = check_view(out[t], out_name[t], batch, seq, dh, true);
    if (s != PB_OK) return s;
    if (in[t]->heads != out[t]->heads)
      return bad(PB_ERR_INVALID_ARG, "%s: input and result have different numbers of heads",
                 in_name[t]);
  }
  for (int t = 0; t < 2; ++t)
    for (int o = 0; o < 2; ++o) {
      if (out[t] == nullptr || in[o] == nullptr) continue;
      if (t == o && same_view(*in[t], *out[t], batch, seq)) continue;
      if (!disjoint(*out[t], *in[o], batch, seq, dh))
        return bad(PB_ERR_INVALID_ARG, "%s overlaps an input without being its own input",
                   out_name[t]);
    }
  if (q_out != nullptr && k_out != nullptr && !disjoint(*q_out, *k_out, batch, seq, dh))
    return record_error(PB_ERR_INVALID_ARG, "q_out and k_out overlap");
  const Flat read[3] = {{gamma_q, size_t(dh) * 2},
                        {gamma_k, size_t(dh) * 2},
                        {positions, size_t(rope->axes) * batch * seq * 4}};
  for (const Flat& r : read)
    for (int t = 0; t < 2; ++t)
      if (!apart(r, out[t], batch, seq, dh))
        return bad(PB_ERR_INVALID_ARG, "%s overlaps a gamma or the positions", out_name[t]);

  Params p{};
  int sms = 0;
  s = fill_params(p, rope, batch, seq, eps, positions, &sms);
  if (s != PB_OK) return s;
  for (int t = 0; t < 2; ++t) {
    if (in[t] == nullptr) continue;
    Job& j = p.job[t];
    j.x = to_view(in[t]);
    j.y = to_view(out[t]);
    j.gamma = static_cast<const __nv_bfloat16*>(gamma[t]);
    j.heads = in[t]->heads;
    set_groups(j, p, int64_t(sms) * 1024);
    const unsigned per_block = THREADS >> p.lanes_log2;
    j.blocks = (j.groups + per_block - 1) / per_block;
  }
  const unsigned grid = p.job[0].blocks + p.job[1].blocks;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool adjacent = rope->pairing == PB_ROPE_ADJACENT;
  const cudaError_t e = p.lanes_log2 == 3   ? launch_forward<3>(adjacent, p, grid, st)
                        : p.lanes_log2 == 2 ? launch_forward<2>(adjacent, p, grid, st)
                                            : launch_forward<-1>(adjacent, p, grid, st);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "qk_norm_rope launch");
}

pb_status pb_qk_norm_rope_scratch_bytes(size_t* bytes) {
  if (bytes == nullptr) return record_error(PB_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = kPartialBytes;
  return PB_OK;
}

pb_status pb_qk_norm_rope_backward(const pb_rope* rope, int32_t batch, int32_t seq,
                                   const pb_heads* q, const pb_heads* k, const void* gamma_q,
                                   const void* gamma_k, float eps, const int32_t* positions,
                                   const pb_heads* dq, const pb_heads* dk,
                                   const pb_heads* dq_out, const pb_heads* dk_out,
                                   float* dgamma_q, float* dgamma_k, int32_t accumulate,
                                   void* scratch, size_t scratch_bytes, void* stream) {
  pb_status s = check_common(rope, batch, seq, eps, gamma_q, gamma_k, positions);
  if (s != PB_OK) return s;
  if ((gamma_q != nullptr || gamma_k != nullptr) && eps < kLeastEpsBackward)
    return record_error(PB_ERR_INVALID_ARG, "eps must be >= 2^-80 for the norm's backward");
  const pb_heads* x[2] = {q, k};
  const pb_heads* dy[2] = {dq, dk};
  const pb_heads* out[2] = {dq_out, dk_out};
  const void* gamma[2] = {gamma_q, gamma_k};
  float* dgamma[2] = {dgamma_q, dgamma_k};
  static const char* const x_name[2] = {"q", "k"};
  static const char* const dy_name[2] = {"dq", "dk"};
  static const char* const out_name[2] = {"dq_out", "dk_out"};
  if (dq == nullptr && dk == nullptr)
    return record_error(PB_ERR_INVALID_ARG, "dq and dk are both NULL");
  const int dh = rope->head_dim;
  const bool none = batch == 0 || seq == 0;
  bool sums = false;
  for (int t = 0; t < 2; ++t) {
    if (dgamma[t] != nullptr && (dy[t] == nullptr || gamma[t] == nullptr))
      return bad(PB_ERR_INVALID_ARG, "%s: a gradient of gamma without gamma", dy_name[t]);
    if ((reinterpret_cast<uintptr_t>(dgamma[t]) & 3) != 0)
      return record_error(PB_ERR_INVALID_ARG, "dgamma_q and dgamma_k must be 4-byte aligned");
    if ((dy[t] == nullptr) != (out[t] == nullptr))
      return bad(PB_ERR_INVALID_ARG, "%s: gradient and result must both be given or both NULL",
                 dy_name[t]);
    if (dy[t] == nullptr || none) continue;
    if (gamma[t] != nullptr && x[t] == nullptr)
      return bad(PB_ERR_INVALID_ARG, "%s is NULL: the norm's backward reads it", x_name[t]);
    s = check_view(dy[t], dy_name[t], batch, seq, dh, false);
    if (s == PB_OK) s = check_view(out[t], out_name[t], batch, seq, dh, true);
    if (s == PB_OK && gamma[t] != nullptr)
      s = check_view(x[t], x_name[t], batch, seq, dh, false);
    if (s != PB_OK) return s;
    if (dy[t]->heads != out[t]->heads || (gamma[t] != nullptr && x[t]->heads != dy[t]->heads))
      return bad(PB_ERR_INVALID_ARG, "%s: the views have different numbers of heads", dy_name[t]);
    sums |= gamma[t] != nullptr;
  }
  if (!none) {
    for (int t = 0; t < 2; ++t)
      for (int o = 0; o < 2; ++o) {
        if (out[t] == nullptr || dy[o] == nullptr) continue;
        const pb_heads* read[2] = {dy[o], gamma[o] != nullptr ? x[o] : nullptr};
        for (const pb_heads* r : read) {
          if (r == nullptr || (t == o && same_view(*r, *out[t], batch, seq))) continue;
          if (!disjoint(*out[t], *r, batch, seq, dh))
            return bad(PB_ERR_INVALID_ARG, "%s overlaps an input without being its own input",
                       out_name[t]);
        }
      }
    if (dq_out != nullptr && dk_out != nullptr && !disjoint(*dq_out, *dk_out, batch, seq, dh))
      return record_error(PB_ERR_INVALID_ARG, "dq_out and dk_out overlap");
    if (sums) {
      if (scratch == nullptr || (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
        return record_error(PB_ERR_INVALID_ARG,
                            "scratch must be a 256-byte aligned device pointer");
      if (scratch_bytes < kPartialBytes)
        return record_error(PB_ERR_WORKSPACE,
                            "scratch is smaller than pb_qk_norm_rope_scratch_bytes");
    }
  }
  // the gammas' gradients and the scratch: apart from one another and from all else
  const Flat written[3] = {{dgamma_q, size_t(dh) * 4},
                           {dgamma_k, size_t(dh) * 4},
                           {sums ? scratch : nullptr, kPartialBytes}};
  const Flat read[3] = {{gamma_q, size_t(dh) * 2},
                        {gamma_k, size_t(dh) * 2},
                        {positions, none ? 0 : size_t(rope->axes) * batch * seq * 4}};
  for (int i = 0; i < 3; ++i) {
    bool clear = true;
    for (int o = 0; o < 3; ++o)
      clear = clear && apart(written[i], read[o]) && (o == i || apart(written[i], written[o]));
    for (int t = 0; t < 2 && !none; ++t) {
      clear = clear && apart(written[i], dy[t], batch, seq, dh) &&
              apart(written[i], out[t], batch, seq, dh) &&
              (dy[t] == nullptr || gamma[t] == nullptr || apart(written[i], x[t], batch, seq, dh));
      if (!apart(read[i], out[t], batch, seq, dh))
        return bad(PB_ERR_INVALID_ARG, "%s overlaps a gamma or the positions", out_name[t]);
    }
    if (!clear)
      return record_error(PB_ERR_INVALID_ARG,
                          "dgamma_q, dgamma_k or scratch overlaps another argument");
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (none) {  // no tokens: the sums over them are zero
    for (float* g : dgamma)
      if (g != nullptr && !accumulate) {
        const cudaError_t e = cudaMemsetAsync(g, 0, size_t(dh) * 4, st);
        if (e != cudaSuccess) return cuda_failed(e, "cudaMemsetAsync(dgamma)");
      }
    return PB_OK;
  }

  Params p{};
  int sms = 0;
  s = fill_params(p, rope, batch, seq, eps, positions, &sms);
  if (s != PB_OK) return s;
  p.partials = static_cast<float*>(scratch);
  GammaSum gs{};
  int heads = 0;
  for (const pb_heads* v : dy) heads += v != nullptr ? v->heads : 0;
  for (int t = 0; t < 2; ++t) {
    if (dy[t] == nullptr) continue;
    Job& j = p.job[t];
    if (gamma[t] != nullptr) j.x = to_view(x[t]);
    j.dy = to_view(dy[t]);
    j.y = to_view(out[t]);
    j.gamma = static_cast<const __nv_bfloat16*>(gamma[t]);
    j.heads = dy[t]->heads;
    // the SMs' two resident blocks, shared by the number of heads
    const unsigned per_block = THREADS >> p.lanes_log2;
    const int64_t items = int64_t(p.tokens) * j.heads;
    int64_t blocks = int64_t(sms) * 2 * j.heads / heads;
    blocks = std::max<int64_t>(1, std::min<int64_t>(blocks, kMaxPartials));
    j.per_group = int((items + blocks * per_block - 1) / (blocks * per_block));
    const int64_t groups = (items + j.per_group - 1) / j.per_group;
    j.blocks = unsigned((groups + per_block - 1) / per_block);
    gs.out[t] = dgamma[t];
    gs.blocks[t] = j.blocks;
  }
  const unsigned grid = p.job[0].blocks + p.job[1].blocks;
  const bool adjacent = rope->pairing == PB_ROPE_ADJACENT;
  cudaError_t e = p.lanes_log2 == 3   ? launch_backward_any<3>(adjacent, p, grid, st)
                  : p.lanes_log2 == 2 ? launch_backward_any<2>(adjacent, p, grid, st)
                                      : launch_backward_any<-1>(adjacent, p, grid, st);
  if (e == cudaSuccess && (gs.out[0] != nullptr || gs.out[1] != nullptr)) {
    e = launch_dependent(gamma_sum_kernel, dim3(unsigned(dh + 31) / 32, 2, 1), dim3(32, 32, 1), 0, 1,
                         st, p.partials, dh, gs, accumulate != 0);
  }
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "qk_norm_rope_backward launch");
}

}  // extern "C"
