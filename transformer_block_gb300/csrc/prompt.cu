// prompt.cu — causal attention of packed prompts of different lengths, with grouped heads, on the
// tensor cores.
//
// Sequence s holds the tokens starts[s] <= i < starts[s + 1]; query head h reads key head h / g.
//   o_i = sum_{k in s, 0 <= i - k < w} softmax_k(scale q_i . k_k) v_k
//
// Rows. The g heads of a key head read the same keys, so a tile of 128 rows holds T = 128 / g
// (rounded down) tokens with all their g heads: row r is head r mod g of token r / g. One TMA box of
// 64 columns x g heads x T tokens writes it. Each tile then needs one key head's keys up to its last
// token, whatever g is, and a short prompt fills its rows with heads instead of padding.
//
// Items. An item is two such tiles that follow one another in a sequence (2 T tokens) and share
// every key and value tile. How many items there are is known on the device only (starts). They are
// dealt out longest first (by the first token's place in its sequence), in rounds of alternating
// direction, to one block an SM. Up to 128 sequences every block finds its own items in that order by
// itself; more are listed by a launch before (counted into buckets by length), beside which the main
// launch sets up.
//
// Inside a block. Warp 0 loads by TMA (K 3 stages, V 2). Warp 1 issues S = Q K^T, warp 3 O += P V,
// each product by one elected lane of the converged warp: issuing from one diverged lane, or all from
// one warp, takes longer than the products (a step of 256 rows x 128 keys: 2048 cycles of products;
// issued by one lane 3960 to 5500 cycles, by one warp 3080, by two 2870). Warp 2 waits for V. Two
// groups of four warps take the softmax, a row a thread. Tensor memory (512 columns) holds
//   S (128) | P0 (64) | P1 (64) | O0 (128) | O1 (128)
// One S serves both row tiles in turn: it is free as soon as the softmax has it in registers, so the
// next tile's scores are computed during this one's softmax. With an S of each tile's own, over which
// its P is written, a tile's S, softmax and P V follow one another (3330 cycles a step). Steps of 64
// keys with two S for each tile need twice the products' starts (16384 tokens: 2277 us, this form
// 1365). P (bf16, as all attention of the library; its error averages over the keys) is handed over in
// two halves. The softmax's maximum, its sum and O are fp32; O is rescaled only where a maximum grows by
// more than 2^8. V comes as it is stored, [keys, head_dim]: the product reads it as an MN-major
// operand, so no transposed copy is made.
//
// A key tile at a sequence's end holds rows of the next sequence, or of nothing. Their scores are
// replaced, not added to; their values would still meet P = 0, and 0 x NaN is NaN, so warp 2 writes
// zeros over those rows of V before the product reads them. Nothing of another sequence reaches a
// result.
//
// Measured (in a graph): 16384 tokens, 32 heads over 8, 1365 to 1416 us on two GPUs (1.55 to 1.61
// PFLOP/s, 80 to 83 % of the library's product rate; tensor pipe 67 % busy; called over and over the
// power limit makes it 1480 to 1530); 15 prompts of 1 to 2049 tokens, 8096 in all, the same heads, 94 us
// (870 TFLOP/s of the pairs that are seen); 4 x 2048 tokens, 16 heads, window 512, 55 us; 128 tokens 6
// us. What is left of the short ones is the start and end of an item, about 6500 cycles: its first
// softmax and last P V have nothing beside them, and its result leaves by plain stores. 168 registers a
// thread, the most that 384 threads may be compiled with, spill 44 bytes of stores and 308 of loads
// (96/200, 104/192 or 120/184 registers a warpgroup; 88/208: 40 and 284).
#include <cuda_bf16.h>

#include <cmath>

#include "heads.h"
#include "kernels.h"
#include "ptx.cuh"

namespace pb {
namespace {

constexpr int BQ = 128, BKV = 128;
constexpr int THREADS = 384;
// Registers a thread: at launch (the most 384 threads may have), then per warpgroup.
constexpr uint32_t kRegsLaunch = 168, kRegsControl = 96, kRegsSoftmax = 200;
static_assert(128 * kRegsControl + 256 * kRegsSoftmax <= THREADS * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t TMEM_COLS = 512;
constexpr int BOX = 128 * 64 * 2;          // 128 rows x 64 columns of 16 bits
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr uint64_t kLimitNs = 2000000000ull;
constexpr int kBuckets = 2048;
constexpr int kOwnItems = 64;       // items that a block lists for itself
constexpr int kOwnSequences = 128;  // of at most so many sequences

// Scratch: the number of entries, then the entries: a pair of tiles of a sequence (every key head
// has one item for it).
struct Entry {
  int first;  // the sequence's first token
  int n;      // its length
  int q0;     // the pair's first token, counted from the sequence's
  int pad;
};
constexpr size_t kHeaderBytes = 256;

struct Params {
  int tokens, sequences;
  int kv_heads, group, tile_tokens;
  int window;  // at least 1
  float scale_log2;
  int shift;      // bucket = pair index >> shift
  int capacity;   // the most pairs that sequences of so many tokens have: entries in scratch
  bool own_list;  // blocks list their items themselves
  const int* starts;  // or null: one sequence
  __nv_bfloat16* out;
  int64_t out_ss, out_hs;
};

// Whether sequence s ends before it begins. Where starts fall, sequences may overlap, and there is no
// bound on their pairs: such a call does nothing.
__device__ __forceinline__ bool falls(const Params& p, int s) {
  return p.starts != nullptr && p.starts[s + 1] < p.starts[s];
}
__device__ __forceinline__ int2 sequence(const Params& p, int s) {
  if (p.starts == nullptr) return make_int2(0, p.tokens);
  const int a = min(max(p.starts[s], 0), p.tokens);
  return make_int2(a, max(min(max(p.starts[s + 1], 0), p.tokens) - a, 0));
}

// Lists the pairs of all sequences, later ones of a sequence (more keys) first. The order of equal
// ones, which atomics decide, changes no result.
__global__ void __launch_bounds__(1024) list_kernel(const Params p, int* count, Entry* entries,
                                                    int* status) {
  __shared__ int at[kBuckets];
  __shared__ int sums[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  for (int b = tid; b < kBuckets; b += 1024) at[b] = 0;
  bool fall = false;
  for (int s = tid; s < p.sequences; s += 1024) fall |= falls(p, s);
  if (__syncthreads_or(fall)) {
    if (tid == 0) {
      *count = 0;
      if (status != nullptr) atomicCAS(status, 0, int(PB_ERR_INVALID_ARG));
    }
    return;
  }
  const int pair_tokens = 2 * p.tile_tokens;
  for (int s = warp; s < p.sequences; s += 32) {
    const int pairs = (sequence(p, s).y + pair_tokens - 1) / pair_tokens;
    for (int i = lane; i < pairs; i += 32) atomicAdd(&at[i >> p.shift], 1);
  }
  __syncthreads();
  // bucket b starts behind all buckets above it: thread t takes buckets kBuckets - 1 - 2t, - 2t - 1
  const int b1 = kBuckets - 1 - 2 * tid, b0 = b1 - 1;
  const int n1 = at[b1], n0 = at[b0];
  int x = n1 + n0;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, d);
    if (lane >= d) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < warp; ++i) before += sums[i];
  x += before;
  at[b1] = x - n1 - n0;
  at[b0] = x - n0;
  if (tid == 1023) *count = x;
  __syncthreads();
  for (int s = warp; s < p.sequences; s += 32) {
    const int2 q = sequence(p, s);
    const int pairs = (q.y + pair_tokens - 1) / pair_tokens;
    for (int i = lane; i < pairs; i += 32) {
      const int e = atomicAdd(&at[i >> p.shift], 1);
      entries[e] = Entry{q.x, q.y, i * pair_tokens, 0};
    }
  }
}

// Half a softmax row of a tile (64 keys from column `first` of s on): p_k = 2^(s_k c - m) rounded to
// bf16 into tensor memory at t_p (column m holds keys 2m and 2m + 1); the fp32 sum of the unrounded
// p_k is added to acc, in four parts of pairs.
__device__ __forceinline__ void probs_to_tmem(const float (&s)[BKV], int first, float c, float m,
                                              uint32_t t_p, uint64_t (&acc)[4]) {
  const uint64_t c2 = f2(c, c), nm2 = f2(-m, -m);
#pragma unroll
  for (int ch = 0; ch < 2; ++ch) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int k = first + ch * 32 + 2 * e;
      const uint64_t x2 = f2_fma(f2(s[k], s[k + 1]), c2, nm2);
      float x0, x1;
      f2_split(x2, x0, x1);
      const uint64_t a2 = f2(ex2_approx(x0), ex2_approx(x1));
      acc[e & 3] = f2_add(acc[e & 3], a2);
      float a0, a1;
      f2_split(a2, a0, a1);
      pk[e] = pack_bf16x2(a0, a1);
    }
    tmem_st16(t_p + uint32_t(ch * 16), pk);
  }
}

// Transposes 16-byte pieces (4 words) inside each group of 4 lanes: piece c of lane l becomes
// piece l of lane c, so that 4 lanes store 64 bytes of one row.
__device__ __forceinline__ void transpose_pieces(uint32_t (&w)[16]) {
  const uint32_t lane = lane_id();
  const bool hi = (lane & 2) != 0, odd = (lane & 1) != 0;
#pragma unroll
  for (int s = 0; s < 2; ++s)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t y = __shfl_xor_sync(0xffffffffu, hi ? w[4 * s + e] : w[4 * (2 + s) + e], 2);
      if (hi)
        w[4 * s + e] = y;
      else
        w[4 * (2 + s) + e] = y;
    }
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t y =
          __shfl_xor_sync(0xffffffffu, odd ? w[4 * (2 * c) + e] : w[4 * (2 * c + 1) + e], 1);
      if (odd)
        w[4 * (2 * c) + e] = y;
      else
        w[4 * (2 * c + 1) + e] = y;
    }
}

// Products issued by the elected lane of a converged warp, descriptors in 32-bit halves (the upper one
// is the same for all operands of a kind): the issuing of a product then costs less than its 64 cycles.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)::"memory");
  return r != 0;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ int item_index(int n, int c, int G) {
  return n * G + ((n & 1) ? G - 1 - c : c);
}

// The same order of pairs, later ones of a sequence first and equal ones by sequence, found by every
// block for its own items alone: no launch before. A lane holds every 32nd sequence's pairs, and the
// pairs behind level L are sum_s max(0, pairs_s - L - 1). Returns the number of all pairs.
__device__ __forceinline__ int list_own(const Params& p, Entry* own, int warp, int lane,
                                        int* status) {
  constexpr int PER = kOwnSequences / 32;
  const int pair_tokens = 2 * p.tile_tokens;
  int2 q[PER];
  int pairs[PER], all = 0, most = 0;
  bool fall = false;
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    q[k] = lane + 32 * k < p.sequences ? sequence(p, lane + 32 * k) : make_int2(0, 0);
    fall |= lane + 32 * k < p.sequences && falls(p, lane + 32 * k);
    pairs[k] = (q[k].y + pair_tokens - 1) / pair_tokens;
    all += pairs[k];
    most = max(most, pairs[k]);
  }
  all = __reduce_add_sync(0xffffffffu, all);
  if (__any_sync(0xffffffffu, fall)) {
    if (lane == 0 && status != nullptr) atomicCAS(status, 0, int(PB_ERR_INVALID_ARG));
    return 0;
  }
  most = __reduce_max_sync(0xffffffffu, most);
  const int items = all * p.kv_heads, G = int(gridDim.x);
  for (int n = warp; n < kOwnItems; n += THREADS / 32) {
    const int r = item_index(n, int(blockIdx.x), G);
    if (r >= items) break;
    const int e = r / p.kv_heads;
    auto behind = [&](int level) {
      int sum = 0;
#pragma unroll
      for (int k = 0; k < PER; ++k) sum += max(0, pairs[k] - level - 1);
      return int(__reduce_add_sync(0xffffffffu, sum));
    };
    int lo = 0, hi = most - 1;  // the lowest level with at most e pairs behind it
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (behind(mid) <= e)
        hi = mid;
      else
        lo = mid + 1;
    }
    int j = e - behind(lo);  // the j-th sequence that has this level
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      const uint32_t m = __ballot_sync(0xffffffffu, pairs[k] > lo);
      if (pairs[k] > lo && __popc(m & ((1u << lane) - 1)) == j)
        own[n] = Entry{q[k].x, q[k].y, lo * pair_tokens, 0};
      j -= __popc(m);  // below zero behind the one that is meant
    }
  }
  return all;
}

template <int DH>
struct Layout {
  static constexpr int Q_TILE = BQ * DH * 2;
  static constexpr int KV_BYTES = BKV * DH * 2;
  static constexpr int K_STAGES = 3, V_STAGES = 2;
  static constexpr int K_OFF = 2 * Q_TILE;
  static constexpr int V_OFF = K_OFF + K_STAGES * KV_BYTES;
  static constexpr int BAR_OFF = V_OFF + V_STAGES * KV_BYTES;
  static constexpr int NUM_BARS = 23;
  static constexpr int OWN_OFF = BAR_OFF + (NUM_BARS * 8 + 16 + 15) / 16 * 16;
  static constexpr size_t NEED = size_t(OWN_OFF) + kOwnItems * sizeof(Entry) + 1024;
  // so much that one block fits an SM: it takes all 512 columns of tensor memory
  static constexpr size_t SMEM = NEED > 200 * 1024 ? NEED : 200 * 1024;
  static_assert(SMEM <= 227 * 1024, "shared memory layout");
};

struct Item {
  int kv;                  // key head
  int first, n, q0;        // as in Entry
  int kb0, ke0, kb1, ke1;  // key tiles [kb, ke] of row tile 0 / 1 (none: ke < kb)
  int U;                   // tiles from kb0 to the last one
};

// Item r of all, the block's n-th.
__device__ __forceinline__ Item make_item(const Params& p, const Entry* entries, int r, int n) {
  Item it;
  const int e = r / p.kv_heads;
  it.kv = r - e * p.kv_heads;
  const int4 v = *reinterpret_cast<const int4*>(entries + (p.own_list ? n : e));
  it.first = v.x;
  it.n = v.y;
  it.q0 = v.z;
  int kb[2], ke[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int qb = it.q0 + h * p.tile_tokens;
    kb[h] = qb < it.n ? max(0, qb - p.window + 1) / BKV : 1;
    ke[h] = qb < it.n ? (min(qb + p.tile_tokens, it.n) - 1) / BKV : 0;
  }
  it.kb0 = kb[0];
  it.ke0 = ke[0];
  it.kb1 = kb[1];
  it.ke1 = ke[1];
  it.U = max(ke[0], ke[1]) - kb[0] + 1;
  return it;
}

__device__ __forceinline__ bool item_needs(const Item& it, int h, int j) {
  return h ? (j >= it.kb1 && j <= it.ke1) : (j >= it.kb0 && j <= it.ke0);
}

template <int DH>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const Params p, const int* count,
                  const Entry* entries0, int* status) {
  using L = Layout<DH>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  const uint32_t q_full = smem_u32(bars + 0);
  const uint32_t q_empty = smem_u32(bars + 1);    // the item's last S products are done
  const uint32_t k_full0 = smem_u32(bars + 2);    // [3]
  const uint32_t k_empty0 = smem_u32(bars + 5);   // [3]
  const uint32_t v_full0 = smem_u32(bars + 8);    // [2]
  const uint32_t v_empty0 = smem_u32(bars + 10);  // [2]
  const uint32_t s_full0 = smem_u32(bars + 12);   // [2] per row tile
  const uint32_t s_free = smem_u32(bars + 14);    // S has been read (4 warps, the row tiles in turn)
  const uint32_t p_half0 = smem_u32(bars + 15);   // [2] per row tile: P of the first 64 keys
  const uint32_t p_full0 = smem_u32(bars + 17);   // [2] and of the others
  const uint32_t o_done0 = smem_u32(bars + 19);   // [2] per row tile: the step's PV is done
  const uint32_t drain0 = smem_u32(bars + 21);    // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + L::NUM_BARS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int G = int(gridDim.x), cta = int(blockIdx.x);

  const uint32_t warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(k_full0 + 8 * s, 1);
      mbar_init(k_empty0 + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(v_full0 + 8 * s, 1);
      mbar_init(v_empty0 + 8 * s, 1);
      mbar_init(s_full0 + 8 * s, 1);
      mbar_init(p_half0 + 8 * s, s == 0 ? 5 : 4);  // row tile 0: and warp 2
      mbar_init(p_full0 + 8 * s, 4);
      mbar_init(o_done0 + 8 * s, 1);
    }
    mbar_init(s_free, 4);
    mbar_init(drain0, 1);
    mbar_init(drain0 + 8, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();  // what the launches before wrote is there, the list too where one of them made it
  Entry* const own = reinterpret_cast<Entry*>(smem + L::OWN_OFF);
  const Entry* const entries = p.own_list ? own : entries0;
  const int num_items =
      (p.own_list ? list_own(p, own, int(warp), int(lane), status) : *count) * p.kv_heads;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const WaitCtl wc{abort_flag, status, kLimitNs};
  const uint64_t drain_ns = kLimitNs > kDrainFloorNs ? kLimitNs : kDrainFloorNs;
  const uint32_t sQ = smem_u32(smem);
  const uint32_t sK = smem_u32(smem + L::K_OFF);
  const uint32_t sV = smem_u32(smem + L::V_OFF);
  if (warp < 4) {
    setmaxnreg_dec<kRegsControl>();
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------------- producer
        // K and V rings run on across items. Per stage: parity of its last load (bit s), ever
        // loaded.
        const uint32_t q_bytes = uint32_t(2 * (DH / 64) * 128) * uint32_t(p.group * p.tile_tokens);
        uint32_t kc = 0, vc = 0;
        uint32_t k_par = 0, v_par = 0, k_used = 0, v_used = 0;
        int n_done = 0;
        bool ok = true;
        for (int n = 0; ok; ++n) {
          const int r = item_index(n, cta, G);
          if (r >= num_items) break;
          const Item it = make_item(p, entries, r, n);
          auto load_k = [&](int idx) -> bool {
            const uint32_t g = kc + uint32_t(idx);
            const uint32_t st = g % 3, par = (g / 3) & 1;
            if (!mbar_wait(k_empty0 + 8 * st, par ^ 1, wc, 11)) return false;
            mbar_arrive_expect_tx(k_full0 + 8 * st, L::KV_BYTES);
#pragma unroll
            for (int hb = 0; hb < DH / 64; ++hb)
              tma_load_3d(sK + st * L::KV_BYTES + hb * BOX, &tmK, k_full0 + 8 * st, hb * 64, it.kv,
                          it.first + (it.kb0 + idx) * BKV);
            k_par = (k_par & ~(1u << st)) | (par << st);
            k_used |= 1u << st;
            return true;
          };
          auto load_v = [&](int idx) -> bool {
            const uint32_t g = vc + uint32_t(idx);
            const uint32_t st = g & 1, par = (g >> 1) & 1;
            if (!mbar_wait(v_empty0 + 8 * st, par ^ 1, wc, 10)) return false;
            mbar_arrive_expect_tx(v_full0 + 8 * st, L::KV_BYTES);
#pragma unroll
            for (int hb = 0; hb < DH / 64; ++hb)
              tma_load_3d(sV + st * L::KV_BYTES + hb * BOX, &tmV, v_full0 + 8 * st, hb * 64, it.kv,
                          it.first + (it.kb0 + idx) * BKV);
            v_par = (v_par & ~(1u << st)) | (par << st);
            v_used |= 1u << st;
            return true;
          };
          // K runs one tile ahead of V: S runs ahead of P V
          ok = load_k(0);  // before Q: its stage is free sooner
          // the Q tiles of the previous item are free once its last S products completed
          if (!ok || !mbar_wait(q_empty, (n & 1) ^ 1, wc, 20)) break;
          mbar_arrive_expect_tx(q_full, q_bytes);
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int hb = 0; hb < DH / 64; ++hb)
              tma_load_3d(sQ + h * L::Q_TILE + hb * BOX, &tmQ, q_full, hb * 64, it.kv * p.group,
                          it.first + it.q0 + h * p.tile_tokens);
          n_done = n + 1;
          for (int idx = 0; ok && idx < it.U; ++idx) {
            if (idx + 1 < it.U) ok = load_k(idx + 1);
            if (ok) ok = load_v(idx);
          }
          kc += uint32_t(it.U);
          vc += uint32_t(it.U);
        }
        if (n_done > 0) mbar_wait_drain(q_full, uint32_t(n_done - 1) & 1, drain_ns);
        for (uint32_t s = 0; s < 3; ++s)
          if (k_used & (1u << s)) mbar_wait_drain(k_full0 + 8 * s, (k_par >> s) & 1u, drain_ns);
        for (uint32_t s = 0; s < 2; ++s)
          if (v_used & (1u << s)) mbar_wait_drain(v_full0 + 8 * s, (v_par >> s) & 1u, drain_ns);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- S = Q K^T
      // The whole warp waits and steps; one lane issues.
      const uint32_t id_s = idesc_bf16_f32(BQ, BKV);
      const uint64_t dQ = sdesc_kmajor_sw128(sQ), dK = sdesc_kmajor_sw128(sK);
      const uint32_t hi = uint32_t(dQ >> 32);
      uint32_t kc = 0;  // K tiles of the items before
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int r = item_index(n, cta, G);
        if (r >= num_items) break;
        const Item it = make_item(p, entries, r, n);
        if (!mbar_wait_warp(q_full, uint32_t(n) & 1, wc, 12)) break;
        for (int idx = 0; ok && idx < it.U; ++idx) {
          const uint32_t g = kc + uint32_t(idx), st = g % 3;
          if (!mbar_wait_warp(k_full0 + 8 * st, (g / 3) & 1, wc, 14)) {
            ok = false;
            break;
          }
          const uint32_t k = uint32_t(dK) + st * uint32_t(L::KV_BYTES >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // the other tile's softmax has read the S before: phases 2 step + h
            if (!mbar_wait_warp(s_free, uint32_t(h ^ 1), wc, 22)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (elect_one()) {
              if (item_needs(it, h, it.kb0 + idx)) {  // nothing where the tile does not need it
                const uint32_t q = uint32_t(dQ) + uint32_t((h * L::Q_TILE) >> 4);
#pragma unroll
                for (int kk = 0; kk < DH / 16; ++kk) {
                  const uint32_t off = uint32_t(((kk >> 2) * BOX) >> 4) + 2 * (kk & 3);
                  mma_ss(tmem_base, q + off, k + off, hi, id_s, kk > 0 ? 1u : 0u);
                }
              }
              mma_commit(s_full0 + 8 * h);
              if (h == 1) {
                mma_commit(k_empty0 + 8 * st);  // both S products have K
                if (idx + 1 == it.U) mma_commit(q_empty);
              }
            }
            __syncwarp();
          }
        }
        kc += uint32_t(it.U);
      }
      if (elect_one()) mma_commit(drain0);
      mbar_wait_drain(drain0, 0, drain_ns);
      __syncwarp();
    } else if (warp == 3) {
      // ---------------------------------------------------------------- O += P V
      constexpr uint32_t T_P = 128, T_O = 256;
      const uint32_t id_o = idesc_f32acc(BQ, DH, false, false, true);
      const uint64_t dV = sdesc_mnmajor_sw128(sV, BOX);
      const uint32_t hi = uint32_t(dV >> 32);
      uint32_t vc = 0;  // V tiles (steps) of the items before
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int r = item_index(n, cta, G);
        if (r >= num_items) break;
        const Item it = make_item(p, entries, r, n);
        for (int idx = 0; ok && idx < it.U; ++idx) {
          const uint32_t g = vc + uint32_t(idx);
          const uint32_t v = uint32_t(dV) + (g & 1) * uint32_t(L::KV_BYTES >> 4);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const bool need = item_needs(it, h, it.kb0 + idx);
            const uint32_t on = it.kb0 + idx > (h ? it.kb1 : it.kb0) ? 1u : 0u;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // P_0's first phase also says that V tile g has landed (warp 2)
              if (!mbar_wait_warp((half ? p_full0 : p_half0) + 8 * h, g & 1, wc, 13)) {
                ok = false;
                break;
              }
              tc_fence_after();
              if (elect_one()) {
                if (need) {
#pragma unroll
                  for (int kk = 4 * half; kk < 4 * half + 4; ++kk)  // 16 keys: two 8-row atoms
                    mma_ts(tmem_base + T_O + uint32_t(h * 128),
                           tmem_base + T_P + uint32_t(h * 64 + kk * 8),
                           v + uint32_t((kk * 2048) >> 4), hi, id_o, kk > 0 ? 1u : on);
                }
                if (half) {
                  mma_commit(o_done0 + 8 * h);
                  if (h == 1) mma_commit(v_empty0 + 8 * (g & 1));  // both PV products have V
                }
              }
              __syncwarp();
            }
            if (!ok) break;
          }
        }
        vc += uint32_t(it.U);
      }
      if (elect_one()) mma_commit(drain0 + 8);
      mbar_wait_drain(drain0 + 8, 0, drain_ns);
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- V's landings
      // Waits for the V tile of each step, writes zeros over its rows behind the sequence, and
      // arrives on row tile 0's first P barrier. The stage cannot be refilled before that phase
      // completes: the products read it only afterwards.
      uint32_t vc = 0;
      bool ok = true;
      for (int n = 0; ok; ++n) {
        const int r = item_index(n, cta, G);
        if (r >= num_items) break;
        const Item it = make_item(p, entries, r, n);
        for (int idx = 0; idx < it.U; ++idx) {
          const uint32_t g = vc + uint32_t(idx);
          if (!mbar_wait_warp(v_full0 + 8 * (g & 1), (g >> 1) & 1, wc, 17)) {
            ok = false;
            break;
          }
          const int live = it.n - (it.kb0 + idx) * BKV;  // rows of the tile in the sequence
          if (live < BKV) {
            uint8_t* v = smem + L::V_OFF + (g & 1) * L::KV_BYTES;
#pragma unroll 1
            for (int hb = 0; hb < DH / 64; ++hb)
#pragma unroll 4
              for (int b = live * 128 + int(lane) * 16; b < BKV * 128; b += 512)
                *reinterpret_cast<uint4*>(v + hb * BOX + b) = make_uint4(0, 0, 0, 0);
            fence_proxy_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(p_half0);
          if (!mbar_wait_warp(p_half0, g & 1, wc, 19)) {
            ok = false;
            break;
          }
        }
        vc += uint32_t(it.U);
      }
      __syncwarp();
    }
  } else {
    setmaxnreg_inc<kRegsSoftmax>();
    // ------------------------------------------------------------------ softmax
    const int h = (warp >= 8) ? 1 : 0;  // row tile of this warpgroup
    const uint32_t quad = warp & 3;
    const int row = int(quad * 32 + lane);  // = lane of tensor memory
    const int tok = row / p.group;
    // the warp's first and last token
    const int warp_tok0 = int(quad * 32) / p.group, warp_tok1 = int(quad * 32 + 31) / p.group;
    const uint32_t lane_addr = (quad * 32u) << 16;
    const uint32_t t_s = tmem_base + lane_addr;
    const uint32_t t_p = tmem_base + lane_addr + 128u + uint32_t(h * 64);
    const uint32_t t_o = tmem_base + lane_addr + 256u + uint32_t(h * 128);
    const uint32_t s_full = s_full0 + 8 * h, p_half = p_half0 + 8 * h, p_full = p_full0 + 8 * h;
    const float c = p.scale_log2;
    uint32_t tb = 0;  // tiles of earlier items
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int ri = item_index(n, cta, G);
      if (ri >= num_items) break;
      const Item it = make_item(p, entries, ri, n);
      const int qb = it.q0 + h * p.tile_tokens;
      const int i = qb + tok;  // place in the sequence
      const int kb_h = h ? it.kb1 : it.kb0, ke_h = h ? it.ke1 : it.ke0;
      const int warp_first = qb + warp_tok0, warp_last = qb + warp_tok1;
      float m_used = -INFINITY, l = 0.f;
      bool has_o = false;
      for (int idx = 0; idx < it.U; ++idx) {
        const int j = it.kb0 + idx;
        if (!mbar_wait_warp(s_full, (tb + uint32_t(idx)) & 1, wc, 16)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (j >= kb_h && j <= ke_h) {
          const int k0 = j * BKV;
          if (k0 + BKV - 1 > warp_first || warp_last - k0 >= p.window) {
            // Scores that the token does not see become -inf where they lie, in a pass of its own:
            // as a branch on the 128 values in registers it costs every tile 260 cycles.
#pragma unroll 1
            for (int ch = 0; ch < BKV / 32; ++ch) {
              const int kf = k0 + ch * 32;
              if (kf + 31 <= warp_first && warp_last - kf < p.window) continue;  // all see these
              uint32_t w[32];
              tmem_ld32(t_s + uint32_t(ch * 32), w);
              tmem_ld_wait(w);
#pragma unroll
              for (int e = 0; e < 32; ++e)  // 0 <= i - k < window in one comparison
                if (uint32_t(i - (kf + e)) >= uint32_t(p.window)) w[e] = 0xff800000u;
              tmem_st32(t_s + uint32_t(ch * 32), w);
            }
            tmem_st_wait();
          }
          uint32_t u[BKV];
#pragma unroll
          for (int ch = 0; ch < BKV / 32; ++ch)
            tmem_ld32(t_s + uint32_t(ch * 32), *reinterpret_cast<uint32_t(*)[32]>(u + ch * 32));
          tmem_ld_wait(*reinterpret_cast<uint32_t(*)[32]>(u));
          tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(u + 32));
          tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(u + 64));
          tmem_ld_wait_regs(*reinterpret_cast<uint32_t(*)[32]>(u + 96));
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_free);  // the other tile's scores may overwrite these
          float s[BKV];
#pragma unroll
          for (int e = 0; e < BKV; ++e) s[e] = __uint_as_float(u[e]);
          float mx4[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            float a = s[32 * q];
#pragma unroll
            for (int e = 1; e < 31; e += 2) a = max3f(a, s[32 * q + e], s[32 * q + e + 1]);
            mx4[q] = fmaxf(a, s[32 * q + 31]);
          }
          const float mx = fmaxf(max3f(mx4[0], mx4[1], mx4[2]), mx4[3]);
          const float mxs = mx * c;
          // the reference maximum moves only when the row's grew by more than 2^8 (from -inf, any
          // finite one does); O is rescaled below, after P is stored
          const bool grow = mxs > m_used + kRescaleThreshold;
          const float alpha = grow ? ex2_approx(m_used - mxs) : 1.f;
          if (grow) {
            l *= alpha;
            m_used = mxs;
          }
          const float m_eff = (m_used == -INFINITY) ? 0.f : m_used;
          uint64_t acc[4] = {0, 0, 0, 0};
          // the product of the step before has read P and added to O
          if (!mbar_wait_warp(o_done0 + 8 * h, (tb + uint32_t(idx) + 1) & 1, wc, 18)) {
            ok = false;
            break;
          }
          tc_fence_after();
          probs_to_tmem(s, 0, c, m_eff, t_p, acc);
          if (has_o && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
            for (int ch = 0; ch < DH / 32; ++ch) {
              uint32_t w[32];
              tmem_ld32(t_o + uint32_t(ch * 32), w);
              tmem_ld_wait(w);
#pragma unroll
              for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * alpha);
              tmem_st32(t_o + uint32_t(ch * 32), w);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_half);
          probs_to_tmem(s, 64, c, m_eff, t_p + 32u, acc);
          const uint64_t a2 = f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3]));
          float a_lo, a_hi;
          f2_split(a2, a_lo, a_hi);
          l += a_lo + a_hi;
          has_o = true;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full);
        } else {
          if (!mbar_wait_warp(o_done0 + 8 * h, (tb + uint32_t(idx) + 1) & 1, wc, 18)) {
            ok = false;
            break;
          }
          if (lane == 0) {
            mbar_arrive(s_free);
            mbar_arrive(p_half);
            mbar_arrive(p_full);
          }
        }
      }
      if (!ok) break;
      tb += uint32_t(it.U);
      if (!mbar_wait_warp(o_done0 + 8 * h, (tb + 1) & 1, wc, 18)) break;
      if (has_o) {
        tc_fence_after();
        const float inv_l = 1.f / l;
        // Four lanes exchange 16-byte pieces and store 64 bytes of one of their rows at a time: a
        // store of one row a lane would touch 32 lines.
        __nv_bfloat16* dst[4];  // this lane's pieces of the four rows, or null
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int rr = int(quad * 32 + (lane & ~3u)) + q, tt = rr / p.group;
          dst[q] = tt < p.tile_tokens && qb + tt < it.n
                       ? p.out + int64_t(it.first + qb + tt) * p.out_ss +
                             int64_t(it.kv * p.group + rr - tt * p.group) * p.out_hs + (lane & 3) * 8
                       : nullptr;
        }
#pragma unroll 1  // once an item: cold instructions cost more than the loop
        for (int ch = 0; ch < DH / 32; ++ch) {
          uint32_t u[32];
          tmem_ld32(t_o + uint32_t(ch * 32), u);
          tmem_ld_wait(u);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            w[e] = pack_bf16x2(__uint_as_float(u[2 * e]) * inv_l,
                               __uint_as_float(u[2 * e + 1]) * inv_l);
          transpose_pieces(w);
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (dst[q] != nullptr)
              reinterpret_cast<uint4*>(dst[q])[ch * 4] =
                  make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
        }
      }
    }  // items
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

int64_t most_entries(int64_t tokens, int64_t sequences, int tile_tokens) {
  return tokens / (2 * tile_tokens) + sequences;
}

template <int DH>
cudaError_t launch(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV,
                   const Params& p, void* scratch, int* status, cudaStream_t stream) {
  using L = Layout<DH>;
  static PerDeviceInit setup;  // per device: the shared-memory opt-in, and the number of SMs
  int sms = 0;
  cudaError_t e = per_device_init(
      setup,
      [](int dev, int* value) {
        const cudaError_t a = cudaFuncSetAttribute(
            prompt_kernel<DH>, cudaFuncAttributeMaxDynamicSharedMemorySize, int(L::SMEM));
        return a != cudaSuccess
                   ? a
                   : cudaDeviceGetAttribute(value, cudaDevAttrMultiProcessorCount, dev);
      },
      &sms);
  if (e != cudaSuccess) return e;
  int* count = static_cast<int*>(scratch);
  Entry* entries = reinterpret_cast<Entry*>(static_cast<uint8_t*>(scratch) + kHeaderBytes);
  const int64_t items = int64_t(p.capacity) * p.kv_heads;
  // Few sequences and items: each block lists its own. With a launch for the list 128 tokens take 7.8
  // us instead of 6.3, the ragged 8096 tokens 96 instead of 94, 128 sequences of 64 tokens 50.0 instead
  // of 45.9 (129, listed by the launch: 50.4), 128 of one token 39 instead of 35. Near 64 items an SM the
  // launch is as good or better, by 2 % at most: 8192 tokens, window 64, 296 heads over 148 (9620 items)
  // 399 us instead of 408, 148 over 148 255 instead of 257, 8 x 1024 with 128 heads 209 instead of 212.
  Params mine = p;
  mine.own_list = p.sequences <= kOwnSequences && items <= int64_t(kOwnItems) * sms;
  if (!mine.own_list) {
    e = launch_dependent(list_kernel, dim3(1), dim3(1024), 0, 1, stream, p, count, entries, status);
    if (e != cudaSuccess) return e;
  }
  return launch_dependent(prompt_kernel<DH>, dim3(unsigned(items < sms ? items : sms)),
                          dim3(THREADS), L::SMEM, 1, stream, tmQ, tmK, tmV, mine,
                          static_cast<const int*>(count), static_cast<const Entry*>(entries), status);
}

}  // namespace
}  // namespace pb

using namespace pb;

extern "C" {

pb_status pb_prompt_attention_scratch_bytes(int32_t tokens, int32_t sequences, size_t* bytes) {
  if (bytes == nullptr) return record_error(PB_ERR_INVALID_ARG, "bytes is NULL");
  if (tokens < 0 || sequences < 0)
    return record_error(PB_ERR_INVALID_ARG, "tokens and sequences must be >= 0");
  *bytes = kHeaderBytes + size_t(most_entries(tokens, sequences, 1)) * sizeof(Entry);
  return PB_OK;
}

pb_status pb_prompt_attention(const pb_prompt_args* args, void* scratch, size_t scratch_bytes,
                              int* status, void* stream) {
  if (args == nullptr) return record_error(PB_ERR_INVALID_ARG, "args is NULL");
  const pb_prompt_args& a = *args;
  if (a.tokens < 0 || a.sequences < 0)
    return record_error(PB_ERR_INVALID_ARG, "tokens and sequences must be >= 0");
  if (a.head_dim != 64 && a.head_dim != 128)
    return record_error(PB_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (a.window < 0) return record_error(PB_ERR_INVALID_ARG, "window must be >= 0");
  if (!(a.scale >= 0.f && a.scale <= 0x1p127f))  // log2(e) times it is finite
    return record_error(PB_ERR_INVALID_ARG, "scale must be between 0 and 2^127");
  if (a.tokens > 0x7fffffff - 1024)  // tiles end up to 256 rows behind the last token
    return record_error(PB_ERR_UNSUPPORTED, "more than 2^31 - 1025 tokens");
  if (a.sequences > (1 << 24))
    return record_error(PB_ERR_UNSUPPORTED, "more than 2^24 sequences");
  if (a.tokens == 0 || a.sequences == 0) return PB_OK;
  if (a.starts == nullptr && a.sequences != 1)
    return record_error(PB_ERR_INVALID_ARG, "starts may be NULL for one sequence only");
  if ((reinterpret_cast<uintptr_t>(a.starts) & 3) != 0)
    return record_error(PB_ERR_INVALID_ARG, "starts must be 4-byte aligned");
  const pb_heads* view[4] = {&a.q, &a.k, &a.v, &a.out};
  static const char* const name[4] = {"q", "k", "v", "out"};
  for (int i = 0; i < 4; ++i) {
    pb_status s = check_view(view[i], name[i], 1, a.tokens, a.head_dim, i == 3);
    if (s != PB_OK) return s;
  }
  if (a.k.heads != a.v.heads)
    return record_error(PB_ERR_INVALID_ARG, "k and v have different numbers of heads");
  if (a.q.heads != a.out.heads)
    return record_error(PB_ERR_INVALID_ARG, "q and out have different numbers of heads");
  if (a.q.heads % a.k.heads != 0)
    return record_error(PB_ERR_INVALID_ARG, "q's heads must be a multiple of k's");
  const int group = a.q.heads / a.k.heads;
  if (group > BQ)
    return record_error(PB_ERR_UNSUPPORTED, "more than 128 heads of q for one of k");
  for (int i = 0; i < 3; ++i)  // a tensor map's strides have 40 bits; broadcast views have none
    if ((a.tokens > 1 && (view[i]->seq_stride < a.head_dim ||
                          view[i]->seq_stride >= (int64_t(1) << 38))) ||
        (view[i]->heads > 1 && (view[i]->head_stride < a.head_dim ||
                                view[i]->head_stride >= (int64_t(1) << 38))))
      return bad(PB_ERR_UNSUPPORTED, "%s: strides must be head_dim at least, and below 2^38",
                 name[i]);
  for (int i = 0; i < 3; ++i)
    if (!disjoint(a.out, *view[i], 1, a.tokens, a.head_dim))
      return bad(PB_ERR_INVALID_ARG, "out overlaps %s", name[i]);
  const int tile_tokens = BQ / group;
  const int64_t capacity = most_entries(a.tokens, a.sequences, tile_tokens);
  const size_t need = kHeaderBytes + size_t(capacity) * sizeof(Entry);
  if (scratch == nullptr || (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
    return record_error(PB_ERR_INVALID_ARG, "scratch must be a 256-byte aligned device pointer");
  if (scratch_bytes < need)
    return record_error(PB_ERR_WORKSPACE, "scratch is smaller than pb_prompt_attention_scratch_bytes");
  if (capacity * a.k.heads > 0x7fffffff - 65536)
    return record_error(PB_ERR_UNSUPPORTED, "more than 2^31 items of work");
  const Flat scr{scratch, need}, starts{a.starts, a.starts ? (size_t(a.sequences) + 1) * 4 : 0};
  for (int i = 0; i < 4; ++i)
    if (!apart(scr, view[i], 1, a.tokens, a.head_dim))
      return bad(PB_ERR_INVALID_ARG, "%s overlaps scratch", name[i]);
  if (!apart(starts, &a.out, 1, a.tokens, a.head_dim) || !apart(starts, scr))
    return record_error(PB_ERR_INVALID_ARG, "starts overlaps out or scratch");

  CUtensorMap tm[3];
  const uint32_t box[3][2] = {{uint32_t(group), uint32_t(tile_tokens)}, {1, BKV}, {1, BKV}};
  for (int i = 0; i < 3; ++i) {
    const pb_status s = make_heads_map(&tm[i], *view[i], a.tokens, a.head_dim, box[i][0], box[i][1]);
    if (s != PB_OK) return s;
  }
  Params p{};
  p.tokens = a.tokens;
  p.sequences = a.sequences;
  p.kv_heads = a.k.heads;
  p.group = group;
  p.tile_tokens = tile_tokens;
  p.window = a.window == 0 ? 0x7fffffff : a.window;
  const double scale = a.scale == 0.f ? 1.0 / std::sqrt(double(a.head_dim)) : double(a.scale);
  p.scale_log2 = float(1.4426950408889634 * scale);
  while (((a.tokens / (2 * tile_tokens)) >> p.shift) >= kBuckets) ++p.shift;
  p.capacity = int(capacity);
  p.starts = a.starts;
  p.out = static_cast<__nv_bfloat16*>(a.out.ptr);
  p.out_ss = a.tokens > 1 ? a.out.seq_stride : 0;
  p.out_hs = a.out.heads > 1 ? a.out.head_stride : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = a.head_dim == 128 ? launch<128>(tm[0], tm[1], tm[2], p, scratch, status, st)
                                          : launch<64>(tm[0], tm[1], tm[2], p, scratch, status, st);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "prompt attention launch");
}

}  // extern "C"
