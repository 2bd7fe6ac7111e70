// cache_attention.cu — attention of new tokens (one of a decoding step, a tree of drafted ones, a
// piece of a prompt) over a paged cache.
//
// New token t of a sequence with b tokens before the new ones, at depth d(t) of its path:
//   out_t = sum_j softmax_j(scale q_t . k_j) v_j
// over the cached tokens j < b with b + d(t) - j < w, and the new tokens u on t's path (itself
// included) with d(t) - d(u) < w. Query head h reads key head h / g.
//
// For few query rows the work is reading k and v once: 4 dh bytes a key and key head for 4 dh g c
// operations (g heads, c new tokens). A block of 4 warps takes MB = 16, 32 or 64 rows (row r: head r
// mod g of token r / g) of one key head, and tiles of 64 keys, two blocks an SM; products by mma.sync,
// whose rate (1024 multiplications a cycle and SM) a block of 64 rows would need 2/3 of at the rate
// of memory. With 64 rows each warp has 16 rows and all keys of a tile; with 32 two warps, with 16 four
// warps share the rows and split the keys, each with a softmax of its own, merged in shared memory at
// the end. (64 rows as one block an SM of 8 or 16 warps and tiles of 128 keys: 61 to 70 us where this
// takes 58.)
//
// Split. All tiles of all (sequence, key head, block of rows) form one line, of which every block
// takes an equal share, whatever it cuts: one long sequence fills the GPU as well as many, and
// ragged lengths cost nothing. A piece of an item that does not hold all of its keys leaves the
// maximum, the sum and the unnormed result in scratch (fp32); a second launch joins the pieces of an
// item in their order. No atomics: the same call gives the same bits.
//
// Pages. The rows of a tile are found by the table, one lookup a row, tiles ahead of its loads, so a
// page may have any size. Rows come by 16-byte asynchronous copies into a ring of stages, chunk c of
// row r at place c ^ (r mod 8), which ldmatrix reads without conflicts. Rows behind the sequence (a
// last page's rest) arrive as zeros: what the pool holds there reaches nothing. Weights are rounded
// to bf16 for the product with v; scores, maximum, sums and results are fp32.
//
// Measured (in a graph): 64 sequences of 500 to 8192 tokens, 32 heads over 8 of 128, 183 us (6.6 TB/s,
// 98 % of a plain copy); one of 131072 tokens 87 us (6.1 TB/s); 8 sequences with 16 drafts each, 58 us
// (3.6 TB/s: bound by latency inside the tiles and 6 us of start, cold instructions among it); one
// token over 500, 4 heads of 64, 6.3 us: five accesses that depend on one another, twice a launch. Many
// tokens in a line read the cache once for 64 rows: the last 512 of 16384, 32 heads over 8, 406 us, the
// last 4096 of 20480 3.5 ms (330 and 350 TFLOP/s).
#include <cuda_bf16.h>

#include <climits>
#include <cmath>

#include "cache.h"
#include "kernels.h"
#include "ptx.cuh"

namespace pb {
namespace {

constexpr int kRing = 8;       // tiles whose rows' places are known
constexpr int kMostTree = 64;  // a bit each
constexpr int kMaxSms = 192;
constexpr float kRescaleThreshold = 8.0f;  // log2 units

constexpr int THREADS = 128, BK = 64, kBlocksPerSm = 2;

// A block of MB query rows.
template <int MB>
struct Shape {
  static constexpr int RW = MB / 16, KW = 4 / RW;  // warps along rows, along keys
  static constexpr int KPW = BK / KW;              // keys of a tile a warp takes
};

// Of one block, two pieces at most do not hold their whole item: the one that it begins with (the
// item began in a block before) and the one that it ends with.
struct Piece {
  int state;        // see below
  int token, row0;  // the item's first new token in the call, its first row
  int rows, kv;     // rows of the sequence (g c), key head
  int pad[3];
};
enum : int { kNone = 0, kGoesOn = 1, kEnds = 2 };

struct Params {
  int n, tokens, group;
  int kv_heads, pages, page_size, page_shift, slots, slot_pages;  // page_shift < 0: no power of two
  int window;
  float scale_log2;
  const __nv_bfloat16 *q, *k, *v;  // k and v: of the layer
  int64_t q_token, q_head;
  __nv_bfloat16* out;
  int64_t out_token, out_head;
  const int *slot, *starts, *parents, *table, *lengths;
  int* status;
  Piece* pieces;  // [blocks][2]
  float* parts;   // [blocks][2][rows][dh + 4]: the result, the maximum, the sum
};

struct Seq {
  int slot, first, count, base, len;
};

// Listed sequence i; count 0 where it has no new tokens or is at fault.
__device__ __forceinline__ Seq sequence(const Params& p, int i, bool report) {
  Seq s;
  s.first = p.starts[i];
  const int64_t count = int64_t(p.starts[i + 1]) - s.first;
  s.slot = p.slot[i];
  s.count = 0;
  s.len = 0;
  int fault = 0;
  if (s.slot < 0 || s.slot >= p.slots) {
    fault = kFaultSlot;
  } else {
    s.len = p.lengths[s.slot];
    if (s.len < 0 || s.len > p.slot_pages * p.page_size)
      fault = kFaultTable;
    else if (s.first < 0 || count < 0 || count > p.tokens - s.first || count > s.len ||
             (p.parents != nullptr && count > kMostTree))
      fault = kFaultCounts;
    else
      s.count = int(count);
  }
  s.base = s.len - s.count;
  if (fault != 0 && report) cache_fault(p.status, fault);
  return s;
}

// a / b for a >= 0, b > 0: in 32 bits where both fit.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? int64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// The end of the keys that block of rows b sees.
template <int MB>
__device__ __forceinline__ int end_of(const Params& p, const Seq& s, int b) {
  return p.parents != nullptr || s.count * p.group <= (b + 1) * MB
             ? s.len
             : s.base + ((b + 1) * MB - 1) / p.group + 1;
}
// Key tiles [from, to) that block of rows b needs: from the first of its first row.
template <int MB>
__device__ __forceinline__ int2 tiles_of(const Params& p, const Seq& s, int b) {
  const int from = s.base + (p.parents == nullptr && b > 0 ? b * MB / p.group : 0);
  return make_int2(max(0, from - p.window + 1) / BK, (end_of<MB>(p, s, b) + BK - 1) / BK);
}
template <int MB>
__device__ __forceinline__ int64_t head_tiles(const Params& p, const Seq& s) {
  int64_t sum = 0;
  for (int b = 0; b * MB < s.count * p.group; ++b) {
    const int2 t = tiles_of<MB>(p, s, b);
    sum += t.y - t.x;
  }
  return sum;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int DH, int MB>
struct Layout {
  static constexpr int TILE = BK * DH * 2;  // of k or v
  static constexpr int STAGES = DH == 128 ? 3 : 6;
  static constexpr int RING_OFF = STAGES * 2 * TILE;
  static constexpr int ROW_OFF = RING_OFF + kRing * BK * 8;  // paths of the new tokens
  static constexpr int SMEM = ROW_OFF + kMostTree * (8 + 4);
  static constexpr int PITCH = DH + 4;  // of the warps' parts
  static_assert(STAGES + 1 < kRing && SMEM <= 111 * 1024, "shared memory");
  static_assert(RING_OFF >= Shape<MB>::KW * MB * (PITCH + 2) * 4, "merge buffer");
};

template <int DH, int MB>
__global__ void __launch_bounds__(THREADS, kBlocksPerSm) attention_kernel(const Params p) {
  using L = Layout<DH, MB>;
  using T = Shape<MB>;
  constexpr int S = L::STAGES, CH = DH / 8;  // 16-byte chunks of a row
  constexpr int RW = T::RW, KW = T::KW, KPW = T::KPW;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ int64_t sums[4];
  __shared__ int64_t found_tile;
  __shared__ Seq found;
  __shared__ int found_i, faulted;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rw = warp % RW, kw = warp / RW;
  int64_t* ring = reinterpret_cast<int64_t*>(smem + L::RING_OFF);
  uint64_t* above = reinterpret_cast<uint64_t*>(smem + L::ROW_OFF);  // tree: a token's path
  int* depth = reinterpret_cast<int*>(above + kMostTree);
  const uint32_t s0 = smem_u32(smem);
  Piece* const mine = p.pieces + 2 * blockIdx.x;
  pdl_wait();
  pdl_trigger();
  if (tid < 2) mine[tid].state = kNone;

  // -------------------------------------------------------------- the block's share of the line
  int status = 0;
  if (tid == 0) status = *reinterpret_cast<volatile int*>(p.status);
  Seq sq{};             // the sequence at which the share begins
  int seq_i = 0;        // its place in the list
  int64_t found_at = 0; // tiles before the share's first in it
  int64_t left = 0;     // tiles to go
  // The share of `all` tiles: its first tile; false where there are fewer tiles than blocks.
  auto share = [&](int64_t all, int64_t* first) {
    const int64_t blocks = all < int64_t(gridDim.x) ? all : int64_t(gridDim.x), b = blockIdx.x;
    if (b >= blocks) return false;
    const int64_t each = divide(all, blocks), more = all - each * blocks;
    *first = each * b + (b < more ? b : more);
    left = each + (b < more ? 1 : 0);
    return true;
  };
  auto scan = [&](int64_t x) {  // inclusive sums over the warp
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
      if (lane >= d) x += y;
    }
    return x;
  };
  if (p.n <= 32) {  // a lane a sequence, every warp for itself
    int64_t x = 0, first = 0;
    if (lane < p.n) {
      sq = sequence(p, lane, blockIdx.x == 0);
      x = head_tiles<MB>(p, sq) * p.kv_heads;
    }
    const int64_t to = scan(x);
    if (!share(__shfl_sync(0xffffffffu, to, 31), &first)) return;
    seq_i = __ffs(int(__ballot_sync(0xffffffffu, first < to))) - 1;
    found_at = first - __shfl_sync(0xffffffffu, to - x, seq_i);
    sq.slot = __shfl_sync(0xffffffffu, sq.slot, seq_i);
    sq.first = __shfl_sync(0xffffffffu, sq.first, seq_i);
    sq.count = __shfl_sync(0xffffffffu, sq.count, seq_i);
    sq.base = __shfl_sync(0xffffffffu, sq.base, seq_i);
    sq.len = __shfl_sync(0xffffffffu, sq.len, seq_i);
  } else {  // a thread a sequence
    int64_t own = 0, all = 0, first = 0, before = 0;
    if (tid < p.n) {
      sq = sequence(p, tid, blockIdx.x == 0);
      own = head_tiles<MB>(p, sq) * p.kv_heads;
    }
    for (int i = tid + THREADS; i < p.n; i += THREADS)
      all += head_tiles<MB>(p, sequence(p, i, blockIdx.x == 0)) * p.kv_heads;
    all = scan(all + own);
    if (lane == 31) sums[warp] = all;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) all += sums[w];
    if (!share(all, &first)) return;
    for (int i0 = 0; i0 < p.n; i0 += THREADS) {
      const int i = i0 + tid;
      int64_t x = own;
      if (i0 > 0) {
        x = 0;
        if (i < p.n) {
          sq = sequence(p, i, false);
          x = head_tiles<MB>(p, sq) * p.kv_heads;
        }
      }
      const int64_t to = scan(x);
      __syncthreads();
      if (lane == 31) sums[warp] = to;
      __syncthreads();
      int64_t at = before + to - x;
      for (int w = 0; w < 4; ++w) {
        at += w < warp ? sums[w] : 0;
        before += sums[w];
      }
      if (first >= at && first < at + x) {
        found = sq;
        found_i = i;
        found_tile = first - at;
      }
      if (before > first) break;  // the same for all threads
    }
    __syncthreads();
    seq_i = found_i;
    sq = found;
    found_at = found_tile;
  }
  // A fault may be recorded while the block's warps read the word: one thread's reading counts for
  // all, and is looked at behind the first barrier that the block comes to anyway. What is read before
  // lies within the tables and tensors, whatever they hold.
  if (tid == 0) faulted = status;
  int kv, blk = 0, t_off;
  {
    const int64_t per = head_tiles<MB>(p, sq);
    kv = int(divide(found_at, per));
    int64_t off = found_at - kv * per;
    int2 t = tiles_of<MB>(p, sq, 0);
    while (off >= t.y - t.x) {
      off -= t.y - t.x;
      t = tiles_of<MB>(p, sq, ++blk);
    }
    t_off = int(off);
  }

  const int c_row = tid / CH, c_chunk = tid % CH;  // loads: rows c_row, c_row + THREADS / CH, ...
  constexpr int ROWS_PASS = THREADS / CH;
  // ldmatrix: this lane's row and chunk inside a group of four 8 x 8 matrices
  const int k_row = ((lane >> 4) << 3) + (lane & 7), k_chunk = (lane >> 3) & 1;
  const int v_row = lane & 15, v_chunk = lane >> 4;

  for (;;) {
    // ------------------------------------------------------------ a piece: tiles [ta, ta + m) of an item
    const int2 range = tiles_of<MB>(p, sq, blk);
    const int whole = range.y - range.x;
    const int m = int(left < whole - t_off ? left : whole - t_off);
    const int ta = range.x + t_off;
    const int rows = sq.count * p.group, row0 = blk * MB;
    const int end = end_of<MB>(p, sq, blk);
    const int* row_table = p.table + int64_t(sq.slot) * p.slot_pages;

    auto page_index = [&](int pos) {
      return p.page_shift >= 0 ? pos >> p.page_shift : pos / p.page_size;
    };
    // key row r of tile i (counted from ta): its page's entry, 0 where there is no such key
    auto entry = [&](int i, int r) {
      const int pos = (ta + i) * BK + r;
      return i < m && pos < end ? row_table[page_index(pos)] : 0;
    };
    // the values before that row in the layer's k, or -1 where there is no such key
    auto place = [&](int page, int i, int r) -> int64_t {
      const int pos = (ta + i) * BK + r;
      if (i >= m || pos >= end) return -1;
      if (page < 0 || page >= p.pages) {
        cache_fault(p.status, kFaultTable);
        return -1;
      }
      const int at = pos - page_index(pos) * p.page_size;
      return ((int64_t(page) * p.kv_heads + kv) * p.page_size + at) * DH;
    };
    auto load = [&](int i) {  // tile i into its stage; always a group of copies
      if (i < m) {
        const uint32_t st = s0 + uint32_t(i % S) * uint32_t(2 * L::TILE);
#pragma unroll
        for (int r = c_row; r < BK; r += ROWS_PASS) {
          const int64_t at = ring[(i % kRing) * BK + r];
          const bool live = at >= 0;
          const int64_t o = (live ? at : 0) + c_chunk * 8;
          const uint32_t dst = st + uint32_t(r * DH * 2) + uint32_t((c_chunk ^ (r & 7)) * 16);
          cp16(dst, p.k + o, live);
          cp16(dst + L::TILE, p.v + o, live);
        }
      }
      cp_commit();
    };

    // What the piece needs from memory first, all on its way at once: pages of the first tiles, the
    // rows' queries, the new tokens' parents.
    constexpr int PLACES = (S * BK + THREADS - 1) / THREADS;
    int first_pages[PLACES];
#pragma unroll
    for (int x = 0; x < PLACES; ++x) {
      const int at = tid + x * THREADS;
      first_pages[x] = at < S * BK ? entry(at / BK, at % BK) : 0;
    }
    int page_ahead = tid < BK ? entry(S, tid) : 0;
    constexpr int QUERIES = MB * CH / THREADS;
    uint4 queries[QUERIES];
#pragma unroll
    for (int x = 0; x < QUERIES; ++x) {
      const int r = (tid + x * THREADS) / CH, ch = tid % CH, rr = row0 + r;
      queries[x] = make_uint4(0, 0, 0, 0);
      if (rr < rows) {
        const int t = rr / p.group, h = rr - t * p.group;
        queries[x] = *reinterpret_cast<const uint4*>(p.q + int64_t(sq.first + t) * p.q_token +
                                                     int64_t(kv * p.group + h) * p.q_head + ch * 8);
      }
    }
    int parent = -1;
    if (p.parents != nullptr && tid < sq.count) parent = p.parents[sq.first + tid];
    __syncthreads();  // the piece before is done with shared memory
    if (faulted != 0) return;
#pragma unroll
    for (int x = 0; x < PLACES; ++x) {
      const int at = tid + x * THREADS;
      if (at < S * BK) ring[at] = place(first_pages[x], at / BK, at % BK);
    }
    // the queries pass through the last stage's place on to registers
    constexpr uint32_t qs = (S - 1) * 2 * L::TILE;
#pragma unroll
    for (int x = 0; x < QUERIES; ++x) {
      const int r = (tid + x * THREADS) / CH, ch = tid % CH;
      *reinterpret_cast<uint4*>(smem + qs + r * DH * 2 + ((ch ^ (r & 7)) * 16)) = queries[x];
    }
    if (p.parents != nullptr && tid < sq.count) depth[tid] = parent;
    __syncthreads();
#pragma unroll 1  // one copy of the code: cold instructions cost more than the loop
    for (int i = 0; i < S - 1; ++i) load(i);
    if (p.parents != nullptr) {
      // walk to the root: 64 steps at most, since a parent comes before its child
      int d = 0;
      uint64_t bits = 0;
      if (tid < sq.count) {
        for (int u = tid;;) {
          if (d < p.window) bits |= uint64_t(1) << u;
          const int up = depth[u];
          if (up < 0 || up >= u) break;
          u = up;
          ++d;
        }
      }
      __syncthreads();
      if (tid < sq.count) {
        above[tid] = bits;
        depth[tid] = d;
      }
    }
    uint32_t qf[DH / 16][4];
#pragma unroll
    for (int ks = 0; ks < DH / 16; ++ks) {
      // A: matrices (rows 0-7, k lo), (rows 8-15, k lo), (rows 0-7, k hi), (rows 8-15, k hi)
      const int r = rw * 16 + (lane & 15), ch = ks * 2 + (lane >> 4);
      ldsm4(s0 + qs + uint32_t(r * DH * 2 + ((ch ^ (r & 7)) * 16)), qf[ks]);
    }
    __syncthreads();
    // this lane's two rows: keys before the new ones from lo on, of the new ones those up to hi (a
    // line) or those in bits (a tree)
    int lo[2], hi[2];
    uint64_t bits[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = row0 + rw * 16 + (lane >> 2) + 8 * e;
      lo[e] = INT_MAX;
      hi[e] = -1;
      bits[e] = 0;
      if (rr < rows) {
        const int t = rr / p.group;
        const int d = p.parents == nullptr ? t : depth[t];
        lo[e] = max(0, sq.base + d - p.window + 1);
        hi[e] = p.parents == nullptr ? sq.base + t : sq.base - 1;
        if (p.parents != nullptr) bits[e] = above[t];
      }
    }
    // keys that all rows of the block see: from all_lo to all_hi
    const int all_hi = p.parents == nullptr ? sq.base + row0 / p.group : sq.base - 1;
    const int all_lo = max(0, sq.len - p.window);

    float o[DH / 8][4];
#pragma unroll
    for (int i = 0; i < DH / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    // the maximum that the weights refer to (log2 units), and their sum
    float mx[2], sum[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[e] = -INFINITY;
      sum[e] = 0.f;
    }

    for (int i = 0; i < m; ++i) {
      cp_wait<S - 2>();
      __syncthreads();  // tile i has landed; everyone is done with the stage that is loaded next
      load(i + S - 1);
      if (tid < BK && i + S < m) {
        ring[((i + S) % kRing) * BK + tid] = place(page_ahead, i + S, tid);
        page_ahead = entry(i + S + 1, tid);
      }
      const uint32_t sk = s0 + uint32_t(i % S) * uint32_t(2 * L::TILE) + uint32_t(kw * KPW * DH * 2);
      float s[KPW / 8][4];
#pragma unroll
      for (int nt = 0; nt < KPW / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < DH / 16; ++ks)
#pragma unroll
        for (int nt = 0; nt < KPW / 16; ++nt) {
          uint32_t b[4];
          const int r = nt * 16 + k_row, ch = ks * 2 + k_chunk;
          ldsm4(sk + uint32_t(r * DH * 2 + ((ch ^ (r & 7)) * 16)), b);
          mma16816(s[2 * nt], qf[ks], b[0], b[1]);
          mma16816(s[2 * nt + 1], qf[ks], b[2], b[3]);
        }
      const int k0 = (ta + i) * BK + kw * KPW;
      if (!(k0 + KPW - 1 <= all_hi && k0 >= all_lo)) {
#pragma unroll
        for (int nt = 0; nt < KPW / 8; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int key = k0 + nt * 8 + (lane & 3) * 2 + (e & 1), w = e >> 1;
            const int u = key - sq.base;
            const bool see = (key >= lo[w] && key <= hi[w]) ||
                             (u >= 0 && u < kMostTree && ((bits[w] >> u) & 1u));
            if (!see) s[nt][e] = -INFINITY;
          }
      }
      // As elsewhere: the reference moves only when a row's maximum grew by more than 2^8 (from
      // -inf, any finite one does), so O is seldom rescaled.
      float ref[2], alpha[2];
      bool moved = false;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        float t = s[0][2 * w];
#pragma unroll
        for (int nt = 0; nt < KPW / 8; ++nt) t = max3f(t, s[nt][2 * w], s[nt][2 * w + 1]);
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 1));
        t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, 2)) * p.scale_log2;
        const bool grow = t > mx[w] + kRescaleThreshold;
        alpha[w] = grow ? ex2_approx(mx[w] - t) : 1.f;
        if (grow) mx[w] = t;
        moved |= grow;
        ref[w] = mx[w] == -INFINITY ? 0.f : mx[w];
      }
      if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          sum[w] *= alpha[w];
#pragma unroll
          for (int j = 0; j < DH / 8; ++j) {
            o[j][2 * w] *= alpha[w];
            o[j][2 * w + 1] *= alpha[w];
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < KPW / 8; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = ex2_approx(fmaf(s[nt][e], p.scale_log2, -ref[e >> 1]));
          sum[e >> 1] += s[nt][e];
        }
      const uint32_t sv = sk + L::TILE;
#pragma unroll
      for (int kt = 0; kt < KPW / 16; ++kt) {
        const uint32_t a[4] = {pack_bf16x2(s[2 * kt][0], s[2 * kt][1]),
                               pack_bf16x2(s[2 * kt][2], s[2 * kt][3]),
                               pack_bf16x2(s[2 * kt + 1][0], s[2 * kt + 1][1]),
                               pack_bf16x2(s[2 * kt + 1][2], s[2 * kt + 1][3])};
#pragma unroll
        for (int j = 0; j < DH / 16; ++j) {
          uint32_t b[4];
          const int r = kt * 16 + v_row, ch = j * 2 + v_chunk;
          ldsm4_t(sv + uint32_t(r * DH * 2 + ((ch ^ (r & 7)) * 16)), b);
          mma16816(o[2 * j], a, b[0], b[1]);
          mma16816(o[2 * j + 1], a, b[2], b[3]);
        }
      }
    }
    cp_wait<0>();
    __syncthreads();  // all tiles are read: shared memory is free for the merge

    // ------------------------------------------------------------ the warps' parts together
    // row r's part of key warp w at (w MB + r)
    constexpr int PITCH = L::PITCH;
    float* parts = reinterpret_cast<float*>(smem);
    float2* stats = reinterpret_cast<float2*>(parts + KW * MB * PITCH);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int at = kw * MB + rw * 16 + (lane >> 2) + 8 * w;
      sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 1);
      sum[w] += __shfl_xor_sync(0xffffffffu, sum[w], 2);
      if ((lane & 3) == 0) stats[at] = make_float2(mx[w], sum[w]);
#pragma unroll
      for (int j = 0; j < DH / 8; ++j)
        *reinterpret_cast<float2*>(parts + at * PITCH + j * 8 + (lane & 3) * 2) =
            make_float2(o[j][2 * w], o[j][2 * w + 1]);
    }
    __syncthreads();
    const bool begins = t_off == 0, ends = t_off + m == whole;
    const int side = begins ? 1 : 0;
    float* part = p.parts + (size_t(blockIdx.x) * 2 + side) * (MB * (DH + 4));
    if (tid == 0 && !(begins && ends)) {
      mine[side].token = sq.first;
      mine[side].row0 = row0;
      mine[side].rows = rows;
      mine[side].kv = kv;
      mine[side].state = ends ? kEnds : kGoesOn;
    }
#pragma unroll
    for (int x0 = 0; x0 < MB * CH; x0 += THREADS) {
      const int r = (x0 + tid) / CH, ch = tid % CH, rr = row0 + r;
      if (rr >= rows) continue;
      float best = -INFINITY, total = 0.f, acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
      float2 st[KW];
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        st[w] = stats[w * MB + r];
        best = fmaxf(best, st[w].x);
      }
      const float ref = best == -INFINITY ? 0.f : best;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float f = ex2_approx(st[w].x - ref);
        total += f * st[w].y;
        const float4* src = reinterpret_cast<const float4*>(parts + (w * MB + r) * PITCH + ch * 8);
        const float4 a = src[0], b = src[1];
        acc[0] += f * a.x;
        acc[1] += f * a.y;
        acc[2] += f * a.z;
        acc[3] += f * a.w;
        acc[4] += f * b.x;
        acc[5] += f * b.y;
        acc[6] += f * b.z;
        acc[7] += f * b.w;
      }
      if (begins && ends) {
        const float inv = 1.f / total;  // a row sees itself at least
        const int t = rr / p.group, h = rr - t * p.group;
        *reinterpret_cast<uint4*>(p.out + int64_t(sq.first + t) * p.out_token +
                                  int64_t(kv * p.group + h) * p.out_head + ch * 8) =
            make_uint4(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv),
                       pack_bf16x2(acc[4] * inv, acc[5] * inv), pack_bf16x2(acc[6] * inv, acc[7] * inv));
      } else {
        float4* dst = reinterpret_cast<float4*>(part + r * (DH + 4) + ch * 8);
        dst[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        dst[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (ch == 0) *reinterpret_cast<float2*>(part + r * (DH + 4) + DH) = make_float2(best, total);
      }
    }

    // ------------------------------------------------------------ on to the next item
    left -= m;
    if (left == 0) break;
    t_off = 0;
    if (++blk * MB >= rows) {
      blk = 0;
      if (++kv == p.kv_heads) {
        kv = 0;
        do sq = sequence(p, ++seq_i, false);
        while (sq.count == 0);
      }
    }
  }
}

// Joins the pieces of the items that several blocks worked on: block (b, y) those of the item that
// begins last in block b, a warp a row.
template <int DH, int MB>
__global__ void __launch_bounds__(128) join_kernel(const Params p) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  const int r = blockIdx.y * 4 + int(threadIdx.x >> 5);
  const Piece head = p.pieces[2 * b + 1];
  // the blocks behind, up to the one in which the item ends
  int pieces = 1;
  for (int i = b + 1;; i += 32) {
    const int state = i + lane < int(gridDim.x) ? p.pieces[2 * (i + lane)].state : kNone;
    if (head.state == kNone || head.row0 + r >= head.rows) return;
    const uint32_t m = __ballot_sync(0xffffffffu, state != kGoesOn);
    if (m != 0) {
      // no end: a block left out its share, since a fault was recorded before it looked
      if (__shfl_sync(0xffffffffu, state, __ffs(int(m)) - 1) != kEnds) return;
      pieces += __ffs(int(m));
      break;
    }
    pieces += 32;
  }
  constexpr int PART = MB * (DH + 4), V = DH / 32, AT_ONCE = 8;
  const float* first = p.parts + (size_t(b) * 2 + 1) * PART + r * (DH + 4);
  float best = -INFINITY, total = 0.f, acc[V];
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.f;
  for (int i0 = 0; i0 < pieces; i0 += AT_ONCE) {
    float2 st[AT_ONCE], x[AT_ONCE][V / 2];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      // piece 0: the block's second; the others: the first of their block
      const int i = i0 + j;
      const float* src = i == 0 ? first : first + size_t(2 * i - 1) * PART;
      st[j] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < V / 2; ++e) x[j][e] = make_float2(0.f, 0.f);
      if (i < pieces) {
        st[j] = *reinterpret_cast<const float2*>(src + DH);
#pragma unroll
        for (int e = 0; e < V / 2; ++e)
          x[j][e] = *reinterpret_cast<const float2*>(src + lane * V + 2 * e);
      }
    }
    float top = best;
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) top = fmaxf(top, st[j].x);
    const float ref = top == -INFINITY ? 0.f : top;
    const float old = ex2_approx(best - ref);
    best = top;
    total *= old;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= old;
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const float f = ex2_approx(st[j].x - ref);
      total += f * st[j].y;
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        acc[2 * e] += f * x[j][e].x;
        acc[2 * e + 1] += f * x[j][e].y;
      }
    }
  }
  const float inv = 1.f / total;
  const int rr = head.row0 + r, t = rr / p.group, h = rr - t * p.group;
  uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + int64_t(head.token + t) * p.out_token +
                                              int64_t(head.kv * p.group + h) * p.out_head + lane * V);
#pragma unroll
  for (int e = 0; e < V; e += 2) dst[e / 2] = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
}

constexpr size_t kMaxBlocks = size_t(kBlocksPerSm) * kMaxSms;
constexpr size_t kPieceBytes = kMaxBlocks * 2 * sizeof(Piece);
size_t scratch_need(int head_dim) { return kPieceBytes + kMaxBlocks * 2 * 64 * (head_dim + 4) * 4; }

template <int DH, int MB>
cudaError_t launch(const Params& p, cudaStream_t stream) {
  using L = Layout<DH, MB>;
  static PerDeviceInit setup;  // per device: the shared-memory opt-in, and the number of SMs
  int sms = 0;
  cudaError_t e = per_device_init(
      setup,
      [](int dev, int* value) {
        const cudaError_t a = cudaFuncSetAttribute(
            attention_kernel<DH, MB>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::SMEM);
        return a != cudaSuccess
                   ? a
                   : cudaDeviceGetAttribute(value, cudaDevAttrMultiProcessorCount, dev);
      },
      &sms);
  if (e != cudaSuccess) return e;
  const unsigned grid = unsigned(kBlocksPerSm * (sms < kMaxSms ? sms : kMaxSms));
  e = launch_dependent(attention_kernel<DH, MB>, dim3(grid), dim3(THREADS), L::SMEM, 1, stream, p);
  if (e != cudaSuccess) return e;
  return launch_dependent(join_kernel<DH, MB>, dim3(grid, MB / 4), dim3(128), 0, 1, stream, p);
}

// The block that holds a sequence's rows, from 8 sequences of 2 to 16 thousand tokens, 8 key heads:
// 16 rows 41.5 us by blocks of 16, 42.7 by 32; 32 rows 57 (16, the cache read twice), 45.9 (32), 54
// (64); 36 rows 58.4 (32), 53.9 (64); 64 rows 68 (32), 58 (64).
// `rows` is the mean of the call's sequences, since their own numbers are on the device only. Where
// they differ much the choice fits the many, and the few with more rows read their cache once for
// every block of theirs: 255 sequences of 2048 tokens with one new token and one of 16384 with 512,
// 4 heads a key head, take 1080 us by blocks of 16 rows (what the mean says) and 801 by 64; 256 with
// one new token each 315 and 411; 15 of 8192 with one and one of 16384 with 16 114 and 120.
template <int DH>
cudaError_t launch_rows(int64_t rows, const Params& p, cudaStream_t stream) {
  return rows <= 16   ? launch<DH, 16>(p, stream)
         : rows <= 32 ? launch<DH, 32>(p, stream)
                      : launch<DH, 64>(p, stream);
}

}  // namespace
}  // namespace pb

using namespace pb;

extern "C" {

pb_status pb_cache_attention_scratch_bytes(const pb_cache* cache, size_t* bytes) {
  if (bytes == nullptr) return record_error(PB_ERR_INVALID_ARG, "bytes is NULL");
  const pb_status s = check_cache_sizes(cache);
  if (s != PB_OK) return s;
  *bytes = scratch_need(cache->head_dim);
  return PB_OK;
}

pb_status pb_cache_attention(const pb_cache* cache, const pb_cache_attention_args* args,
                             void* scratch, size_t scratch_bytes, void* stream) {
  pb_status s = check_cache(cache);
  if (s != PB_OK) return s;
  if (args == nullptr) return record_error(PB_ERR_INVALID_ARG, "args is NULL");
  const pb_cache& c = *cache;
  const pb_cache_attention_args& a = *args;
  if (a.layer < 0 || a.layer >= c.layers)
    return record_error(PB_ERR_INVALID_ARG, "layer is not one of the cache's");
  if (a.sequences < 0 || a.sequences > c.slots)
    return record_error(PB_ERR_INVALID_ARG, "sequences must be between 0 and the cache's slots");
  if (a.tokens < 0 || a.tokens > (1 << 30))
    return record_error(PB_ERR_INVALID_ARG, "tokens must be between 0 and 2^30");
  if (a.window < 0) return record_error(PB_ERR_INVALID_ARG, "window must be >= 0");
  if (!(a.scale >= 0.f && a.scale <= 0x1p127f))  // log2(e) times it is finite
    return record_error(PB_ERR_INVALID_ARG, "scale must be between 0 and 2^127");
  if (a.sequences == 0 || a.tokens == 0) return PB_OK;
  s = check_view(&a.q, "q", 1, a.tokens, c.head_dim, false);
  if (s == PB_OK) s = check_view(&a.out, "out", 1, a.tokens, c.head_dim, true);
  if (s != PB_OK) return s;
  if (a.q.heads != a.out.heads)
    return record_error(PB_ERR_INVALID_ARG, "q and out have different numbers of heads");
  if (a.q.heads % c.kv_heads != 0)
    return record_error(PB_ERR_INVALID_ARG, "q's heads must be a multiple of the cache's kv_heads");
  const int group = a.q.heads / c.kv_heads;
  if (int64_t(a.tokens) * group > (1 << 30))
    return record_error(PB_ERR_UNSUPPORTED, "more than 2^30 rows of q for a head of the cache");
  if (!disjoint(a.out, a.q, 1, a.tokens, c.head_dim))
    return record_error(PB_ERR_INVALID_ARG, "out overlaps q");
  const size_t need = scratch_need(c.head_dim);
  if (scratch == nullptr || (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
    return record_error(PB_ERR_INVALID_ARG, "scratch must be a 256-byte aligned device pointer");
  if (scratch_bytes < need)
    return record_error(PB_ERR_WORKSPACE, "scratch is smaller than pb_cache_attention_scratch_bytes");
  const Flat scr{scratch, need};
  Dim d[3];
  const Flat out{a.out.ptr, size_t(extent(a.out, 1, a.tokens, c.head_dim, d)) * 2};
  if (!apart(scr, &a.q, 1, a.tokens, c.head_dim) || !apart(scr, out) || !apart_from_cache(scr, c))
    return record_error(PB_ERR_INVALID_ARG, "scratch overlaps q, out or the cache");
  if (!apart_from_cache(out, c))
    return record_error(PB_ERR_INVALID_ARG, "out overlaps a buffer of the cache");
  const Flat words[3] = {{a.slots, size_t(a.sequences) * 4},
                         {a.starts, (size_t(a.sequences) + 1) * 4},
                         {a.parents, size_t(a.tokens) * 4}};
  static const char* const name[3] = {"slots", "starts", "parents"};
  for (int i = 0; i < 3; ++i) {
    if ((i < 2 && words[i].p == nullptr) || !aligned4(words[i].p))
      return bad(PB_ERR_INVALID_ARG, "%s must be a 4-byte aligned device pointer", name[i]);
    if (!apart(words[i], out) || !apart(words[i], scr))
      return bad(PB_ERR_INVALID_ARG, "%s overlaps out or scratch", name[i]);
  }
  Params p{};
  p.n = a.sequences;
  p.tokens = a.tokens;
  p.group = group;
  p.kv_heads = c.kv_heads;
  p.pages = c.pages;
  p.page_size = c.page_size;
  p.page_shift = -1;
  for (int i = 0; i < 31; ++i)
    if (c.page_size == 1 << i) p.page_shift = i;
  p.slots = c.slots;
  p.slot_pages = c.slot_pages;
  p.window = a.window == 0 ? INT_MAX : a.window;
  const double scale = a.scale == 0.f ? 1.0 / std::sqrt(double(c.head_dim)) : double(a.scale);
  p.scale_log2 = float(1.4426950408889634 * scale);
  const int64_t layer = int64_t(a.layer) * c.pages * page_values(c);
  p.q = static_cast<const __nv_bfloat16*>(a.q.ptr);
  p.k = static_cast<const __nv_bfloat16*>(c.k) + layer;
  p.v = static_cast<const __nv_bfloat16*>(c.v) + layer;
  p.q_token = a.q.seq_stride;
  p.q_head = a.q.head_stride;
  p.out = static_cast<__nv_bfloat16*>(a.out.ptr);
  p.out_token = a.out.seq_stride;
  p.out_head = a.out.head_stride;
  p.slot = a.slots;
  p.starts = a.starts;
  p.parents = a.parents;
  p.table = c.table;
  p.lengths = c.lengths;
  p.status = c.status;
  p.pieces = static_cast<Piece*>(scratch);
  p.parts = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + kPieceBytes);
  // the mean rows of a sequence (padding counts): any choice is right, not all are as fast
  const int64_t rows = (int64_t(a.tokens) + a.sequences - 1) / a.sequences * group;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = c.head_dim == 128 ? launch_rows<128>(rows, p, st) : launch_rows<64>(rows, p, st);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache attention launch");
}

}  // extern "C"
