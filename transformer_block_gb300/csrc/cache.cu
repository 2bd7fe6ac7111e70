// cache.cu — a paged cache of keys and values: room for new tokens, their rows, the accepted ones of
// drafted tokens moved together, sequences forked and cut.
//
// The table, the lengths and the pages' counts of users live on the device and are changed there, so
// that a decoding loop whose numbers of accepted tokens come out of the model needs no word from the
// host, and can be a captured graph.
//
// Bookkeeping is small (a few thousand words): one block checks a whole call, so that a call at fault
// changes nothing, and does it. It waits for memory, so it takes few steps that depend on one
// another: a thread a sequence for its words, then 16 lanes a sequence for its pages. Free pages are
// those whose count is zero, found in rising order by a scan (one block scan for 4096 pages): their
// numbers depend on nothing but the counts, whatever the order in which sequences came and went, and
// there is no list that could disagree with them. A fork reads all its sources' rows of the table
// before it writes one, since a slot may be read and written in one call.
//
// Data moves by 16-byte accesses, a row of a head (128 or 256 bytes) by 8 or 16 lanes.
//
// Measured (in a graph): 64 sequences, 16 drafts each, 8 layers of 8 heads of 128: cut, extended,
// written and kept in 37 us, of which the 67 MB that the write moves take 12 (a plain copy: 10) and
// the 27 MB of the kept rows 8; the rest is three bookkeeping launches of 3 to 5 us, bound by the four
// to six accesses that depend on one another. 8 sequences of 4096 tokens forked into 64, extended by
// a token and written: 32 us, the copies of the partly filled pages (105 MB, mostly in L2) 12 of them.
// One sequence, 7 drafts, one layer: 17 us, the six launches. A layer's rows alone, as a model has
// them: 2.5 to 4 us a call for 1 to 1024 tokens.
// More sequences or pages than lanes cost turns of the one block. Extended by 20 tokens and cut again:
// 1 to 64 sequences of 100 tokens 7 to 8 us, 256 10, 1000 23. Freed and made anew: one of 131072 tokens
// in pages of 16 72 us, eight 286.
#include <cuda_bf16.h>

#include "cache.h"
#include "kernels.h"
#include "ptx.cuh"

namespace pb {
namespace {

struct Job {  // a listed sequence
  int slot;   // -1: none, or at fault
  int len;    // its length
  int a, b, c, d;  // by the call
};
struct Copy {
  int from, to, rows, pad;
};

// Scratch: header, Job [slots], Copy [slots], free pages [pages] or rows of the table [slots,
// slot_pages].
struct Header {
  int go;      // the call is sound
  int copies;  // pages to copy
};
constexpr size_t kHeaderBytes = 256;

struct Cache {
  int layers, pages, page_size, kv_heads, head_dim, slots, slot_pages;
  __nv_bfloat16 *k, *v;
  int *table, *lengths, *refs, *status;
  Header* header;
  Job* jobs;
  Copy* copies;
  int* list;
};

size_t scratch_need(const pb_cache& c) {
  const size_t list = size_t(c.slots) * c.slot_pages;
  return kHeaderBytes + size_t(c.slots) * (sizeof(Job) + sizeof(Copy)) +
         4 * (list > size_t(c.pages) ? list : size_t(c.pages));
}

Cache device_view(const pb_cache& c, void* scratch) {
  uint8_t* s = static_cast<uint8_t*>(scratch);
  Cache d{c.layers,  c.pages,   c.page_size, c.kv_heads, c.head_dim, c.slots, c.slot_pages,
          static_cast<__nv_bfloat16*>(c.k), static_cast<__nv_bfloat16*>(c.v),
          c.table,   c.lengths, c.refs,      c.status,   nullptr,    nullptr, nullptr, nullptr};
  if (s != nullptr) {
    d.header = reinterpret_cast<Header*>(s);
    d.copies = reinterpret_cast<Copy*>(s + kHeaderBytes);
    d.jobs = reinterpret_cast<Job*>(d.copies + c.slots);
    d.list = reinterpret_cast<int*>(d.jobs + c.slots);
  }
  return d;
}

constexpr int BLOCK = 1024, WARPS = BLOCK / 32;
constexpr int LANES = 16, GROUPS = BLOCK / LANES;  // lanes of a sequence
constexpr int kListed = 2048;                      // free pages listed in shared memory

struct Shared {
  uint32_t seen[kMaxSlots / 32];  // slots listed
  Job job[BLOCK];                 // of the 1024 sequences at work
  int sums[WARPS];
  int list[kListed];
  int fault;
};

__device__ __forceinline__ int pages_of(const Cache& c, int tokens) {
  return (tokens + c.page_size - 1) / c.page_size;
}
// Threads of one block agree on the first fault seen.
__device__ __forceinline__ void set_fault(Shared& sh, int fault) { atomicCAS(&sh.fault, 0, fault); }

// Exclusive sum of x over the block, and the total.
__device__ int block_scan(int x, Shared& sh, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();  // the sums of the scan before are read
  if (lane == 31) sh.sums[warp] = inc;
  __syncthreads();
  const int s = sh.sums[lane];
  int run = s;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, run, d);
    if (lane >= d) run += y;
  }
  *total = __shfl_sync(0xffffffffu, run, 31);
  const int before = __shfl_sync(0xffffffffu, run - s, warp);
  return before + inc - x;
}

// Clears the bits of the slots and tells whether the cache is free of faults (all threads). What a
// thread has read from memory before is on its way meanwhile.
__device__ bool begin(const Cache& c, Shared& sh) {
  for (int i = threadIdx.x; i < (c.slots + 31) / 32; i += BLOCK) sh.seen[i] = 0;
  if (threadIdx.x == 0) {
    sh.fault = *reinterpret_cast<volatile int*>(c.status) != 0 ? -1 : 0;
    if (sh.fault != 0) *c.header = Header{0, 0};
  }
  __syncthreads();
  const bool sound = sh.fault == 0;
  __syncthreads();  // read by all before anyone records a fault
  return sound;
}
// After all checks: records a fault, and whether the call goes on (all threads).
__device__ bool decide(const Cache& c, Shared& sh, int copies) {
  __syncthreads();
  const int fault = sh.fault;
  if (threadIdx.x == 0) {
    c.header->go = fault == 0;
    c.header->copies = fault == 0 ? copies : 0;
    if (fault > 0) cache_fault(c.status, fault);
  }
  return fault == 0;
}
__device__ __forceinline__ bool good_length(const Cache& c, int len) {
  return len >= 0 && len <= c.slot_pages * c.page_size;
}
__device__ __forceinline__ bool good_page(const Cache& c, int page) {
  return page >= 0 && page < c.pages;
}
// A slot of the list, which must not come again: whether it may be used, and its length.
__device__ bool check_slot(const Cache& c, Shared& sh, int slot, int* len) {
  if (slot < 0 || slot >= c.slots ||
      ((atomicOr(&sh.seen[slot >> 5], 1u << (slot & 31)) >> (slot & 31)) & 1u) != 0) {
    set_fault(sh, kFaultSlot);
    return false;
  }
  *len = c.lengths[slot];
  if (!good_length(c, *len)) {
    set_fault(sh, kFaultTable);
    return false;
  }
  return true;
}
// The pages [a, z) of a slot lose a user; LANES lanes.
__device__ __forceinline__ void release(const Cache& c, int slot, int a, int z) {
  const int* row = c.table + int64_t(slot) * c.slot_pages;
#pragma unroll 4
  for (int i = a + int(threadIdx.x % LANES); i < z; i += LANES) atomicSub(&c.refs[row[i]], 1);
}
// Whether the pages [a, z) of a slot are pages; LANES lanes.
__device__ __forceinline__ void check_pages(const Cache& c, Shared& sh, int slot, int a, int z) {
  const int* row = c.table + int64_t(slot) * c.slot_pages;
  bool sound = true;
#pragma unroll 4
  for (int i = a + int(threadIdx.x % LANES); i < z; i += LANES) sound &= good_page(c, row[i]);
  if (!sound) set_fault(sh, kFaultTable);
}
// For every sequence of the list, 1024 at a time: a thread fills its job, kept in scratch too where
// there are more, or where the launch behind reads it; or (filled) the jobs are those of before. Then
// LANES lanes work on each.
template <class Fill, class Work>
__device__ __forceinline__ void each(const Cache& c, Shared& sh, int n, bool keep, Fill&& fill,
                                     Work&& work) {
  const int tid = threadIdx.x;
  for (int i0 = 0; i0 < n; i0 += BLOCK) {
    __syncthreads();
    Job job{-1, 0, 0, 0, 0, 0};
    if (i0 + tid < n) fill(i0 + tid, job);
    sh.job[tid] = job;
    if ((keep || n > BLOCK) && i0 + tid < n) c.jobs[i0 + tid] = job;
    __syncthreads();
    for (int g = tid / LANES; g < min(BLOCK, n - i0); g += GROUPS)
      if (sh.job[g].slot >= 0) work(i0 + g, sh.job[g]);
  }
}
template <class Work>
__device__ __forceinline__ void each_again(const Cache& c, Shared& sh, int n, Work&& work) {
  const int tid = threadIdx.x;
  for (int i0 = 0; i0 < n; i0 += BLOCK) {
    if (n > BLOCK) {
      __syncthreads();
      if (i0 + tid < n) sh.job[tid] = c.jobs[i0 + tid];
      __syncthreads();
    }
    for (int g = tid / LANES; g < min(BLOCK, n - i0); g += GROUPS) work(i0 + g, sh.job[g]);
  }
}

// ------------------------------------------------------------------ extend

__global__ void __launch_bounds__(BLOCK) extend_kernel(const Cache c, int n, const int* slots,
                                                       const int* starts) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int tid = threadIdx.x, lane = tid % LANES;
  pdl_wait();
  pdl_trigger();
  // the first pages' counts: whether they are free is needed last
  int ahead[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) ahead[e] = 4 * tid + e < c.pages ? c.refs[4 * tid + e] : 1;
  const int slot0 = tid < n ? slots[tid] : 0;
  const int start0 = tid < n ? starts[tid] : 0, start1 = tid < n ? starts[tid + 1] : 0;
  if (!begin(c, sh)) return;
  int need_all = 0, copies = 0;
  // job: a: tokens more, b: rank of the first new page, c: whether the last page is copied, d: place
  // in the list of copies
  for (int i0 = 0; i0 < n; i0 += BLOCK) {
    const int i = i0 + tid;
    Job job{-1, 0, 0, 0, 0, 0};
    int need = 0;
    if (i < n) {
      const int slot = i0 == 0 ? slot0 : slots[i];
      const int64_t count =
          i0 == 0 ? int64_t(start1) - start0 : int64_t(starts[i + 1]) - starts[i];
      if (check_slot(c, sh, slot, &job.len)) {
        if (count < 0) {
          set_fault(sh, kFaultCounts);
        } else if (job.len + count > int64_t(c.slot_pages) * c.page_size) {
          set_fault(sh, kFaultRow);
        } else {
          if (count > 0 && job.len % c.page_size != 0) {
            const int page = c.table[int64_t(slot) * c.slot_pages + job.len / c.page_size];
            if (!good_page(c, page))
              set_fault(sh, kFaultTable);
            else
              job.c = c.refs[page] > 1;
          }
          job.slot = slot;
          job.a = int(count);
          need = pages_of(c, int(job.len + count)) - pages_of(c, job.len) + job.c;
        }
      }
    }
    // a page more than there are is as many as any: 1024 of them stay below 2^31
    int total, ctotal;
    job.b = need_all + block_scan(min(need, c.pages + 1), sh, &total);
    job.d = copies + block_scan(job.c, sh, &ctotal);
    sh.job[tid] = job;
    if (n > BLOCK && i < n) c.jobs[i] = job;
    need_all += total;
    copies += ctotal;
    if (need_all > c.pages) {
      set_fault(sh, kFaultPages);
      break;  // the same for all threads
    }
  }
  __syncthreads();
  // the need_all free pages of lowest number
  const bool listed = need_all <= kListed;
  if (sh.fault == 0) {
    int found = 0;
    for (int p0 = 0; p0 < c.pages && found < need_all; p0 += 4 * BLOCK) {
      const int p = p0 + 4 * tid;
      int used[4], zeros = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        used[e] = p0 == 0 ? ahead[e] : p + e < c.pages ? c.refs[p + e] : 1;
        zeros += used[e] == 0;
      }
      int total;
      int rank = found + block_scan(zeros, sh, &total);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (used[e] == 0) {
          if (rank < need_all) (listed ? sh.list : c.list)[rank] = p + e;
          ++rank;
        }
      found += total;
    }
    __syncthreads();  // all have read that there was no fault
    if (found < need_all && tid == 0) set_fault(sh, kFaultPages);
  }
  if (!decide(c, sh, copies)) return;
  const int* list = listed ? sh.list : c.list;
  each_again(c, sh, n, [&](int, const Job& job) {
    int* row = c.table + int64_t(job.slot) * c.slot_pages;
    const int have = pages_of(c, job.len), more = pages_of(c, job.len + job.a) - have;
    for (int j = lane; j < more; j += LANES) {
      const int page = list[job.b + job.c + j];
      row[have + j] = page;
      c.refs[page] = 1;
    }
    if (lane == 0) {
      if (job.c != 0) {
        const int at = job.len / c.page_size, old = row[at], page = list[job.b];
        c.copies[job.d] = Copy{old, page, job.len % c.page_size, 0};
        row[at] = page;
        c.refs[page] = 1;
        atomicSub(&c.refs[old], 1);
      }
      c.lengths[job.slot] = job.len + job.a;
    }
  });
}

// u = quotient d + remainder: in 32 bits where u fits (64-bit divisions by every thread were half of
// the copy's instructions).
__device__ __forceinline__ int64_t divide(int64_t u, int d, int* remainder) {
  if ((u >> 32) == 0) {
    const uint32_t q = uint32_t(u) / uint32_t(d);
    *remainder = int(uint32_t(u) - q * uint32_t(d));
    return q;
  }
  const int64_t q = u / d;
  *remainder = int(u - q * d);
  return q;
}

// Copies the rows of the listed pages, a head of a layer of k or v at a time.
__global__ void __launch_bounds__(256) copy_kernel(const Cache c) {
  pdl_wait();
  pdl_trigger();
  const int64_t units = int64_t(c.header->copies) * c.layers * 2 * c.kv_heads;
  const int64_t plane = int64_t(c.page_size) * c.head_dim;  // values of a head of a page
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    int h, layer;
    const int64_t w = divide(u, c.kv_heads, &h);
    const int which = int(w & 1);
    const Copy t = c.copies[divide(w >> 1, c.layers, &layer)];
    __nv_bfloat16* pool = which ? c.v : c.k;
    const uint4* src = reinterpret_cast<const uint4*>(
        pool + ((int64_t(layer) * c.pages + t.from) * c.kv_heads + h) * plane);
    uint4* dst = reinterpret_cast<uint4*>(
        pool + ((int64_t(layer) * c.pages + t.to) * c.kv_heads + h) * plane);
    const int64_t m = int64_t(t.rows) * (c.head_dim / 8);
    for (int64_t i = threadIdx.x; i < m; i += 1024) {
      uint4 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + 256 * e < m) x[e] = src[i + 256 * e];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + 256 * e < m) dst[i + 256 * e] = x[e];
    }
  }
}

// ------------------------------------------------------------------ write

struct Rows {
  const __nv_bfloat16* p;
  int64_t layer, token, head;  // strides
};

// A warp a token and layer: finds the token's sequence, then copies its heads of k and v.
__global__ void __launch_bounds__(256, 4) write_kernel(const Cache c, int layer0, int layers, int n,
                                                    const int* slots, const int* starts,
                                                    int tokens, const Rows k, const Rows v) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t units = int64_t(tokens) * layers;
  // the warp as a whole: another may record a fault meanwhile
  if (__any_sync(0xffffffffu, *reinterpret_cast<volatile int*>(c.status) != 0)) return;
  for (int64_t u = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units;
       u += int64_t(gridDim.x) * 8) {
    int layer;
    const int t = int(divide(u, layers, &layer));
    // the rows are on their way while their place is found
    const int per = c.head_dim / 8, chunks = c.kv_heads * per;
    const __nv_bfloat16* const ks = k.p + layer * k.layer + t * k.token;
    const __nv_bfloat16* const vs = v.p + layer * v.layer + t * v.token;
    uint4 x[2][4];
    auto fetch = [&](int i) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = i + 32 * e, h = j / per, d = (j - h * per) * 8;
        if (j < chunks) {
          x[0][e] = *reinterpret_cast<const uint4*>(ks + h * k.head + d);
          x[1][e] = *reinterpret_cast<const uint4*>(vs + h * v.head + d);
        }
      }
    };
    fetch(lane);
    if (t < starts[0] || t >= starts[n]) continue;
    // the last i with starts[i] <= t, 32 candidates at a time (starts that fall find any): it is
    // among lo .. lo + span - 1
    int lo = 0, span = n;
    while (span > 1) {
      const int step = (span + 31) / 32;
      const int i = lane * step;
      const uint32_t m = __ballot_sync(0xffffffffu, i < span && starts[lo + i] <= t);
      const int last = m == 0 ? 0 : 31 - __clz(int(m));
      lo += last * step;
      span = min(step, span - last * step);
    }
    const int slot = slots[lo], first = starts[lo];
    const int64_t count = int64_t(starts[lo + 1]) - first;
    if (slot < 0 || slot >= c.slots) {
      if (lane == 0) cache_fault(c.status, kFaultSlot);
      continue;
    }
    const int len = c.lengths[slot];
    if (!good_length(c, len)) {
      if (lane == 0) cache_fault(c.status, kFaultTable);
      continue;
    }
    if (first < 0 || first > t || t - first >= count || count > tokens - first || count > len) {
      if (lane == 0) cache_fault(c.status, kFaultCounts);
      continue;
    }
    const int pos = len - int(count) + (t - first);
    const int at = pos / c.page_size, row = pos - at * c.page_size;
    const int page = c.table[int64_t(slot) * c.slot_pages + at];
    if (!good_page(c, page)) {
      if (lane == 0) cache_fault(c.status, kFaultTable);
      continue;
    }
    const int64_t plane = int64_t(c.page_size) * c.head_dim;
    const int64_t dst0 =
        (int64_t(layer0 + layer) * c.pages + page) * c.kv_heads * plane + int64_t(row) * c.head_dim;
    for (int i = lane; i < chunks; i += 128) {
      if (i != lane) fetch(i);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = i + 32 * e, h = j / per, d = (j - h * per) * 8;
        if (j < chunks) {
          *reinterpret_cast<uint4*>(c.k + dst0 + h * plane + d) = x[0][e];
          *reinterpret_cast<uint4*>(c.v + dst0 + h * plane + d) = x[1][e];
        }
      }
    }
  }
}

// ------------------------------------------------------------------ keep

// Checks, new lengths and released pages; the rows are moved by the launch behind it, which finds
// them by the table: entries behind a sequence's end stay in it.
__global__ void __launch_bounds__(BLOCK) keep_kernel(const Cache c, int n, const int* slots,
                                                     const int* starts, int tokens,
                                                     const int* path, const int* kept) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x % LANES;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  // job: a: tokens before the new ones, b: new ones, c: those kept, d: the first one's row
  each(
      c, sh, n, true,
      [&](int i, Job& job) {
        const int slot = slots[i], first = starts[i], a = kept[i];
        const int64_t count = int64_t(starts[i + 1]) - first;
        if (!check_slot(c, sh, slot, &job.len)) return;
        if (count < 0 || first < 0 || first + count > tokens || count > job.len) {
          set_fault(sh, kFaultCounts);
        } else if (a < 0 || a > count) {
          set_fault(sh, kFaultPath);
        } else {
          job = Job{slot, job.len, job.len - int(count), int(count), a, first};
        }
      },
      [&](int, const Job& job) {
        const int* row = c.table + int64_t(job.slot) * c.slot_pages;
        check_pages(c, sh, job.slot, job.a / c.page_size, pages_of(c, job.len));
        bool rises = true;
        int moved = job.c;  // the first that moves: all behind it do
        for (int j = lane; j < job.c; j += LANES) {
          const int at = path[job.d + j], before = j > 0 ? path[job.d + j - 1] : -1;
          rises &= at > before && at < job.b;
          if (at != j) moved = min(moved, j);
        }
        if (!rises) set_fault(sh, kFaultPath);
        // the lanes of this sequence among the warp's that are here
        moved = __reduce_min_sync(0xffffu << (threadIdx.x & 16), moved);
        if (moved < job.c)
          for (int q = (job.a + moved) / c.page_size + lane; q < pages_of(c, job.a + job.c);
               q += LANES)
            if (good_page(c, row[q]) && c.refs[row[q]] != 1) set_fault(sh, kFaultShared);
      });
  if (!decide(c, sh, 0)) return;
  each_again(c, sh, n, [&](int, const Job& job) {
    release(c, job.slot, pages_of(c, job.a + job.c), pages_of(c, job.len));
    if (lane == 0) c.lengths[job.slot] = job.a + job.c;
  });
}

// A group of head_dim / 8 lanes a head of a layer of k or v of a sequence: rows move forward or stay,
// in rising order, so a row is read before anything is written over it, eight at a time too.
__global__ void __launch_bounds__(256) move_kernel(const Cache c, int n, const int* path) {
  pdl_wait();
  pdl_trigger();
  if (c.header->go == 0) return;
  const int per = c.head_dim / 8;  // 8 or 16 lanes
  const int groups = 256 / per, lane = threadIdx.x % per;
  const int64_t units = int64_t(n) * c.layers * 2 * c.kv_heads;
  const int64_t plane = int64_t(c.page_size) * c.head_dim;
  for (int64_t u = int64_t(blockIdx.x) * groups + threadIdx.x / per; u < units;
       u += int64_t(gridDim.x) * groups) {
    int h, layer;
    const int64_t w = divide(u, c.kv_heads, &h);
    const int which = int(w & 1);
    const Job f = c.jobs[divide(w >> 1, c.layers, &layer)];
    const int* row = c.table + int64_t(f.slot) * c.slot_pages;
    const int* from = path + f.d;
    __nv_bfloat16* pool = (which ? c.v : c.k) +
                          (int64_t(layer) * c.pages * c.kv_heads + h) * plane + lane * 8;
    auto place = [&](int t) {
      const int at = t / c.page_size;
      return reinterpret_cast<uint4*>(pool + int64_t(row[at]) * c.kv_heads * plane +
                                      int64_t(t - at * c.page_size) * c.head_dim);
    };
    for (int j = 0; j < f.c; j += 8) {
      uint4 x[8];
      uint32_t move = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < f.c && from[j + e] != j + e) {
          x[e] = *place(f.a + from[j + e]);
          move |= 1u << e;
        }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((move >> e) & 1u) *place(f.a + j + e) = x[e];
    }
  }
}

// ------------------------------------------------------------------ fork

// A call's sources and targets checked. ALL: the whole call in this one block; else the launches
// behind go on.
template <bool ALL>
__global__ void __launch_bounds__(BLOCK) fork_kernel(const Cache c, int n, const int* from,
                                                     const int* to) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x % LANES;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  // job: slot, len: the target and what it holds; a: the source, b: its length
  each(
      c, sh, n, true,
      [&](int i, Job& job) {
        const int src = from[i], dst = to[i];
        if (!check_slot(c, sh, dst, &job.len)) return;
        if (src < 0 || src >= c.slots) {
          set_fault(sh, kFaultSlot);
          return;
        }
        job.a = src;
        job.b = c.lengths[src];
        if (good_length(c, job.b))
          job.slot = dst;
        else
          set_fault(sh, kFaultTable);
      },
      [&](int, const Job& job) {
        check_pages(c, sh, job.a, 0, pages_of(c, job.b));
        check_pages(c, sh, job.slot, 0, pages_of(c, job.len));
      });
  if (!decide(c, sh, 0) || !ALL) return;
  each_again(c, sh, n, [&](int i, const Job& job) {
    const int* row = c.table + int64_t(job.a) * c.slot_pages;
    const int m = pages_of(c, job.b);
#pragma unroll 4
    for (int j = lane; j < m; j += LANES) {
      const int page = row[j];
      c.list[int64_t(i) * c.slot_pages + j] = page;
      atomicAdd(&c.refs[page], 1);
    }
  });
  __syncthreads();
  each_again(c, sh, n, [&](int i, const Job& job) {
    int* row = c.table + int64_t(job.slot) * c.slot_pages;
    release(c, job.slot, 0, pages_of(c, job.len));
    __syncwarp(0xffffu << (threadIdx.x & 16));  // the old pages are read
    const int m = pages_of(c, job.b);
#pragma unroll 4
    for (int j = lane; j < m; j += LANES) row[j] = c.list[int64_t(i) * c.slot_pages + j];
    if (lane == 0) c.lengths[job.slot] = job.b;
  });
}

// The sources' rows into scratch; their pages get a user more.
__global__ void __launch_bounds__(256) fork_read_kernel(const Cache c) {
  pdl_wait();
  pdl_trigger();
  if (c.header->go == 0) return;
  const Job job = c.jobs[blockIdx.x];
  const int* row = c.table + int64_t(job.a) * c.slot_pages;
  int* save = c.list + int64_t(blockIdx.x) * c.slot_pages;
  const int m = pages_of(c, job.b);
  for (int j = threadIdx.x; j < m; j += 256) {
    const int page = row[j];
    save[j] = page;
    atomicAdd(&c.refs[page], 1);
  }
}

__global__ void __launch_bounds__(256) fork_write_kernel(const Cache c) {
  pdl_wait();
  pdl_trigger();
  if (c.header->go == 0) return;
  const Job job = c.jobs[blockIdx.x];
  int* row = c.table + int64_t(job.slot) * c.slot_pages;
  const int* save = c.list + int64_t(blockIdx.x) * c.slot_pages;
  const int m = pages_of(c, job.b), old = pages_of(c, job.len);
  for (int j = threadIdx.x; j < max(m, old); j += 256) {
    if (j < old) atomicSub(&c.refs[row[j]], 1);
    if (j < m) row[j] = save[j];
  }
  if (threadIdx.x == 0) c.lengths[job.slot] = job.b;
}

// ------------------------------------------------------------------ truncate

__global__ void __launch_bounds__(BLOCK) truncate_kernel(const Cache c, int n, const int* slots,
                                                         const int* lengths) {
  extern __shared__ __align__(16) uint8_t raw[];
  Shared& sh = *reinterpret_cast<Shared*>(raw);
  const int lane = threadIdx.x % LANES;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  each(
      c, sh, n, false,
      [&](int i, Job& job) {  // a: the new length
        const int slot = slots[i], to = lengths[i];
        if (!check_slot(c, sh, slot, &job.len)) return;
        job.slot = slot;
        job.a = min(job.len, max(0, to));
      },
      [&](int, const Job& job) {
        check_pages(c, sh, job.slot, pages_of(c, job.a), pages_of(c, job.len));
      });
  if (!decide(c, sh, 0)) return;
  each_again(c, sh, n, [&](int, const Job& job) {
    release(c, job.slot, pages_of(c, job.a), pages_of(c, job.len));
    if (lane == 0) c.lengths[job.slot] = job.a;
  });
}

// ------------------------------------------------------------------ arguments

// Device arrays of a call.
struct Words {
  const char* name;
  const void* p;
  size_t count;
};

template <int N>
pb_status check_call(const pb_cache* cache, int32_t n, const Words (&w)[N], const void* scratch,
                     size_t scratch_bytes, bool needs_scratch) {
  const pb_status s = check_cache(cache);
  if (s != PB_OK) return s;
  if (n < 0 || n > cache->slots)
    return record_error(PB_ERR_INVALID_ARG, "n must be between 0 and the cache's slots");
  if (n == 0) return PB_OK;
  const size_t need = needs_scratch ? scratch_need(*cache) : 0;
  if (needs_scratch) {
    if (scratch == nullptr || (reinterpret_cast<uintptr_t>(scratch) & 255) != 0)
      return record_error(PB_ERR_INVALID_ARG, "scratch must be a 256-byte aligned device pointer");
    if (scratch_bytes < need)
      return record_error(PB_ERR_WORKSPACE, "scratch is smaller than pb_cache_scratch_bytes");
    if (!apart_from_cache(Flat{scratch, need}, *cache))
      return record_error(PB_ERR_INVALID_ARG, "scratch overlaps a buffer of the cache");
  }
  for (const Words& x : w) {
    if ((x.p == nullptr && x.count > 0) || !aligned4(x.p))
      return bad(PB_ERR_INVALID_ARG, "%s must be a 4-byte aligned device pointer", x.name);
    const Flat f{x.p, x.count * 4};
    if (!apart_from_cache(f, *cache) || (needs_scratch && !apart(f, Flat{scratch, need})))
      return bad(PB_ERR_INVALID_ARG, "%s overlaps a buffer of the cache or scratch", x.name);
  }
  return PB_OK;
}

pb_status sm_count(int* sms) {
  static PerDeviceInit setup;
  const cudaError_t e = per_device_init(
      setup,
      [](int dev, int* value) {
        return cudaDeviceGetAttribute(value, cudaDevAttrMultiProcessorCount, dev);
      },
      sms);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cudaDeviceGetAttribute");
}

// A bookkeeping launch: one block.
template <class... P, class... A>
cudaError_t launch_one(void (*kernel)(P...), cudaStream_t st, const A&... args) {
  return launch_dependent(kernel, dim3(1), dim3(BLOCK), sizeof(Shared), 1, st, args...);
}
static_assert(sizeof(Shared) <= 48 * 1024, "no opt-in");

// A fork is one block's work for up to 128 sequences if no lane group of it has more than 128 entries
// of the table, and three launches beyond. In a graph, pages of 16, all rows full (one launch, three):
// 8 x 128 entries 5.0 and 6.4 us, 64 x 64 5.7 and 6.7, 64 x 96 7.1 and 7.4, 64 x 128 7.7 and 7.3, 64 x 160
// 9.0 and 8.2, 64 x 256 14.2 and 8.6, 128 x 48 8.1 and 8.9, 128 x 64 8.6 and 7.7, 256 x 16 10.4 and 9.5, 2 x
// 8192 204 and 66. With short sequences, whose entries the host does not know, 64 x 128 takes 4.9 and 6.8,
// 128 x 64 7.2 and 7.9, 256 x 32 11.0 and 9.5. (Few long rows would do up to 256: 8 x 256 6.2 and 7.9.)
constexpr int kForkRows = 128, kForkEntries = 128;

unsigned blocks_for(int64_t units, int64_t per_block, int64_t most) {
  const int64_t b = (units + per_block - 1) / per_block;
  return unsigned(b < most ? b : most);
}

}  // namespace
}  // namespace pb

using namespace pb;

extern "C" {

pb_status pb_cache_scratch_bytes(const pb_cache* cache, size_t* bytes) {
  if (bytes == nullptr) return record_error(PB_ERR_INVALID_ARG, "bytes is NULL");
  const pb_status s = check_cache_sizes(cache);
  if (s != PB_OK) return s;
  *bytes = scratch_need(*cache);
  return PB_OK;
}

pb_status pb_cache_extend(const pb_cache* cache, int32_t n, const int32_t* slots,
                          const int32_t* starts, void* scratch, size_t scratch_bytes,
                          void* stream) {
  const Words w[2] = {{"slots", slots, size_t(n)}, {"starts", starts, size_t(n) + 1}};
  pb_status s = check_call(cache, n, w, scratch, scratch_bytes, true);
  if (s != PB_OK || n == 0) return s;
  int sms = 0;
  s = sm_count(&sms);
  if (s != PB_OK) return s;
  const Cache c = device_view(*cache, scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_one(extend_kernel, st, c, n, slots, starts);
  // most calls copy nothing, and then the blocks only look; eight an SM keep enough on its way where
  // they copy (fork of 8 to 64: 32.6 us, with four 34.9)
  const unsigned grid = blocks_for(int64_t(n) * c.layers * 2 * c.kv_heads, 1, 8 * sms);
  if (e == cudaSuccess) e = launch_dependent(copy_kernel, dim3(grid), dim3(256), 0, 1, st, c);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache extend launch");
}

pb_status pb_cache_write(const pb_cache* cache, int32_t layer, int32_t layers, int32_t n,
                         const int32_t* slots, const int32_t* starts, int32_t tokens,
                         const pb_heads* k, const pb_heads* v, void* stream) {
  const Words w[2] = {{"slots", slots, size_t(n)}, {"starts", starts, size_t(n) + 1}};
  pb_status s = check_call(cache, n, w, nullptr, 0, false);
  if (s != PB_OK) return s;
  if (layer < 0 || layers < 0 || layers > cache->layers - layer)
    return record_error(PB_ERR_INVALID_ARG, "layers outside the cache's");
  if (tokens < 0 || tokens > (1 << 30))
    return record_error(PB_ERR_INVALID_ARG, "tokens must be between 0 and 2^30");
  if (n == 0 || layers == 0 || tokens == 0) return PB_OK;
  const pb_heads* view[2] = {k, v};
  static const char* const name[2] = {"k", "v"};
  Rows rows[2];
  for (int i = 0; i < 2; ++i) {
    if (view[i] == nullptr) return bad(PB_ERR_INVALID_ARG, "%s is NULL", name[i]);
    s = check_view(view[i], name[i], layers, tokens, cache->head_dim, false);
    if (s != PB_OK) return s;
    if (view[i]->heads != cache->kv_heads)
      return bad(PB_ERR_INVALID_ARG, "%s: its heads are not the cache's kv_heads", name[i]);
    Dim d[3];
    const Flat f{view[i]->ptr, size_t(extent(*view[i], layers, tokens, cache->head_dim, d)) * 2};
    if (!apart_from_cache(f, *cache))
      return bad(PB_ERR_INVALID_ARG, "%s overlaps a buffer of the cache", name[i]);
    rows[i] = Rows{static_cast<const __nv_bfloat16*>(view[i]->ptr), view[i]->batch_stride,
                   view[i]->seq_stride, view[i]->head_stride};
  }
  int sms = 0;
  s = sm_count(&sms);
  if (s != PB_OK) return s;
  const Cache c = device_view(*cache, nullptr);
  const unsigned grid = blocks_for(int64_t(tokens) * layers, 8, 16 * sms);
  const cudaError_t e =
      launch_dependent(write_kernel, dim3(grid), dim3(256), 0, 1, static_cast<cudaStream_t>(stream),
                       c, layer, layers, n, slots, starts, tokens, rows[0], rows[1]);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache write launch");
}

pb_status pb_cache_keep(const pb_cache* cache, int32_t n, const int32_t* slots,
                        const int32_t* starts, int32_t tokens, const int32_t* path,
                        const int32_t* kept, void* scratch, size_t scratch_bytes, void* stream) {
  if (tokens < 0) return record_error(PB_ERR_INVALID_ARG, "tokens must be >= 0");
  const Words w[4] = {{"slots", slots, size_t(n)},
                      {"starts", starts, size_t(n) + 1},
                      {"path", path, size_t(tokens)},
                      {"kept", kept, size_t(n)}};
  pb_status s = check_call(cache, n, w, scratch, scratch_bytes, true);
  if (s != PB_OK || n == 0) return s;
  int sms = 0;
  s = sm_count(&sms);
  if (s != PB_OK) return s;
  const Cache c = device_view(*cache, scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_one(keep_kernel, st, c, n, slots, starts, tokens, path, kept);
  const unsigned grid =
      blocks_for(int64_t(n) * c.layers * 2 * c.kv_heads, 256 / (c.head_dim / 8), 8 * sms);
  if (e == cudaSuccess)
    e = launch_dependent(move_kernel, dim3(grid), dim3(256), 0, 1, st, c, n, path);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache keep launch");
}

pb_status pb_cache_fork(const pb_cache* cache, int32_t n, const int32_t* from, const int32_t* to,
                        void* scratch, size_t scratch_bytes, void* stream) {
  const Words w[2] = {{"from", from, size_t(n)}, {"to", to, size_t(n)}};
  const pb_status s = check_call(cache, n, w, scratch, scratch_bytes, true);
  if (s != PB_OK || n == 0) return s;
  const Cache c = device_view(*cache, scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n <= kForkRows && int64_t((n + GROUPS - 1) / GROUPS) * c.slot_pages <= kForkEntries) {
    const cudaError_t one = launch_one(fork_kernel<true>, st, c, n, from, to);
    return one == cudaSuccess ? PB_OK : cuda_failed(one, "cache fork launch");
  }
  cudaError_t e = launch_one(fork_kernel<false>, st, c, n, from, to);
  if (e == cudaSuccess)
    e = launch_dependent(fork_read_kernel, dim3(unsigned(n)), dim3(256), 0, 1, st, c);
  if (e == cudaSuccess)
    e = launch_dependent(fork_write_kernel, dim3(unsigned(n)), dim3(256), 0, 1, st, c);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache fork launch");
}

pb_status pb_cache_truncate(const pb_cache* cache, int32_t n, const int32_t* slots,
                            const int32_t* lengths, void* scratch, size_t scratch_bytes,
                            void* stream) {
  const Words w[2] = {{"slots", slots, size_t(n)}, {"lengths", lengths, size_t(n)}};
  const pb_status s = check_call(cache, n, w, scratch, scratch_bytes, true);
  if (s != PB_OK || n == 0) return s;
  const Cache c = device_view(*cache, scratch);
  const cudaError_t e = launch_one(truncate_kernel, static_cast<cudaStream_t>(stream), c, n, slots,
                                   lengths);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache truncate launch");
}

}  // extern "C"
