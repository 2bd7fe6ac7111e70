// cache.cu — a paged cache of keys and values: room for new tokens, their rows, the accepted ones of
// drafted tokens moved together, sequences forked and cut.
//
// The table, the lengths and the pages' counts of users live on the device and are changed there, so
// that a decoding loop whose numbers of accepted tokens come out of the model needs no word from the
// host, and can be a captured graph.
//
// Bookkeeping is small (a few thousand words): one block checks a whole call, so that a call at fault
// changes nothing, and does it, a warp a sequence. Free pages are those whose count is zero, found
// in rising order by a scan (one block scan for 4096 pages): their numbers depend on nothing but the
// counts, whatever the order in which sequences came and went, and there is no list that could
// disagree with them. A fork copies rows of the table, which a block a sequence does, in two launches
// (read all, then write), since a slot may be read and written in one call.
//
// Data moves by 16-byte accesses, a row of a head (128 or 256 bytes) by 8 or 16 lanes: bound by
// memory for many sequences and by the launch for few.
#include <cuda_bf16.h>

#include "cache.h"
#include "kernels.h"
#include "ptx.cuh"

namespace pb {
namespace {

struct Info {  // of a listed sequence, for the launch that moves data
  int base;    // keep: tokens before the new ones; extend: rank of its first new page; fork: length
  int count;   // keep: tokens to keep; extend: 1 where its last page is copied
  int copy;    // extend: place in the list of copies
  int pad;
};
struct Copy {
  int from, to, rows, pad;
};

// Scratch: header, Info [slots], Copy [slots], free pages [pages] or rows of the table [slots,
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
  Info* info;
  Copy* copies;
  int* list;
};

size_t scratch_need(const pb_cache& c) {
  const size_t list = size_t(c.slots) * c.slot_pages;
  return kHeaderBytes + size_t(c.slots) * (sizeof(Info) + sizeof(Copy)) +
         4 * (list > size_t(c.pages) ? list : size_t(c.pages));
}

Cache device_view(const pb_cache& c, void* scratch) {
  uint8_t* s = static_cast<uint8_t*>(scratch);
  Cache d{c.layers,  c.pages,   c.page_size, c.kv_heads, c.head_dim, c.slots, c.slot_pages,
          static_cast<__nv_bfloat16*>(c.k), static_cast<__nv_bfloat16*>(c.v),
          c.table,   c.lengths, c.refs,      c.status,   nullptr,    nullptr, nullptr, nullptr};
  if (s != nullptr) {
    d.header = reinterpret_cast<Header*>(s);
    d.info = reinterpret_cast<Info*>(s + kHeaderBytes);
    d.copies = reinterpret_cast<Copy*>(d.info + c.slots);
    d.list = reinterpret_cast<int*>(d.copies + c.slots);
  }
  return d;
}

constexpr int BLOCK = 1024, WARPS = BLOCK / 32;

struct Shared {
  uint32_t seen[kMaxSlots / 32];  // slots listed
  int sums[WARPS];
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

// Clears the bits of the slots and tells whether the cache is free of faults (all threads).
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
// A slot of the list: whether it may be used.
__device__ bool check_slot(const Cache& c, Shared& sh, int slot) {
  if (slot < 0 || slot >= c.slots ||
      ((atomicOr(&sh.seen[slot >> 5], 1u << (slot & 31)) >> (slot & 31)) & 1u) != 0) {
    set_fault(sh, kFaultSlot);
    return false;
  }
  if (!good_length(c, c.lengths[slot])) {
    set_fault(sh, kFaultTable);
    return false;
  }
  return true;
}
// The pages [a, z) of a slot lose a user; one warp.
__device__ void release(const Cache& c, int slot, int a, int z) {
  const int* row = c.table + int64_t(slot) * c.slot_pages;
  for (int i = a + int(threadIdx.x & 31); i < z; i += 32) atomicSub(&c.refs[row[i]], 1);
}
// Whether the pages [a, z) of a slot are pages; one warp, its lanes together.
__device__ void check_pages(const Cache& c, Shared& sh, int slot, int a, int z) {
  const int* row = c.table + int64_t(slot) * c.slot_pages;
  for (int i = a + int(threadIdx.x & 31); i < z; i += 32)
    if (!good_page(c, row[i])) set_fault(sh, kFaultTable);
}

// ------------------------------------------------------------------ extend

__global__ void __launch_bounds__(BLOCK) extend_kernel(const Cache c, int n, const int* slots,
                                                       const int* starts) {
  __shared__ Shared sh;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  int need_all = 0, copies = 0;
  for (int i0 = 0; i0 < n; i0 += BLOCK) {
    const int i = i0 + tid;
    int need = 0, copy = 0;
    if (i < n) {
      const int slot = slots[i];
      const int64_t count = int64_t(starts[i + 1]) - starts[i];
      if (check_slot(c, sh, slot)) {
        const int len = c.lengths[slot];
        if (count < 0) {
          set_fault(sh, kFaultCounts);
        } else if (len + count > int64_t(c.slot_pages) * c.page_size) {
          set_fault(sh, kFaultRow);
        } else {
          if (count > 0 && len % c.page_size != 0) {
            const int page = c.table[int64_t(slot) * c.slot_pages + len / c.page_size];
            if (!good_page(c, page))
              set_fault(sh, kFaultTable);
            else
              copy = c.refs[page] > 1;
          }
          need = pages_of(c, int(len + count)) - pages_of(c, len) + copy;
        }
      }
    }
    // a page more than there are is as many as any: 1024 of them stay below 2^31
    int total, ctotal;
    const int first = block_scan(min(need, c.pages + 1), sh, &total);
    const int cfirst = block_scan(copy, sh, &ctotal);
    if (i < n) c.info[i] = Info{need_all + first, copy, copies + cfirst, 0};
    copies += ctotal;
    need_all += total;
    if (need_all > c.pages) {
      set_fault(sh, kFaultPages);
      break;  // the same for all threads
    }
  }
  __syncthreads();
  // the need_all free pages of lowest number
  if (sh.fault == 0) {
    int found = 0;
    for (int p0 = 0; p0 < c.pages && found < need_all; p0 += 4 * BLOCK) {
      const int p = p0 + 4 * tid;
      int used[4], zeros = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        used[e] = p + e < c.pages ? c.refs[p + e] : 1;
        zeros += used[e] == 0;
      }
      int total;
      int rank = found + block_scan(zeros, sh, &total);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (used[e] == 0) {
          if (rank < need_all) c.list[rank] = p + e;
          ++rank;
        }
      found += total;
    }
    __syncthreads();  // all have read that there was no fault
    if (found < need_all && tid == 0) set_fault(sh, kFaultPages);
  }
  if (!decide(c, sh, copies)) return;
  for (int i = warp; i < n; i += WARPS) {
    const int slot = slots[i], count = starts[i + 1] - starts[i];
    const int len = c.lengths[slot];
    const Info f = c.info[i];
    int* row = c.table + int64_t(slot) * c.slot_pages;
    const int have = pages_of(c, len), more = pages_of(c, len + count) - have;
    for (int j = lane; j < more; j += 32) {
      const int page = c.list[f.base + f.count + j];
      row[have + j] = page;
      c.refs[page] = 1;
    }
    __syncwarp();  // all lanes have read the length
    if (lane == 0) {
      if (f.count != 0) {
        const int at = len / c.page_size, old = row[at], page = c.list[f.base];
        c.copies[f.copy] = Copy{old, page, len % c.page_size, 0};
        row[at] = page;
        c.refs[page] = 1;
        atomicSub(&c.refs[old], 1);
      }
      c.lengths[slot] = len + count;
    }
  }
}

// Copies the rows of the listed pages, a head of a layer of k or v at a time.
__global__ void __launch_bounds__(256) copy_kernel(const Cache c) {
  pdl_wait();
  pdl_trigger();
  const int64_t units = int64_t(c.header->copies) * c.layers * 2 * c.kv_heads;
  const int64_t plane = int64_t(c.page_size) * c.head_dim;  // values of a head of a page
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int h = int(u % c.kv_heads);
    const int64_t w = u / c.kv_heads;
    const int which = int(w & 1), layer = int((w >> 1) % c.layers);
    const Copy t = c.copies[(w >> 1) / c.layers];
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
__global__ void __launch_bounds__(256) write_kernel(const Cache c, int layer0, int layers, int n,
                                                    const int* slots, const int* starts,
                                                    int tokens, const Rows k, const Rows v) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t units = int64_t(tokens) * layers;
  if (*reinterpret_cast<volatile int*>(c.status) != 0) return;
  for (int64_t u = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5); u < units;
       u += int64_t(gridDim.x) * 8) {
    const int t = int(u / layers), layer = int(u % layers);
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
    const int per = c.head_dim / 8;
    const int64_t plane = int64_t(c.page_size) * c.head_dim;
    const int64_t dst0 =
        (int64_t(layer0 + layer) * c.pages + page) * c.kv_heads * plane + int64_t(row) * c.head_dim;
    const int chunks = c.kv_heads * per;
    for (int i = lane; i < chunks; i += 128) {
      uint4 x[2][4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = i + 32 * e, h = j / per, d = (j - h * per) * 8;
        if (j < chunks) {
          x[0][e] = *reinterpret_cast<const uint4*>(k.p + layer * k.layer + t * k.token + h * k.head + d);
          x[1][e] = *reinterpret_cast<const uint4*>(v.p + layer * v.layer + t * v.token + h * v.head + d);
        }
      }
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
  __shared__ Shared sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  for (int i = warp; i < n; i += WARPS) {
    const int slot = slots[i], first = starts[i], a = kept[i];
    const int64_t count = int64_t(starts[i + 1]) - first;
    int sound = 0;
    if (lane == 0 && check_slot(c, sh, slot)) {
      if (count < 0 || first < 0 || first + count > tokens || count > c.lengths[slot])
        set_fault(sh, kFaultCounts);
      else if (a < 0 || a > count)
        set_fault(sh, kFaultPath);
      else
        sound = 1;
    }
    if (__shfl_sync(0xffffffffu, sound, 0) == 0) continue;
    const int len = c.lengths[slot], base = len - int(count);
    check_pages(c, sh, slot, base / c.page_size, pages_of(c, len));
    bool moved = false;
    for (int j = lane; j < a; j += 32) {
      const int at = path[first + j], before = j > 0 ? path[first + j - 1] : -1;
      if (at <= before || at >= count) set_fault(sh, kFaultPath);
      moved |= at != j;
    }
    if (__any_sync(0xffffffffu, moved)) {
      const int* row = c.table + int64_t(slot) * c.slot_pages;
      for (int q = base / c.page_size + lane; q < pages_of(c, base + a); q += 32)
        if (good_page(c, row[q]) && c.refs[row[q]] != 1) set_fault(sh, kFaultShared);
    }
    if (lane == 0) c.info[i] = Info{base, a, 0, 0};
  }
  if (!decide(c, sh, 0)) return;
  for (int i = warp; i < n; i += WARPS) {
    const int slot = slots[i];
    const Info f = c.info[i];
    release(c, slot, pages_of(c, f.base + f.count), pages_of(c, c.lengths[slot]));
    __syncwarp();
    if (lane == 0) c.lengths[slot] = f.base + f.count;
  }
}

// A group of head_dim / 8 lanes a head of a layer of k or v of a sequence: rows move forward or stay,
// in rising order, so a row is read before anything is written over it, eight at a time too.
__global__ void __launch_bounds__(256) move_kernel(const Cache c, int n, const int* slots,
                                                   const int* starts, const int* path) {
  pdl_wait();
  pdl_trigger();
  if (c.header->go == 0) return;
  const int per = c.head_dim / 8;  // 8 or 16 lanes
  const int groups = 256 / per, lane = threadIdx.x % per;
  const int64_t units = int64_t(n) * c.layers * 2 * c.kv_heads;
  const int64_t plane = int64_t(c.page_size) * c.head_dim;
  for (int64_t u = int64_t(blockIdx.x) * groups + threadIdx.x / per; u < units;
       u += int64_t(gridDim.x) * groups) {
    const int h = int(u % c.kv_heads);
    const int64_t w = u / c.kv_heads;
    const int which = int(w & 1), layer = int((w >> 1) % c.layers), i = int((w >> 1) / c.layers);
    const Info f = c.info[i];
    const int* row = c.table + int64_t(slots[i]) * c.slot_pages;
    const int* from = path + starts[i];
    __nv_bfloat16* pool = (which ? c.v : c.k) +
                          (int64_t(layer) * c.pages * c.kv_heads + h) * plane + lane * 8;
    auto place = [&](int t) {
      const int at = t / c.page_size;
      return reinterpret_cast<uint4*>(pool + int64_t(row[at]) * c.kv_heads * plane +
                                      int64_t(t - at * c.page_size) * c.head_dim);
    };
    for (int j = 0; j < f.count; j += 8) {
      uint4 x[8];
      uint32_t move = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < f.count && from[j + e] != j + e) {
          x[e] = *place(f.base + from[j + e]);
          move |= 1u << e;
        }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((move >> e) & 1u) *place(f.base + j + e) = x[e];
    }
  }
}

// ------------------------------------------------------------------ fork

__global__ void __launch_bounds__(BLOCK) fork_check_kernel(const Cache c, int n, const int* from,
                                                           const int* to) {
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  for (int i = warp; i < n; i += WARPS) {
    const int src = from[i], dst = to[i];
    int sound = 0;
    if (lane == 0 && check_slot(c, sh, dst)) {
      if (src < 0 || src >= c.slots)
        set_fault(sh, kFaultSlot);
      else if (!good_length(c, c.lengths[src]))
        set_fault(sh, kFaultTable);
      else
        sound = 1;
    }
    if (__shfl_sync(0xffffffffu, sound, 0) == 0) continue;
    check_pages(c, sh, src, 0, pages_of(c, c.lengths[src]));
    check_pages(c, sh, dst, 0, pages_of(c, c.lengths[dst]));
    if (lane == 0) c.info[i] = Info{c.lengths[src], 0, 0, 0};
  }
  decide(c, sh, 0);
}

// The sources' rows into scratch; their pages get a user more.
__global__ void __launch_bounds__(256) fork_read_kernel(const Cache c, const int* from) {
  pdl_wait();
  pdl_trigger();
  if (c.header->go == 0) return;
  const int i = blockIdx.x;
  const int* row = c.table + int64_t(from[i]) * c.slot_pages;
  int* save = c.list + int64_t(i) * c.slot_pages;
  const int m = pages_of(c, c.info[i].base);
  for (int j = threadIdx.x; j < m; j += 256) {
    const int page = row[j];
    save[j] = page;
    atomicAdd(&c.refs[page], 1);
  }
}

__global__ void __launch_bounds__(256) fork_write_kernel(const Cache c, const int* to) {
  pdl_wait();
  pdl_trigger();
  if (c.header->go == 0) return;
  const int i = blockIdx.x, slot = to[i];
  int* row = c.table + int64_t(slot) * c.slot_pages;
  const int* save = c.list + int64_t(i) * c.slot_pages;
  const int m = pages_of(c, c.info[i].base), old = pages_of(c, c.lengths[slot]);
  for (int j = threadIdx.x; j < max(m, old); j += 256) {
    if (j < old) atomicSub(&c.refs[row[j]], 1);
    if (j < m) row[j] = save[j];
  }
  __syncthreads();  // every thread has read the length
  if (threadIdx.x == 0) c.lengths[slot] = c.info[i].base;
}

// ------------------------------------------------------------------ truncate

__global__ void __launch_bounds__(BLOCK) truncate_kernel(const Cache c, int n, const int* slots,
                                                         const int* lengths) {
  __shared__ Shared sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  if (!begin(c, sh)) return;
  for (int i = warp; i < n; i += WARPS) {
    const int slot = slots[i];
    const int sound = lane == 0 ? int(check_slot(c, sh, slot)) : 0;
    if (__shfl_sync(0xffffffffu, sound, 0) == 0) continue;
    const int len = c.lengths[slot], to = min(len, max(0, lengths[i]));
    check_pages(c, sh, slot, pages_of(c, to), pages_of(c, len));
  }
  if (!decide(c, sh, 0)) return;
  for (int i = warp; i < n; i += WARPS) {
    const int slot = slots[i], len = c.lengths[slot], to = min(len, max(0, lengths[i]));
    release(c, slot, pages_of(c, to), pages_of(c, len));
    __syncwarp();
    if (lane == 0) c.lengths[slot] = to;
  }
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
  cudaError_t e = launch_dependent(extend_kernel, dim3(1), dim3(BLOCK), 0, 1, st, c, n, slots, starts);
  // few blocks an SM: most calls copy nothing, and then these only look
  const unsigned grid = blocks_for(int64_t(n) * c.layers * 2 * c.kv_heads, 1, 4 * sms);
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
  cudaError_t e = launch_dependent(keep_kernel, dim3(1), dim3(BLOCK), 0, 1, st, c, n, slots, starts,
                                   tokens, path, kept);
  const unsigned grid =
      blocks_for(int64_t(n) * c.layers * 2 * c.kv_heads, 256 / (c.head_dim / 8), 8 * sms);
  if (e == cudaSuccess)
    e = launch_dependent(move_kernel, dim3(grid), dim3(256), 0, 1, st, c, n, slots, starts, path);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache keep launch");
}

pb_status pb_cache_fork(const pb_cache* cache, int32_t n, const int32_t* from, const int32_t* to,
                        void* scratch, size_t scratch_bytes, void* stream) {
  const Words w[2] = {{"from", from, size_t(n)}, {"to", to, size_t(n)}};
  const pb_status s = check_call(cache, n, w, scratch, scratch_bytes, true);
  if (s != PB_OK || n == 0) return s;
  const Cache c = device_view(*cache, scratch);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = launch_dependent(fork_check_kernel, dim3(1), dim3(BLOCK), 0, 1, st, c, n, from, to);
  if (e == cudaSuccess)
    e = launch_dependent(fork_read_kernel, dim3(unsigned(n)), dim3(256), 0, 1, st, c, from);
  if (e == cudaSuccess)
    e = launch_dependent(fork_write_kernel, dim3(unsigned(n)), dim3(256), 0, 1, st, c, to);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache fork launch");
}

pb_status pb_cache_truncate(const pb_cache* cache, int32_t n, const int32_t* slots,
                            const int32_t* lengths, void* scratch, size_t scratch_bytes,
                            void* stream) {
  const Words w[2] = {{"slots", slots, size_t(n)}, {"lengths", lengths, size_t(n)}};
  const pb_status s = check_call(cache, n, w, scratch, scratch_bytes, true);
  if (s != PB_OK || n == 0) return s;
  const Cache c = device_view(*cache, scratch);
  const cudaError_t e = launch_dependent(truncate_kernel, dim3(1), dim3(BLOCK), 0, 1,
                                         static_cast<cudaStream_t>(stream), c, n, slots, lengths);
  return e == cudaSuccess ? PB_OK : cuda_failed(e, "cache truncate launch");
}

}  // extern "C"
