// tables.hip -- a serving step's page tables, slots, positions and row ranges from the
// requests' lengths (lutgemm_batch_tables; the rules are in lutgemm.h).
//
// Integers only, a few megabytes at most: bound by latency. scan_kernel, one workgroup,
// walks the sequences 1024 at a time with running sums of new rows, of pages taken and of
// pages given back; a sequence's rows and pages then follow from its sums alone. Sums
// saturate at 2^30, above every limit that they are compared with.
#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kScan = 1024;      // threads of scan_kernel: sequences of one turn
constexpr int kFill = 256;       // threads of fill_kernel
constexpr int kFillRows = 1024;  // rows of one of its workgroups
constexpr uint32_t kFull = 1u << 30;

struct TablesParams {
  const int32_t* change;
  const int32_t* lens;
  const int32_t* offsets;
  const int32_t* range;
  int32_t* table;
  int32_t* ring;
  int64_t* positions;
  int64_t* slots;
  int32_t* lens_out;
  int32_t* starts;
  int32_t* range_out;
  int32_t* ws;  // [seqs][2]: keys before the step, and the place in the ring of the first page taken
  int64_t table_stride;
  int32_t seqs, page, width, capacity, tokens;
};

__device__ __forceinline__ uint32_t add_full(uint32_t a, uint32_t b) {
  const uint32_t s = a + b;
  return s < kFull ? s : kFull;
}

// Inclusive sums over the workgroup's threads; *total: of all of them.
__device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t* waves, uint32_t* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t u = __shfl_up(v, d, 64);
    if (lane >= d) v = add_full(v, u);
  }
  if (lane == 63) waves[wave] = v;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kScan / 64; ++w) {
    if (w < wave) before = add_full(before, waves[w]);
    all = add_full(all, waves[w]);
  }
  __syncthreads();
  *total = all;
  return add_full(v, before);
}

// Where the ring's entry `nth` behind `first` lies (nth up to the capacity).
__device__ __forceinline__ int around(int first, uint32_t nth, int capacity) {
  const uint32_t at = (uint32_t)first + nth;
  return (int)(at < (uint32_t)capacity ? at : at - (uint32_t)capacity);
}

struct Range {
  int first, count;
};

__device__ __forceinline__ Range free_range(const TablesParams& p) {
  Range r = {0, 0};
  if (!p.ring) return r;
  r.first = p.range[0] % p.capacity;
  if (r.first < 0) r.first += p.capacity;
  r.count = p.range[1];
  r.count = r.count < 0 ? 0 : r.count > p.capacity ? p.capacity : r.count;
  return r;
}

__global__ __launch_bounds__(kScan) void scan_kernel(TablesParams p) {
  __shared__ uint32_t waves[kScan / 64];
  __shared__ uint32_t served_rows, served_pages;
  fetch(p);
  const Range free = free_range(p);
  const int limit = p.width * p.page, lane = threadIdx.x & 63;
  const uint32_t room = (uint32_t)(p.capacity - free.count);
  const int behind = around(free.first, (uint32_t)free.count, p.capacity);
  uint32_t rows = 0, pages = 0, given = 0;  // sums of the turns before
  if (threadIdx.x == 0) {
    served_rows = served_pages = 0;
    p.starts[0] = 0;
  }
  for (int s0 = 0; s0 < p.seqs; s0 += kScan) {
    const int s = s0 + threadIdx.x;
    int n = 0, change = 0;
    if (s < p.seqs) {
      n = p.lens[s];
      n = n < 0 ? 0 : n > limit ? limit : n;
      change = p.change[s];
    }
    uint32_t grow = change > 0 && change <= limit - n ? (uint32_t)change : 0;
    const int held = (n + p.page - 1) / p.page;
    uint32_t need = 0, back = 0;
    int after = n;
    if (change < 0) after = n + change < 0 ? 0 : n + change;
    if (p.ring) {
      need = (uint32_t)((n + (int)grow + p.page - 1) / p.page - held);
      back = (uint32_t)(held - (after + p.page - 1) / p.page);
    }
    uint32_t all_rows, all_pages, all_given;
    const uint32_t end = add_full(rows, scan(grow, waves, &all_rows));
    const uint32_t page_end = add_full(pages, scan(need, waves, &all_pages));
    const uint32_t given_end = add_full(given, scan(back, waves, &all_given));
    const bool served = end <= (uint32_t)p.tokens && page_end <= (uint32_t)free.count;
    if (s < p.seqs && served) {
      atomicMax(&served_rows, end);
      atomicMax(&served_pages, page_end);
    }
    __syncthreads();
    if (s < p.seqs) {
      if (!served) grow = 0;
      p.starts[s + 1] = (int)(served ? end : served_rows);
      p.lens_out[s] = after + (int)grow;
      p.ws[2 * s] = n;
      p.ws[2 * s + 1] = served && p.ring ? around(free.first, page_end - need, p.capacity) : 0;
    }
    // pages given back, a wave to a sequence at a time
    uint64_t givers = __ballot(back > 0);
    while (givers) {
      const int from = __builtin_ctzll(givers);
      givers &= givers - 1;
      const int count = __builtin_amdgcn_readlane((int)back, from);
      const uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)(given_end - back), from);
      const int first = __builtin_amdgcn_readlane(held, from) - count;
      const int32_t* row = p.table + (int64_t)(s0 + (int)(threadIdx.x & ~63u) + from) * p.table_stride;
      for (int j = lane; j < count; j += 64)
        if (at + (uint32_t)j < room)
          p.ring[around(behind, at + (uint32_t)j, p.capacity)] = row[first + j];
    }
    rows = add_full(rows, all_rows);
    pages = add_full(pages, all_pages);
    given = add_full(given, all_given);
    __syncthreads();
  }
  if (threadIdx.x == 0 && p.ring) {
    const uint32_t put = given < room ? given : room;
    p.range_out[0] = around(free.first, served_pages, p.capacity);
    p.range_out[1] = free.count - (int)served_pages + (int)put;
  }
}

// The rows' positions and slots, and the table's new entries: by the row whose key is
// its page's first.
__global__ __launch_bounds__(kFill) void fill_kernel(TablesParams p) {
  fetch(p);
  const int row0 = blockIdx.x * kFillRows;
  for (int row = row0 + threadIdx.x; row < min(row0 + kFillRows, p.tokens); row += kFill) {
    // the sequence: the last one whose first row is not behind this one
    int lo = 0, hi = p.seqs;  // starts[lo] <= row
    if (row >= p.starts[p.seqs]) {
      p.positions[row] = 0;
      p.slots[row] = -1;
      continue;
    }
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.starts[mid] <= row) lo = mid; else hi = mid;
    }
    const int n = p.ws[2 * lo], at = n + row - p.starts[lo];
    const int page = at / p.page, held = (n + p.page - 1) / p.page;
    int32_t* entry = p.table + (int64_t)lo * p.table_stride + page;
    int id;
    if (p.ring && page >= held) {
      id = p.ring[around(p.ws[2 * lo + 1], (uint32_t)(page - held), p.capacity)];
      if (at % p.page == 0) *entry = id;
    } else {
      id = *entry;
    }
    p.positions[row] = (p.offsets ? (int64_t)p.offsets[lo] : 0) + at;
    p.slots[row] = (int64_t)id * p.page + at % p.page;
  }
}

// ------------------------------------------------------------------ host side

int check_tables(const lutgemm_tables* t) {
  if (!t) return LUTGEMM_ERR_NULL;
  if (t->seqs < 0 || t->seqs >= (1 << 20) || t->tokens < 0 || t->tokens >= (1 << 24))
    return LUTGEMM_ERR_SHAPE;
  if (t->page_size < 1 || t->page_size > 65536 || t->table_width < 1 ||
      (int64_t)t->table_width * t->page_size > ((int64_t)1 << 30))
    return LUTGEMM_ERR_SHAPE;
  if (t->capacity < 0 || t->capacity >= (1 << 29)) return LUTGEMM_ERR_SHAPE;
  if (t->table_stride < (t->seqs > 1 ? t->table_width : 0) || t->table_stride >= ((int64_t)1 << 40))
    return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_batch_tables_workspace(const lutgemm_tables* t, size_t* bytes) {
  const int st = check_tables(t);
  if (st) return st;
  if (!bytes) return LUTGEMM_ERR_NULL;
  *bytes = (size_t)t->seqs * 2 * sizeof(int32_t);
  return LUTGEMM_OK;
}

extern "C" int lutgemm_batch_tables(const lutgemm_tables* t, const int32_t* d_change,
                                    const int32_t* d_lens, const int32_t* d_offsets, int32_t* d_table,
                                    int32_t* d_ring, const int32_t* d_range, int64_t* d_positions,
                                    int64_t* d_slots, int32_t* d_lens_out, int32_t* d_starts,
                                    int32_t* d_range_out, void* d_workspace, size_t workspace_bytes,
                                    void* stream) {
  try {
    int st = check_tables(t);
    if (st) return st;
    if (!d_starts || (t->tokens && (!d_positions || !d_slots))) return LUTGEMM_ERR_NULL;
    if (t->seqs && (!d_change || !d_lens || !d_table || !d_lens_out || !d_workspace))
      return LUTGEMM_ERR_NULL;
    if (t->capacity && (!d_ring || !d_range || !d_range_out)) return LUTGEMM_ERR_NULL;
    for (const void* at : {(const void*)d_change, (const void*)d_lens, (const void*)d_offsets,
                           (const void*)d_table, (const void*)d_ring, (const void*)d_range,
                           (const void*)d_lens_out, (const void*)d_starts, (const void*)d_range_out,
                           (const void*)d_workspace})
      if (!aligned(at, 4)) return LUTGEMM_ERR_ALIGN;
    if (!aligned(d_positions, 8) || !aligned(d_slots, 8)) return LUTGEMM_ERR_ALIGN;
    if (workspace_bytes < (size_t)t->seqs * 2 * sizeof(int32_t)) return LUTGEMM_ERR_BUFFER;
    const int64_t seqs4 = 4 * (int64_t)t->seqs, rows8 = 8 * t->tokens;
    const bool same_lens = d_lens_out == d_lens, same_range = d_range_out == d_range;
    const Flat all[] = {{d_positions, rows8},
                        {d_slots, rows8},
                        {d_starts, seqs4 + 4},
                        {d_lens_out, seqs4},
                        {t->capacity ? d_range_out : nullptr, 8},
                        {t->capacity ? d_ring : nullptr, 4 * (int64_t)t->capacity},
                        {d_workspace, 2 * seqs4},
                        {d_change, seqs4},
                        {d_offsets, seqs4},
                        {same_lens ? nullptr : d_lens, seqs4},
                        {same_range || !t->capacity ? nullptr : d_range, 8}};
    if (clash(all, 7)) return LUTGEMM_ERR_SHAPE;
    int cus = 0;
    st = serve::check_device(&cus);
    if (st) return st;
    TablesParams p{};
    p.change = d_change;
    p.lens = d_lens;
    p.offsets = d_offsets;
    p.range = d_range;
    p.table = d_table;
    p.ring = t->capacity ? d_ring : nullptr;
    p.positions = d_positions;
    p.slots = d_slots;
    p.lens_out = d_lens_out;
    p.starts = d_starts;
    p.range_out = d_range_out;
    p.ws = (int32_t*)d_workspace;
    p.table_stride = t->table_stride;
    p.seqs = t->seqs;
    p.page = t->page_size;
    p.width = t->table_width;
    p.capacity = t->capacity;
    p.tokens = t->tokens;
    hipStream_t strm = (hipStream_t)stream;
    st = launch(scan_kernel, dim3(1), kScan, p, strm);
    if (st || !t->tokens) return st;
    return launch(fill_kernel, dim3((unsigned)((t->tokens + kFillRows - 1) / kFillRows)), kFill, p, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
