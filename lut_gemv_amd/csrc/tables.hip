// tables.hip -- a serving step's page tables, slots, positions and row ranges from the
// requests' lengths (lutgemm_batch_tables; the rules are in lutgemm.h).
//
// Integers only, a few megabytes at most: bound by latency. scan_kernel, one workgroup,
// walks the sequences a workgroup's width at a time with running sums of new rows, of pages
// taken and of pages given back; a sequence's rows and pages then follow from its sums alone.
// Sums saturate at 2^30 + 2^29: above every limit that they are compared with, also less a
// sequence's own pages (2^30 at most; a ring has fewer than 2^29), and an int with a thread's
// number added. Up to kFewRows rows it also writes the rows, those of a few tokens by the
// sequence's own thread; more are fill_kernel's, whose workgroups look for the sequences of
// their rows.
#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kFill = 256;       // threads of fill_kernel
constexpr int kFillRows = 512;   // rows of one of its workgroups
constexpr int kFewRows = 4096;   // that scan_kernel writes itself
constexpr int kOwnRows = 4;      // of a sequence, by its own thread
constexpr uint32_t kFull = 3u << 29;

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

struct Sums {
  uint32_t rows, pages, given;
  __device__ __forceinline__ void add(const Sums& o) {
    rows = add_full(rows, o.rows);
    pages = add_full(pages, o.pages);
    given = add_full(given, o.given);
  }
};

template <int Control, int Rows>
__device__ __forceinline__ void add_from(Sums& v) {
  auto from = [](uint32_t x) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, Control, Rows, 0xF, false);
  };
  const Sums o = {from(v.rows), from(v.pages), from(v.given)};
  v.add(o);
}

// Inclusive sums over the workgroup's threads; *total: of all of them.
template <int Waves>
__device__ __forceinline__ Sums scan(Sums v, Sums* waves, Sums* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  add_from<0x111, 0xF>(v);
  add_from<0x112, 0xF>(v);
  add_from<0x114, 0xF>(v);
  add_from<0x118, 0xF>(v);
  add_from<0x142, 0xA>(v);
  add_from<0x143, 0xC>(v);
  if (lane == 63) waves[wave] = v;
  __syncthreads();
  Sums before = {0, 0, 0}, all = {0, 0, 0};
#pragma unroll
  for (int w = 0; w < Waves; ++w) {
    if (w < wave) before.add(waves[w]);
    all.add(waves[w]);
  }
  *total = all;
  v.add(before);
  return v;
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

// The row of a sequence's ith new token: its position and slot, and the table's new entry, by
// the row whose key is its page's first.
__device__ __forceinline__ void write_row(const TablesParams& p, int s, int row, int n, int held,
                                          int taken, int64_t offset, int i) {
  const int at = n + i, page = at / p.page, place = at - page * p.page;
  int32_t* const entry = p.table + (int64_t)s * p.table_stride + page;
  int id;
  if (p.ring && page >= held) {
    id = p.ring[around(taken, (uint32_t)(page - held), p.capacity)];
    if (place == 0) *entry = id;
  } else {
    id = *entry;
  }
  p.positions[row] = offset + at;
  p.slots[row] = (int64_t)id * p.page + place;
}

// Bound by latency: the lengths' reads, two barriers a turn, the table's and the ring's entries behind
// them. One sequence 2.8 to 3.0 us; 400, of which 9 end and 31 take keys back, 6.8 to 7.2 (a wave's
// sequences that give pages back wait for one another, a read and a write each); 64 chunks beside 96
// single tokens, whose rows are fill_kernel's, 4.0.
template <int Threads>
__global__ __launch_bounds__(Threads) void scan_kernel(TablesParams p) {
  __shared__ Sums waves[2][Threads / 64];
  __shared__ int32_t of_row[Threads], of_len[Threads], of_ring[Threads];
  __shared__ uint32_t served_rows, served_pages;
  fetch(p);
  const int limit = p.width * p.page, lane = threadIdx.x & 63;
  const bool all_rows = p.tokens <= kFewRows;  // fill_kernel is not launched
  int n = 0, change = 0;
  auto read = [&](int s) {
    if (s >= p.seqs) return;
    n = p.lens[s];
    change = p.change[s];
  };
  read(threadIdx.x);
  const Range free = free_range(p);
  const uint32_t room = (uint32_t)(p.capacity - free.count);
  const int behind = around(free.first, (uint32_t)free.count, p.capacity);
  Sums sums = {0, 0, 0};  // of the turns before
  if (threadIdx.x == 0) {
    served_rows = served_pages = 0;
    p.starts[0] = 0;
  }
  for (int s0 = 0, turn = 0; s0 < p.seqs; s0 += Threads, turn ^= 1) {
    const int s = s0 + threadIdx.x;
    if (s0) read(s);
    const bool here = s < p.seqs;
    n = !here || n < 0 ? 0 : n > limit ? limit : n;
    if (!here) change = 0;
    uint32_t grow = change > 0 && change <= limit - n ? (uint32_t)change : 0;
    const int held = (n + p.page - 1) / p.page;
    uint32_t need = 0, back = 0;
    int after = n;
    if (change < 0) after = n + change < 0 ? 0 : n + change;
    if (p.ring) {
      if (grow) need = (uint32_t)((n + (int)grow + p.page - 1) / p.page - held);
      if (change < 0) back = (uint32_t)(held - (after + p.page - 1) / p.page);
    }
    Sums all;
    Sums end = scan<Threads / 64>({grow, need, back}, waves[turn], &all);
    end.add(sums);
    const bool served = end.rows <= (uint32_t)p.tokens && end.pages <= (uint32_t)free.count;
    // sums rise: the last sequence served of a wave has its largest
    const uint64_t votes = __ballot(here && served);
    if (votes && lane == 63 - __builtin_clzll(votes)) {
      atomicMax(&served_rows, end.rows);
      atomicMax(&served_pages, end.pages);
    }
    __syncthreads();
    const int first_row = (int)(end.rows - grow);
    if (!served) grow = 0;
    int taken = 0;
    if (here) {
      p.starts[s + 1] = (int)(served ? end.rows : served_rows);
      p.lens_out[s] = after + (int)grow;
      if (served && p.ring) taken = around(free.first, end.pages - need, p.capacity);
      if (!all_rows) {
        p.ws[2 * s] = n;
        p.ws[2 * s + 1] = taken;
      }
    }
    // pages given back, a wave to a sequence at a time
    for (uint64_t givers = __ballot(back > 0); givers; givers &= givers - 1) {
      const int from = __builtin_ctzll(givers);
      const int all_back = __builtin_amdgcn_readlane((int)back, from);
      const uint32_t at = (uint32_t)__builtin_amdgcn_readlane((int)(end.given - back), from);
      const int first = __builtin_amdgcn_readlane(held, from) - all_back;
      if (at >= room) break;  // no room for these, nor for those behind
      const int count = min(all_back, (int)(room - at));
      const int32_t* row = p.table + (int64_t)(s0 + (int)(threadIdx.x & ~63u) + from) * p.table_stride;
      constexpr int kTogether = 8;  // reads under way
      for (int j0 = lane; j0 < count; j0 += 64 * kTogether) {
        int32_t id[kTogether];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) id[k] = row[first + min(j0 + 64 * k, count - 1)];
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          const uint32_t nth = at + (uint32_t)(j0 + 64 * k);
          if (j0 + 64 * k < count) p.ring[around(behind, nth, p.capacity)] = id[k];
        }
      }
    }
    if (all_rows) {
      if (grow && grow <= kOwnRows) {
        const int64_t offset = p.offsets ? (int64_t)p.offsets[s] : 0;
        for (int i = 0; i < (int)grow; ++i) write_row(p, s, first_row + i, n, held, taken, offset, i);
      }
      of_row[threadIdx.x] = here && served ? first_row : INT32_MAX;
      of_len[threadIdx.x] = n;
      of_ring[threadIdx.x] = taken;
      if (__syncthreads_or(grow > kOwnRows))
        for (int row = (int)sums.rows + threadIdx.x; row < (int)served_rows; row += Threads) {
          int a = 0, b = Threads;  // the sequence: the last one that begins here or before
          while (b - a > 1) {
            const int mid = (a + b) >> 1;
            if (of_row[mid] <= row)
              a = mid;
            else
              b = mid;
          }
          const int next = a + 1 < Threads ? min(of_row[a + 1], (int)served_rows) : (int)served_rows;
          if (next - of_row[a] <= kOwnRows) continue;  // written already
          write_row(p, s0 + a, row, of_len[a], (of_len[a] + p.page - 1) / p.page, of_ring[a],
                    p.offsets ? (int64_t)p.offsets[s0 + a] : 0, row - of_row[a]);
        }
    }
    sums.add(all);
  }
  __syncthreads();
  if (threadIdx.x == 0 && p.ring) {
    const uint32_t put = sums.given < room ? sums.given : room;
    p.range_out[0] = around(free.first, served_pages, p.capacity);
    p.range_out[1] = free.count - (int)served_pages + (int)put;
  }
  if (all_rows)
    for (int row = (int)served_rows + threadIdx.x; row < p.tokens; row += Threads) {
      p.positions[row] = 0;
      p.slots[row] = -1;
    }
}

// The last sequence of which the first row is not behind `row`, which the last one's end
// is: by whole waves, 64 starts at a time.
__device__ __forceinline__ int owner(const TablesParams& p, int row, int lane) {
  int lo = 0, n = p.seqs;  // among [lo, lo + n)
  while (n > 1) {
    const int step = (n + 63) / 64, at = lo + lane * step;
    const uint64_t votes = __ballot(at < lo + n && p.starts[min(at, p.seqs)] <= row);
    const int found = __popcll(votes) - 1;
    lo += found * step;
    n = min(step, n - found * step);
  }
  return lo;
}

// Bound by its beginning (the search, 2 us) and its writes: 196608 rows, 3.1 MB, 5.1 to 5.6 us.
__global__ __launch_bounds__(kFill) void fill_kernel(TablesParams p) {
  __shared__ int32_t starts[kFillRows + 1];
  fetch(p);
  const int lane = threadIdx.x & 63, rows = p.starts[p.seqs];
  const int row0 = blockIdx.x * kFillRows, end = min(row0 + kFillRows, p.tokens);
  const int last = min(end, rows) - 1;
  int lo = 0, hi = 0;
  bool near = true;
  if (last >= row0) {
    lo = owner(p, row0, lane);
    hi = owner(p, last, lane);
    near = hi - lo < kFillRows;  // sequences without rows may lie between
    if (near)
      for (int i = threadIdx.x; i <= hi - lo; i += kFill) starts[i] = p.starts[lo + i];
  }
  __syncthreads();
  for (int row = row0 + threadIdx.x; row < end; row += kFill) {
    if (row > last) {
      p.positions[row] = 0;
      p.slots[row] = -1;
      continue;
    }
    int a = lo, b = hi + 1;
    while (b - a > 1) {
      const int mid = (a + b) >> 1;
      if ((near ? starts[mid - lo] : p.starts[mid]) <= row)
        a = mid;
      else
        b = mid;
    }
    const int n = p.ws[2 * a], held = (n + p.page - 1) / p.page;
    write_row(p, a, row, n, held, p.ws[2 * a + 1], p.offsets ? (int64_t)p.offsets[a] : 0,
              row - (near ? starts[a - lo] : p.starts[a]));
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

size_t workspace(const lutgemm_tables* t) {
  return t->tokens <= kFewRows ? 0 : (size_t)t->seqs * 2 * sizeof(int32_t);
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_batch_tables_workspace(const lutgemm_tables* t, size_t* bytes) {
  const int st = check_tables(t);
  if (st) return st;
  if (!bytes) return LUTGEMM_ERR_NULL;
  *bytes = workspace(t);
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
    const size_t need = workspace(t);
    if (t->seqs && (!d_change || !d_lens || !d_table || !d_lens_out)) return LUTGEMM_ERR_NULL;
    if (need && !d_workspace) return LUTGEMM_ERR_NULL;
    if (t->capacity && (!d_ring || !d_range || !d_range_out)) return LUTGEMM_ERR_NULL;
    for (const void* at : {(const void*)d_change, (const void*)d_lens, (const void*)d_offsets,
                           (const void*)d_table, (const void*)d_ring, (const void*)d_range,
                           (const void*)d_lens_out, (const void*)d_starts, (const void*)d_range_out,
                           (const void*)d_workspace})
      if (!aligned(at, 4)) return LUTGEMM_ERR_ALIGN;
    if (!aligned(d_positions, 8) || !aligned(d_slots, 8)) return LUTGEMM_ERR_ALIGN;
    if (workspace_bytes < need) return LUTGEMM_ERR_BUFFER;
    const int64_t seqs4 = 4 * (int64_t)t->seqs, rows8 = 8 * t->tokens;
    const bool same_lens = d_lens_out == d_lens, same_range = d_range_out == d_range;
    const Flat all[] = {{d_positions, rows8},
                        {d_slots, rows8},
                        {d_starts, seqs4 + 4},
                        {d_lens_out, seqs4},
                        {t->capacity ? d_range_out : nullptr, 8},
                        {t->capacity ? d_ring : nullptr, 4 * (int64_t)t->capacity},
                        {d_workspace, (int64_t)need},
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
    // fewer waves begin and meet sooner (one sequence: 2.8 us), more take fewer turns (400: 7.6
    // us, in two turns of 256 8.5)
    st = t->seqs <= 256 ? launch(scan_kernel<256>, dim3(1), 256, p, strm)
                        : launch(scan_kernel<1024>, dim3(1), 1024, p, strm);
    if (st || t->tokens <= kFewRows) return st;
    return launch(fill_kernel, dim3((unsigned)((t->tokens + kFillRows - 1) / kFillRows)), kFill, p, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
