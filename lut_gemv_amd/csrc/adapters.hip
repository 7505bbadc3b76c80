// adapters.hip -- low-rank adapters of many requests added to a projection's output
// (lutgemm_adapters_add; the formula is in lutgemm.h).
//
// Two products on the matrix cores, t = A[a] x and out = y + s B[a] t, over tiles of
// up to 16 or 32 rows that share an adapter. Memory and the latency of a few dependent
// reads bound both: a decode step reads each adapter it uses once, a prompt reads x and y.
// Rows come in any order; up to 64 of them every wave groups for itself (one row per lane),
// up to 1024 every workgroup, above that one workgroup sorts them first (sort_kernel).
//
// shrink_kernel splits K over workgroups and waves; its parts are summed when
// expand_kernel reads them, in a fixed order. t is rounded for the second product to
// a pair of numbers, high + low, of the element type: the pair's error is far below
// the rounding of the output, for two small matrix products in place of one.
//
// 61 rows of 24 adapters of rank 64, K = 11008, N = 4096 (49 MB): 16.8 us, 2.9 TB/s;
// 4096 rows of 8, K = N = 8192, rank 32 (210 MB): 56 us, 3.7 TB/s, of them 8 sorting.
#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 256;
constexpr int kTileRows = 16;    // of a set of rows
constexpr int kLaneRows = 64;    // up to so many rows are sorted by each wave itself
constexpr int kFindRows = 1024;  // up to so many, of up to kFindBins - 1 adapters, by each workgroup
constexpr int kFindBins = 256;
constexpr int kSortThreads = 1024;
constexpr int kMaxAdapters = 4096;
constexpr int kTileCols = 64;    // output columns of a wave at a time
constexpr int kTurns = 2;        // expand_kernel: how many times
constexpr int kFusedWaves = 16;

struct AdapterParams {
  const uint16_t* x;
  const uint16_t* y;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int32_t* ids;
  uint16_t* out;
  float* part;       // [split][row][rank]
  int32_t* order;    // rows sorted by adapter, NULL if workgroups find theirs
  int32_t* tiles;    // [tile][3]: adapter (-1: none, -2: no such tile), start, count
  int32_t x_row, y_row, out_row;
  uint32_t x_bytes, y_bytes, out_bytes;
  int32_t rows, K, N, rank, adapters, splits, split_k, n_tiles;
  int32_t wide;      // y and out can be read 16 bytes at a time, and N is a multiple of 8
  int32_t in_place;
  int32_t id_bits;   // of the numbers 0 .. adapters
  int32_t tile_rows;
};

// R sets of sixteen rows.
template <int R>
struct Tile {
  int adapter;  // -1: rows without one; -2: no such tile
  int count;
  int row[R];   // of this lane's columns (16 set + lane % 16); one of the tile's rows in any case

  __device__ __forceinline__ bool has(int set) const {
    return 16 * set + (int)(threadIdx.x & 15) < count;
  }
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Buffers with 32-bit offsets: few instructions an address, and words past the end
// read as zeros and are not written. All of an address is in the vector offset, the
// one that is checked against the buffer's size; buffers are below 2 GiB, so kNowhere
// and a few words from it are past the end of each.
constexpr uint32_t kNowhere = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, (int)bytes, 0x00027000);
}
template <int Hint = 0>
__device__ __forceinline__ u4v load16(__amdgpu_buffer_rsrc_t b, uint32_t at) {
  return __builtin_bit_cast(u4v, __builtin_amdgcn_raw_buffer_load_b128(b, at, 0, Hint));
}

// The hint (non-temporal) for y and out where many rows pass through: it keeps B and t in
// the L2 (4096 rows, K = N = 8192, rank 32: 60.4 us without it, 57.0 with; for x as well
// 58.9). Few rows stay in the L2 for the next reader.
template <int R>
constexpr int kOnce = R == 2 ? 2 : 0;

__device__ __forceinline__ int at_most(int v, int most) { return v < most ? v : most; }

__device__ __forceinline__ int id_of(const AdapterParams& p, int row) {
  const int id = p.ids[row];
  return (uint32_t)id < (uint32_t)p.adapters ? id : -1;
}

// The lanes whose `v`, a number of so many bits, is this lane's.
__device__ __forceinline__ uint64_t lanes_with(int v, int bits) {
  uint64_t same = ~(uint64_t)0;
  for (int b = 0; b < bits; ++b) {
    const bool one = (v >> b) & 1;
    const uint64_t ones = __ballot(one);
    same &= one ? ones : ~ones;
  }
  return same;
}

// Tile `g` of up to 64 rows grouped by adapter, sixteen rows to a tile: each wave finds it
// from the ids, one to a lane.
__device__ __forceinline__ Tile<1> lane_tile(const AdapterParams& p, int g) {
  const int lane = threadIdx.x & 63;
  Tile<1> t;
  const bool here = lane < p.rows;
  const int id = here ? id_of(p, lane) : -1;
  const uint64_t same = lanes_with(id < 0 ? p.adapters : id, p.id_bits) & __ballot(here);
  const int rank = __popcll(same & (((uint64_t)1 << lane) - 1));
  // every sixteenth row of an adapter heads a tile
  const uint64_t heads = __ballot(here && rank % kTileRows == 0);
  t.adapter = -2;
  t.count = 0;
  t.row[0] = 0;
  if (g >= __popcll(heads)) return t;
  const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(heads >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)heads, 0));
  const int head = __builtin_ctzll(__ballot(((heads >> lane) & 1) && before == g));
  t.adapter = __builtin_amdgcn_readlane(id, head);
  const int place = rank - __builtin_amdgcn_readlane(rank, head);
  const bool member = here && id == t.adapter && place >= 0 && place < kTileRows;
  t.count = __popcll(__ballot(member));
  // row number to the lane of its column; the others' go to a lane that is not read
  const int placed = __builtin_amdgcn_ds_permute(4 * (member ? place : 63), lane);
  t.row[0] = __shfl(placed, t.has(0) ? lane & 15 : 0, 64);
  return t;
}

// Tile `g` of up to kFindRows rows, found by a workgroup of four waves: each counts the
// adapters of its quarter of the rows, all waves find the tile from the counts, and the
// rows of the tile's adapter place themselves, in their order. Sorting in a launch of its
// own costs more up to some 1700 rows (117 rows of 5 adapters: 17.7 us, so 15.0; 1076 of 3:
// 26.4 and 24.6; 1723 of 9: 28.0 and 28.3; 4096 of 8: 61 and 73).
struct Found {
  int count[4][kFindBins];
  int row[32];
};

template <int R>
__device__ __forceinline__ Tile<R> group_tile(const AdapterParams& p, int g, Found& found) {
  constexpr int kIds = kFindRows / kThreads;  // of a lane
  constexpr int kRows = 16 * R;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int each = (p.rows + kThreads - 1) / kThreads * 64;  // rows of a wave
  const int row0 = wave * each + lane;
  int bin[kIds], before[kIds];  // the last bin: rows without an adapter; -1: no such row
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    bin[i] = -1;
    if (64 * i < each) bin[i] = p.ids[at_most(row0 + 64 * i, p.rows - 1)];
  }
  for (int i = threadIdx.x; i < 4 * kFindBins; i += kThreads) (&found.count[0][0])[i] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    if (64 * i >= each) break;
    const bool here = row0 + 64 * i < p.rows;
    bin[i] = !here ? -1 : (uint32_t)bin[i] < (uint32_t)p.adapters ? bin[i] : p.adapters;
    // the wave's rows of a bin are counted at once; no other wave has its counters
    const uint64_t same = lanes_with(here ? bin[i] : 0, p.id_bits) & __ballot(here);
    const int old = here ? found.count[wave][bin[i]] : 0;
    before[i] = old + __popcll(same & (((uint64_t)1 << lane) - 1));
    if (here && lane == __builtin_ctzll(same)) found.count[wave][bin[i]] = old + __popcll(same);
  }
  __syncthreads();
  // four bins to a lane: the tiles before them, and the one that holds tile g
  int count[4], tiles = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    count[e] = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) count[e] += found.count[w][4 * lane + e];
    tiles += (count[e] + kRows - 1) / kRows;
  }
  int until = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(until, d, 64);
    until += lane >= d ? x : 0;
  }
  Tile<R> t;
  t.adapter = -2;
  t.count = 0;
#pragma unroll
  for (int j = 0; j < R; ++j) t.row[j] = 0;
  const uint64_t holds = __ballot(g < until && g >= until - tiles);
  if (!holds) return t;
  int nth = g - (until - tiles), its = 0, rows = 0;
  bool open = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int n = (count[e] + kRows - 1) / kRows;
    if (open && nth < n) {
      open = false;
      its = 4 * lane + e;
      rows = count[e];
    } else if (open) {
      nth -= n;
    }
  }
  const int owner = __builtin_ctzll(holds);
  its = __builtin_amdgcn_readlane(its, owner);
  const int first = __builtin_amdgcn_readlane(nth, owner) * kRows;
  t.adapter = its == p.adapters ? -1 : its;
  t.count = at_most(__builtin_amdgcn_readlane(rows, owner) - first, kRows);
  int earlier = -first;
  for (int w = 0; w < wave; ++w) earlier += found.count[w][its];
#pragma unroll
  for (int i = 0; i < kIds; ++i) {
    if (64 * i >= each) break;
    const int place = before[i] + earlier;
    if (bin[i] == its && place >= 0 && place < t.count) found.row[place] = row0 + 64 * i;
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < R; ++j) t.row[j] = found.row[t.has(j) ? 16 * j + (lane & 15) : 0];
  return t;
}

template <int R>
__device__ __forceinline__ Tile<R> find_tile(const AdapterParams& p, int g, Found& found) {
  if (p.rows > kLaneRows && !p.order) return group_tile<R>(p, g, found);
  if constexpr (R == 1)
    if (p.rows <= kLaneRows) return lane_tile(p, g);
  const int lane = threadIdx.x & 63;
  Tile<R> t;
  t.adapter = uniform(p.tiles[3 * g]);
  const int start = uniform(p.tiles[3 * g + 1]);
  t.count = uniform(p.tiles[3 * g + 2]);
#pragma unroll
  for (int j = 0; j < R; ++j)
    t.row[j] = t.adapter == -2 ? 0 : p.order[start + (t.has(j) ? 16 * j + (lane & 15) : 0)];
  return t;
}

// ---------------------------------------------------------------------- sorting

// One workgroup counts the rows of each adapter, places the adapters one after the
// other, describes the tiles and puts the rows in order. Rows of one adapter often stand
// together, so a wave adds its rows to a counter at once: 4096 rows of 8 adapters take 8.4
// us in place of 11.7 with an atomic for each.
__global__ __launch_bounds__(kSortThreads) void sort_kernel(AdapterParams p) {
  __shared__ int count[kMaxAdapters + 1], row_at[kMaxAdapters + 1], tile_at[kMaxAdapters + 2];
  __shared__ int sums[2][kSortThreads / 64];
  fetch(p);
  const int bins = p.adapters + 1, tid = threadIdx.x;  // the last bin: rows without one
  const int lane = tid & 63, wave = tid >> 6;
  // the bin of a row, -1 past the last row
  auto bin_of = [&](int row) {
    const int id = id_of(p, at_most(row, p.rows - 1));
    return row >= p.rows ? -1 : id < 0 ? p.adapters : id;
  };
  // counters[bin] raised by the wave's rows of each bin; *at: this row's place in its bin
  auto add = [&](int* counters, int bin, int* at) {
    const uint64_t same = lanes_with(bin < 0 ? 0 : bin, p.id_bits) & __ballot(bin >= 0);
    const int first = bin >= 0 ? __builtin_ctzll(same) : lane;
    int old = 0;
    if (bin >= 0 && lane == first) old = atomicAdd(&counters[bin], __popcll(same));
    *at = __shfl(old, first, 64) + __popcll(same & (((uint64_t)1 << lane) - 1));
  };
  for (int i = tid; i < bins; i += kSortThreads) count[i] = 0;
  __syncthreads();
  // four rows of a thread are read before the first is counted
  constexpr int kBatch = 4;
  auto each_row = [&](auto use) {
    for (int i = wave * 64; i < p.rows; i += kBatch * kSortThreads) {
      int bin[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) bin[j] = bin_of(i + j * kSortThreads + lane);
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (i + j * kSortThreads < p.rows) use(i + j * kSortThreads + lane, bin[j]);
    }
  };
  int at;
  each_row([&](int, int bin) { add(count, bin, &at); });
  __syncthreads();
  // running sums of rows and of tiles over the bins, a few bins to a thread
  const int each = (bins + kSortThreads - 1) / kSortThreads;
  const int b0 = tid * each, b1 = b0 + each < bins ? b0 + each : bins;
  int rows = 0, tiles = 0;
  for (int i = b0; i < b1; ++i) {
    rows += count[i];
    tiles += (count[i] + p.tile_rows - 1) / p.tile_rows;
  }
  int row = rows, tile = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int x = __shfl_up(row, d, 64), y = __shfl_up(tile, d, 64);
    row += lane >= d ? x : 0;
    tile += lane >= d ? y : 0;
  }
  if (lane == 63) {
    sums[0][wave] = row;
    sums[1][wave] = tile;
  }
  __syncthreads();
  row -= rows;
  tile -= tiles;
  for (int w = 0; w < wave; ++w) {
    row += sums[0][w];
    tile += sums[1][w];
  }
  for (int i = b0; i < b1; ++i) {
    row_at[i] = row;
    tile_at[i] = tile;
    row += count[i];
    tile += (count[i] + p.tile_rows - 1) / p.tile_rows;
  }
  if (b0 < bins && b1 == bins) tile_at[bins] = tile;
  __syncthreads();
  for (int t = tid; t < p.n_tiles; t += kSortThreads) {
    int* to = p.tiles + 3 * t;
    if (t >= tile_at[bins]) {
      to[0] = -2;
      to[1] = to[2] = 0;
      continue;
    }
    int lo = 0, hi = bins;  // the last bin that begins at or before t, which has a tile there
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_at[mid] <= t) lo = mid; else hi = mid;
    }
    const int in_bin = (t - tile_at[lo]) * p.tile_rows;
    to[0] = lo == p.adapters ? -1 : lo;
    to[1] = row_at[lo] + in_bin;
    to[2] = count[lo] - in_bin < p.tile_rows ? count[lo] - in_bin : p.tile_rows;
  }
  __syncthreads();
  // the order within a bin changes from run to run; no row's result depends on it
  each_row([&](int row, int bin) {
    add(row_at, bin, &at);
    if (bin >= 0) p.order[at] = row;
  });
}

// ------------------------------------------------------------------ t = A[a] x
//
// NB blocks of 16 ranks, R sets of 16 rows; W waves take turns at kStep k each. A wave brings
// whole rows of its step to its own LDS and reads both operands from there (eight
// consecutive k per lane). Read from memory in the operands' own layout, 64 bytes of each
// of sixteen rows at a time, every line is asked for twice, and a compute unit waits for
// its lines (one row, K = 4096, rank 16, in one workgroup: 8.3 us, so 5.6; 4096 rows, rank 32: 26
// us, so 20). Entry e of acc[j][i]: rank 16 i + 4 (lane / 16) + e of the row of column
// lane % 16 of set j.

template <int NB, int R>
struct Stage {
  static constexpr int kStep = NB == 8 ? 64 : 128;    // k of a step
  static constexpr int kWords = kStep / 8;            // 16-byte words of a row
  static constexpr int kRows = 64 / kWords;           // rows of one load
  static constexpr int kBytes = (NB + R) * 16 * kStep * 2;
  // the place of a word in its row of LDS, so that the rows read together differ in banks
  static __device__ __forceinline__ int place(int row, int word) {
    return word ^ (kWords == 16 ? row & 15 : (row >> 1) & 7);
  }
};

template <class T, int NB, int R>
__device__ __forceinline__ void shrink(const AdapterParams& p, const Tile<R>& t, int from, int to,
                                       int stride, char* lds, f4v (&acc)[R][NB]) {
  using S = Stage<NB, R>;
  const int lane = threadIdx.x & 63, c = lane >> 4, col = lane & 15;
  const __amdgpu_buffer_rsrc_t x = buffer(p.x, p.x_bytes);
  const __amdgpu_buffer_rsrc_t a =
      buffer(p.a + (int64_t)t.adapter * p.rank * p.K, 2u * (uint32_t)p.rank * (uint32_t)p.K);
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[j][i] = f4v{0.f, 0.f, 0.f, 0.f};
  char* const a_lds = lds + R * 16 * S::kStep * 2;
  // this lane's row of each load and the word that belongs in its place
  constexpr int kLoads = 16 / S::kRows;
  uint32_t x_at[R][kLoads], a_at[kLoads];
#pragma unroll
  for (int l = 0; l < kLoads; ++l) {
    const int row = S::kRows * l + lane / S::kWords;
    const uint32_t word = 16 * S::place(row, lane % S::kWords);
    a_at[l] = 2 * (uint32_t)row * (uint32_t)p.K + word;
#pragma unroll
    for (int j = 0; j < R; ++j)
      x_at[j][l] = 2 * (uint32_t)__shfl(t.row[j], row, 64) * (uint32_t)p.x_row + word;
  }
  const uint32_t a_block = 32 * (uint32_t)p.K;
  int k0 = from;
  for (; k0 + S::kStep <= to; k0 += stride) {
    // rows past the tile's last are those of its first again, or not read; ranks past the
    // last are the last rows' again: both only reach entries that are not used
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
      for (int l = 0; l < kLoads; ++l)
        if (16 * j + S::kRows * l < t.count)
          load_to_lds(x, x_at[j][l] + 2 * k0, lds + (16 * j + S::kRows * l) * S::kStep * 2);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int l = 0; l < kLoads; ++l)
        if (16 * i + S::kRows * l < p.rank)
          load_to_lds(a, a_at[l] + i * a_block + 2 * k0,
                      a_lds + (16 * i + S::kRows * l) * S::kStep * 2);
    wait_for_loads();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < S::kStep / 32; ++s) {
      const int word = 16 * S::place(col, 4 * s + c);
      u4v xw[R];
#pragma unroll
      for (int j = 0; j < R; ++j) xw[j] = *(const u4v*)(lds + (16 * j + col) * S::kStep * 2 + word);
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const u4v aw = *(const u4v*)(a_lds + (16 * i + col) * S::kStep * 2 + word);
#pragma unroll
        for (int j = 0; j < R; ++j) acc[j][i] = T::mfma16(aw, xw[j], acc[j][i]);
      }
    }
    // the next step's loads come after these reads
    wait_for_lds();
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
  // the end of K, less than a step, straight to the operands
  for (; k0 < to; k0 += 32) {
    const bool in = k0 + 8 * c < to;
    const uint32_t at = 2 * k0 + 16 * c;
    u4v xw[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
      xw[j] = load16(x, in && t.has(j) ? 2 * (uint32_t)t.row[j] * (uint32_t)p.x_row + at : kNowhere);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const u4v aw = load16(
          a, in && 16 * i + col < p.rank ? 2 * (uint32_t)(16 * i + col) * (uint32_t)p.K + at : kNowhere);
#pragma unroll
      for (int j = 0; j < R; ++j) acc[j][i] = T::mfma16(aw, xw[j], acc[j][i]);
    }
  }
}

template <class T, int NB, int R>
__global__ __launch_bounds__(kThreads) void shrink_kernel(AdapterParams p) {
  using S = Stage<NB, R>;
  __shared__ __attribute__((aligned(16))) char stage[4 * S::kBytes];
  static_assert(S::kBytes >= R * NB * 1024, "the waves' sums fit their stage");
  fetch(p);
  static_assert(sizeof(Found) <= sizeof stage, "both use the same memory");
  const Tile<R> t = find_tile<R>(p, blockIdx.x, *(Found*)stage);
  if (t.adapter < 0) return;
  __syncthreads();
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int from = blockIdx.y * p.split_k;
  const int to = from + p.split_k < p.K ? from + p.split_k : p.K;
  f4v acc[R][NB];
  shrink<T, NB, R>(p, t, from + S::kStep * wave, to, 4 * S::kStep, stage + wave * S::kBytes, acc);
  __syncthreads();
  float(*sums)[R * NB][64][4] = (float(*)[R * NB][64][4])stage;
#pragma unroll
  for (int j = 0; j < R; ++j)
#pragma unroll
    for (int i = 0; i < NB; ++i) *(f4v*)sums[wave][j * NB + i][lane] = acc[j][i];
  __syncthreads();
  for (int e = wave; e < R * NB; e += 4) {
    const int j = e / NB, r = 16 * (e % NB) + 4 * (lane >> 4);
    f4v v = *(f4v*)sums[0][e][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += *(f4v*)sums[w][e][lane];
    int row = t.row[0];
#pragma unroll
    for (int i = 1; i < R; ++i) row = j == i ? t.row[i] : row;
    if (t.has(j) && r < p.rank)
      *(f4v*)(p.part + ((int64_t)blockIdx.y * p.rows + row) * p.rank + r) = v;
  }
}

// ------------------------------------------------------------- out = y + s B[a] t
//
// 64 output columns to a wave at a time. Row i of column block k's operand is output
// column 32 (k / 2) + 8 (i / 4) + 4 (k % 2) + i % 4, so a lane's results are twice eight
// consecutive columns of its row, and four lanes' together 64 bytes of y and out. Lanes of
// neighbouring rows exchange halves, so that a load or store moves 128 bytes of a row
// (4096 rows, K = N = 8192, rank 32: 63.0 us, so 60.5). y and B are read before t is
// needed. Where rows do not begin at multiples of 16 bytes, whole tiles of columns are
// read and written by unaligned words of 16 bytes (156 rows, N = 10925: 12.4 us, by single
// elements 20.5), the last tile by single elements.

// The neighbouring lane's v.
__device__ __forceinline__ uint32_t neighbour(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true);
}

// From a lane's two halves of its own row to the two rows of a pair of lanes, half
// lane % 2 of each, and back.
__device__ __forceinline__ void exchange(u4v (&w)[2]) {
  const bool odd = threadIdx.x & 1;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t got = neighbour(odd ? w[0][e] : w[1][e]);
    w[0][e] = odd ? got : w[0][e];
    w[1][e] = odd ? w[1][e] : got;
  }
}

// Where column n of row i of this pair of lanes is in y or out.
template <int R>
__device__ __forceinline__ uint32_t place(const Tile<R>& t, int j, int i, int n, int row_step,
                                          int N) {
  const int odd = threadIdx.x & 1, row = (int)neighbour((uint32_t)t.row[j]);
  const bool in = 16 * j + (int)(threadIdx.x & 14) + i < t.count && n < N;
  return in ? 2 * ((uint32_t)(i == odd ? t.row[j] : row) * (uint32_t)row_step + n) : kNowhere;
}

template <class T, int NB, int R>
struct Columns {
  static constexpr int kSteps = (NB + 1) / 2;  // products of 32 ranks
  u4v b[kSteps][4], y[R][2];

  __device__ __forceinline__ void load(const AdapterParams& p, const Tile<R>& t, int n0) {
    const int lane = threadIdx.x & 63, c = lane >> 4, col = lane & 15;
    const int n = n0 + 8 * c, odd = lane & 1;
    const __amdgpu_buffer_rsrc_t from = buffer(p.y, p.y_bytes);
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (p.wide) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
          y[j][i] = load16<kOnce<R>>(from, place(t, j, i, n + 32 * odd, p.y_row, p.N));
        continue;
      }
      if (n0 + kTileCols <= p.N) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t at = place(t, j, i, n + 32 * odd, p.y_row, p.N);
          __builtin_memcpy(&y[j][i], (const char*)p.y + (at == kNowhere ? 0 : at), 16);
        }
        continue;
      }
      const uint32_t at = 2 * ((uint32_t)t.row[j] * (uint32_t)p.y_row + n);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = n + 32 * i + 2 * e;
          const uint32_t to = at + 64 * i + 4 * e;
          const uint32_t e0 = __builtin_amdgcn_raw_buffer_load_b16(
              from, t.has(j) && m < p.N ? to : kNowhere, 0, 0);
          const uint32_t e1 = __builtin_amdgcn_raw_buffer_load_b16(
              from, t.has(j) && m + 1 < p.N ? to + 2 : kNowhere, 0, 0);
          y[j][i][e] = (e0 & 0xFFFF) | (e1 << 16);
        }
      }
    }
    if (t.adapter < 0) return;
    const __amdgpu_buffer_rsrc_t rows =
        buffer(p.b + (int64_t)t.adapter * p.N * p.rank, 2u * (uint32_t)p.N * (uint32_t)p.rank);
    const uint32_t b_at = 2 * (uint32_t)(n0 + 8 * (col >> 2) + (col & 3)) * (uint32_t)p.rank + 16 * c;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        b[s][i] = load16(rows, 32 * s + 8 * c < p.rank
                                   ? b_at + 64 * s + (32 * (i / 2) + 4 * (i % 2)) * 2 * (uint32_t)p.rank
                                   : kNowhere);
  }
};

// t of sixteen rows, from fp32 in LDS to pairs high + low of the element type in operand
// layout. fp16: the row's largest entry is brought to [512, 1024) by a power of two, so
// neither half overflows and the low half keeps its digits; `factor` undoes it.
template <class T, int NB>
struct Inner {
  static constexpr int kSteps = (NB + 1) / 2;
  u4v hi[kSteps], lo[kSteps];
  float factor;

  __device__ __forceinline__ void read(const AdapterParams& p, int adapter, bool here,
                                       const float* inner) {
    const int lane = threadIdx.x & 63, c = lane >> 4;
    float v[kSteps][8], top = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int e = 0; e < 8; e += 4) {
        const bool in = 32 * s + 8 * c < p.rank && here;
        const f4v w = *(const f4v*)(inner + at_most(32 * s + 8 * c, p.rank - 8) + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[s][e + i] = in ? w[i] : 0.f;
          top = fmaxf(top, fabsf(v[s][e + i]));
        }
      }
    factor = p.scales ? p.scales[adapter] : 1.f;
    if (T::kHalf) {
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const bool plain = !(top > 0.f) || top == INFINITY;
      const int e = plain ? 0 : 10 - __builtin_amdgcn_frexp_expf(top);
      factor *= __builtin_amdgcn_ldexpf(1.f, -e);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[s][i] = __builtin_amdgcn_ldexpf(v[s][i], e);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[s][i] = T::pack(v[s][2 * i], v[s][2 * i + 1]);
        const f2v h = T::unpack(hi[s][i]);
        const float l0 = v[s][2 * i] - h.x, l1 = v[s][2 * i + 1] - h.y;
        // of an infinity or NaN the high half says all
        lo[s][i] = T::pack(fabsf(h.x) < INFINITY ? l0 : 0.f, fabsf(h.y) < INFINITY ? l1 : 0.f);
      }
  }
};

template <class T, int NB, int R>
__device__ __forceinline__ void expand(const AdapterParams& p, const Tile<R>& t,
                                       const Columns<T, NB, R>& w, const Inner<T, NB> (&v)[R],
                                       int n0) {
  const int lane = threadIdx.x & 63, c = lane >> 4;
  const int n = n0 + 8 * c;
  const __amdgpu_buffer_rsrc_t to = buffer(p.out, p.out_bytes);
#pragma unroll
  for (int j = 0; j < R; ++j) {
    f4v acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
    u4v r[2] = {w.y[j][0], w.y[j][1]};
    const bool whole = p.wide || n0 + kTileCols <= p.N;
    if (whole) exchange(r);
    if (t.adapter >= 0) {
#pragma unroll
      for (int s = 0; s < Inner<T, NB>::kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[i] = T::mfma16(w.b[s][i], v[j].hi[s], acc[i]);
          acc[i] = T::mfma16(w.b[s][i], v[j].lo[s], acc[i]);
        }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f2v f = T::unpack(r[i / 4][i % 4]);
        r[i / 4][i % 4] = T::pack(f.x + acc[i / 2][2 * (i % 2)] * v[j].factor,
                                  f.y + acc[i / 2][2 * (i % 2) + 1] * v[j].factor);
      }
    }
    if (whole) {
      exchange(r);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = place(t, j, i, n + 32 * (lane & 1), p.out_row, p.N);
        if (p.wide)
          __builtin_amdgcn_raw_buffer_store_b128(r[i], to, at, 0, kOnce<R>);
        else if (at != kNowhere)
          __builtin_memcpy((char*)p.out + at, &r[i], 16);
      }
      continue;
    }
    const uint32_t at = 2 * ((uint32_t)t.row[j] * (uint32_t)p.out_row + n);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        __builtin_amdgcn_raw_buffer_store_b16(
            (short)(r[i][e / 2] >> (16 * (e % 2))), to,
            t.has(j) && n + 32 * i + e < p.N ? at + 64 * i + 2 * e : kNowhere, 0, 0);
  }
}

// Two turns of 64 columns to a wave; the workgroup sums the parts of t once. Workgroups
// go to the eight XCDs in turn, the column blocks first: an XCD's L2 then holds its own
// columns' part of B (4096 rows, N = 8192: 39 us with the tiles first, so 35).
template <class T, int NB, int R>
__global__ __launch_bounds__(kThreads) void expand_kernel(AdapterParams p) {
  constexpr int kPitch = 16 * NB + 4;
  __shared__ __attribute__((aligned(16))) float inner[16 * R * kPitch];
  __shared__ int row_of[16 * R];
  fetch(p);
  __shared__ Found found;
  const Tile<R> t = find_tile<R>(p, blockIdx.y, found);
  if (t.adapter == -2 || (t.adapter == -1 && p.in_place)) return;
  const int wave = uniform(threadIdx.x >> 6), col = threadIdx.x & 15;
  const int n0 = ((int)blockIdx.x * 4 + wave) * kTurns * kTileCols;
  Columns<T, NB, R> w;
  if (n0 < p.N) w.load(p, t, n0);
  Inner<T, NB> v[R];
  if (t.adapter >= 0) {
    if (threadIdx.x < 16) {
#pragma unroll
      for (int j = 0; j < R; ++j) row_of[16 * j + col] = t.row[j];
    }
    __syncthreads();
    const int words = p.rank / 4;
    for (int e = threadIdx.x; e < 16 * R * words; e += kThreads) {
      const int at = e / words, r = e % words * 4;
      const float* from = p.part + (int64_t)row_of[at] * p.rank + r;
      const int64_t step = (int64_t)p.rows * p.rank;
      f4v sum = f4v{0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < p.splits; j += 4) {
        f4v x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *(const f4v*)(from + at_most(j + i, p.splits - 1) * step);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (j + i < p.splits) sum += x[i];
      }
      *(f4v*)(inner + at * kPitch + r) = sum;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < R; ++j)
      v[j].read(p, t.adapter, t.has(j), inner + (16 * j + col) * kPitch);
  }
#pragma unroll
  for (int i = 0; i < kTurns; ++i) {
    const int at = n0 + i * kTileCols;
    if (at >= p.N) return;
    if (i) w.load(p, t, at);
    expand<T, NB, R>(p, t, w, v, at);
  }
}

// ------------------------------------------------------------ both in one launch
//
// For few rows with small adapters: sixteen waves compute t of a tile over all of K, in
// every workgroup again for its 1024 output columns. Reading A again for each of them costs less
// than a second launch and the way of t through memory.

template <class T>
__global__ __launch_bounds__(64 * kFusedWaves) void fused_kernel(AdapterParams p) {
  constexpr int NB = 1, kPitch = 16 * NB + 4;
  using S = Stage<NB, 1>;
  __shared__ __attribute__((aligned(16))) char stage[kFusedWaves * S::kBytes];
  __shared__ __attribute__((aligned(16))) float inner[16 * kPitch];
  fetch(p);
  const Tile<1> t = lane_tile(p, blockIdx.y);
  if (t.adapter == -2 || (t.adapter == -1 && p.in_place)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int n0 = ((int)blockIdx.x * kFusedWaves + wave) * kTileCols;
  Columns<T, NB, 1> w;
  if (n0 < p.N) w.load(p, t, n0);
  Inner<T, NB> v[1];
  if (t.adapter >= 0) {
    f4v acc[1][NB];
    shrink<T, NB, 1>(p, t, S::kStep * wave, p.K, kFusedWaves * S::kStep, stage + wave * S::kBytes,
                     acc);
    __syncthreads();
    float* sums = (float*)stage;
#pragma unroll
    for (int i = 0; i < NB; ++i) *(f4v*)(sums + ((wave * NB + i) * 64 + lane) * 4) = acc[0][i];
    __syncthreads();
    if (threadIdx.x < NB * 256) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kFusedWaves; ++i) sum += sums[i * NB * 256 + threadIdx.x];
      const int l = threadIdx.x / 4 % 64, r = threadIdx.x / 256 * 16 + 4 * (l >> 4) + threadIdx.x % 4;
      inner[(l & 15) * kPitch + r] = sum;
    }
    __syncthreads();
    v[0].read(p, t.adapter, t.has(0), inner + (lane & 15) * kPitch);
  }
  if (n0 < p.N) expand<T, NB, 1>(p, t, w, v, n0);
}

// ------------------------------------------------------------------- host side

constexpr int64_t kMostBytes = 0x7FFFFF00;

// Bytes from the first element of `rows` rows of n elements to the last.
int64_t extent(int64_t rows, int64_t stride, int64_t n) {
  if (rows < 1 || n < 1) return 0;
  return stride > kMostBytes ? kMostBytes + 1 : 2 * ((rows - 1) * stride + n);
}

int check_adapters(const lutgemm_adapters* l) {
  if (!l) return LUTGEMM_ERR_NULL;
  if (l->type != LUTGEMM_F16 && l->type != LUTGEMM_BF16) return LUTGEMM_ERR_SHAPE;
  if (l->rows < 0 || l->rows > 65535) return LUTGEMM_ERR_SHAPE;
  if (l->K < 0 || l->K % 8 || l->K >= (1 << 23) || l->N < 0 || l->N >= (1 << 23))
    return LUTGEMM_ERR_SHAPE;
  if (l->rank < 8 || l->rank > 128 || l->rank % 8) return LUTGEMM_ERR_SHAPE;
  if (l->adapters < 0 || l->adapters > kMaxAdapters) return LUTGEMM_ERR_SHAPE;
  // the kernels address x, y and out with 32-bit offsets
  if (!stride_ok(l->x_row) || l->y_row < 0 || l->out_row < 0) return LUTGEMM_ERR_SHAPE;
  if (l->rows > 1 && l->out_row < l->N) return LUTGEMM_ERR_SHAPE;  // output rows that overlap
  if (extent(l->rows, l->x_row, l->K) > kMostBytes || extent(l->rows, l->y_row, l->N) > kMostBytes ||
      extent(l->rows, l->out_row, l->N) > kMostBytes)
    return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

struct AdapterPlan {
  bool fused, sorted;
  int tile_rows, tiles, splits, split_k;
  size_t part_at, ws_bytes;
};

AdapterPlan plan(const lutgemm_adapters* l) {
  AdapterPlan r{};
  const int groups = l->adapters + 1 < l->rows ? l->adapters + 1 : l->rows;
  // many rows to an adapter: two sets of sixteen in a tile share A and B (4096 rows of 8
  // adapters of rank 32: 63 us against 66; 1000 rows of 10, rank 16: 24.3 against 25.3)
  r.tile_rows = l->rows > kLaneRows && l->rows >= 32 * (l->adapters + 1) ? 32 : 16;
  r.tiles = l->rows / r.tile_rows + groups;
  if (r.tiles > l->rows) r.tiles = l->rows;
  // fused_kernel reads A again for every 1024 columns: with ranks up to 16, up to 128 KB a
  // workgroup and 64 MB in all it is the faster way (K = N = 4096, one row: 5.6 us against 8.4; 32
  // rows of 16 adapters, N = 12288, 30 MB: 8.3 against 9.9)
  const int64_t a_bytes = (int64_t)l->K * l->rank * 2;
  const int64_t blocks = (int64_t)r.tiles * ((l->N + 1023) / 1024);
  r.fused = l->rows <= kLaneRows && l->rank <= 16 && a_bytes <= 128 << 10 &&
            a_bytes * blocks <= 64 << 20;
  if (r.fused) return r;
  // enough workgroups to use every compute unit, twice with the larger tiles, each wave
  // with a full step at least
  const int fill = r.tile_rows == 32 ? 512 : 256;
  int splits = r.tiles > 0 ? (fill + r.tiles - 1) / r.tiles : 1;
  constexpr int kStepK = 128;
  const int most = (l->K + 4 * kStepK - 1) / (4 * kStepK);
  if (splits > most) splits = most;
  if (splits > 16) splits = 16;
  if (splits < 1) splits = 1;
  r.split_k = (l->K / 8 + splits - 1) / splits * 8;
  r.split_k = (r.split_k + 4 * kStepK - 1) / (4 * kStepK) * (4 * kStepK);
  r.splits = l->K > 0 ? (l->K + r.split_k - 1) / r.split_k : 0;
  r.sorted = l->rows > kFindRows || (l->rows > kLaneRows && l->adapters >= kFindBins);
  if (r.sorted)
    r.part_at = (((size_t)l->rows + 3 * (size_t)r.tiles) * sizeof(int32_t) + 15) / 16 * 16;
  r.ws_bytes = r.part_at + (size_t)r.splits * l->rows * l->rank * sizeof(float);
  return r;
}

template <class T, int NB, int R>
int run_tiles(const AdapterPlan& r, const AdapterParams& p, hipStream_t stream) {
  int st = LUTGEMM_OK;
  if (r.splits > 0 && p.adapters > 0)
    st = launch(shrink_kernel<T, NB, R>, dim3((unsigned)r.tiles, (unsigned)r.splits), kThreads, p,
                stream);
  constexpr int cols = 4 * kTurns * kTileCols;
  if (!st)
    st = launch(expand_kernel<T, NB, R>,
                dim3((unsigned)((p.N + cols - 1) / cols), (unsigned)r.tiles), kThreads, p, stream);
  return st;
}

template <class T, int NB>
int run_adapters(const AdapterPlan& r, const AdapterParams& p, hipStream_t stream) {
  if constexpr (NB == 1)
    if (r.fused) {
      constexpr int cols = kFusedWaves * kTileCols;
      return launch(fused_kernel<T>,
                    dim3((unsigned)((p.N + cols - 1) / cols), (unsigned)r.tiles),
                    64 * kFusedWaves, p, stream);
    }
  if (r.sorted) {
    const int st = launch(sort_kernel, dim3(1), kSortThreads, p, stream);
    if (st) return st;
  }
  return r.tile_rows == 32 ? run_tiles<T, NB, 2>(r, p, stream) : run_tiles<T, NB, 1>(r, p, stream);
}

template <class T>
int run_adapters(const AdapterPlan& r, const AdapterParams& p, hipStream_t stream) {
  if (p.rank <= 16) return run_adapters<T, 1>(r, p, stream);
  if (p.rank <= 32) return run_adapters<T, 2>(r, p, stream);
  if (p.rank <= 64) return run_adapters<T, 4>(r, p, stream);
  return run_adapters<T, 8>(r, p, stream);
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_adapters_workspace(const lutgemm_adapters* l, size_t* bytes) {
  const int st = check_adapters(l);
  if (st) return st;
  if (!bytes) return LUTGEMM_ERR_NULL;
  *bytes = plan(l).ws_bytes;
  return LUTGEMM_OK;
}

extern "C" int lutgemm_adapters_add(const lutgemm_adapters* l, const void* d_x, const void* d_y,
                                    const void* d_a, const void* d_b, const float* d_scales,
                                    const int32_t* d_ids, void* d_out, void* d_workspace,
                                    size_t workspace_bytes, void* stream) {
  try {
    int st = check_adapters(l);
    if (st) return st;
    if (l->rows == 0 || l->N == 0) return LUTGEMM_OK;
    if (!d_y || !d_out || !d_ids) return LUTGEMM_ERR_NULL;
    if (l->adapters > 0 && ((l->K > 0 && (!d_x || !d_a)) || !d_b)) return LUTGEMM_ERR_NULL;
    if (!aligned(d_x, 16) || !aligned(d_a, 16) || !aligned(d_b, 16) || !aligned(d_ids, 4) ||
        !aligned(d_scales, 4) || !aligned(d_y, 2) || !aligned(d_out, 2))
      return LUTGEMM_ERR_ALIGN;
    if (d_y == d_out && l->y_row != l->out_row) return LUTGEMM_ERR_SHAPE;
    // workgroups read x, and y where it is not theirs, while others write their part of out
    const Rows out{d_out, l->rows, l->out_row, l->N};
    if ((d_y != d_out && overlap(out, {d_y, l->rows, l->y_row, l->N})) ||
        (l->adapters > 0 && overlap(out, {d_x, l->rows, l->x_row, l->K})))
      return LUTGEMM_ERR_SHAPE;
    const AdapterPlan r = plan(l);
    if (r.ws_bytes) {
      if (!d_workspace) return LUTGEMM_ERR_NULL;
      if (workspace_bytes < r.ws_bytes) return LUTGEMM_ERR_BUFFER;
      if (!aligned(d_workspace, 16)) return LUTGEMM_ERR_ALIGN;
    }
    int cus = 0;
    st = serve::check_device(&cus);
    if (st) return st;
    AdapterParams p{};
    p.x = (const uint16_t*)d_x;
    p.y = (const uint16_t*)d_y;
    p.a = (const uint16_t*)d_a;
    p.b = (const uint16_t*)d_b;
    p.scales = d_scales;
    p.ids = d_ids;
    p.out = (uint16_t*)d_out;
    if (r.sorted) {
      p.order = (int32_t*)d_workspace;
      p.tiles = p.order + l->rows;
    }
    p.part = (float*)((char*)d_workspace + r.part_at);
    p.x_row = (int32_t)l->x_row;
    p.y_row = (int32_t)l->y_row;
    p.out_row = (int32_t)l->out_row;
    p.x_bytes = (uint32_t)extent(l->rows, l->x_row, l->K);
    p.y_bytes = (uint32_t)extent(l->rows, l->y_row, l->N);
    p.out_bytes = (uint32_t)extent(l->rows, l->out_row, l->N);
    p.rows = l->rows;
    p.K = l->K;
    p.N = l->N;
    p.rank = l->rank;
    p.adapters = l->adapters;
    p.splits = r.splits;
    p.split_k = r.split_k;
    p.n_tiles = r.tiles;
    p.tile_rows = r.tile_rows;
    p.wide = aligned(d_y, 16) && aligned(d_out, 16) && l->y_row % 8 == 0 && l->out_row % 8 == 0 &&
             l->N % 8 == 0;
    p.in_place = d_y == d_out;
    while ((p.adapters >> p.id_bits) != 0) ++p.id_bits;
    return l->type == LUTGEMM_F16 ? run_adapters<serve::F16>(r, p, (hipStream_t)stream)
                                  : run_adapters<serve::BF16>(r, p, (hipStream_t)stream);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
