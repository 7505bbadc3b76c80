// adapters.hip -- low-rank adapters of many requests added to a projection's output
// (lutgemm_adapters_add; the formula is in lutgemm.h).
//
// Two products on the matrix cores, t = A[a] x and out = y + s B[a] t, over tiles of
// up to 16 rows that share an adapter. Memory bounds both: a decode step reads each
// adapter it uses once, a prompt reads x and y. Rows come in any order; up to 64 of
// them every workgroup sorts for itself (one row per lane, no extra launch), above
// that one workgroup sorts them first (sort_kernel).
//
// shrink_kernel splits K over workgroups and waves; its parts are summed when
// expand_kernel reads them, in a fixed order. t is rounded for the second product to
// a pair of numbers, high + low, of the element type: the pair's error is far below
// the rounding of the output, for two small matrix products in place of one.
#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 256;
constexpr int kTileRows = 16;
constexpr int kLaneRows = 64;    // up to so many rows are sorted by each wave itself
constexpr int kStepK = 128;      // K that a wave reads before the next wave's share
constexpr int kSortThreads = 1024;
constexpr int kMaxAdapters = 4096;
constexpr int kTileCols = 64;    // output columns of a wave

struct AdapterParams {
  const uint16_t* x;
  const uint16_t* y;
  const uint16_t* a;
  const uint16_t* b;
  const float* scales;
  const int32_t* ids;
  uint16_t* out;
  float* part;       // [split][row][rank]
  int32_t* order;    // rows sorted by adapter (above kLaneRows rows)
  int32_t* tiles;    // [tile][3]: adapter (-1: none, -2: no such tile), start, count
  int64_t x_row, y_row, out_row;
  int32_t rows, K, N, rank, adapters, splits, split_k, n_tiles;
  int32_t wide;      // y and out rows can be read 16 bytes at a time
  int32_t in_place;
};

struct Tile {
  int adapter;  // -1: rows without one; -2: no such tile
  int count;
  int row;      // of this lane's column (lane % 16); one of the tile's rows in any case
};

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int id_of(const AdapterParams& p, int row) {
  const int id = p.ids[row];
  return (uint32_t)id < (uint32_t)p.adapters ? id : -1;
}

// Tile `g` of the rows grouped by adapter. Up to 64 rows: a row's rank among those of
// its adapter makes every sixteenth of them the head of a tile.
__device__ __forceinline__ Tile find_tile(const AdapterParams& p, int g) {
  const int lane = threadIdx.x & 63;
  Tile t;
  if (p.rows > kLaneRows) {
    t.adapter = uniform(p.tiles[3 * g]);
    const int start = uniform(p.tiles[3 * g + 1]);
    t.count = uniform(p.tiles[3 * g + 2]);
    const int col = lane & 15;
    t.row = t.adapter == -2 ? 0 : p.order[start + (col < t.count ? col : 0)];
    return t;
  }
  const bool here = lane < p.rows;
  const int id = here ? id_of(p, lane) : -2;
  int rank = 0;
  for (int j = 0; j < p.rows; ++j)
    rank += __builtin_amdgcn_readlane(id, j) == id && j < lane ? 1 : 0;
  const uint64_t heads = __ballot(here && rank % kTileRows == 0);
  t.adapter = -2;
  t.count = 0;
  t.row = 0;
  if (g >= __popcll(heads)) return t;
  const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(heads >> 32),
                                               __builtin_amdgcn_mbcnt_lo((uint32_t)heads, 0));
  const uint64_t mine = __ballot(((heads >> lane) & 1) && before == g);
  const int head = __builtin_ctzll(mine);
  t.adapter = __builtin_amdgcn_readlane(id, head);
  const int first = __builtin_amdgcn_readlane(rank, head);
  const bool member = here && id == t.adapter && rank >= first && rank < first + kTileRows;
  t.count = __popcll(__ballot(member));
  const int placed = __builtin_amdgcn_ds_permute(4 * (member ? rank - first : 63), lane);
  const int col = lane & 15;
  t.row = __shfl(placed, col < t.count ? col : 0, 64);
  return t;
}

// ---------------------------------------------------------------------- sorting

__global__ __launch_bounds__(kSortThreads) void sort_kernel(AdapterParams p) {
  __shared__ int count[kMaxAdapters + 1], row_at[kMaxAdapters + 1], tile_at[kMaxAdapters + 2];
  __shared__ int sums[2][kSortThreads];
  const int bins = p.adapters + 1, tid = threadIdx.x;  // the last bin: rows without one
  for (int i = tid; i < bins; i += kSortThreads) count[i] = 0;
  __syncthreads();
  for (int i = tid; i < p.rows; i += kSortThreads) {
    const int id = id_of(p, i);
    atomicAdd(&count[id < 0 ? p.adapters : id], 1);
  }
  __syncthreads();
  // running sums of rows and of tiles over the bins, a few bins to a thread
  const int each = (bins + kSortThreads - 1) / kSortThreads;
  const int b0 = tid * each, b1 = b0 + each < bins ? b0 + each : bins;
  int rows = 0, tiles = 0;
  for (int i = b0; i < b1; ++i) {
    rows += count[i];
    tiles += (count[i] + kTileRows - 1) / kTileRows;
  }
  sums[0][tid] = rows;
  sums[1][tid] = tiles;
  __syncthreads();
  for (int d = 1; d < kSortThreads; d <<= 1) {
    const int x = tid >= d ? sums[0][tid - d] : 0, y = tid >= d ? sums[1][tid - d] : 0;
    __syncthreads();
    sums[0][tid] += x;
    sums[1][tid] += y;
    __syncthreads();
  }
  int row = sums[0][tid] - rows, tile = sums[1][tid] - tiles;
  for (int i = b0; i < b1; ++i) {
    row_at[i] = row;
    tile_at[i] = tile;
    row += count[i];
    tile += (count[i] + kTileRows - 1) / kTileRows;
  }
  if (tid == 0) tile_at[bins] = sums[1][kSortThreads - 1];
  __syncthreads();
  for (int t = tid; t < p.n_tiles; t += kSortThreads) {
    int* to = p.tiles + 3 * t;
    if (t >= tile_at[bins]) {
      to[0] = -2;
      to[1] = to[2] = 0;
      continue;
    }
    int lo = 0, hi = bins;  // the last bin that begins at or before t and has a tile there
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (tile_at[mid] <= t) lo = mid; else hi = mid;
    }
    const int at = (t - tile_at[lo]) * kTileRows;
    to[0] = lo == p.adapters ? -1 : lo;
    to[1] = row_at[lo] + at;
    to[2] = count[lo] - at < kTileRows ? count[lo] - at : kTileRows;
  }
  __syncthreads();
  // the order within a bin changes from run to run; no row's result depends on it
  for (int i = tid; i < p.rows; i += kSortThreads) {
    const int id = id_of(p, i);
    p.order[atomicAdd(&row_at[id < 0 ? p.adapters : id], 1)] = i;
  }
}

// ------------------------------------------------------------------ t = A[a] x
//
// NB blocks of 16 ranks. Both operands come straight from memory in their layout
// (eight consecutive k per lane), so nothing is staged; the four waves take turns at
// 128 k each and join their sums through LDS.

template <class T, int NB>
__global__ __launch_bounds__(kThreads) void shrink_kernel(AdapterParams p) {
  __shared__ float sums[4][NB][64][4];
  const Tile t = find_tile(p, blockIdx.x);
  if (t.adapter < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane >> 4, col = lane & 15;
  const int from = blockIdx.y * p.split_k;
  const int to = from + p.split_k < p.K ? from + p.split_k : p.K;
  const uint16_t* x = p.x + t.row * p.x_row + 8 * c;
  const uint16_t* a = p.a + (int64_t)t.adapter * p.rank * p.K + 8 * c;
  int64_t a_row[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int r = 16 * i + col;
    a_row[i] = (int64_t)(r < p.rank ? r : p.rank - 1) * p.K;
  }
  f4v acc[NB];
#pragma unroll
  for (int i = 0; i < NB; ++i) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
  for (int k0 = from + kStepK * wave; k0 < to; k0 += 4 * kStepK) {
    u4v xw[kStepK / 32], aw[kStepK / 32][NB];
#pragma unroll
    for (int s = 0; s < kStepK / 32; ++s) {
      const bool in = k0 + 32 * s + 8 * c < to;
      xw[s] = in ? *(const u4v*)(x + k0 + 32 * s) : u4v{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < NB; ++i)
        aw[s][i] = in ? *(const u4v*)(a + a_row[i] + k0 + 32 * s) : u4v{0, 0, 0, 0};
    }
#pragma unroll
    for (int s = 0; s < kStepK / 32; ++s)
#pragma unroll
      for (int i = 0; i < NB; ++i) acc[i] = T::mfma16(aw[s][i], xw[s], acc[i]);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) *(f4v*)sums[wave][i][lane] = acc[i];
  __syncthreads();
  // entry e of lane l: rank 16 i + 4 (l / 16) + e of the row of column l % 16
  for (int i = wave; i < NB; i += 4) {
    const int r = 16 * i + 4 * c;
    f4v v = *(f4v*)sums[0][i][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += *(f4v*)sums[w][i][lane];
    if (col < t.count && r < p.rank)
      *(f4v*)(p.part + ((int64_t)blockIdx.y * p.rows + t.row) * p.rank + r) = v;
  }
}

// ------------------------------------------------------------- out = y + s B[a] t
//
// A wave serves 64 output columns. Row i of the four column blocks' operands is
// output column 16 (i / 4) + 4 block + i % 4, so a lane's results are sixteen
// consecutive columns of its row: 32 bytes of y and out.

template <class T, int NB>
__global__ __launch_bounds__(kThreads) void expand_kernel(AdapterParams p) {
  constexpr int kSteps = (NB + 1) / 2;  // products of 32 ranks
  const Tile t = find_tile(p, blockIdx.x);
  if (t.adapter == -2 || (t.adapter == -1 && p.in_place)) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane >> 4, col = lane & 15;
  const int n0 = ((int)blockIdx.y * 4 + wave) * kTileCols;
  if (n0 >= p.N) return;
  f4v acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f4v{0.f, 0.f, 0.f, 0.f};
  float scale = 0.f;
  if (t.adapter >= 0) {
    const uint16_t* b = p.b + (int64_t)t.adapter * p.N * p.rank + 8 * c;
    u4v bw[kSteps][4];
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + 16 * (col >> 2) + 4 * i + (col & 3);
        bw[s][i] = 32 * s + 8 * c < p.rank
                       ? *(const u4v*)(b + (int64_t)(n < p.N ? n : p.N - 1) * p.rank + 32 * s)
                       : u4v{0, 0, 0, 0};
      }
    // this row's t, eight ranks per step, the parts summed in order
    float v[kSteps][8];
    float top = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[s][e] = 0.f;
      if (32 * s + 8 * c < p.rank) {
        const float* from = p.part + (int64_t)t.row * p.rank + 32 * s + 8 * c;
        for (int j = 0; j < p.splits; ++j) {
          const f4v lo = *(const f4v*)from, hi = *(const f4v*)(from + 4);
          from += (int64_t)p.rows * p.rank;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[s][e] += lo[e];
            v[s][4 + e] += hi[e];
          }
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[s][e]));
    }
    scale = p.scales ? p.scales[t.adapter] : 1.f;
    float down = 1.f;
    if (T::kHalf) {
      // fp16: the row's largest entry brought to [512, 1024) by a power of two, so
      // neither half of a pair overflows and the low half keeps its digits
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const bool plain = !(top > 0.f) || top == INFINITY;
      const int e = plain ? 0 : 10 - __builtin_amdgcn_frexp_expf(top);
      down = __builtin_amdgcn_ldexpf(1.f, -e);
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[s][i] = __builtin_amdgcn_ldexpf(v[s][i], e);
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u4v hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        hi[i] = T::pack(v[s][2 * i], v[s][2 * i + 1]);
        const f2v h = T::unpack(hi[i]);
        const float l0 = v[s][2 * i] - h.x, l1 = v[s][2 * i + 1] - h.y;
        // of an infinity or NaN the high half says all
        lo[i] = T::pack(fabsf(h.x) < INFINITY ? l0 : 0.f, fabsf(h.y) < INFINITY ? l1 : 0.f);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i] = T::mfma16(bw[s][i], hi, acc[i]);
        acc[i] = T::mfma16(bw[s][i], lo, acc[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = acc[i][e] * down * scale;
  }
  if (col >= t.count) return;
  const int n = n0 + 16 * c;
  const uint16_t* y = p.y + t.row * p.y_row + n;
  uint16_t* out = p.out + t.row * p.out_row + n;
  if (p.wide && n + 16 <= p.N) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      u4v w = *(const u4v*)(y + 8 * i);
      if (t.adapter >= 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f2v f = T::unpack(w[e]);
          const int at = 2 * i + e / 2, el = 2 * (e % 2);
          w[e] = T::pack(f.x + acc[at][el], f.y + acc[at][el + 1]);
        }
      }
      *(u4v*)(out + 8 * i) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (n + i < p.N)
        out[i] = t.adapter >= 0 ? T::one(T::wide(y[i]) + acc[i / 4][i % 4]) : y[i];
  }
}

// ------------------------------------------------------------------- host side

int check_adapters(const lutgemm_adapters* l) {
  if (!l) return LUTGEMM_ERR_NULL;
  if (l->type != LUTGEMM_F16 && l->type != LUTGEMM_BF16) return LUTGEMM_ERR_SHAPE;
  if (l->rows < 0 || l->rows > 65535) return LUTGEMM_ERR_SHAPE;
  if (l->K < 0 || l->K % 8 || l->K >= (1 << 24) || l->N < 0 || l->N >= (1 << 23))
    return LUTGEMM_ERR_SHAPE;
  if (l->rank < 8 || l->rank > 128 || l->rank % 8) return LUTGEMM_ERR_SHAPE;
  if (l->adapters < 0 || l->adapters > kMaxAdapters) return LUTGEMM_ERR_SHAPE;
  constexpr int64_t far = (int64_t)1 << 40;
  if (!stride_ok(l->x_row) || l->y_row < 0 || l->y_row >= far || l->out_row < 0 || l->out_row >= far)
    return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

struct AdapterPlan {
  int tiles, splits, split_k;
  size_t part_at, ws_bytes;
};

AdapterPlan plan(const lutgemm_adapters* l) {
  AdapterPlan r{};
  const int groups = l->adapters + 1 < l->rows ? l->adapters + 1 : l->rows;
  r.tiles = l->rows / kTileRows + groups;
  if (r.tiles > l->rows) r.tiles = l->rows;
  // enough workgroups to use every compute unit, each wave with a full step at least
  constexpr int kFill = 256;
  int splits = r.tiles > 0 ? (kFill + r.tiles - 1) / r.tiles : 1;
  const int most = (l->K + 4 * kStepK - 1) / (4 * kStepK);
  if (splits > most) splits = most;
  if (splits > 16) splits = 16;
  if (splits < 1) splits = 1;
  r.split_k = (l->K / 8 + splits - 1) / splits * 8;
  r.split_k = (r.split_k + 4 * kStepK - 1) / (4 * kStepK) * (4 * kStepK);
  r.splits = l->K > 0 ? (l->K + r.split_k - 1) / r.split_k : 0;
  if (l->rows > kLaneRows)
    r.part_at = (((size_t)l->rows + 3 * (size_t)r.tiles) * sizeof(int32_t) + 15) / 16 * 16;
  r.ws_bytes = r.part_at + (size_t)r.splits * l->rows * l->rank * sizeof(float);
  return r;
}

template <class T, int NB>
int run_adapters(const AdapterPlan& r, const AdapterParams& p, hipStream_t stream) {
  int st = LUTGEMM_OK;
  if (p.rows > kLaneRows) st = launch(sort_kernel, dim3(1), kSortThreads, p, stream);
  if (!st && r.splits > 0 && p.adapters > 0)
    st = launch(shrink_kernel<T, NB>, dim3((unsigned)r.tiles, (unsigned)r.splits), kThreads, p,
                stream);
  if (!st)
    st = launch(expand_kernel<T, NB>,
                dim3((unsigned)r.tiles, (unsigned)((p.N + 4 * kTileCols - 1) / (4 * kTileCols))),
                kThreads, p, stream);
  return st;
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
    if (l->rows > kLaneRows) {
      p.order = (int32_t*)d_workspace;
      p.tiles = p.order + l->rows;
    }
    p.part = (float*)((char*)d_workspace + r.part_at);
    p.x_row = l->x_row;
    p.y_row = l->y_row;
    p.out_row = l->out_row;
    p.rows = l->rows;
    p.K = l->K;
    p.N = l->N;
    p.rank = l->rank;
    p.adapters = l->adapters;
    p.splits = r.splits;
    p.split_k = r.split_k;
    p.n_tiles = r.tiles;
    p.wide = aligned(d_y, 16) && aligned(d_out, 16) && l->y_row % 8 == 0 && l->out_row % 8 == 0;
    p.in_place = d_y == d_out;
    return l->type == LUTGEMM_F16 ? run_adapters<serve::F16>(r, p, (hipStream_t)stream)
                                  : run_adapters<serve::BF16>(r, p, (hipStream_t)stream);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
