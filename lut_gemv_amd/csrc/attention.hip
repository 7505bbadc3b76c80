// attention.hip -- attention of new tokens over a paged key/value cache
// (lutgemm_paged_attention; the formula is in lutgemm.h).
//
// The query rows of one key head -- every new token times the group of query heads
// that share the key head -- are packed into tiles, row = token * group + member, so
// keys and values are read once for the whole group. Scores are computed transposed,
// S^T = K Q^T: a lane then holds one row's scores for several keys, the softmax's
// maximum and sum stay in the lane but for one exchange, and the weights are already
// in the operand layout of the second product, O^T = V^T P^T, whose V columns come
// from LDS by transposing reads. Softmax runs in base 2 with a running maximum that
// is raised only when a score passes it by more than 8: until then weights stay below
// 2^8, inside fp16's range, and the accumulators need no rescaling.
//
// Two kernels, chosen per sequence by its rows (tokens x group):
//   few_kernel   up to 16 rows, memory-bound: each wave streams its own 32-key tiles
//   many_kernel  more rows: 128 rows x 64 keys per step, keys and values through LDS
// Both split a long key axis over workgroups; combine_kernel joins the parts.
#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 256;
constexpr int kFewRows = 16;
constexpr int kManyRows = 128;
constexpr int kSplitKeys = 128;   // a part of the key axis is a multiple of this
constexpr int kMaxSplits = 128;
constexpr float kRaise = 8.0f;

struct AttnParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  uint16_t* out;
  float* part_o;  // [split][token][head][dim], the parts' sums, not yet divided
  float* part_ml;  // [split][token][head][2], their maximum and sum of weights
  int64_t table_stride, q_token, q_head, o_token, o_head;
  int64_t k_page, k_head, v_page, v_head;
  int32_t k_slot, v_slot;
  int32_t tokens, seqs, heads, kv_heads, group, pages, page_log2, table_keys, window;
  int32_t splits, chunk;
  int32_t few_rows;  // sequences of up to so many rows are few_kernel's
  int32_t tiles;     // row tiles of many_kernel, an upper bound
  float scale2;      // scale * log2(e)
};

// One sequence's new tokens and keys, brought inside the arrays.
struct Seq {
  int begin, len, n;
  bool bad;
};

__device__ __forceinline__ int start_of(const AttnParams& p, int s) {
  if (!p.q_starts) return s;
  const int v = p.q_starts[s];
  return v < 0 ? 0 : v > p.tokens ? p.tokens : v;
}

__device__ __forceinline__ Seq sequence(const AttnParams& p, int s) {
  Seq q;
  q.begin = start_of(p, s);
  const int end = start_of(p, s + 1);
  q.len = end > q.begin ? end - q.begin : 0;
  const int n = p.kv_lens[s];
  q.bad = n > p.table_keys;
  q.n = n < 0 ? 0 : n > p.table_keys ? p.table_keys : n;
  return q;
}

// The keys [lo, hi) that rows r0 .. r1 - 1 of a sequence see between them, lo brought
// down to a multiple of 64, and how they are split: parts of `chunk` keys each.
struct Span {
  int lo, hi, chunk, parts;
};

__device__ __forceinline__ Span span_of(const AttnParams& p, const Seq& q, int r0, int r1) {
  Span a;
  const int first = q.n - q.len + r0 / p.group, last = q.n - q.len + (r1 - 1) / p.group;
  a.hi = last + 1 < 0 ? 0 : last + 1;
  int lo = p.window > 0 ? first - p.window + 1 : 0;
  a.lo = lo < 0 ? 0 : lo & ~63;
  const int keys = a.hi > a.lo ? a.hi - a.lo : 0;
  // a sequence longer than the launch was made for takes longer parts
  const int need = (keys + p.splits - 1) / p.splits;
  a.chunk = need > p.chunk ? (need + kSplitKeys - 1) / kSplitKeys * kSplitKeys : p.chunk;
  a.parts = keys > a.chunk ? (keys + a.chunk - 1) / a.chunk : 1;
  return a;
}

// Where the sixteen keys from key 16 * blk on lie in their page: the page's number
// and the element offset of the first of them.
__device__ __forceinline__ int page_of(const AttnParams& p, const int32_t* row, int blk, bool* bad) {
  const int id = row[blk >> (p.page_log2 - 4)];
  const bool out = (uint32_t)id >= (uint32_t)p.pages;
  *bad |= out;
  return out ? 0 : id;
}

__device__ __forceinline__ int slot_of(const AttnParams& p, int blk) {
  return (blk & ((1 << (p.page_log2 - 4)) - 1)) << 4;
}

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int min_of(int a, int b) { return a < b ? a : b; }

// LDS rows of D elements, in which 16-byte words (keys) or 32-byte blocks (values) are
// placed at their index xor a function of the row, so that the rows that one read
// touches lie in different banks.
template <int D>
__device__ __forceinline__ int k_word(int row, int word) {
  return row * (2 * D) + ((word ^ (D == 128 ? row & 15 : (row >> 1) & 7)) << 4);
}
template <int D>
__device__ __forceinline__ int v_word(int row, int word) {
  const int turn = D == 128 ? row & 7 : (row >> 1) & 3;
  return row * (2 * D) + (((word >> 1) ^ turn) << 5) + ((word & 1) << 4);
}

// ------------------------------------------------------------------- few rows
//
// Bound by reading the cache. The four waves of a workgroup take turns at 32-key
// tiles of its part and keep their own softmax; a tile's keys go straight from
// memory to the operand registers, its values through the wave's own 32 rows of LDS,
// so the loop has no barrier. The next tile's loads are in flight while a tile is
// computed: with two workgroups on a compute unit 128 KB per unit.

template <int D>
struct FewTile {
  u4v k[2][D / 32];
  u4v v[2][D / 32];
};

template <class T, int D>
__device__ __forceinline__ void few_load(const AttnParams& p, FewTile<D>& t, const int32_t* table,
                                         int kvh, int kt, int n, int lane, bool* bad) {
  const int last = (n - 1) >> 4;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int blk = min_of(2 * kt + i, last), most = n - 1 - 16 * blk;
    const int id = uniform(page_of(p, table, blk, bad));
    const int slot = slot_of(p, blk);
    const uint16_t* kb = p.k + (int64_t)id * p.k_page + (int64_t)slot * p.k_slot + kvh * p.k_head;
    const uint16_t* vb = p.v + (int64_t)id * p.v_page + (int64_t)slot * p.v_slot + kvh * p.v_head;
    const uint32_t ko = (uint32_t)min_of(lane & 15, most) * (uint32_t)p.k_slot + 8 * (lane >> 4);
#pragma unroll
    for (int ks = 0; ks < D / 32; ++ks) t.k[i][ks] = *(const u4v*)(kb + ko + 32 * ks);
    constexpr int words = D / 8, rows = 64 / words;  // rows of values that one load covers
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const int row = min_of(rows * j + lane / words, most);
      t.v[i][j] = *(const u4v*)(vb + (uint32_t)row * (uint32_t)p.v_slot + 8 * (lane % words));
    }
  }
}

template <class T, int D>
__global__ __launch_bounds__(kThreads, 2) void few_kernel(AttnParams p) {
  constexpr int kPitch = D + 4;
  constexpr int kOut = 4 * kFewRows * kPitch * 4, kVal = 4 * 32 * D * 2;
  __shared__ __attribute__((aligned(16))) char mem[kOut > kVal ? kOut : kVal];
  __shared__ float wave_m[4][kFewRows], wave_l[4][kFewRows];
  __shared__ int any_bad;

  const int s = blockIdx.x / p.kv_heads, kvh = blockIdx.x % p.kv_heads, split = blockIdx.y;
  const Seq seq = sequence(p, s);
  const int rows = seq.len * p.group;
  if (rows > p.few_rows) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane >> 4;
  const int32_t* table = p.table + s * p.table_stride;

  for (int r0 = 0; r0 < rows; r0 += kFewRows) {
    const int r1 = min_of(r0 + kFewRows, rows);
    const Span span = span_of(p, seq, r0, r1);
    if (split >= span.parts) continue;
    const int from = span.lo + split * span.chunk;
    const int to = min_of(span.hi, from + span.chunk);
    if (threadIdx.x == 0) any_bad = seq.bad;
    __syncthreads();

    // this lane's row: its query operand and the keys [row_lo, row_hi) it sees
    const int r = r0 + (lane & 15);
    const int rc = min_of(r, r1 - 1);
    const int tok = rc / p.group, head = kvh * p.group + rc % p.group;
    const int pos = seq.n - seq.len + tok;
    const int row_hi = r < r1 ? pos + 1 : 0;
    const int row_lo = p.window > 0 ? pos - p.window + 1 : 0;
    u4v q[D / 32];
    {
      const uint16_t* qp = p.q + (int64_t)(seq.begin + tok) * p.q_token + head * p.q_head + 8 * c;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) q[ks] = *(const u4v*)(qp + 32 * ks);
    }
    f4v o[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] = f4v{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    char* vals = mem + wave * (32 * D * 2);

    auto step = [&](const FewTile<D>& t, int kt) {
      f4v sc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) {
        sc[0] = T::mfma16(t.k[0][ks], q[ks], sc[0]);
        sc[1] = T::mfma16(t.k[1][ks], q[ks], sc[1]);
      }
      constexpr int words = D / 8, vr = 64 / words;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          *(u4v*)(vals + v_word<D>(16 * i + vr * j + lane / words, lane % words)) = t.v[i][j];
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 32 * kt + 16 * i + 4 * c + e;
          const float x = sc[i][e] * p.scale2;
          sc[i][e] = key < row_hi && key >= row_lo ? x : -INFINITY;
          top = fmaxf(top, sc[i][e]);
        }
      if (__any(top > m + kRaise)) {
        top = fmaxf(top, __shfl_xor(top, 16, 64));
        top = fmaxf(top, __shfl_xor(top, 32, 64));
        const float raised = fmaxf(m, top);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - raised);
        m = raised;
        l *= f;
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][e] *= f;
      }
      const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[i][e] = __builtin_amdgcn_exp2f(sc[i][e] - base);
          l += sc[i][e];
        }
      // keys of the operand: 4c .. 4c+3 of the first sixteen, then of the second
      u4v w;
      w[0] = T::pack(sc[0][0], sc[0][1]);
      w[1] = T::pack(sc[0][2], sc[0][3]);
      w[2] = T::pack(sc[1][0], sc[1][1]);
      w[3] = T::pack(sc[1][2], sc[1][3]);
      // the wave's own stores to LDS are complete and visible to its other lanes
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      const int row = 4 * c + ((lane & 15) >> 2), col = lane & 3;  // col: 8-byte words
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        const u2v a = read_column(vals + v_word<D>(row, 2 * d + (col >> 1)) + 8 * (col & 1));
        const u2v b = read_column(vals + v_word<D>(row + 16, 2 * d + (col >> 1)) + 8 * (col & 1));
        o[d] = T::mfma16(u4v{a.x, a.y, b.x, b.y}, w, o[d]);
      }
      // the next tile's stores come after these reads
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    };

    const int end = (to + 31) >> 5;
    int kt = (from >> 5) + wave;
    if (kt < end) {
      FewTile<D> t0, t1;
      few_load<T, D>(p, t0, table, kvh, kt, seq.n, lane, &bad);
      while (true) {
        if (kt + 4 < end) few_load<T, D>(p, t1, table, kvh, kt + 4, seq.n, lane, &bad);
        step(t0, kt);
        kt += 4;
        if (kt >= end) break;
        if (kt + 4 < end) few_load<T, D>(p, t0, table, kvh, kt + 4, seq.n, lane, &bad);
        step(t1, kt);
        kt += 4;
        if (kt >= end) break;
      }
    }
    // join the four waves
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (bad && lane == 0) any_bad = 1;
    if (c == 0) {
      wave_m[wave][lane] = m;
      wave_l[wave][lane] = l;
    }
    __syncthreads();
    float* sums = (float*)mem;
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
      *(f4v*)(sums + (wave * kFewRows + (lane & 15)) * kPitch + 16 * d + 4 * c) = o[d];
    __syncthreads();
    const int jr = threadIdx.x >> 4, jc = (threadIdx.x & 15) * (D / 16);
    if (r0 + jr < r1) {
      float top = -INFINITY, total = 0.f, f[4];
#pragma unroll
      for (int w = 0; w < 4; ++w) top = fmaxf(top, wave_m[w][jr]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        f[w] = wave_m[w][jr] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(wave_m[w][jr] - top);
        total += wave_l[w][jr] * f[w];
      }
      float sum[D / 16];
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        sum[e] = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w)
          sum[e] += sums[(w * kFewRows + jr) * kPitch + jc + e] * f[w];
      }
      if (any_bad) total = __builtin_nanf("");
      const int token = seq.begin + (r0 + jr) / p.group, hd = kvh * p.group + (r0 + jr) % p.group;
      if (span.parts == 1) {
        const float inv = total == 0.f ? 0.f : 1.f / total;
        uint32_t* to32 = (uint32_t*)(p.out + (int64_t)token * p.o_token + hd * p.o_head + jc);
#pragma unroll
        for (int e = 0; e < D / 32; ++e) to32[e] = T::pack(sum[2 * e] * inv, sum[2 * e + 1] * inv);
      } else {
        const int64_t at = ((int64_t)split * p.tokens + token) * p.heads + hd;
#pragma unroll
        for (int e = 0; e < D / 16; e += 4)
          *(f4v*)(p.part_o + at * D + jc + e) = f4v{sum[e], sum[e + 1], sum[e + 2], sum[e + 3]};
        if (jc == 0) *(f2v*)(p.part_ml + 2 * at) = f2v{top, total};
      }
    }
    __syncthreads();  // before the next row tile takes the shared memory
  }
}

// ------------------------------------------------------------------ many rows
//
// Bound by the matrix cores and the softmax between them. A wave owns 32 rows; the
// four share 64 keys and values in LDS, in two buffers: the next tile's loads are
// issued before a tile is computed and stored to the other buffer after it, one
// barrier a tile. Two workgroups share a compute unit, so one's products run beside
// the other's exponentials.

template <class T, int D>
__global__ __launch_bounds__(kThreads, 2) void many_kernel(AttnParams p) {
  constexpr int kTile = 64 * D * 2;
  __shared__ __attribute__((aligned(16))) char keys[2][kTile];
  __shared__ __attribute__((aligned(16))) char vals[2][kTile];
  __shared__ int any_bad;

  const int kvh = blockIdx.x % p.kv_heads, split = blockIdx.y;
  const int tile = p.tiles - 1 - (int)(blockIdx.x / p.kv_heads);  // the longest rows first
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int h = lane >> 5;

  // the sequence of this row tile: tiles of sequence s begin at start * group / 128 + s,
  // which leaves each at least as many as its rows need
  int found = 0;
  for (int s0 = 0; s0 < p.seqs; s0 += 64) {
    const bool begun = s0 + lane < p.seqs &&
        (int)((int64_t)start_of(p, s0 + lane) * p.group / kManyRows) + s0 + lane <= tile;
    const uint64_t votes = __ballot(begun);
    found += __popcll(votes);
    if (votes != ~0ull) break;
  }
  if (found == 0) return;
  const int s = uniform(found - 1);
  const Seq seq = sequence(p, s);
  const int rows = seq.len * p.group;
  if (rows <= p.few_rows) return;
  const int r0 = (tile - (int)((int64_t)seq.begin * p.group / kManyRows) - s) * kManyRows;
  if (r0 < 0 || r0 >= rows) return;
  const int r1 = min_of(r0 + kManyRows, rows);
  const Span span = span_of(p, seq, r0, r1);
  if (split >= span.parts) return;
  const int from = span.lo + split * span.chunk;
  const int to = min_of(span.hi, from + span.chunk);
  const int32_t* table = p.table + s * p.table_stride;
  if (threadIdx.x == 0) any_bad = seq.bad;

  // this lane's row, and the wave's rows together
  const int w0 = r0 + 32 * wave, r = w0 + (lane & 31);
  const int rc = min_of(r, r1 - 1);
  const int tok = rc / p.group, head = kvh * p.group + rc % p.group;
  const int pos = seq.n - seq.len + tok;
  const int row_hi = pos + 1;
  const int row_lo = p.window > 0 ? pos - p.window + 1 : 0;
  const int first = uniform(seq.n - seq.len + min_of(w0, r1 - 1) / p.group);
  const int last = uniform(seq.n - seq.len + min_of(w0 + 31, r1 - 1) / p.group);
  // keys that some row sees [wave_lo, wave_hi), and that every row sees [all_lo, all_hi)
  const int wave_hi = w0 < r1 ? last + 1 : 0, all_hi = first + 1;
  const int wave_lo = p.window > 0 ? first - p.window + 1 : 0;
  const int all_lo = p.window > 0 ? last - p.window + 1 : 0;
  u4v q[D / 16];
  {
    const uint16_t* qp = p.q + (int64_t)(seq.begin + tok) * p.q_token + head * p.q_head + 8 * h;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) q[ks] = *(const u4v*)(qp + 16 * ks);
  }
  f16v o[D / 32];
#pragma unroll
  for (int d = 0; d < D / 32; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
  float m = -INFINITY, l = 0.f;
  bool bad = false;

  // a thread's share of a tile: one 16-byte word of each of kLoads row groups
  constexpr int kWords = D / 8, kRowsEach = kThreads / kWords, kLoads = 64 / kRowsEach;
  const int my_row = threadIdx.x / kWords, my_word = threadIdx.x % kWords;
  u4v kr[kLoads], vr[kLoads];
  const int end_blk = (seq.n - 1) >> 4;
  auto load = [&](int kt) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = kRowsEach * i + my_row;
      const int blk = uniform(min_of(4 * kt + (row >> 4), end_blk));
      const int id = uniform(page_of(p, table, blk, &bad));
      const int slot = slot_of(p, blk);
      const uint32_t in_blk = (uint32_t)min_of(row & 15, seq.n - 1 - 16 * blk);
      const uint16_t* kb = p.k + (int64_t)id * p.k_page + (int64_t)slot * p.k_slot + kvh * p.k_head;
      const uint16_t* vb = p.v + (int64_t)id * p.v_page + (int64_t)slot * p.v_slot + kvh * p.v_head;
      kr[i] = *(const u4v*)(kb + in_blk * (uint32_t)p.k_slot + 8 * my_word);
      vr[i] = *(const u4v*)(vb + in_blk * (uint32_t)p.v_slot + 8 * my_word);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = kRowsEach * i + my_row;
      *(u4v*)(keys[buf] + k_word<D>(row, my_word)) = kr[i];
      *(u4v*)(vals[buf] + v_word<D>(row, my_word)) = vr[i];
    }
  };
  auto step = [&](int buf, int kt) {
    const int k0 = 64 * kt;
    f16v sc[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int e = 0; e < 16; ++e) sc[b][e] = 0.f;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const u4v a = *(const u4v*)(keys[buf] + k_word<D>(32 * b + (lane & 31), 2 * ks + h));
        sc[b] = T::mfma32(a, q[ks], sc[b]);
      }
    }
    if (k0 + 64 > all_hi || k0 < all_lo) {
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int key = k0 + 32 * b + 8 * (e >> 2) + 4 * h + (e & 3);
          if (key >= row_hi || key < row_lo) sc[b][e] = -INFINITY;
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[b][e]);
    top *= p.scale2;
    if (__any(top > m + kRaise)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float raised = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - raised);
      m = raised;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= f;
    }
    const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        sc[b][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[b][e], p.scale2, -base));
        l += sc[b][e];
      }
    const int vrow = 4 * h + ((lane & 15) >> 2), col = lane & 3, half = (lane >> 4) & 1;
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        u4v w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = T::pack(sc[b][8 * u + 2 * e], sc[b][8 * u + 2 * e + 1]);
        const int row = 32 * b + 16 * u + vrow;
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          const int word = 4 * d + 2 * half + (col >> 1);
          const u2v x = read_column(vals[buf] + v_word<D>(row, word) + 8 * (col & 1));
          const u2v y = read_column(vals[buf] + v_word<D>(row + 8, word) + 8 * (col & 1));
          o[d] = T::mfma32(u4v{x.x, x.y, y.x, y.y}, w, o[d]);
        }
      }
  };

  const int begin = from >> 6, end = (to + 63) >> 6;
  if (begin < end) {
    load(begin);
    store(0);
    __syncthreads();
    for (int kt = begin; kt < end; ++kt) {
      const int buf = (kt - begin) & 1;
      if (kt + 1 < end) load(kt + 1);
      if (64 * kt < wave_hi && 64 * kt + 64 > wave_lo) step(buf, kt);
      if (kt + 1 < end) store(buf ^ 1);
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  if (bad && lane == 0) any_bad = 1;
  __syncthreads();
  if (r >= r1) return;
  l += __shfl_xor(l, 32, 64);
  if (any_bad) l = __builtin_nanf("");
  const int token = seq.begin + tok;
  if (span.parts == 1) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* dst = p.out + (int64_t)token * p.o_token + head * p.o_head + 4 * h;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(u2v*)(dst + 32 * d + 8 * e) = u2v{T::pack(o[d][4 * e] * inv, o[d][4 * e + 1] * inv),
                                            T::pack(o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv)};
  } else {
    const int64_t at = ((int64_t)split * p.tokens + token) * p.heads + head;
    float* dst = p.part_o + at * D + 4 * h;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(f4v*)(dst + 32 * d + 8 * e) =
            f4v{o[d][4 * e], o[d][4 * e + 1], o[d][4 * e + 2], o[d][4 * e + 3]};
    if (h == 0) *(f2v*)(p.part_ml + 2 * at) = f2v{m, l};
  }
}

// -------------------------------------------------------------- joining parts
//
// One wave for each row that was split: the parts' sums brought to one maximum.

template <class T, int D>
__global__ __launch_bounds__(kThreads) void combine_kernel(AttnParams p) {
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + uniform(threadIdx.x >> 6);
  if (row >= (int64_t)p.tokens * p.heads) return;
  const int token = (int)(row / p.heads), head = (int)(row % p.heads);
  int s = token;
  if (p.q_starts) {
    s = 0;
    for (int s0 = 0; s0 < p.seqs; s0 += 64) {
      const uint64_t votes =
          __ballot(s0 + lane < p.seqs && start_of(p, s0 + lane + 1) <= token);
      s += __popcll(votes);
      if (votes != ~0ull) break;
    }
    s = uniform(s);
    if (s >= p.seqs) return;
  }
  const Seq seq = sequence(p, s);
  if (token < seq.begin || token >= seq.begin + seq.len) return;
  const int rows = seq.len * p.group;
  const int tile = rows <= p.few_rows ? kFewRows : kManyRows;
  const int r0 = ((token - seq.begin) * p.group + head % p.group) / tile * tile;
  const Span span = span_of(p, seq, r0, min_of(r0 + tile, rows));
  if (span.parts == 1) return;
  const int64_t step = (int64_t)p.tokens * p.heads;
  float top = -INFINITY;
  for (int j = 0; j < span.parts; ++j) top = fmaxf(top, p.part_ml[2 * (row + j * step)]);
  float total = 0.f, sum[D / 64] = {};
  for (int j = 0; j < span.parts; ++j) {
    const float m = p.part_ml[2 * (row + j * step)], l = p.part_ml[2 * (row + j * step) + 1];
    const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top);
    total += l != l ? l : l * f;
#pragma unroll
    for (int e = 0; e < D / 64; ++e)
      sum[e] += f * p.part_o[(row + j * step) * D + lane * (D / 64) + e];
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  uint16_t* dst = p.out + (int64_t)token * p.o_token + head * p.o_head + lane * (D / 64);
  if constexpr (D == 128)
    *(uint32_t*)dst = T::pack(sum[0] * inv, sum[1] * inv);
  else
    *dst = T::one(sum[0] * inv);
}

// ------------------------------------------------------------------ host side

int check_attention(const lutgemm_attention* a) {
  if (!a) return LUTGEMM_ERR_NULL;
  if (a->type != LUTGEMM_F16 && a->type != LUTGEMM_BF16) return LUTGEMM_ERR_SHAPE;
  if (a->head_dim != 64 && a->head_dim != 128) return LUTGEMM_ERR_SHAPE;
  if (a->kv_heads < 1 || a->heads < 1 || a->heads > 1024 || a->heads % a->kv_heads)
    return LUTGEMM_ERR_SHAPE;
  if (a->page_size < 16 || a->page_size > 65536 || (a->page_size & (a->page_size - 1)))
    return LUTGEMM_ERR_SHAPE;
  if (a->seqs < 0 || a->seqs >= (1 << 20) || a->tokens < 0 || a->tokens >= (1 << 24))
    return LUTGEMM_ERR_SHAPE;
  if (a->table_width < 1 || (int64_t)a->table_width * a->page_size >= ((int64_t)1 << 31) - 128 ||
      a->table_stride < 0 || a->table_stride >= ((int64_t)1 << 40))
    return LUTGEMM_ERR_SHAPE;
  if (a->pages < 1 || a->pages >= ((int64_t)1 << 31)) return LUTGEMM_ERR_SHAPE;
  if (a->window < 0 || a->max_q < 0 || a->max_kv < 0) return LUTGEMM_ERR_SHAPE;
  if (!(a->scale > 0.0f) || !isfinite(a->scale)) return LUTGEMM_ERR_VALUE;
  if (!stride_ok(a->q_token) || !stride_ok(a->q_head) || !stride_ok(a->o_token) ||
      !stride_ok(a->o_head) || !stride_ok(a->k_page) || !stride_ok(a->k_slot) ||
      !stride_ok(a->k_head) || !stride_ok(a->v_page) || !stride_ok(a->v_slot) ||
      !stride_ok(a->v_head))
    return LUTGEMM_ERR_SHAPE;
  if (a->k_slot >= (1 << 24) || a->v_slot >= (1 << 24)) return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

struct AttnPlan {
  bool few, many;
  int splits, chunk;
  int64_t tiles;
  size_t ws_bytes;
};

// Which kernels run and how many parts the longest key axis is cut into: enough to
// fill the card twice over, of at least kSplitKeys keys (few rows) or 512 (many).
AttnPlan plan(const lutgemm_attention* a) {
  AttnPlan r{};
  if (a->tokens == 0 || a->seqs == 0) return r;  // nothing runs
  constexpr int64_t kFill = 512;  // workgroups: two on each of 256 compute units
  const int64_t group = a->heads / a->kv_heads;
  const int64_t table_keys = (int64_t)a->table_width * a->page_size;
  int64_t max_q = a->max_q < a->tokens ? a->max_q : a->tokens;
  if (a->seqs == 1) max_q = a->tokens;
  if (max_q < 1) max_q = 1;
  int64_t keys = a->max_kv < table_keys ? a->max_kv : table_keys;
  if (a->window > 0 && keys > a->window + max_q + 64) keys = a->window + max_q + 64;
  if (keys < 1) keys = 1;
  r.many = max_q * group > kFewRows;
  r.few = !r.many || a->seqs > 1;
  r.tiles = a->tokens * group / kManyRows + a->seqs;
  const int64_t base = (r.many ? a->tokens * group / kManyRows + 1 : a->seqs) * a->kv_heads;
  const int64_t least = r.many ? 512 : kSplitKeys;
  int64_t splits = (kFill + base - 1) / base;
  const int64_t most = (keys + least - 1) / least;
  if (splits > most) splits = most;
  if (splits > kMaxSplits) splits = kMaxSplits;
  if (splits < 1) splits = 1;
  int64_t chunk = (keys + splits - 1) / splits;
  chunk = (chunk + kSplitKeys - 1) / kSplitKeys * kSplitKeys;
  r.splits = (int)((keys + chunk - 1) / chunk);
  r.chunk = (int)chunk;
  if (r.splits > 1)
    r.ws_bytes = (size_t)r.splits * (size_t)a->tokens * (size_t)a->heads *
                 (size_t)(a->head_dim + 2) * sizeof(float);
  return r;
}

template <class T, int D>
int run_attention(const AttnPlan& r, const AttnParams& p, hipStream_t stream) {
  int st = LUTGEMM_OK;
  if (r.many)
    st = launch(many_kernel<T, D>, dim3((unsigned)(r.tiles * p.kv_heads), (unsigned)r.splits),
                kThreads, p, stream);
  if (!st && r.few)
    st = launch(few_kernel<T, D>, dim3((unsigned)(p.seqs * p.kv_heads), (unsigned)r.splits),
                kThreads, p, stream);
  if (!st && r.splits > 1)
    st = launch(combine_kernel<T, D>,
                dim3((unsigned)(((int64_t)p.tokens * p.heads + 3) / 4)), kThreads, p, stream);
  return st;
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_paged_attention_workspace(const lutgemm_attention* a, size_t* bytes) {
  const int st = check_attention(a);
  if (st) return st;
  if (!bytes) return LUTGEMM_ERR_NULL;
  *bytes = plan(a).ws_bytes;
  return LUTGEMM_OK;
}

extern "C" int lutgemm_paged_attention(const lutgemm_attention* a, const void* d_q, const void* d_k,
                                       const void* d_v, const int32_t* d_table,
                                       const int32_t* d_kv_lens, const int32_t* d_q_starts,
                                       void* d_out, void* d_workspace, size_t workspace_bytes,
                                       void* stream) {
  try {
    int st = check_attention(a);
    if (st) return st;
    if (!d_q_starts && a->tokens != a->seqs) return LUTGEMM_ERR_SHAPE;
    if (a->tokens == 0 || a->seqs == 0) return LUTGEMM_OK;
    if (!d_q || !d_k || !d_v || !d_table || !d_kv_lens || !d_out) return LUTGEMM_ERR_NULL;
    if (!aligned(d_q, 16) || !aligned(d_k, 16) || !aligned(d_v, 16) || !aligned(d_out, 16) ||
        !aligned(d_table, 4) || !aligned(d_kv_lens, 4) || !aligned(d_q_starts, 4))
      return LUTGEMM_ERR_ALIGN;
    const AttnPlan r = plan(a);
    // a launch has fewer than 2^32 threads along each axis of its grid
    constexpr int64_t kMost = (int64_t)1 << 24;
    if (r.tiles * a->kv_heads >= kMost || (int64_t)a->seqs * a->kv_heads >= kMost ||
        (r.splits > 1 && a->tokens * a->heads / 4 + 1 >= kMost))
      return LUTGEMM_ERR_SHAPE;
    if (r.ws_bytes) {
      if (!d_workspace) return LUTGEMM_ERR_NULL;
      if (workspace_bytes < r.ws_bytes) return LUTGEMM_ERR_BUFFER;
      if (!aligned(d_workspace, 16)) return LUTGEMM_ERR_ALIGN;
    }
    int cus = 0;
    st = serve::check_device(&cus);
    if (st) return st;
    AttnParams p{};
    p.q = (const uint16_t*)d_q;
    p.k = (const uint16_t*)d_k;
    p.v = (const uint16_t*)d_v;
    p.table = d_table;
    p.kv_lens = d_kv_lens;
    p.q_starts = d_q_starts;
    p.out = (uint16_t*)d_out;
    p.part_o = (float*)d_workspace;
    p.part_ml = r.ws_bytes ? (float*)d_workspace +
                                 (size_t)r.splits * a->tokens * a->heads * a->head_dim
                           : nullptr;
    p.table_stride = a->table_stride;
    p.q_token = a->q_token;
    p.q_head = a->q_head;
    p.o_token = a->o_token;
    p.o_head = a->o_head;
    p.k_page = a->k_page;
    p.k_head = a->k_head;
    p.v_page = a->v_page;
    p.v_head = a->v_head;
    p.k_slot = (int32_t)a->k_slot;
    p.v_slot = (int32_t)a->v_slot;
    p.tokens = (int32_t)a->tokens;
    p.seqs = a->seqs;
    p.heads = a->heads;
    p.kv_heads = a->kv_heads;
    p.group = a->heads / a->kv_heads;
    p.pages = (int32_t)a->pages;
    for (p.page_log2 = 4; (1 << p.page_log2) < a->page_size;) ++p.page_log2;
    p.table_keys = a->table_width * a->page_size;
    p.window = a->window;
    p.splits = r.splits;
    p.chunk = r.chunk;
    p.few_rows = !r.many ? 0x7FFFFFFF : r.few ? kFewRows : 0;
    p.tiles = (int32_t)r.tiles;
    p.scale2 = a->scale * 1.4426950408889634f;
    const bool f16 = a->type == LUTGEMM_F16;
    hipStream_t strm = (hipStream_t)stream;
    if (a->head_dim == 64)
      return f16 ? run_attention<serve::F16, 64>(r, p, strm)
                 : run_attention<serve::BF16, 64>(r, p, strm);
    return f16 ? run_attention<serve::F16, 128>(r, p, strm)
               : run_attention<serve::BF16, 128>(r, p, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
