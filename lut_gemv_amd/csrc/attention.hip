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
// is raised only when a score passes it by more than 8: until then the accumulators need
// no rescaling. fp16's weights are all multiplied by 2^7 (kLift), which their sum divides
// out again: at most 2^15 then, they are inside its range, and lose digits only below 2^-21
// of the running maximum's and vanish only below 2^-32. Unlifted, those below 2^-25 would
// vanish from the products while their sum counts them: of 131072 keys at 2^-25.4 beside a
// large one, 0.3% of the output.
//
// The weights are rounded to the element type for the second product, their sum is not:
// outputs are 1.2 to 1.4 times as far from 64 bits as with weights in fp32. Pairs of numbers
// would double that product's matrix instructions, which bound many_rows.
//
// Two bodies, chosen per sequence by its rows (tokens x group):
//   few_rows   up to 16 rows, memory-bound: each wave streams its own 32-key tiles
//   many_rows  more rows: 128 rows x 64 keys per step, keys and values through LDS
// in a kernel each, and in one together for a batch that has both. Both split a long key
// axis over workgroups; the combine kernels join the parts.
#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 256;
constexpr int kFewRows = 16;
constexpr int kFewWaves = 4;      // few_kernel's waves
constexpr int kLoneWaves = 8;     // with one workgroup to a compute unit at most
constexpr int kShortWaves = 2;    // for parts of up to kShortKeys keys
constexpr int kShortKeys = 128;
constexpr int kManyRows = 128;
constexpr int kSplitKeys = 128;   // a part of the key axis is a multiple of this
constexpr int kMaxSplits = 128;
constexpr float kRaise = 8.0f;
template <class T>
constexpr float kLift = T::kHalf ? 7.0f : 0.0f;  // bf16 has fp32's range

struct AttnParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const int32_t* table;
  const int32_t* kv_lens;
  const int32_t* q_starts;
  uint16_t* out;
  float* part_o;  // [part row][dim], the parts' sums, not yet divided
  float* part_ml;  // [part row][2], their maximum and sum of weights
  int64_t few_step, many_step, many_at;  // part rows of one split; where many_rows' begin
  int64_t table_stride, q_token, q_head, o_token, o_head;
  int64_t k_page, k_head, v_page, v_head;
  int32_t k_slot, v_slot;
  int32_t tokens, seqs, heads, kv_heads, group, pages, page_log2, table_keys, window;
  int32_t splits[2], chunk[2];  // of few_rows and of many_rows
  int32_t few_rows;             // sequences of up to so many rows are few_rows'
  int32_t tiles;                // row tiles of many_rows, an upper bound
  int32_t many_blocks;          // mixed_kernel: the workgroups of its first kind
  int32_t join_blocks;          // combine_kernel: likewise
  int32_t join_rows;            // combine_few: workgroups to a sequence and key head
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

// The first key that a row at this position sees.
__device__ __forceinline__ int first_key(const AttnParams& p, int pos) {
  return p.window > 0 && pos >= p.window ? pos - p.window + 1 : 0;
}

// The keys [first, hi) that rows r0 .. r1 - 1 of a sequence see between them, first
// brought down to a multiple of 64 (lo), and how they are split: parts of `chunk` keys
// each. Blocks of sixteen keys before first's and from hi on are never asked for: their
// pages may be gone. first's or the last one stands in for them, and no row sees it there.
struct Span {
  int first, lo, hi, chunk, parts;
  __device__ __forceinline__ int block(int blk) const {
    const int least = first >> 4, most = (hi - 1) >> 4;
    return blk < least ? least : blk > most ? most : blk;
  }
};

template <int Kind>  // 0: few_rows', 1: many_rows'
__device__ __forceinline__ Span span_of(const AttnParams& p, const Seq& q, int r0, int r1) {
  Span a;
  const int first = q.n - q.len + r0 / p.group, last = q.n - q.len + (r1 - 1) / p.group;
  a.hi = last + 1 < 0 ? 0 : last + 1;
  a.first = first_key(p, first);
  a.lo = a.first & ~63;
  const int keys = a.hi > a.lo ? a.hi - a.lo : 0;
  // a sequence longer than the launch was made for takes longer parts
  int need = (keys + p.splits[Kind] - 1) / p.splits[Kind];
  // few_rows has room for the parts of so many rows; a longer chunk, which a launch made
  // for short ones meets, is not split
  if (Kind == 0 && q.len * p.group > kFewRows) need = keys;
  a.chunk = need > p.chunk[Kind] ? (need + kSplitKeys - 1) / kSplitKeys * kSplitKeys
                                 : p.chunk[Kind];
  a.parts = keys > a.chunk ? (keys + a.chunk - 1) / a.chunk : 1;
  return a;
}

// The part row of split 0 of row r of a sequence's key head in few_rows.
__device__ __forceinline__ int64_t few_part(const AttnParams& p, int s, int kvh, int r) {
  return ((int64_t)s * p.kv_heads + kvh) * kFewRows + r;
}

// A row of the page table, read by scalar loads: they do not wait in turn behind the
// keys and values under way.
typedef const __attribute__((address_space(4))) int32_t* TableRow;

__device__ __forceinline__ TableRow table_row(const AttnParams& p, int s) {
  return (TableRow)(p.table + s * p.table_stride);
}

// The page of the sixteen keys from key 16 * blk on, and the slot of the first of them.
__device__ __forceinline__ int page_of(const AttnParams& p, int id, bool* bad) {
  const bool out = (uint32_t)id >= (uint32_t)p.pages;
  *bad |= out;
  return out ? 0 : id;
}

__device__ __forceinline__ int table_at(const AttnParams& p, int blk) {
  return blk >> (p.page_log2 - 4);
}

__device__ __forceinline__ int slot_of(const AttnParams& p, int blk) {
  return (blk & ((1 << (p.page_log2 - 4)) - 1)) << 4;
}

// What a row's sums are divided by: its weights' total, which is zero for a row that stands
// before the first key (its output is zero), and for one whose scores are all minus
// infinity, which has no softmax (0 / 0: NaN).
__device__ __forceinline__ float inverse(float total, int pos) {
  return total == 0.f && pos < 0 ? 0.f : 1.f / total;
}

// What a workgroup met: a page outside the cache or more keys than the table holds;
// infinities or NaN that were taken out of the values.
constexpr int kBad = 1, kFound = 2;

// Key k's value, for the seldom path that takes them one by one.
template <class Row>
__device__ __forceinline__ const uint16_t* value_at(const AttnParams& p, Row table, int k, int kvh,
                                                    bool* bad) {
  const int id = page_of(p, table[table_at(p, k >> 4)], bad);
  return p.v + (int64_t)id * p.v_page + (int64_t)(slot_of(p, k >> 4) + (k & 15)) * p.v_slot +
         kvh * p.v_head;
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
  // four rows of two blocks (many_rows) and eight of one (few_rows) cover all banks
  const int turn = D == 128 ? (row & 3) << 1 | ((row >> 2) & 1) : (row & 2) | ((row >> 2) & 1);
  return row * (2 * D) + (((word >> 1) ^ turn) << 5) + ((word & 1) << 4);
}

// The sixteen rows from `base` on, of `slot` elements' distance and D elements each.
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t sixteen_rows(const uint16_t* base, int slot) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, 30 * slot + 2 * D, 0x00027000);
}

// ------------------------------------------------------------------- few rows
//
// Bound by reading the cache. The waves of a workgroup take turns at 32-key tiles of its
// part and keep their own softmax. A tile's keys and values pass through
// the wave's own 64 rows of LDS, so the loop has no barrier; the next tile's loads
// follow at once into the registers that this frees and are in flight while the tile is
// computed, 128 KB per compute unit. Loads cover whole
// rows of the cache: keys loaded in the matrix operand's own layout (64 bytes of each
// of 16 rows at a time) needed no LDS and were slower.

// One tile's 32 keys and values in registers as they lie in memory: a load covers
// whole rows, 64 / (D / 8) of them.
template <int D>
struct FewTile {
  u4v k[D / 16], v[D / 16];
};

template <int D>
__device__ __forceinline__ void few_load(const AttnParams& p, FewTile<D>& t, const int (&ids)[2],
                                         int kvh, int kt, const Span& span, int lane, bool* bad) {
  constexpr int words = D / 8, rows = 64 / words, each = 16 / rows;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int blk = span.block(2 * kt + i), most = span.hi - 1 - 16 * blk;
    const int id = page_of(p, ids[i], bad), slot = slot_of(p, blk);
    const uint16_t* kb = p.k + (int64_t)id * p.k_page + (int64_t)slot * p.k_slot + kvh * p.k_head;
    const uint16_t* vb = p.v + (int64_t)id * p.v_page + (int64_t)slot * p.v_slot + kvh * p.v_head;
#pragma unroll
    for (int j = 0; j < each; ++j) {
      const uint32_t row = (uint32_t)min_of(rows * j + lane / words, most);
      const uint32_t col = 8 * (lane % words);
      t.k[each * i + j] =
          __builtin_nontemporal_load((const u4v*)(kb + row * (uint32_t)p.k_slot + col));
      t.v[each * i + j] =
          __builtin_nontemporal_load((const u4v*)(vb + row * (uint32_t)p.v_slot + col));
    }
  }
}

// W waves; region(w): the LDS of wave w, 64 rows of D elements.
template <int W>
struct FewShared {
  float m[W][kFewRows], l[W][kFewRows];
  int marks;
};

template <class T, int D, int W, class Region>
__device__ __forceinline__ void few_rows(const AttnParams& p, int block, Region region,
                                         FewShared<W>& shared) {
  constexpr int kPitch = D + 4;
  static_assert(kFewRows * kPitch * 4 <= 64 * D * 2, "a wave's sums fit its region");
  const int part = block / p.kv_heads, kvh = block % p.kv_heads;
  const int s = part % p.seqs, split = part / p.seqs;
  const Seq seq = sequence(p, s);
  const int rows = seq.len * p.group;
  if (rows > p.few_rows) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int c = lane >> 4;
  const TableRow table = table_row(p, s);

  for (int r0 = 0; r0 < rows; r0 += kFewRows) {
    const int r1 = min_of(r0 + kFewRows, rows);
    const Span span = span_of<0>(p, seq, r0, r1);
    if (split >= span.parts) continue;
    const int from = span.lo + split * span.chunk;
    const int to = min_of(span.hi, from + span.chunk);
    if (threadIdx.x == 0) shared.marks = seq.bad ? kBad : 0;
    __syncthreads();

    // this lane's row: its query operand and the keys [row_lo, row_hi) it sees
    const int r = r0 + (lane & 15);
    const int rc = min_of(r, r1 - 1);
    const int tok = rc / p.group, head = kvh * p.group + rc % p.group;
    const int pos = seq.n - seq.len + tok;
    const int row_hi = r < r1 ? pos + 1 : 0;
    const int row_lo = first_key(p, pos);
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
    bool bad = false, found = false;
    // Values that some row of the tile may not see must be finite in the product, where a
    // hidden one is multiplied by zero: infinities and NaN among them are taken out here
    // and added at the end to the rows that see them.
    const int all_hi = seq.n - seq.len + r0 / p.group + 1;
    const int all_lo = first_key(p, seq.n - seq.len + (r1 - 1) / p.group);
    auto partly = [&](int kt) { return 32 * kt + 32 > all_hi || 32 * kt < all_lo; };
    char* keys = region(wave);
    char* vals = keys + 32 * D * 2;
    FewTile<D> t;
    int ids[2];
    const int end = (to + 31) >> 5;
    auto next_ids = [&](int kt) {
#pragma unroll
      for (int i = 0; i < 2; ++i) ids[i] = table[table_at(p, span.block(2 * kt + i))];
    };
    int kt = (from >> 5) + wave;
    if (kt < end) {
      next_ids(kt);
      few_load<D>(p, t, ids, kvh, kt, span, lane, &bad);
      next_ids(kt + W);
    }
    for (; kt < end; kt += W) {
      constexpr int words = D / 8, vr = 64 / words;
      if (partly(kt) && __any(any_non_finite<T>(t.v))) {
        found = true;
#pragma unroll
        for (int j = 0; j < D / 16; ++j) t.v[j] = finite<T>(t.v[j]);
      }
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        *(u4v*)(keys + k_word<D>(vr * j + lane / words, lane % words)) = t.k[j];
        *(u4v*)(vals + v_word<D>(vr * j + lane / words, lane % words)) = t.v[j];
      }
      if (kt + W < end) {
        few_load<D>(p, t, ids, kvh, kt + W, span, lane, &bad);
        next_ids(kt + 2 * W);
      }
      // the wave's own stores to LDS are complete and visible to its other lanes
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
      f4v sc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          sc[i] = T::mfma16(*(const u4v*)(keys + k_word<D>(16 * i + (lane & 15), 4 * ks + c)), q[ks],
                            sc[i]);
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
      const float base = m == -INFINITY ? 0.f : m - kLift<T>;
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
    }
    // join the waves
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    const int marks = (__any(bad) ? kBad : 0) | (found ? kFound : 0);
    if (marks && lane == 0) atomicOr(&shared.marks, marks);
    if (c == 0) {
      shared.m[wave][lane] = m;
      shared.l[wave][lane] = l;
    }
    __syncthreads();
    float* sums = (float*)region(wave);
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
      *(f4v*)(sums + (lane & 15) * kPitch + 16 * d + 4 * c) = o[d];
    __syncthreads();
    constexpr int E = kFewRows * D / (64 * W);  // outputs of a thread
    const int jr = threadIdx.x / (D / E), jc = threadIdx.x % (D / E) * E;
    if (r0 + jr < r1) {
      float top = -INFINITY, total = 0.f, f[W], sum[E] = {};
#pragma unroll
      for (int w = 0; w < W; ++w) top = fmaxf(top, shared.m[w][jr]);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        f[w] = shared.m[w][jr] == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(shared.m[w][jr] - top);
        total += shared.l[w][jr] * f[w];
#pragma unroll
        for (int e = 0; e < E; ++e)
          sum[e] += ((const float*)region(w))[jr * kPitch + jc + e] * f[w];
      }
      if (shared.marks & kBad) total = __builtin_nanf("");
      const int token = seq.begin + (r0 + jr) / p.group, hd = kvh * p.group + (r0 + jr) % p.group;
      if (shared.marks & kFound) {
        const int at = seq.n - seq.len + (r0 + jr) / p.group;
        for (int k = from; k < to; ++k) {
          if (!partly(k >> 5) || k > at || k < first_key(p, at)) continue;
          const uint16_t* v = value_at(p, table, k, kvh, &bad) + jc;
#pragma unroll
          for (int e = 0; e < E; ++e) sum[e] = with_non_finite<T>(sum[e], v[e]);
        }
      }
      if (span.parts == 1) {
        const float inv = inverse(total, seq.n - seq.len + (r0 + jr) / p.group);
        uint32_t* to32 = (uint32_t*)(p.out + (int64_t)token * p.o_token + hd * p.o_head + jc);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) to32[e] = T::pack(sum[2 * e] * inv, sum[2 * e + 1] * inv);
      } else {
        const int64_t at = split * p.few_step + few_part(p, s, kvh, r0 + jr);
#pragma unroll
        for (int e = 0; e < E; ++e) p.part_o[at * D + jc + e] = sum[e];
        if (jc == 0) *(f2v*)(p.part_ml + 2 * at) = f2v{top, total};
      }
    }
    __syncthreads();  // before the next row tile takes the shared memory
  }
}

template <class T, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void few_kernel(AttnParams p) {
  __shared__ __attribute__((aligned(16))) char mem[W * 64 * D * 2];
  __shared__ FewShared<W> shared;
  fetch(p);
  few_rows<T, D, W>(p, blockIdx.x, [&](int w) { return mem + w * (64 * D * 2); }, shared);
}

// ------------------------------------------------------------------ many rows
//
// Bound by the matrix cores, the exponentials beside them and the power both draw:
// 2048 tokens x 32 heads on 16384 keys take 483 to 526 us by the machine, up to 1070
// TFLOP/s, at a clock that the card lowers from 2.0 to 1.7 GHz meanwhile (a large library product in bf16 reaches 1200).
// A wave owns 32 rows; the four share 64 keys and values in LDS, in two buffers that
// loads fill without passing registers, one barrier a tile. (Through registers, with
// the operands' LDS reads waiting on them: 605 us.) The scores of one block of 32 keys are computed
// beside the exponentials of the block before it, which costs 32 registers and saves
// a third of the cycles; two workgroups share a compute unit. The buffers are arrays of
// their own, so that the compiler sees that a load into one and a read of the other
// need not wait for each other.

// The nth row tile in the order in which they start: the sequence and the first row.
// Long sequences first, and each from its last rows, so that no long tile begins when
// the others end (10 chunks of 253 tokens x 32 heads on 820 .. 4099 keys beside 6
// single tokens: 114 us in the sequences' order, 108 so). More sequences than
// lanes are taken from the last to the first.
struct RowTile {
  int s, r0;  // s < 0: there is no such tile
};

__device__ __forceinline__ RowTile row_tile(const AttnParams& p, int nth, int lane) {
  if (p.seqs <= 64) {
    const Seq q = sequence(p, min_of(lane, p.seqs - 1));
    const int rows = lane < p.seqs && q.len * p.group > p.few_rows ? q.len * p.group : 0;
    const int tiles = (rows + kManyRows - 1) / kManyRows;
    int before = 0;
    for (int s = 0; s < p.seqs; ++s) {
      const int n = __builtin_amdgcn_readlane(q.n, s);
      if (n > q.n || (n == q.n && s < lane)) before += __builtin_amdgcn_readlane(tiles, s);
    }
    const uint64_t mine = __ballot(nth >= before && nth < before + tiles);
    if (!mine) return {-1, 0};
    const int s = __builtin_ctzll(mine);
    const int left = __builtin_amdgcn_readlane(before + tiles, s) - 1 - nth;
    return {s, left * kManyRows};
  }
  // tiles of sequence s begin at start * group / 128 + s, which leaves each at least as
  // many as its rows need
  const int tile = p.tiles - 1 - nth;
  int found = 0;
  for (int s0 = 0; s0 < p.seqs; s0 += 64) {
    const bool begun = s0 + lane < p.seqs &&
        (int)((int64_t)start_of(p, s0 + lane) * p.group / kManyRows) + s0 + lane <= tile;
    const uint64_t votes = __ballot(begun);
    found += __popcll(votes);
    if (votes != ~0ull) break;
  }
  const int s = uniform(found - 1);
  if (s < 0) return {-1, 0};
  return {s, (tile - (int)((int64_t)start_of(p, s) * p.group / kManyRows) - s) * kManyRows};
}

template <class T, int D>
__device__ __forceinline__ void many_rows(const AttnParams& p, int block, char* keys0, char* vals0,
                                          char* keys1, char* vals1, int& marks) {
  const int kvh = block % p.kv_heads;
  const int nth = block / p.kv_heads % p.tiles, split = block / p.kv_heads / p.tiles;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int h = lane >> 5;

  const RowTile at = row_tile(p, nth, lane);
  if (at.s < 0) return;
  const int s = at.s, r0 = at.r0;
  const Seq seq = sequence(p, s);
  const int rows = seq.len * p.group;
  if (rows <= p.few_rows || r0 < 0 || r0 >= rows) return;
  const int r1 = min_of(r0 + kManyRows, rows);
  const Span span = span_of<1>(p, seq, r0, r1);
  if (split >= span.parts) return;
  const int from = span.lo + split * span.chunk;
  const int to = min_of(span.hi, from + span.chunk);
  const int32_t* table = p.table + s * p.table_stride;
  if (threadIdx.x == 0) marks = seq.bad ? kBad : 0;

  // this lane's row, and the wave's rows together
  const int w0 = r0 + 32 * wave, r = w0 + (lane & 31);
  const int rc = min_of(r, r1 - 1);
  const int tok = rc / p.group, head = kvh * p.group + rc % p.group;
  const int pos = seq.n - seq.len + tok;
  const int row_hi = pos + 1;
  const int row_lo = first_key(p, pos);
  const int first = uniform(seq.n - seq.len + min_of(w0, r1 - 1) / p.group);
  const int last = uniform(seq.n - seq.len + min_of(w0 + 31, r1 - 1) / p.group);
  // the keys that every row of the wave sees
  const int all_hi = first + 1;
  const int all_lo = first_key(p, last);
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
  float m = -INFINITY, l = 0.f, base = 0.f;
  bool bad = false, found = false;

  // A wave brings sixteen of a tile's keys and values, straight from memory to LDS:
  // a load places 1 KB of whole rows there in lane order, so each lane reads the word
  // whose place in the LDS layout its own is.
  constexpr int kWords = D / 8, kRowsEach = 64 / kWords, kLoads = 16 / kRowsEach;
  // lane i: the page of this wave's values of tile ids_from + i - 1, lanes' keys being two
  // blocks of sixteen further on
  int k_ids = 0, v_ids = 0, ids_from = 0;
  auto read_ids = [&](int kt) {
    ids_from = kt - 1;
    k_ids = table[table_at(p, span.block(4 * (ids_from + lane) + 2 + wave))];
    v_ids = table[table_at(p, span.block(4 * (ids_from + lane) + wave))];
    asm volatile("" : "+v"(k_ids), "+v"(v_ids));  // they arrive here, not behind later loads
  };
  auto load = [&](int blk, int id, const uint16_t* cache, int64_t page_step, int64_t head_step,
                  int slot_step, char* to, auto word_of) {
    const int page = page_of(p, id, &bad);
    const __amdgpu_buffer_rsrc_t rows = sixteen_rows<D>(
        cache + page * page_step + (int64_t)slot_of(p, blk) * slot_step + kvh * head_step, slot_step);
    const int most = span.hi - 1 - 16 * blk;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = kRowsEach * j + lane / kWords, place = lane % kWords;
      const uint32_t word = (uint32_t)(word_of(row, place) - row * 2 * D);
      load_to_lds(rows, 2 * __umul24(min_of(row, most), slot_step) + word,
                  to + (16 * wave + kRowsEach * j) * 2 * D);
    }
  };
  auto load_keys = [&](int kt, char* to) {
    if (kt - ids_from >= 64) read_ids(kt);
    load(span.block(4 * kt + 2 + wave), __builtin_amdgcn_readlane(k_ids, kt - ids_from), p.k, p.k_page,
         p.k_head, p.k_slot, to, [](int r, int w) { return k_word<D>(r, w); });
  };
  auto load_values = [&](int kt, char* to) {
    load(span.block(4 * kt + wave), __builtin_amdgcn_readlane(v_ids, kt - ids_from), p.v, p.v_page,
         p.v_head, p.v_slot, to, [](int r, int w) { return v_word<D>(r, w); });
  };
  constexpr int kSteps = D / 16;
  // S^T of 32 keys in LDS
  auto scores = [&](const char* keys) {
    f16v sc;
#pragma unroll
    for (int e = 0; e < 16; ++e) sc[e] = 0.f;
#pragma unroll
    for (int ks = 0; ks < kSteps; ++ks)
      sc = T::mfma32(*(const u4v*)(keys + k_word<D>(lane & 31, 2 * ks + h)), q[ks], sc);
    return sc;
  };
  // of the keys from k0 on: hidden ones out, and the running maximum
  auto settle = [&](f16v& sc, int k0) {
    if (k0 + 32 > all_hi || k0 < all_lo) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int key = k0 + 8 * (e >> 2) + 4 * h + (e & 3);
        if (key >= row_hi || key < row_lo) sc[e] = -INFINITY;
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[e]);
    top *= p.scale2;
    if (__any(top > m + kRaise)) {
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float raised = fmaxf(m, top);
      const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - raised);
      m = raised;
      base = m == -INFINITY ? 0.f : m - kLift<T>;
      l *= f;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] *= f;
    }
  };
  // the weights of 32 keys and their products with the values in LDS
  auto weigh = [&](const f16v& sc, const char* vals) {
    const int vrow = 4 * h + ((lane & 15) >> 2), col = lane & 3, half = (lane >> 4) & 1;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      u4v w;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          x[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[8 * g + 2 * e + i], p.scale2, -base));
          l += x[i];
        }
        w[e] = T::pack(x[0], x[1]);
      }
#pragma unroll
      for (int d = 0; d < D / 32; ++d) {
        const int row = 16 * g + vrow, word = 4 * d + 2 * half + (col >> 1);
        const u2v x = read_column(vals + v_word<D>(row, word) + 8 * (col & 1));
        const u2v y = read_column(vals + v_word<D>(row + 8, word) + 8 * (col & 1));
        o[d] = T::mfma32(u4v{x.x, x.y, y.x, y.y}, w, o[d]);
      }
    }
  };

  const int begin = from >> 6, end = (to + 63) >> 6;
  constexpr int kHalf = 32 * D * 2;
  // As in few_rows: of a tile that not every row of the workgroup sees whole, infinities
  // and NaN are taken out of the values before the products, by the lanes that brought
  // them and before the barrier that hands the tile over.
  const int group_hi = seq.n - seq.len + r0 / p.group + 1;
  const int group_lo = first_key(p, seq.n - seq.len + (r1 - 1) / p.group);
  auto partly = [&](int kt) { return 64 * kt + 64 > group_hi || 64 * kt < group_lo; };
  auto clean = [&](int kt, char* vals) {
    if (!partly(kt)) return;
    u4v* const mine = (u4v*)(vals + 16 * wave * 2 * D) + lane;
    u4v w[kLoads];
#pragma unroll
    for (int j = 0; j < kLoads; ++j) w[j] = mine[64 * j];
    if (!__any(any_non_finite<T>(w))) return;
#pragma unroll
    for (int j = 0; j < kLoads; ++j) mine[64 * j] = finite<T>(w[j]);
    found = true;
  };
  if (begin < end) {
    read_ids(begin);
    load_keys(begin - 1, keys1);
    load_keys(begin, keys0);
    load_values(begin, vals0);
    // the queries have arrived before the loop: a wait for them in it would be one
    // for the loads under way as well
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) asm volatile("" : "+v"(q[ks]));
    wait_for_loads();
    clean(begin, vals0);
    __syncthreads();
    if (w0 < r1) {
      f16v s0, s1;
      // Two steps of 32 keys, in each the weights of one block and the scores of the
      // next: independent, so the products of one run beside the exponentials of the
      // other. LDS holds the values of blocks 2 kt and 2 kt + 1 and the keys of the
      // blocks after them.
      auto turn = [&](int kt, char* keys, char* next_keys, char* vals, char* next_vals) {
        load_keys(kt + 1, next_keys);
        load_values(kt + 1, next_vals);
        __builtin_amdgcn_sched_barrier(0);
        s1 = scores(keys);
        weigh(s0, vals);
        settle(s1, 64 * kt + 32);
        s0 = scores(keys + kHalf);
        weigh(s1, vals + kHalf);
        settle(s0, 64 * kt + 64);
        wait_for_loads();
        clean(kt + 1, next_vals);
        __syncthreads();
      };
      auto last = [&](int kt, char* keys, char* vals) {
        s1 = scores(keys);
        weigh(s0, vals);
        settle(s1, 64 * kt + 32);
        weigh(s1, vals + kHalf);
      };
      s0 = scores(keys1 + kHalf);
      settle(s0, 64 * begin);
      __syncthreads();
      int kt = begin;
      for (; kt + 2 < end; kt += 2) {
        turn(kt, keys0, keys1, vals0, vals1);
        turn(kt + 1, keys1, keys0, vals1, vals0);
      }
      const bool two = kt + 1 < end;
      if (two) turn(kt, keys0, keys1, vals0, vals1);
      last(end - 1, two ? keys1 : keys0, two ? vals1 : vals0);
    } else {  // a wave without rows only loads
      __syncthreads();
      for (int kt = begin; kt + 1 < end; ++kt) {
        const bool even = ((kt - begin) & 1) == 0;
        load_keys(kt + 1, even ? keys1 : keys0);
        load_values(kt + 1, even ? vals1 : vals0);
        wait_for_loads();
        clean(kt + 1, even ? vals1 : vals0);
        __syncthreads();
      }
    }
  } else {
    __syncthreads();
  }
  // a barrier lies between the word's first value and these
  const int met = (__any(bad) ? kBad : 0) | (found ? kFound : 0);
  if (met && lane == 0) atomicOr(&marks, met);
  __syncthreads();
  if (r >= r1) return;
  l += __shfl_xor(l, 32, 64);
  if (marks & kFound) {
    for (int k = from; k < to; ++k) {
      if (!partly(k >> 6) || k >= row_hi || k < row_lo) continue;
      const uint16_t* v = value_at(p, table, k, kvh, &bad) + 4 * h;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          o[d][e] = with_non_finite<T>(o[d][e], v[32 * d + 8 * (e >> 2) + (e & 3)]);
    }
  }
  if (marks & kBad) l = __builtin_nanf("");
  const int token = seq.begin + tok;
  if (span.parts == 1) {
    const float inv = inverse(l, pos);
    uint16_t* dst = p.out + (int64_t)token * p.o_token + head * p.o_head + 4 * h;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(u2v*)(dst + 32 * d + 8 * e) = u2v{T::pack(o[d][4 * e] * inv, o[d][4 * e + 1] * inv),
                                            T::pack(o[d][4 * e + 2] * inv, o[d][4 * e + 3] * inv)};
  } else {
    const int64_t at = p.many_at + split * p.many_step + (int64_t)token * p.heads + head;
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

template <class T, int D>
__global__ __launch_bounds__(kThreads, 2) void many_kernel(AttnParams p) {
  constexpr int kTile = 64 * D * 2;
  __shared__ __attribute__((aligned(16))) char keys0[kTile], vals0[kTile], keys1[kTile], vals1[kTile];
  __shared__ int marks;
  fetch(p);
  many_rows<T, D>(p, blockIdx.x, keys0, vals0, keys1, vals1, marks);
}

// A batch with sequences of both kinds in one launch: the reading of the one runs
// beside the products of the other.
template <class T, int D>
__global__ __launch_bounds__(kThreads, 2) void mixed_kernel(AttnParams p) {
  constexpr int kTile = 64 * D * 2;
  __shared__ __attribute__((aligned(16))) char keys0[kTile], vals0[kTile], keys1[kTile], vals1[kTile];
  __shared__ FewShared<kThreads / 64> shared;
  fetch(p);
  const int block = (int)blockIdx.x - p.many_blocks;
  if (block < 0)
    many_rows<T, D>(p, blockIdx.x, keys0, vals0, keys1, vals1, shared.marks);
  else
    few_rows<T, D, kThreads / 64>(
        p, block,
        [&](int w) { return w == 0 ? keys0 : w == 1 ? vals0 : w == 2 ? keys1 : vals1; }, shared);
}

// -------------------------------------------------------------- joining parts
//
// The parts' sums of a row brought to one maximum. Here by one wave for each row: the
// lanes read the parts' maxima together, and the sums of kAhead parts are under way with them.

template <class T, int D>
__device__ __forceinline__ void combine_row(const AttnParams& p, int parts, int64_t row, int token,
                                            int head, int pos) {
  constexpr int E = D / 64, kAhead = 16;
  typedef float fE __attribute__((ext_vector_type(E)));
  const int lane = threadIdx.x & 63;
  const int64_t step = p.few_step;
  const float* from = p.part_o + row * D + lane * E;
  fE o[kAhead];
  auto read = [&](int j) {  // parts past the last one are the last again
#pragma unroll
    for (int i = 0; i < kAhead; ++i) o[i] = *(const fE*)(from + min_of(j + i, parts - 1) * step * D);
  };
  read(0);
  float top = -INFINITY, total = 0.f;
  fE sum = {};
  for (int j0 = 0; j0 < parts; j0 += 64) {
    const bool here = j0 + lane < parts;
    f2v ml = f2v{-INFINITY, 0.f};
    if (here) ml = *(const f2v*)(p.part_ml + 2 * (row + (j0 + lane) * step));
    float most = ml.x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
    const float raised = fmaxf(top, most);
    const float old = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - raised);
    const float f = ml.x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml.x - raised);
    top = raised;
    float l = ml.y != ml.y ? ml.y : ml.y * f;  // NaN marks a part that met a bad page
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) l += __shfl_xor(l, d, 64);
    total = total * old + l;
    sum *= old;
    const int n = min_of(parts - j0, 64);
    for (int j = 0; j < n; j += kAhead) {
      if (j0 + j) read(j0 + j);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float w = __shfl(f, j + i, 64);
        if (j + i < n) sum += o[i] * w;
      }
    }
  }
  const float inv = inverse(total, pos);
  uint16_t* dst = p.out + (int64_t)token * p.o_token + head * p.o_head + lane * E;
  if constexpr (D == 128)
    *(uint32_t*)dst = T::pack(sum[0] * inv, sum[1] * inv);
  else
    *dst = T::one(sum[0] * inv);
}

// few_rows' rows: four of one sequence and key head at a time.
template <class T, int D>
__device__ __forceinline__ void combine_few(const AttnParams& p, int block) {
  const int first = block % p.join_rows;
  const int s = block / p.join_rows / p.kv_heads, kvh = block / p.join_rows % p.kv_heads;
  const Seq seq = sequence(p, s);
  const int rows = seq.len * p.group;
  if (rows > p.few_rows) return;
  const int wave = uniform(threadIdx.x >> 6);
  for (int r = first * 4 + wave; r < rows; r += 4 * p.join_rows) {
    const int r0 = r / kFewRows * kFewRows;
    const Span span = span_of<0>(p, seq, r0, min_of(r0 + kFewRows, rows));
    const int token = seq.begin + r / p.group, head = kvh * p.group + r % p.group;
    if (span.parts > 1)
      combine_row<T, D>(p, span.parts, few_part(p, s, kvh, r), token, head,
                        seq.n - seq.len + r / p.group);
  }
}

// many_rows' rows, kJoinRows of one row tile and key head: all have as many parts, and
// D / 4 lanes join a row. (One wave to a row, which looked for its sequence by itself: 25
// us for 1002 tokens x 32 heads in two parts; 10 us so.)
constexpr int kJoinRows = 32;

template <class T, int D>
__device__ __forceinline__ void combine_many(const AttnParams& p, int block) {
  constexpr int G = D / 4, kAhead = 4;
  const int kvh = block % p.kv_heads, sub = block / p.kv_heads % (kManyRows / kJoinRows);
  const RowTile at = row_tile(p, block / p.kv_heads / (kManyRows / kJoinRows), threadIdx.x & 63);
  if (at.s < 0) return;
  const Seq seq = sequence(p, at.s);
  const int rows = seq.len * p.group;
  if (rows <= p.few_rows || at.r0 < 0 || at.r0 >= rows) return;
  const int end = min_of(at.r0 + kManyRows, rows);
  const int parts = span_of<1>(p, seq, at.r0, end).parts;
  if (parts == 1) return;
  const int64_t step = p.many_step;
  const int c = threadIdx.x % G, first = at.r0 + sub * kJoinRows;
  for (int r = first + threadIdx.x / G; r < min_of(first + kJoinRows, end); r += kThreads / G) {
    const int token = seq.begin + r / p.group, head = kvh * p.group + r % p.group;
    const int64_t row = p.many_at + (int64_t)token * p.heads + head;
    const f2v* const ml = (const f2v*)p.part_ml + row;
    const f4v* const from = (const f4v*)(p.part_o + row * D) + c;
    f4v o[kAhead];
    float m[kAhead];
    auto read = [&](int j) {  // parts past the last one are the last again
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int64_t part = min_of(j + i, parts - 1) * step;
        m[i] = ml[part].x;
        o[i] = from[part * G];
      }
    };
    read(0);
    float top = -INFINITY, total = 0.f;
    for (int i = c; i < parts; i += G) top = fmaxf(top, ml[i * step].x);
#pragma unroll
    for (int d = 1; d < G; d <<= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    auto weight = [&](float m) { return m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - top); };
    for (int i = c; i < parts; i += G) {
      const f2v x = ml[i * step];
      total += x.y != x.y ? x.y : x.y * weight(x.x);  // NaN marks a part that met a bad page
    }
#pragma unroll
    for (int d = 1; d < G; d <<= 1) total += __shfl_xor(total, d, 64);
    f4v sum = {};
    for (int j = 0; j < parts; j += kAhead) {
      if (j) read(j);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (j + i < parts) sum += o[i] * weight(m[i]);
    }
    sum *= inverse(total, seq.n - seq.len + r / p.group);
    *(u2v*)(p.out + (int64_t)token * p.o_token + head * p.o_head + 4 * c) =
        u2v{T::pack(sum[0], sum[1]), T::pack(sum[2], sum[3])};
  }
}

template <class T, int D>
__global__ __launch_bounds__(kThreads) void combine_kernel(AttnParams p) {
  fetch(p);
  if ((int)blockIdx.x < p.join_blocks)
    combine_few<T, D>(p, blockIdx.x);
  else
    combine_many<T, D>(p, blockIdx.x - p.join_blocks);
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
  if (a->table_width < 1 || (int64_t)a->table_width * a->page_size > ((int64_t)1 << 30) ||
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
  if (!serve::apart({{a->tokens, a->o_token}, {a->heads, a->o_head}}, a->head_dim))
    return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

struct AttnPlan {
  bool few, many;
  int splits[2], chunk[2];
  int64_t tiles;
  int64_t few_step, part_rows;  // part rows of one of few_rows' splits, and all of them
  size_t ws_bytes;
};

// The length of n parts of `keys` keys, and how many of that length there are.
int64_t part_keys(int64_t keys, int64_t n) {
  return ((keys + n - 1) / n + kSplitKeys - 1) / kSplitKeys * kSplitKeys;
}
int64_t most_parts(int64_t keys) {  // none shorter than 512 keys
  const int64_t most = (keys + 511) / 512;
  return most < kMaxSplits ? most : kMaxSplits;
}
void split_keys(int64_t keys, int64_t n, int* splits, int* chunk) {
  const int64_t most = most_parts(keys);
  if (n > most) n = most;
  if (n < 1) n = 1;
  const int64_t each = part_keys(keys, n);
  *splits = (int)((keys + each - 1) / each);
  *chunk = (int)each;
}

// The number of parts for `base` row tiles of as many keys, of which `slots` run at a time:
// the one that takes least time, where a part costs as much as `more` keys besides its
// own (one token x 64 heads of 8 on 32768 keys: 30 us, with four rounds of parts 36; 300
// tokens x 32 heads of 8 on 16384: 106 us, with as many parts as cover the slots 121).
int64_t parts_for(int64_t keys, int64_t base, int64_t slots, int64_t more) {
  int64_t best = 1, least = INT64_MAX;
  const int64_t most = most_parts(keys);
  for (int64_t n = 1; n <= most && base * (n - 1) < 4 * slots; ++n) {
    const int64_t each = part_keys(keys, n);
    const int64_t rounds = (base * keys + each * slots - 1) / (each * slots);
    const int64_t time = rounds * (each + more * (n > 1));
    if (time < least) {
      least = time;
      best = n;
    }
  }
  return best;
}

// Which kernels run and how many parts the longest key axis is cut into.
AttnPlan plan(const lutgemm_attention* a) {
  AttnPlan r{};
  if (a->tokens == 0 || a->seqs == 0) return r;  // nothing runs
  const int64_t group = a->heads / a->kv_heads;
  const int64_t table_keys = (int64_t)a->table_width * a->page_size;
  int64_t max_q = a->max_q < a->tokens ? a->max_q : a->tokens;
  if (a->seqs == 1) max_q = a->tokens;
  if (max_q < 1) max_q = 1;
  int64_t keys = a->max_kv < table_keys ? a->max_kv : table_keys;
  if (a->window > 0 && keys > a->window + max_q + 64) keys = a->window + max_q + 64;
  if (keys < 1) keys = 1;
  r.many = max_q * group > kFewRows;
  r.few = !r.many || (a->seqs > 1 && group <= kFewRows);  // a token alone has `group` rows
  r.tiles = a->tokens * group / kManyRows + a->seqs;
  const int64_t few = (int64_t)a->seqs * a->kv_heads;
  int64_t few_parts = 1, many_parts = 1;
  if (a->seqs == 1) {
    if (r.few)
      few_parts = parts_for(keys, few, 256, 200);
    else
      many_parts = parts_for(
          keys, (a->tokens * group + kManyRows - 1) / kManyRows * a->kv_heads, 512, 300);
  } else {
    // Lengths that differ even out over a few rounds of workgroups (48 sequences of 800 ..
    // 8000 keys: 197 us in one part, 168 in three, 164 in four, 162 in six, 177 in
    // sixteen; equal ones, 4 of 128k keys: 318 us in 8, 329 in 32, 345 in 64). Beside
    // many_rows' they start last and short parts fill what the long tiles leave (row_tile's
    // batch: in one part 106 us, in three 98); that batch's own tiles in two parts take 120.
    few_parts = few > 256 ? (1536 + few - 1) / few : (r.many ? 1536 : 1024) / few;
    const int64_t many = (a->tokens * group / kManyRows + (a->seqs + 1) / 2) * a->kv_heads;
    many_parts = (512 + many - 1) / many;
  }
  split_keys(keys, few_parts, &r.splits[0], &r.chunk[0]);
  split_keys(keys, many_parts, &r.splits[1], &r.chunk[1]);
  if (!r.few) r.splits[0] = 1;
  if (!r.many) r.splits[1] = 1;
  const int64_t rows = a->tokens * a->heads;
  r.few_step = r.splits[0] > 1 ? (int64_t)a->seqs * a->kv_heads * kFewRows : 0;
  r.part_rows = r.splits[0] * r.few_step + (r.splits[1] > 1 ? r.splits[1] * rows : 0);
  r.ws_bytes = (size_t)r.part_rows * (size_t)(a->head_dim + 2) * sizeof(float);
  return r;
}

// Two workgroups of four waves share a compute unit, so that one begins or ends while the
// other reads (4 sequences of 128k keys: 329 us, with eight waves and one workgroup
// 332; 48 of 800 .. 8000: 164 and 167). Where there is only one to a unit it takes
// eight waves (one sequence of 512 keys x 32 heads: 8.6 us, with four 9.5). Short parts leave
// most waves idle, and their LDS keeps other workgroups from the unit (39 x 32 heads of
// up to 50 keys: 23.4 us with eight, with two 9.8).
template <class T, int D>
int launch_few(const AttnPlan& r, int64_t few, const AttnParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)few);
  if (r.chunk[0] <= kShortKeys)
    return launch(few_kernel<T, D, kShortWaves>, grid, 64 * kShortWaves, p, stream);
  if (few <= 256) return launch(few_kernel<T, D, kLoneWaves>, grid, 64 * kLoneWaves, p, stream);
  return launch(few_kernel<T, D, kFewWaves>, grid, 64 * kFewWaves, p, stream);
}

template <class T, int D>
int run_attention(const AttnPlan& r, const AttnParams& p, hipStream_t stream) {
  const int64_t few = (int64_t)p.seqs * r.splits[0] * p.kv_heads;
  const int64_t many = r.tiles * p.kv_heads * r.splits[1];
  int st;
  if (r.few && r.many)
    st = launch(mixed_kernel<T, D>, dim3((unsigned)(few + many)), kThreads, p, stream);
  else if (r.many)
    st = launch(many_kernel<T, D>, dim3((unsigned)many), kThreads, p, stream);
  else
    st = launch_few<T, D>(r, few, p, stream);
  const int64_t joined = r.splits[1] > 1 ? r.tiles * p.kv_heads * (kManyRows / kJoinRows) : 0;
  if (!st && p.join_blocks + joined > 0)
    st = launch(combine_kernel<T, D>, dim3((unsigned)(p.join_blocks + joined)), kThreads, p, stream);
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
    // a workgroup has read its own rows of q before it writes them, but no other's
    const bool in_place = d_out == d_q && (a->tokens == 1 || a->o_token == a->q_token) &&
                          (a->heads == 1 || a->o_head == a->q_head);
    auto tokens_of = [&](const void* at, int64_t token, int64_t head) {
      return Rows{at, a->tokens, token, (a->heads - 1) * head + a->head_dim};
    };
    auto heads_of = [&](const void* at, int64_t token, int64_t head) {
      return Rows{at, a->heads, head, (a->tokens - 1) * token + a->head_dim};
    };
    if (!in_place &&
        overlap(tokens_of(d_out, a->o_token, a->o_head), tokens_of(d_q, a->q_token, a->q_head)) &&
        overlap(heads_of(d_out, a->o_token, a->o_head), heads_of(d_q, a->q_token, a->q_head)))
      return LUTGEMM_ERR_SHAPE;
    const AttnPlan r = plan(a);
    // a launch has fewer than 2^32 threads along each axis of its grid
    constexpr int64_t kMost = (int64_t)1 << 24;
    const int64_t few = (int64_t)a->seqs * r.splits[0] * a->kv_heads;
    const int64_t joined = (r.splits[0] > 1 ? (int64_t)a->seqs * a->kv_heads * 4 : 0) +
                           (r.splits[1] > 1 ? r.tiles * a->kv_heads * (kManyRows / kJoinRows) : 0);
    if (r.tiles * a->kv_heads * r.splits[1] + few >= kMost / 2 || joined >= kMost)
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
    p.part_ml = r.ws_bytes ? (float*)d_workspace + r.part_rows * a->head_dim : nullptr;
    p.few_step = r.few_step;
    p.many_step = a->tokens * a->heads;
    p.many_at = r.splits[0] * r.few_step;
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
    for (int i = 0; i < 2; ++i) {
      p.splits[i] = r.splits[i];
      p.chunk[i] = r.chunk[i];
    }
    p.many_blocks = (int32_t)(r.tiles * a->kv_heads * r.splits[1]);
    p.join_rows = r.many || p.group >= kFewRows ? kFewRows / 4 : (p.group + 3) / 4;
    p.join_blocks = r.few && r.splits[0] > 1 ? a->seqs * a->kv_heads * p.join_rows : 0;
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
