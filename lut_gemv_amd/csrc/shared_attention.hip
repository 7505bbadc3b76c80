// shared_attention.hip -- attention of a batch whose sequences share long prefixes
// (lutgemm_shared_attention; the formula is in lutgemm.h).
//
// A softmax over a prefix and a sequence's own keys is joined from parts of both, each
// with its own maximum and sum, so the prefix is one more sequence for the bodies of
// attention_kernel.h: its rows are the new tokens of the whole group, all of which see all
// of its keys. Its keys are read once for 128 rows, not once for each sequence. One
// launch runs the prefixes of small groups (few_rows), the row tiles of others (many_rows),
// then the own keys of chunks (many_rows) and of single tokens (few_rows); all leave their
// parts in the workspace, and join_kernel brings each row's to one maximum.
//
// Measured (keys of 128, prefix of 32768, 64 sequences with 450 keys of their own on average, 64
// heads of 8, bf16): 69 G multiplications and additions, 57 us at a large matrix product's
// rate, take 105 and the join 10. 40 sequences in 5 groups on 4099 keys (32 heads of 64, fp16):
// 470 MB, 70 us at a copy's rate, take 95 and the join 5. 8 chunks of 253 tokens on 16384 keys (32
// heads of 8, bf16): 348 us at the product's rate, take 438 to 473 by the machine's clock and the
// join 29. (Kernels by themselves, in a trace; calls in a row take 107 to 117, 98 to 100 and 432
// to 457 us.)
#include "attention_kernel.h"

namespace lutgemm {
namespace {

struct SharedParams : AttnParams {
  const int32_t* prefix_table;
  const int32_t* prefix_lens;
  const int32_t* group_starts;
  int64_t prefix_stride, prefix_at;  // prefix_at: where the prefixes' part rows begin
  int32_t groups, prefix_keys, prefix_tiles, prefix_splits, prefix_chunk;
  int32_t prefix_few;     // groups of up to so many rows are few_rows'
  int32_t blocks[4];      // workgroups of the prefixes' few_rows, their many_rows, the own keys'
                          // many_rows and few_rows
};

// A sequence's own keys. Part row of split s: (s * tokens + token) * heads + head.
struct OwnView : PagedView {
  typedef SharedParams Params;
  static constexpr bool kDirect = false;
  static __device__ __forceinline__ int64_t few_at(const SharedParams& p, int split, int, int, int,
                                                   int token, int head) {
    return split * p.many_step + (int64_t)token * p.heads + head;
  }
  static __device__ __forceinline__ int64_t many_at(const SharedParams&) { return 0; }
};

__device__ __forceinline__ int group_start(const SharedParams& p, int g) {
  if (!p.group_starts) return g > 0 ? p.seqs : 0;
  const int v = p.group_starts[g];
  return v < 0 ? 0 : v > p.seqs ? p.seqs : v;
}

// A group's prefix, seen whole by each of the group's rows.
struct PrefixView {
  typedef SharedParams Params;
  static constexpr bool kDirect = false;
  static __device__ __forceinline__ int count(const SharedParams& p) { return p.groups; }
  static __device__ __forceinline__ int start(const SharedParams& p, int g) {
    return start_of(p, group_start(p, g));
  }
  static __device__ __forceinline__ Seq seq(const SharedParams& p, int g) {
    Seq q;
    q.begin = start(p, g);
    const int end = start(p, g + 1);
    q.len = end > q.begin ? end - q.begin : 0;
    const int n = p.prefix_lens[g];
    q.bad = n > p.prefix_keys;
    q.n = n < 0 ? 0 : n > p.prefix_keys ? p.prefix_keys : n;
    return q;
  }
  static __device__ __forceinline__ int few(const SharedParams& p) { return p.prefix_few; }
  static __device__ __forceinline__ int tiles(const SharedParams& p) { return p.prefix_tiles; }
  static __device__ __forceinline__ Cut cut(const SharedParams& p, int) {
    return {p.prefix_splits, p.prefix_chunk};
  }
  static __device__ __forceinline__ const int32_t* table(const SharedParams& p, int g) {
    return p.prefix_table + g * p.prefix_stride;
  }
  static __device__ __forceinline__ int pos(const Seq& q, int) { return q.n - 1; }
  static __device__ __forceinline__ int64_t few_at(const SharedParams& p, int split, int, int, int,
                                                   int token, int head) {
    return p.prefix_at + split * p.many_step + (int64_t)token * p.heads + head;
  }
  static __device__ __forceinline__ int64_t many_at(const SharedParams& p) { return p.prefix_at; }
};

// Which bodies a launch has: the prefixes' (one, none, or both where groups of few rows may
// stand beside larger ones), and whether single tokens and chunks are among the own keys. A
// kernel of all of them at once is slower at each (64 sequences on 32768 keys 146 us, so
// 106). Bound by the matrix cores where a group has many rows
// (the prefix alone of those 64: 94 us, 730 TFLOP/s of many_rows on 14 parts of 2341 keys, whose
// beginnings and ends it pays 14 times), by the reading where it has few.
enum { kNoPrefix, kManyPrefix, kFewPrefix, kBothPrefixes };

template <class T, int D, int Prefix, bool Few, bool Many>
__global__ __launch_bounds__(kThreads, 2) void shared_kernel(SharedParams p) {
  constexpr int kTile = 64 * D * 2;
  __shared__ __attribute__((aligned(16))) char keys0[kTile], vals0[kTile], keys1[kTile], vals1[kTile];
  __shared__ FewShared<kThreads / 64> shared;
  fetch(p);
  auto region = [&](int w) { return w == 0 ? keys0 : w == 1 ? vals0 : w == 2 ? keys1 : vals1; };
  int block = blockIdx.x;
  if constexpr (Prefix == kFewPrefix || Prefix == kBothPrefixes) {
    if (block < p.blocks[0]) {
      few_rows<PrefixView, T, D, kThreads / 64>(p, block, region, shared);
      return;
    }
    block -= p.blocks[0];
  }
  if constexpr (Prefix == kManyPrefix || Prefix == kBothPrefixes) {
    if (block < p.blocks[1]) {
      many_rows<PrefixView, T, D>(p, block, keys0, vals0, keys1, vals1, shared.marks);
      return;
    }
    block -= p.blocks[1];
  }
  if constexpr (Many) {
    if (block < p.blocks[2]) {
      many_rows<OwnView, T, D>(p, block, keys0, vals0, keys1, vals1, shared.marks);
      return;
    }
    block -= p.blocks[2];
  }
  if constexpr (Few) few_rows<OwnView, T, D, kThreads / 64>(p, block, region, shared);
}

// The last i in [0, count) whose start is at most `token`, -1 for none; all lanes ask together.
template <class V>
__device__ __forceinline__ int owner(const SharedParams& p, int count, int token, int lane) {
  int found = 0;
  for (int i0 = 0; i0 < count; i0 += 64) {
    const uint64_t votes = __ballot(i0 + lane < count && V::start(p, i0 + lane) <= token);
    found += __popcll(votes);
    if (votes != ~0ull) break;
  }
  return uniform(found - 1);
}

// Joins the parts of rows of one token: D / 4 lanes to a row. Bound by reading them: 36 MB for
// 64 tokens x 64 heads of 128 in 17 parts, 9.7 us. (Parts asked for before it is known how
// many there are: 10 to 11 us.)
template <class T, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(SharedParams p) {
  constexpr int G = D / 4, kRows = kThreads / G, kAhead = 4;
  fetch(p);
  const int per = (p.heads + kRows - 1) / kRows;
  const int token = (int)(blockIdx.x / per), head = (int)(blockIdx.x % per) * kRows + threadIdx.x / G;
  const int lane = threadIdx.x & 63, c = threadIdx.x % G;
  const int s = p.q_starts ? owner<OwnView>(p, p.seqs, token, lane) : token;
  if (s < 0) return;
  const Seq seq = sequence(p, s);
  if (token >= seq.begin + seq.len) return;  // behind the last sequence
  int g = -1;
  for (int i0 = 0, found = 0; i0 < p.groups; i0 += 64) {
    const uint64_t votes = __ballot(i0 + lane < p.groups && group_start(p, i0 + lane) <= s);
    found += __popcll(votes);
    g = uniform(found - 1);
    if (votes != ~0ull) break;
  }
  int prefix_parts = 0, prefix_n = 0;
  if (g >= 0 && s < group_start(p, g + 1)) {
    const Seq pre = PrefixView::seq(p, g);
    prefix_parts = span_of<PrefixView, 1>(p, pre, 0, 1).parts;
    prefix_n = pre.n;
  }
  if (head >= p.heads) return;
  const int rows = seq.len * p.group, r = (token - seq.begin) * p.group + head % p.group;
  int parts;
  if (rows > p.few_rows) {
    const int r0 = r / kManyRows * kManyRows;
    parts = span_of<OwnView, 1>(p, seq, r0, min_of(r0 + kManyRows, rows)).parts;
  } else {
    const int r0 = r / kFewRows * kFewRows;
    parts = span_of<OwnView, 0>(p, seq, r0, min_of(r0 + kFewRows, rows)).parts;
  }
  const int64_t row = (int64_t)token * p.heads + head;
  const int all = parts + prefix_parts;
  auto part_of = [&](int i) {  // parts past the last one are the last again
    i = min_of(i, all - 1);
    return row + (i < parts ? i * p.many_step : p.prefix_at + (i - parts) * p.many_step);
  };
  float top = -INFINITY, total = 0.f;
  f4v sum = {};
  for (int j = 0; j < all; j += kAhead) {
    f4v o[kAhead];
    f2v ml[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int64_t at = part_of(j + i);
      ml[i] = *((const f2v*)p.part_ml + at);
      o[i] = *((const f4v*)(p.part_o + at * D) + c);
    }
    float most = top;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) most = fmaxf(most, ml[i].x);
    const float old = top == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(top - most);
    top = most;
    total *= old;
    sum *= old;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (j + i >= all) continue;
      const float w = ml[i].x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[i].x - top);
      total += ml[i].y != ml[i].y ? ml[i].y : ml[i].y * w;  // NaN marks a bad page
      sum += o[i] * w;
    }
  }
  // a row that sees no key at all is zero
  sum *= inverse(total, prefix_n > 0 ? 0 : PagedView::pos(seq, token - seq.begin));
  *(u2v*)(p.out + (int64_t)token * p.o_token + head * p.o_head + 4 * c) =
      u2v{T::pack(sum[0], sum[1]), T::pack(sum[2], sum[3])};
}

// ------------------------------------------------------------------ host side

int check_shared(const lutgemm_shared* a) {
  if (!a) return LUTGEMM_ERR_NULL;
  const int st = check_attention(&a->own);
  if (st) return st;
  if (a->own.window != 0) return LUTGEMM_ERR_SHAPE;
  if (a->groups < 0 || a->groups >= (1 << 20) || a->prefix_width < 1 ||
      (int64_t)a->prefix_width * a->own.page_size > ((int64_t)1 << 30) || a->prefix_stride < 0 ||
      a->prefix_stride >= ((int64_t)1 << 40) || a->max_prefix < 0)
    return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

// A launch has fewer workgroups: below 2^32 threads along each axis of its grid.
constexpr int64_t kMostBlocks = (int64_t)1 << 23;

// Workgroups that run at a time: two to a compute unit. (Heads of 64 have room for three, and for four
// in 128 registers: 40 sequences in 5 groups 104 and 111 to 118 us, so 100.)
constexpr int64_t kSlots = 512;

struct SharedPlan {
  bool few, many;
  int prefix;  // which kernel
  int splits[3], chunk[3];  // of few_rows, many_rows and the prefixes
  int64_t tiles, prefix_tiles;
  int64_t rows, part_rows;
  int64_t blocks[4];  // as SharedParams'
  size_t ws_bytes;
};

int64_t grid_of(const SharedPlan& r) { return r.blocks[0] + r.blocks[1] + r.blocks[2] + r.blocks[3]; }

// Cuts `keys` keys of `base` row tiles into the number of parts that takes least time on
// `slots` workgroups at once, where a part costs as much as `more` keys besides its own.
void cut_keys(int64_t keys, int64_t base, int64_t slots, int64_t more, int* splits, int* chunk) {
  int64_t best = 1, least = INT64_MAX;
  for (int64_t n = 1; n <= kMaxSplits && base * (n - 1) < 4 * slots; ++n) {
    const int64_t each = part_keys(keys, n), parts = (keys + each - 1) / each;
    const int64_t time = (base * parts + slots - 1) / slots * (each + more);
    if (time < least) {
      least = time;
      best = parts;
    }
  }
  const int64_t each = part_keys(keys, best);
  *splits = (int)((keys + each - 1) / each);
  *chunk = (int)each;
}

SharedPlan plan(const lutgemm_shared* s) {
  const lutgemm_attention* a = &s->own;
  SharedPlan r{};
  if (a->tokens == 0 || a->seqs == 0) return r;  // nothing runs
  const int64_t group = a->heads / a->kv_heads;
  auto at_most = [](int64_t v, int64_t most) { return v < 1 ? 1 : v < most ? v : most; };
  const int64_t max_q = a->seqs == 1 ? a->tokens : at_most(a->max_q, a->tokens);
  const int64_t keys = at_most(a->max_kv, (int64_t)a->table_width * a->page_size);
  const int64_t prefix = at_most(s->max_prefix, (int64_t)s->prefix_width * a->page_size);
  r.many = max_q * group > kFewRows;
  r.few = !r.many || (a->seqs > 1 && group <= kFewRows);
  r.tiles = r.many ? a->tokens * group / kManyRows + a->seqs : 0;
  // A group of up to sixteen rows to a key head reads its prefix as a single token does: 16 rows on
  // heads of 64 57 us so and 59 by row tiles of 128, on heads of 128 97 and 101, 16 on 16000 keys in
  // 16 groups 178 and 237; 32 rows 43 and 40, 68 and 62. Where few rows are the mean, each group goes
  // by its own: 512 rows beside 63 groups of 8 on 4096 keys 143 us, all by few_rows 1420, all by
  // row tiles 150. Even batches pay up to 4% for workgroups that find no tile (63 groups of 8 rows
  // 92 to 94 us, with one of 16 99 to 103). Where more are the mean, all go by row tiles.
  const int64_t rows = a->tokens * group;
  const bool small = s->groups && (a->tokens + s->groups - 1) / s->groups * group <= kFewRows;
  r.prefix = !s->groups ? kNoPrefix : !small ? kManyPrefix
             : s->groups > 1 && rows > kFewRows ? kBothPrefixes : kFewPrefix;
  // the row tiles of groups of more rows; of more than 64 groups row_tile gives one more to each
  r.prefix_tiles = r.prefix == kManyPrefix
                       ? s->groups == 1 ? (rows + kManyRows - 1) / kManyRows : rows / kManyRows + s->groups
                   : r.prefix == kBothPrefixes
                       ? rows / kManyRows + (s->groups > 64 ? s->groups
                                                            : std::min<int64_t>(s->groups, rows / (kFewRows + 1)))
                       : 0;
  const int64_t few = (int64_t)a->seqs * a->kv_heads;
  const int64_t many = (a->tokens * group / kManyRows + (a->seqs + 1) / 2) * a->kv_heads;
  const int64_t shared_tiles = small            ? s->groups
                               : s->groups == 1 ? r.prefix_tiles
                                                : a->tokens * group / kManyRows + (s->groups + 1) / 2;
  const int64_t shared = shared_tiles * a->kv_heads;
  cut_keys(keys, few, kSlots, 256, &r.splits[0], &r.chunk[0]);
  cut_keys(keys, many, kSlots, 256, &r.splits[1], &r.chunk[1]);
  // The prefixes' tiles begin first; an eighth of the slots is left for the single tokens'
  // own keys to run beside them (64 sequences on 32768 keys, 64 heads of 8: 14 parts 112 to
  // 116 us, 16, which fill the slots, 119 to 122, 8, which fill half of them, 118). Both
  // in turn from the start was slower: the tiles then end late (125 to 146 us).
  cut_keys(prefix, shared, r.many || small ? kSlots : kSlots / 8 * 7, 256, &r.splits[2], &r.chunk[2]);
  if (!r.few) r.splits[0] = 0;
  if (!r.many) r.splits[1] = 0;
  if (!s->groups) r.splits[2] = 0;
  r.rows = a->tokens * a->heads;
  r.part_rows = (std::max(r.splits[0], r.splits[1]) + r.splits[2]) * r.rows;
  r.ws_bytes = (size_t)r.part_rows * (size_t)(a->head_dim + 2) * sizeof(float);
  r.blocks[0] = small ? (int64_t)s->groups * a->kv_heads * r.splits[2] : 0;
  r.blocks[1] = r.prefix_tiles * a->kv_heads * r.splits[2];
  r.blocks[2] = r.tiles * a->kv_heads * r.splits[1];
  r.blocks[3] = few * r.splits[0];
  if (r.prefix == kBothPrefixes && grid_of(r) >= kMostBlocks) {  // by few_rows all fit, or none
    r.prefix = kFewPrefix;
    r.blocks[1] = 0;
  }
  return r;
}

template <class T, int D, int Prefix>
int launch_shared(const SharedPlan& r, const SharedParams& p, hipStream_t stream) {
  const dim3 grid((unsigned)grid_of(r));
  if (r.few && r.many) return launch(shared_kernel<T, D, Prefix, true, true>, grid, kThreads, p, stream);
  if (r.many) return launch(shared_kernel<T, D, Prefix, false, true>, grid, kThreads, p, stream);
  return launch(shared_kernel<T, D, Prefix, true, false>, grid, kThreads, p, stream);
}

template <class T, int D>
int run_shared(const SharedPlan& r, const SharedParams& p, hipStream_t stream) {
  constexpr int kRows = kThreads / (D / 4);
  const int64_t joins = (int64_t)p.tokens * ((p.heads + kRows - 1) / kRows);
  const int st = r.prefix == kNoPrefix       ? launch_shared<T, D, kNoPrefix>(r, p, stream)
                 : r.prefix == kManyPrefix ? launch_shared<T, D, kManyPrefix>(r, p, stream)
                 : r.prefix == kFewPrefix  ? launch_shared<T, D, kFewPrefix>(r, p, stream)
                                           : launch_shared<T, D, kBothPrefixes>(r, p, stream);
  return st ? st : launch(join_kernel<T, D>, dim3((unsigned)joins), kThreads, p, stream);
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_shared_attention_workspace(const lutgemm_shared* a, size_t* bytes) {
  const int st = check_shared(a);
  if (st) return st;
  if (!bytes) return LUTGEMM_ERR_NULL;
  *bytes = plan(a).ws_bytes;
  return LUTGEMM_OK;
}

extern "C" int lutgemm_shared_attention(const lutgemm_shared* s, const void* d_q, const void* d_k,
                                        const void* d_v, const int32_t* d_prefix_table,
                                        const int32_t* d_prefix_lens, const int32_t* d_group_starts,
                                        const int32_t* d_table, const int32_t* d_kv_lens,
                                        const int32_t* d_q_starts, void* d_out, void* d_workspace,
                                        size_t workspace_bytes, void* stream) {
  try {
    int st = check_shared(s);
    if (st) return st;
    const lutgemm_attention* a = &s->own;
    if (!d_q_starts && a->tokens != a->seqs) return LUTGEMM_ERR_SHAPE;
    if (!d_group_starts && s->groups > 1) return LUTGEMM_ERR_SHAPE;
    if (a->tokens == 0 || a->seqs == 0) return LUTGEMM_OK;
    if (!d_q || !d_k || !d_v || !d_table || !d_kv_lens || !d_out) return LUTGEMM_ERR_NULL;
    if (s->groups && (!d_prefix_table || !d_prefix_lens)) return LUTGEMM_ERR_NULL;
    if (!aligned(d_q, 16) || !aligned(d_k, 16) || !aligned(d_v, 16) || !aligned(d_out, 16) ||
        !aligned(d_table, 4) || !aligned(d_kv_lens, 4) || !aligned(d_q_starts, 4) ||
        !aligned(d_prefix_table, 4) || !aligned(d_prefix_lens, 4) || !aligned(d_group_starts, 4))
      return LUTGEMM_ERR_ALIGN;
    const SharedPlan r = plan(s);
    if (grid_of(r) >= kMostBlocks || a->tokens * ((a->heads + 7) / 8) >= 2 * kMostBlocks)
      return LUTGEMM_ERR_SHAPE;
    if (!d_workspace) return LUTGEMM_ERR_NULL;
    if (workspace_bytes < r.ws_bytes) return LUTGEMM_ERR_BUFFER;
    if (!aligned(d_workspace, 16)) return LUTGEMM_ERR_ALIGN;
    int cus = 0;
    st = serve::check_device(&cus);
    if (st) return st;
    SharedParams p{};
    p.q = (const uint16_t*)d_q;
    p.k = (const uint16_t*)d_k;
    p.v = (const uint16_t*)d_v;
    p.table = d_table;
    p.kv_lens = d_kv_lens;
    p.q_starts = d_q_starts;
    p.prefix_table = d_prefix_table;
    p.prefix_lens = d_prefix_lens;
    p.group_starts = d_group_starts;
    p.out = (uint16_t*)d_out;
    p.part_o = (float*)d_workspace;
    p.part_ml = (float*)d_workspace + r.part_rows * a->head_dim;
    p.many_step = r.rows;
    p.prefix_at = std::max(r.splits[0], r.splits[1]) * r.rows;
    p.table_stride = a->table_stride;
    p.prefix_stride = s->prefix_stride;
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
    p.prefix_keys = s->prefix_width * a->page_size;
    for (int i = 0; i < 2; ++i) {
      p.splits[i] = std::max(r.splits[i], 1);
      p.chunk[i] = r.chunk[i];
    }
    p.prefix_splits = std::max(r.splits[2], 1);
    p.prefix_chunk = r.chunk[2];
    p.groups = s->groups;
    p.prefix_tiles = (int32_t)r.prefix_tiles;
    p.prefix_few = r.prefix == kManyPrefix ? 0 : r.prefix == kFewPrefix ? 0x7FFFFFFF : kFewRows;
    for (int i = 0; i < 4; ++i) p.blocks[i] = (int32_t)r.blocks[i];
    p.few_rows = !r.many ? 0x7FFFFFFF : r.few ? kFewRows : 0;
    p.tiles = (int32_t)r.tiles;
    p.scale2 = a->scale * 1.4426950408889634f;
    const bool f16 = a->type == LUTGEMM_F16;
    hipStream_t strm = (hipStream_t)stream;
    if (a->head_dim == 64)
      return f16 ? run_shared<serve::F16, 64>(r, p, strm) : run_shared<serve::BF16, 64>(r, p, strm);
    return f16 ? run_shared<serve::F16, 128>(r, p, strm) : run_shared<serve::BF16, 128>(r, p, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
