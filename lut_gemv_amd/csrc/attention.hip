// attention.hip -- attention of new tokens over a paged key/value cache
// (lutgemm_paged_attention; the formula is in lutgemm.h).
//
// The two bodies of attention_kernel.h, in a kernel each and in one together for a batch
// that has sequences of both kinds; the combine kernels join the parts of split key axes.
#include "attention_kernel.h"

namespace lutgemm {
namespace {

template <class T, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void few_kernel(AttnParams p) {
  __shared__ __attribute__((aligned(16))) char mem[W * 64 * D * 2];
  __shared__ FewShared<W> shared;
  fetch(p);
  few_rows<PagedView, T, D, W>(p, blockIdx.x, [&](int w) { return mem + w * (64 * D * 2); }, shared);
}

template <class T, int D>
__global__ __launch_bounds__(kThreads, 2) void many_kernel(AttnParams p) {
  constexpr int kTile = 64 * D * 2;
  __shared__ __attribute__((aligned(16))) char keys0[kTile], vals0[kTile], keys1[kTile], vals1[kTile];
  __shared__ int marks;
  fetch(p);
  many_rows<PagedView, T, D>(p, blockIdx.x, keys0, vals0, keys1, vals1, marks);
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
    many_rows<PagedView, T, D>(p, blockIdx.x, keys0, vals0, keys1, vals1, shared.marks);
  else
    few_rows<PagedView, T, D, kThreads / 64>(
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
    const Span span = span_of<PagedView, 0>(p, seq, r0, min_of(r0 + kFewRows, rows));
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
  const RowTile at = row_tile<PagedView>(p, block / p.kv_heads / (kManyRows / kJoinRows), threadIdx.x & 63);
  if (at.s < 0) return;
  const Seq seq = sequence(p, at.s);
  const int rows = seq.len * p.group;
  if (rows <= p.few_rows || at.r0 < 0 || at.r0 >= rows) return;
  const int end = min_of(at.r0 + kManyRows, rows);
  const int parts = span_of<PagedView, 1>(p, seq, at.r0, end).parts;
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

struct AttnPlan {
  bool few, many;
  int splits[2], chunk[2];
  int64_t tiles;
  int64_t few_step, part_rows;  // part rows of one of few_rows' splits, and all of them
  size_t ws_bytes;
};

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
