// heads.hip -- per-head norms of queries and keys, rotation by position, and the
// append of keys and values to the paged cache, in one pass over a fused QKV
// output (lutgemm_qk_norm_rotate; the formulas are in lutgemm.h).
//
// Memory bounds it: every element is read once and written once, with a few fp32
// operations between. 8192 tokens of 64 + 2 x 8 heads of 128 (340 MB) take 56.6 to
// 58.9 us by the machine, 5.8 to 6.0 TB/s; a plain copy of the same bytes takes 63. A
// thread owns sixteen entries of a head as two 16-byte words, chosen so that both halves of
// each rotated pair are its own (entries 8u .. 8u+7 and R/2 + 8u .. for pairs of halves,
// 16u .. 16u+15 for neighbours); the only exchange between lanes is the norm's sum over a
// head. A workgroup serves one token, so its slot and angles are looked up once for all the
// heads that it walks; reading several heads ahead (64 to 66 us) or a workgroup for each
// group of heads (87 us) did not gain.
#include <type_traits>

#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

struct HeadsParams {
  const uint16_t* qkv;
  const int64_t* positions;
  const float* table;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  uint16_t* q;
  uint16_t* k;
  uint16_t* v;
  const int64_t* slots;
  int64_t n_positions, n_slots;
  int64_t qkv_token, q_token;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;
  int32_t heads, kv_heads, dim, rotary, interleaved, page_size;
  int32_t lanes_log2;  // lanes of a head: the power of two from dim / 16 up
  int32_t walk;        // head groups that one workgroup serves
  int32_t all;         // heads served: of queries, keys and, into a cache, values
  float eps, inv_dim;
};

constexpr int kThreads = 256;

template <class T>
__device__ __forceinline__ void unpack16(u4v w, float (&a)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f2v x = T::unpack(w[i]);
    a[2 * i] = x.x;
    a[2 * i + 1] = x.y;
  }
}

// The rotation of a thread's sixteen entries. Pairs of halves: (a[i], b[i]);
// neighbours: the entries a[0..7], b[0..7] in order, two by two.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float (&cs)[8],
                                     const float (&sn)[8], bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = x * cs[i] - y * sn[i];
      a[2 * i + 1] = y * cs[i] + x * sn[i];
      const float z = b[2 * i], w = b[2 * i + 1];
      b[2 * i] = z * cs[4 + i] - w * sn[4 + i];
      b[2 * i + 1] = w * cs[4 + i] + z * sn[4 + i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = x * cs[i] - y * sn[i];
      b[i] = y * cs[i] + x * sn[i];
    }
  }
}

// A value summed over aligned groups of 1 << log2 lanes, up to sixteen, without LDS.
__device__ __forceinline__ float sum_lanes(float v, int log2) {
  auto moved = [&](auto control) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                 decltype(control)::value, 0xF, 0xF,
                                                                 true));
  };
  if (log2 > 0) v += moved(std::integral_constant<int, 0xB1>{});   // lanes 1, 0, 3, 2 of each four
  if (log2 > 1) v += moved(std::integral_constant<int, 0x4E>{});   // lanes 2, 3, 0, 1
  if (log2 > 2) v += moved(std::integral_constant<int, 0x141>{});  // eight lanes mirrored
  if (log2 > 3) v += moved(std::integral_constant<int, 0x140>{});  // sixteen mirrored
  return v;
}

// 1 / sqrt(v). The instruction takes v below the normal numbers for zero.
template <bool Tiny>
__device__ __forceinline__ float inverse_root(float v) {
  const bool small = Tiny && v < 0x1p-126f;
  return __builtin_amdgcn_rsqf(small ? v * 0x1p64f : v) * (small ? 0x1p32f : 1.f);
}

// Once: the heads do not stay in the L2 until their next reader, and pass it by
// (8192 tokens: 60.3 us, without the hint 64.2). Tiny: eps lies below the normal numbers, and
// mean squares may (a kernel of its own: with the test for it, or a branch on the launch's
// eps, it takes 73 registers in place of 72, a wave less to a SIMD, and 59.5 us in place of 58.8).
template <class T, bool Once, bool Tiny>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadsParams p) {
  fetch(p);
  const int64_t t = blockIdx.x;
  const int lanes = 1 << p.lanes_log2;
  const int u = threadIdx.x & (lanes - 1);            // which sixteen entries of the head
  const int per_group = kThreads >> p.lanes_log2;     // heads served together
  const bool active = u < p.dim / 16;
  const bool turned = u < p.rotary / 16;
  const bool halves = turned && !p.interleaved;
  const uint32_t c0 = !active ? 0 : halves ? 8 * u : 16 * u;
  const uint32_t c1 = !active ? 8 : halves ? 8 * u + p.rotary / 2 : 16 * u + 8;
  const uint16_t* src = p.qkv + t * p.qkv_token;
  const int64_t slot = p.slots ? p.slots[t] : 0;
  const int64_t pos = p.rotary ? p.positions[t] : 0;
  const int first = (int)blockIdx.y * p.walk * per_group + (int)(threadIdx.x >> p.lanes_log2);

  // the first head's words are on their way while the slot and the angles are looked up
  auto head_at = [&](int h) { return src + (uint32_t)min(h, p.all - 1) * (uint32_t)p.dim; };
  auto read = [](const uint16_t* from) {
    return Once ? __builtin_nontemporal_load((const u4v*)from) : *(const u4v*)from;
  };
  auto write = [](uint16_t* to, u4v w) {
    if constexpr (Once)
      __builtin_nontemporal_store(w, (u4v*)to);
    else
      *(u4v*)to = w;
  };
  u4v w0 = read(head_at(first) + c0), w1 = read(head_at(first) + c1);
  u4v qw0 = {}, qw1 = {}, kw0 = {}, kw1 = {};
  if (p.q_weight) {
    qw0 = *(const u4v*)(p.q_weight + c0);
    qw1 = *(const u4v*)(p.q_weight + c1);
    kw0 = *(const u4v*)(p.k_weight + c0);
    kw1 = *(const u4v*)(p.k_weight + c1);
  }
  const bool kept = !p.slots || (slot >= 0 && slot < p.n_slots);
  int64_t page = t, in_page = 0;
  if (p.slots && kept) {
    page = (p.n_slots >> 32) ? slot / p.page_size : (uint32_t)slot / (uint32_t)p.page_size;
    in_page = slot - page * p.page_size;
  }
  uint16_t* const q_to = p.q + t * p.q_token;
  uint16_t* const k_to = p.k + page * p.k_page + in_page * p.k_slot;
  uint16_t* const v_to = p.v + page * p.v_page + in_page * p.v_slot;
  float cs[8], sn[8];
  if (turned) {
    const bool known = pos >= 0 && pos < p.n_positions;
    const float* row = p.table + (known ? pos : 0) * p.rotary + 8 * u;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f4v c = *(const f4v*)(row + 4 * i), s = *(const f4v*)(row + p.rotary / 2 + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        cs[4 * i + j] = known ? c[j] : __builtin_nanf("");
        sn[4 * i + j] = known ? s[j] : __builtin_nanf("");
      }
    }
  }
  // whole heads step together, so every lane of a head is here or none is
  for (int g = 0; g < p.walk; ++g) {
    const int h = first + g * per_group;
    if (h >= p.all) break;
    if (g) {
      w0 = read(head_at(h) + c0);
      w1 = read(head_at(h) + c1);
    }
    const bool is_q = h < p.heads, is_v = h >= p.heads + p.kv_heads;
    if (!is_v) {
      float a[8], b[8];
      unpack16<T>(w0, a);
      unpack16<T>(w1, b);
      if (p.q_weight) {
        float wa[8], wb[8], sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          sum = __builtin_fmaf(a[i], a[i], sum);
          sum = __builtin_fmaf(b[i], b[i], sum);
        }
        sum = sum_lanes(active ? sum : 0.f, p.lanes_log2);
        const float r = inverse_root<Tiny>(__builtin_fmaf(sum, p.inv_dim, p.eps));
        unpack16<T>(is_q ? qw0 : kw0, wa);
        unpack16<T>(is_q ? qw1 : kw1, wb);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] *= r * wa[i];
          b[i] *= r * wb[i];
        }
      }
      if (turned) turn(a, b, cs, sn, p.interleaved);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        w0[i] = T::pack(a[2 * i], a[2 * i + 1]);
        w1[i] = T::pack(b[2 * i], b[2 * i + 1]);
      }
    }
    if (!active || (!is_q && !kept)) continue;
    uint16_t* to = is_q ? q_to + (uint32_t)h * (uint32_t)p.dim
                 : is_v ? v_to + (int64_t)(h - p.heads - p.kv_heads) * p.v_head
                        : k_to + (int64_t)(h - p.heads) * p.k_head;
    write(to + c0, w0);
    write(to + c1, w1);
  }
}

template <class T>
auto pick(bool once, bool tiny) {
  return once ? tiny ? heads_kernel<T, true, true> : heads_kernel<T, true, false>
              : tiny ? heads_kernel<T, false, true> : heads_kernel<T, false, false>;
}

int check_heads(const lutgemm_heads* h, bool paged) {
  if (!h) return LUTGEMM_ERR_NULL;
  if (h->type != LUTGEMM_F16 && h->type != LUTGEMM_BF16) return LUTGEMM_ERR_SHAPE;
  if (h->heads < 1 || h->kv_heads < 1 || h->heads > (1 << 16) || h->kv_heads > (1 << 16))
    return LUTGEMM_ERR_SHAPE;
  if (h->head_dim < 16 || h->head_dim > 256 || h->head_dim % 16) return LUTGEMM_ERR_SHAPE;
  if (h->rotary < 0 || h->rotary > h->head_dim || h->rotary % 16) return LUTGEMM_ERR_SHAPE;
  if (h->interleaved != 0 && h->interleaved != 1) return LUTGEMM_ERR_SHAPE;
  if (!(h->eps >= 0.0f) || !isfinite(h->eps)) return LUTGEMM_ERR_VALUE;
  if (h->tokens < 0 || h->tokens >= (1 << 24)) return LUTGEMM_ERR_SHAPE;
  if (h->rotary && (h->positions < 1 || h->positions >= ((int64_t)1 << 40)))
    return LUTGEMM_ERR_SHAPE;
  if (!stride_ok(h->qkv_token) || !stride_ok(h->q_token) || !stride_ok(h->k_page) ||
      !stride_ok(h->k_head))
    return LUTGEMM_ERR_SHAPE;
  const int64_t dim = h->head_dim;
  if (!serve::apart({{h->tokens, h->q_token}}, h->heads * dim)) return LUTGEMM_ERR_SHAPE;
  if (!paged && !serve::apart({{h->tokens, h->k_page}, {h->kv_heads, h->k_head}}, dim))
    return LUTGEMM_ERR_SHAPE;
  if (paged) {
    if (h->page_size < 1 || h->pages < 0 || h->pages >= ((int64_t)1 << 31)) return LUTGEMM_ERR_SHAPE;
    if (!stride_ok(h->k_slot) || !stride_ok(h->v_page) || !stride_ok(h->v_slot) ||
        !stride_ok(h->v_head))
      return LUTGEMM_ERR_SHAPE;
    if (!serve::apart({{h->pages, h->k_page}, {h->page_size, h->k_slot}, {h->kv_heads, h->k_head}},
                      dim) ||
        !serve::apart({{h->pages, h->v_page}, {h->page_size, h->v_slot}, {h->kv_heads, h->v_head}},
                      dim))
      return LUTGEMM_ERR_SHAPE;
  }
  return LUTGEMM_OK;
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_qk_norm_rotate(const lutgemm_heads* h, const void* d_qkv,
                                      const int64_t* d_positions, const float* d_table,
                                      const void* d_q_weight, const void* d_k_weight, void* d_q,
                                      void* d_k, void* d_v, const int64_t* d_slots, void* stream) {
  try {
    int st = check_heads(h, d_slots != nullptr);
    if (st) return st;
    if (h->tokens == 0) return LUTGEMM_OK;
    if (!d_qkv || !d_q || !d_k || (d_slots && !d_v)) return LUTGEMM_ERR_NULL;
    if (h->rotary && (!d_positions || !d_table)) return LUTGEMM_ERR_NULL;
    if ((d_q_weight == nullptr) != (d_k_weight == nullptr)) return LUTGEMM_ERR_NULL;
    if (!aligned(d_qkv, 16) || !aligned(d_q, 16) || !aligned(d_k, 16) || !aligned(d_v, 16) ||
        !aligned(d_table, 16) || !aligned(d_q_weight, 16) || !aligned(d_k_weight, 16) ||
        !aligned(d_positions, 8) || !aligned(d_slots, 8))
      return LUTGEMM_ERR_ALIGN;
    // a thread writes the queries that it has read, where other threads' heads do not lie
    const int64_t dim = h->head_dim;
    if (!(d_q == d_qkv && (h->tokens == 1 || h->q_token == h->qkv_token)) &&
        overlap({d_q, h->tokens, h->q_token, h->heads * dim},
                {d_qkv, h->tokens, h->qkv_token, (h->heads + 2 * (int64_t)h->kv_heads) * dim}))
      return LUTGEMM_ERR_SHAPE;
    int cus = 0;
    st = serve::check_device(&cus);
    if (st) return st;
    HeadsParams p{};
    p.qkv = (const uint16_t*)d_qkv;
    p.positions = d_positions;
    p.table = d_table;
    p.q_weight = (const uint16_t*)d_q_weight;
    p.k_weight = (const uint16_t*)d_k_weight;
    p.q = (uint16_t*)d_q;
    p.k = (uint16_t*)d_k;
    p.v = (uint16_t*)d_v;
    p.slots = d_slots;
    p.n_positions = h->positions;
    p.n_slots = h->pages * h->page_size;
    p.qkv_token = h->qkv_token;
    p.q_token = h->q_token;
    p.k_page = h->k_page;
    p.k_slot = h->k_slot;
    p.k_head = h->k_head;
    p.v_page = h->v_page;
    p.v_slot = h->v_slot;
    p.v_head = h->v_head;
    p.heads = h->heads;
    p.kv_heads = h->kv_heads;
    p.dim = h->head_dim;
    p.rotary = h->rotary;
    p.interleaved = h->interleaved;
    p.page_size = h->page_size;
    p.eps = h->eps;
    p.inv_dim = 1.0f / (float)h->head_dim;
    while ((16 << p.lanes_log2) < h->head_dim) ++p.lanes_log2;
    const int per_group = kThreads >> p.lanes_log2;
    const int all = h->heads + h->kv_heads * (d_slots ? 2 : 1);
    const int groups = (all + per_group - 1) / per_group;
    // few tokens: a workgroup for each group of heads; many: one walks them all
    p.walk = (int64_t)h->tokens * groups <= 8 * (int64_t)cus ? 1 : groups;
    p.all = all;
    const dim3 grid((unsigned)h->tokens, (unsigned)((groups + p.walk - 1) / p.walk));
    const bool once = (int64_t)h->tokens * all * h->head_dim * 2 > (int64_t)32 << 20;  // the L2s
    const bool tiny = d_q_weight && h->eps < 0x1p-126f;
    return serve::launch(h->type == LUTGEMM_F16 ? pick<serve::F16>(once, tiny)
                                                : pick<serve::BF16>(once, tiny),
                         grid, kThreads, p, (hipStream_t)stream);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
