// sample.hip -- next tokens from logits by temperature, top-k, top-p and min-p and one
// given random number a row (lutgemm_sample_tokens; the definition is in lutgemm.h).
//
// All three filters keep the first tokens of one order (value falling, index rising), so
// a row's kept tokens are those before one border: a value, and among the tokens that
// have it an index. Borders and the drawn token follow from sums of weights, and of
// 100000 tokens whose sums are off by 2^-24 the wrong one is taken in 1 of 100 rows.
// So weights are computed in 64 bits, 2^y = m 2^e from a table of 2^(i/1024) and a cubic
// polynomial, and all sums are integers, exact and the same in any order: by value, m 2^40 in
// bins of a sixteenth of an octave, where the bin tells e; in the order of the tokens,
// 2^S m 2^e with S = 62 - log2(vocab). Tokens below 2^-63 of the largest weight count as none.
//
// chunk_kernel takes a piece of a row to each workgroup and holds it in registers: its
// largest value, and relative to that (brought up to a whole octave, so that the
// pieces' bins and integers are each other's but for shifts) what the row's settings ask for:
// the sums of the bins (top_p, large top_k), the numbers of tokens in them (top_k), or the sums
// by place (no filter). row_kernel joins them, finds the bin of the border, reads the row
// once more for the tokens of this bin and the ones above, and ends on these in LDS where
// they are few (a radix select by weight, on 64-bit codes of value and index, then on
// the index); where they are many, the bins' sums say in which piece the drawn token lies,
// and only that is weighed again.
#include <type_traits>

#include "serve.h"

// A weight has the same bits wherever it is computed, and Scale's two parts of a product are
// its parts: products and sums are joined only where this is written.
#pragma clang fp contract(off)

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kSteps = 1024;       // table entries of an octave
constexpr int kBins = 1024;        // sixteenths of octaves below the largest weight
constexpr int kList = 4096;        // tokens of a list
constexpr int kMine = kList / kThreads;
constexpr int kStripes = 4;        // words of 16 bytes of a piece that a thread holds at most
constexpr int kLeastPiece = 4096;
constexpr int kMostPieces = 64;
constexpr int64_t kMostTokens = 1 << 20;
constexpr int kIndexBits = 20;

struct SampleParams {
  const void* logits;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t* tokens;
  float* logprobs;
  char* ws;  // [row][piece] of kRecord bytes
  int64_t row_step, record;
  int32_t rows, vocab, pieces, piece, parts, scale;  // parts: of a piece; scale: S
};

struct F32 {
  typedef uint32_t Raw;
  static constexpr int kKeyBits = 32;
  static constexpr Raw kNone = 0xFF800000;  // -infinity
  static __device__ __forceinline__ float wide(uint32_t a) { return __builtin_bit_cast(float, a); }
};
template <class T>
struct Logit16 : T {
  typedef uint16_t Raw;
  static constexpr int kKeyBits = 16;
  static constexpr Raw kNone = T::kHalf ? 0xFC00 : 0xFF80;
};

// An integer that rises with the value; the zeros are equal.
template <class T>
__device__ __forceinline__ uint32_t key_of(typename T::Raw raw) {
  constexpr uint32_t sign = 1u << (T::kKeyBits - 1);
  uint32_t b = raw;
  if (b == sign) b = 0;
  return b & sign ? ~b & (sign | (sign - 1)) : b | sign;
}

// The tokens' order as one number: falling values, then rising indices.
template <class T>
__device__ __forceinline__ uint64_t code_of(typename T::Raw raw, int index) {
  constexpr uint32_t all = T::kKeyBits == 32 ? ~0u : (1u << (T::kKeyBits & 31)) - 1;
  return (uint64_t)(~key_of<T>(raw) & all) << kIndexBits | (uint32_t)index;
}

// 16 bytes at any element's address: rows of odd lengths lie anywhere.
typedef uint32_t WordOf4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t WordOf2 __attribute__((ext_vector_type(4), aligned(2)));

// `n` tokens of a row: stripes of kThreads words of kPer tokens.
template <class T>
struct Piece {
  typedef typename T::Raw Raw;
  static constexpr int kPer = 16 / sizeof(Raw);
  const Raw* at;
  int n;
  __device__ __forceinline__ int stripes() const { return (n + kThreads * kPer - 1) / (kThreads * kPer); }
  __device__ __forceinline__ int first(int stripe) const {
    return (stripe * kThreads + (int)threadIdx.x) * kPer;
  }
  // The thread's word of a stripe, with -infinity past the end.
  __device__ __forceinline__ u4v word(int stripe) const {
    typedef typename std::conditional<sizeof(Raw) == 4, WordOf4, WordOf2>::type Any;
    const int i = first(stripe);
    if (i + kPer <= n) return *(const Any*)(at + i);
    u4v w;
    Raw* const e = (Raw*)&w;
#pragma unroll
    for (int j = 0; j < kPer; ++j) e[j] = i + j < n ? at[i + j] : T::kNone;
    return w;
  }
  // An element of which the place is only known when it runs.
  static __device__ __forceinline__ Raw any(const u4v& w, int e) {
    const int at = e * (int)sizeof(Raw) / 4;
    const uint32_t x = at < 2 ? (at == 0 ? w[0] : w[1]) : (at == 2 ? w[2] : w[3]);
    return sizeof(Raw) == 4 ? (Raw)x : (Raw)(x >> (16 * (e & 1)));
  }
  static __device__ __forceinline__ Raw element(const u4v& w, int e) {
    if constexpr (sizeof(Raw) == 4) return w[e];
    return (Raw)(w[e >> 1] >> (16 * (e & 1)));
  }
};

// What values are measured against: 2^top (a whole octave) is at least the weight of
// `ref`, whose own distance from it is `shift` in 1024ths of an octave.
struct Scale {
  double ref, step, shift, top;
  __device__ __forceinline__ void set(float largest, float temperature) {
    const double octaves = 1.4426950408889634074 / (double)temperature;
    ref = (double)largest;
    step = octaves * kSteps;
    const double p = ref * octaves;
    if (__builtin_fabs(p) < 0x1p40) {
      top = __builtin_ceil(p);
      shift = ((p - top) + __builtin_fma(ref, octaves, -p)) * kSteps;
    } else {  // other values are more than 64 octaves away
      top = p;
      shift = 0.0;
    }
  }
  // The weight m 2^(k >> 10) of a value of at most ref, m in [1, 2] but for rounding.
  __device__ __forceinline__ double weigh(double x, const double* steps, int* k) const {
    constexpr double kRound = 0x1.8p52, c = 0.69314718055994530942 / kSteps;
    double y = __builtin_fma(x - ref, step, shift);
    y = y < -1e6 ? -1e6 : y;
    const double s = y + kRound;
    *k = (int)(uint32_t)__builtin_bit_cast(uint64_t, s);
    const double f = y - (s - kRound);
    const double p = __builtin_fma(
        f, __builtin_fma(f, __builtin_fma(f, c * c * c / 6, c * c / 2), c), 1.0);
    return steps[*k & (kSteps - 1)] * p;
  }
};

// Sixteenths of octaves below the top, and the octave of such a bin.
__device__ __forceinline__ int bin_of(int k) { return -(k >> 6); }
__device__ __forceinline__ int octave_of(int bin) { return (-bin) >> 4; }

// x to the nearest integer, x below 2^51.
__device__ __forceinline__ uint64_t whole(double x) {
  constexpr double kOne = 0x1p52;
  return __builtin_bit_cast(uint64_t, x + kOne) - __builtin_bit_cast(uint64_t, kOne);
}
// A weight in a bin's sum: m 2^40.
__device__ __forceinline__ uint64_t term_of(double m) {
  constexpr double kUnit = 0x1p12;  // the last place of 2^12 + m is 2^-40
  return __builtin_bit_cast(uint64_t, m + kUnit) - __builtin_bit_cast(uint64_t, kUnit);
}
// A weight in a sum by place: m 2^(S + e).
__device__ __forceinline__ uint64_t place_of(double m, int k, int scale) {
  return whole(__builtin_ldexp(m, scale + (k >> 10)));
}
// v 2^by, without what falls below 1.
__device__ __forceinline__ uint64_t shifted(uint64_t v, int by) {
  return by >= 64 || by <= -64 ? 0 : by >= 0 ? v << by : v >> -by;
}

// The largest whole number of at most a * v, a in [0, 1); `up`: the smallest of at least.
__device__ __forceinline__ uint64_t share(float a, uint64_t v, bool up) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, a);
  const int e = (int)(bits >> 23);
  const uint64_t m = e ? (bits & 0x7FFFFF) | 0x800000 : bits & 0x7FFFFF;
  const int down = 150 - (e ? e : 1);  // a = m 2^-down
  const unsigned __int128 product = (unsigned __int128)v * m;
  if (down >= 100) return up && product ? 1 : 0;
  const unsigned __int128 rest = up ? (((unsigned __int128)1) << down) - 1 : 0;
  return (uint64_t)((product + rest) >> down);
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d, 64);
  return v;
}

// Sums of the threads before this one and itself, in order; *total: of all.
template <class V>
__device__ __forceinline__ V block_scan(V v, V* waves, V* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const V u = __shfl_up(v, d, 64);
    if (lane >= d) v += u;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = v;
  __syncthreads();
  V before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += waves[w];
    all += waves[w];
  }
  *total = all;
  return v + before;
}

// A row's settings, and what they make of it.
struct Settings {
  float u, temperature, top_p, min_p;
  int top_k;
  bool bad, by_count, by_weight, by_least;
  __device__ __forceinline__ Settings(const SampleParams& p, int64_t r) {
    u = p.u[r];
    temperature = p.temperature ? p.temperature[r] : 1.f;
    top_p = p.top_p ? p.top_p[r] : 1.f;
    min_p = p.min_p ? p.min_p[r] : 0.f;
    top_k = p.top_k ? p.top_k[r] : 0;
    bad = !(u >= 0.f && u < 1.f) || !(temperature >= 0.f && temperature < INFINITY) ||
          top_p != top_p || min_p != min_p;
    by_count = top_k > 0 && top_k < p.vocab;
    by_weight = top_p < 1.f;
    by_least = min_p > 0.f;
  }
  __device__ __forceinline__ bool greedy() const { return temperature == 0.f; }
  // whether the tokens that top_k leaves go into a list, weighed there
  __device__ __forceinline__ bool few() const { return by_count && top_k <= kList / 2; }
  __device__ __forceinline__ bool counts() const { return by_count; }
  __device__ __forceinline__ bool sums() const { return by_count ? !few() : by_weight; }
  __device__ __forceinline__ bool places() const { return !by_count && !by_weight && !by_least; }
};

// A piece's record in the workspace: this, then the bins' sums and counts or the parts' sums.
struct Head {
  double top;
  float largest;
  int32_t bad, at, pad;  // at: greedy: the first token of the largest value
};
constexpr int kSumsAt = 64, kCountsAt = kSumsAt + kBins * 8, kPartsAt = kSumsAt;
constexpr int kRecord = kCountsAt + kBins * 4;

template <class T>
__global__ __launch_bounds__(kThreads, 8) void chunk_kernel(SampleParams p) {
  typedef Piece<T> P;
  __shared__ double steps[kSteps];
  __shared__ uint64_t sums[kBins];
  __shared__ uint32_t counts[kBins];
  __shared__ float waves[kWaves];
  __shared__ int32_t first;
  fetch(p);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t r = blockIdx.x / (unsigned)p.pieces;
  const int c = (int)(blockIdx.x % (unsigned)p.pieces);
  const int begin = c * p.piece;
  P piece;
  piece.at = (const typename T::Raw*)p.logits + r * p.row_step + begin;
  piece.n = min(p.piece, p.vocab - begin);
  const int stripes = piece.stripes();
  u4v w[kStripes];
#pragma unroll
  for (int s = 0; s < kStripes; ++s)
    if (s < stripes) w[s] = piece.word(s);
  const Settings set(p, r);
  // while the loads are under way
  if (set.sums() || set.places()) steps[t] = exp2((double)t / kSteps);
  if (set.sums()) sums[t] = 0;
  if (set.counts()) counts[t] = 0;
  if (t == 0) first = INT32_MAX;
  float most = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int s = 0; s < kStripes; ++s)
    if (s < stripes)
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) {
        const float x = T::wide(P::element(w[s], e));
        bad |= !(x < INFINITY);
        most = fmaxf(most, x);
      }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
  if (lane == 0) waves[wave] = most;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int v = 0; v < kWaves; ++v) most = fmaxf(most, waves[v]);
  char* const record = p.ws + (r * p.pieces + c) * p.record;
  if (set.greedy()) {
    int least = INT32_MAX;
#pragma unroll
    for (int s = 0; s < kStripes; ++s)
      if (s < stripes)
#pragma unroll
        for (int e = 0; e < P::kPer; ++e) {
          const int i = piece.first(s) + e;
          if (T::wide(P::element(w[s], e)) == most && i < least) least = i;
        }
    if (least < piece.n) atomicMin(&first, least);
    __syncthreads();
  }
  Scale scale;
  scale.set(most, set.temperature);
  if (t == 0) *(Head*)record = Head{scale.top, most, bad, begin + first, 0};
  if (set.bad || bad || set.greedy() || most == -INFINITY) return;
  if (set.places()) {
    uint64_t* const parts = (uint64_t*)(record + kPartsAt);
#pragma unroll
    for (int s = 0; s < kStripes; ++s) {
      if (s >= stripes) continue;
      uint64_t sum = 0;
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) {
        int k;
        const double m = scale.weigh((double)T::wide(P::element(w[s], e)), steps, &k);
        sum += place_of(m, k, p.scale);
      }
      sum = wave_sum(sum);
      if (lane == 0) parts[s * kWaves + wave] = sum;
    }
    for (int i = stripes * kWaves + t; i < p.parts; i += kThreads) parts[i] = 0;
    return;
  }
  if (!set.sums() && !set.counts()) return;
  auto fill = [&](auto with_sums, auto with_counts) {
#pragma unroll
    for (int s = 0; s < kStripes; ++s) {
      if (s >= stripes) continue;
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) {
        int k;
        const double m = scale.weigh((double)T::wide(P::element(w[s], e)), steps, &k);
        const int bin = bin_of(k);
        if (bin >= kBins) continue;
        if (with_sums) atomicAdd((unsigned long long*)&sums[bin], (unsigned long long)term_of(m));
        if (with_counts) atomicAdd(&counts[bin], 1u);
      }
    }
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  if (!set.sums())
    fill(no, yes);
  else if (!set.counts())
    fill(yes, no);
  else
    fill(yes, yes);
  __syncthreads();
  if (set.sums()) ((uint64_t*)(record + kSumsAt))[t] = sums[t];
  if (set.counts()) ((uint32_t*)(record + kCountsAt))[t] = counts[t];
}

// ------------------------------------------------------------------ rows

struct RowShared {
  double steps[kSteps];
  uint64_t list[kList];   // codes; or the parts' sums
  uint64_t inside[kList]; // codes of the border's bin
  uint64_t sums[256];
  uint32_t counts[256];
  uint64_t qwaves[kWaves];
  uint32_t waves[kWaves];
  uint64_t found_sum, found_code;
  int32_t found, found_count;
  uint32_t above, within;  // tokens of the lists
};

// The first code, of those that `members` hands to its argument with a value each, up to which
// the values sum to `target` (at least 1), in the order of the codes; *before: the sum
// ahead of it. If the sum is less, the last code. By eight bits at a time from the
// highest of `bits`, until one code is left.
template <class Members>
__device__ uint64_t select(RowShared& sh, int bits, uint64_t target, uint64_t* before, Members members) {
  const int t = threadIdx.x;
  uint64_t prefix = 0, passed = 0;
  int shift = (bits + 7) / 8 * 8;
  while (shift > 0) {
    shift -= 8;
    __syncthreads();
    if (t < 256) {
      sh.sums[t] = 0;
      sh.counts[t] = 0;
    }
    __syncthreads();
    members([&](uint64_t code, uint64_t value) {
      if (code >> (shift + 8) != prefix) return;
      const int byte = (int)(code >> shift) & 255;
      atomicAdd((unsigned long long*)&sh.sums[byte], (unsigned long long)value);
      atomicAdd(&sh.counts[byte], 1u);
    });
    __syncthreads();
    const uint64_t v = t < 256 ? sh.sums[t] : 0;
    const uint32_t n = t < 256 ? sh.counts[t] : 0;
    uint64_t all;
    const uint64_t up = block_scan(v, sh.qwaves, &all);
    const uint64_t want = target < all ? target : all;
    if (n && v && up >= want && up - v < want) {
      sh.found = t;
      sh.found_sum = up - v;
      sh.found_count = (int)n;
    }
    if (all == 0 && t == 0) {  // nothing has a value: there is no such code
      sh.found = 255;
      sh.found_sum = 0;
      sh.found_count = 2;
    }
    __syncthreads();
    prefix = prefix << 8 | (uint32_t)sh.found;
    passed += sh.found_sum;
    target = want - sh.found_sum;
    if (sh.found_count == 1 && shift > 0) {
      members([&](uint64_t code, uint64_t) {
        if (code >> shift == prefix) sh.found_code = code;
      });
      __syncthreads();
      *before = passed;
      return sh.found_code;
    }
  }
  __syncthreads();
  *before = passed;
  return prefix;
}

template <class T>
__global__ __launch_bounds__(kThreads) void row_kernel(SampleParams p) {
  typedef Piece<T> P;
  typedef typename T::Raw Raw;
  constexpr int kCodeBits = T::kKeyBits + kIndexBits;
  constexpr uint32_t kKeyAll = T::kKeyBits == 32 ? ~0u : (1u << (T::kKeyBits & 31)) - 1;
  __shared__ RowShared sh;
  fetch(p);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t r = blockIdx.x;
  const Settings set(p, r);
  const char* const records = p.ws + r * p.pieces * p.record;
  // the pieces' heads, one to a lane
  Head head = {0.0, -INFINITY, 0, 0, 0};
  if (lane < p.pieces) head = *(const Head*)(records + lane * p.record);
  float most = head.largest;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
  if (set.bad || __any(head.bad) || most == -INFINITY) {
    if (t == 0) {
      p.tokens[r] = -1;
      if (p.logprobs) p.logprobs[r] = __builtin_nanf("");
    }
    return;
  }
  if (set.greedy()) {
    const int c = __builtin_ctzll(__ballot(head.largest == most && lane < p.pieces));
    if (t == c) {
      p.tokens[r] = head.at;
      if (p.logprobs) p.logprobs[r] = 0.f;
    }
    return;
  }
  sh.steps[t] = exp2((double)t / kSteps);
  Scale scale;
  scale.set(most, set.temperature);
  // octaves of the pieces below the row's, 64 for those without weight
  const double lower = scale.top - head.top;
  const int down = head.largest > -INFINITY && lower < 64.0 ? (int)lower : 64;
  const int S = p.scale;
  P row;
  row.at = (const Raw*)p.logits + r * p.row_step;
  row.n = p.vocab;

  int owner_token = -1;   // of the thread that has found the token
  float owner_value = 0.f;
  uint64_t total = 0;     // kept weights, 2^S each

  // the first token up to which `weight` of the tokens of [at, at + 64 kPer) sums to `goal`, by one wave
  auto pick = [&](const P& piece, int stripe, int part_wave, uint64_t goal, int offset, auto weight) {
    if (wave != part_wave) return;
    const u4v w = piece.word(stripe);
    const int i0 = piece.first(stripe);
    uint64_t mine[P::kPer], sum = 0;
#pragma unroll 1
    for (int e = 0; e < P::kPer; ++e) {
      const uint64_t v = i0 + e < piece.n ? weight(P::any(w, e), i0 + e) : 0;
#pragma unroll
      for (int j = 0; j < P::kPer; ++j)
        if (j == e) mine[j] = v;
      sum += v;
    }
    uint64_t up = sum;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint64_t o = __shfl_up(up, d, 64);
      if (lane >= d) up += o;
    }
    uint64_t cursor = up - sum;
    int token = -1, last = -1;
    float value = 0.f, last_value = 0.f;
#pragma unroll
    for (int e = 0; e < P::kPer; ++e) {
      cursor += mine[e];
      if (!mine[e]) continue;
      last = i0 + e;
      last_value = T::wide(P::element(w, e));
      if (token < 0 && cursor >= goal) {
        token = last;
        value = last_value;
      }
    }
    const uint64_t have = __ballot(token >= 0), some = __ballot(last >= 0);
    const int owner = have ? __builtin_ctzll(have) : some ? 63 - __builtin_clzll(some) : -1;
    if (lane == owner) {
      owner_token = offset + (have ? token : last);
      owner_value = have ? value : last_value;
    }
  };

  if (set.places()) {
    // parts in order, a few to a thread
    const int all = p.pieces * p.parts, each = (all + kThreads - 1) / kThreads;
    auto part_at = [&](int i) -> uint64_t {
      const int at = min(i, all - 1), c = at / p.parts;
      const int by = __shfl(down, c, 64);  // by all lanes
      if (i >= all || by >= 64) return 0;
      return shifted(((const uint64_t*)(records + c * p.record + kPartsAt))[at % p.parts], -by);
    };
    uint64_t sum = 0;
    for (int j = 0; j < each; ++j) sum += part_at(t * each + j);
    const uint64_t up = block_scan(sum, sh.qwaves, &total);
    const uint64_t goal = share(set.u, total, false) + 1;
    if (t == 0) sh.found = 0;
    __syncthreads();
    if (sum && up >= goal && up - sum < goal) {
      sh.found = t;
      sh.found_sum = up - sum;
    }
    __syncthreads();
    uint64_t before = sh.found_sum;
    int part = sh.found * each;
    for (;; ++part) {  // every thread by itself
      const uint64_t v = part_at(part);
      if (before + v >= goal || part + 1 >= all) break;
      before += v;
    }
    const int c = part / p.parts, by = __shfl(down, c, 64);
    Scale own;
    own.set(__shfl(head.largest, c, 64), set.temperature);
    P piece;
    piece.at = row.at + c * p.piece;
    piece.n = min(p.piece, p.vocab - c * p.piece);
    pick(piece, part % p.parts / kWaves, part % p.parts % kWaves, (goal - before) << by, c * p.piece,
         [&](Raw raw, int) {
           int k;
           const double m = own.weigh((double)T::wide(raw), sh.steps, &k);
           return place_of(m, k, S);
         });
  } else {
    // the bins of all pieces: sums in their own octave's unit and in 2^S
    uint64_t sum = 0;
    uint32_t count = 0;
    for (int c = 0; c < p.pieces; ++c) {
      const int by = __builtin_amdgcn_readlane(down, c);
      const int bin = t - 16 * by;
      if (by >= 64 || bin < 0) continue;
      if (set.sums()) sum += ((const uint64_t*)(records + c * p.record + kSumsAt))[bin];
      if (set.counts()) count += ((const uint32_t*)(records + c * p.record + kCountsAt))[bin];
    }
    const int octave = octave_of(t);
    const uint64_t mine = shifted(sum, S - 40 + octave);
    uint64_t all_sum = 0;
    uint32_t all_count = 0;
    const uint64_t upto = block_scan(mine, sh.qwaves, &all_sum);
    const uint32_t upto_count = block_scan(count, sh.waves, &all_count);

    // the first bin whose sum or count from the top passes what is asked for, kBins if none
    auto bin_where = [&](bool passes) {
      if (t == 0) sh.found = kBins;
      __syncthreads();
      if (passes) atomicMin(&sh.found, t);
      __syncthreads();
      const int bin = sh.found;
      __syncthreads();
      return bin;
    };
    // a value that no token of the bins up to this one is below
    auto least_of = [&](double bin) {
      const double x = scale.ref + (-64.0 * bin - 0.5 - scale.shift) / scale.step;
      return (float)(x - 1e-6 * (__builtin_fabs(x) + __builtin_fabs(scale.ref)) - 1e-30);
    };
    // f(raw, index) of every token of at least `least`
    auto each_from = [&](float least, auto f) {
      const int stripes = row.stripes();
      constexpr int kAhead = 4;
      for (int s0 = 0; s0 < stripes; s0 += kAhead) {
        u4v w[kAhead];
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
          if (s0 + a < stripes) w[a] = row.word(s0 + a);
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          if (s0 + a >= stripes) continue;
          const int i0 = row.first(s0 + a);
          uint32_t some = 0;
#pragma unroll
          for (int e = 0; e < P::kPer; ++e) some |= (T::wide(P::element(w[a], e)) >= least) << e;
          for (; some; some &= some - 1) {
            const int e = __builtin_ctz(some);
            if (i0 + e < row.n) f(P::any(w[a], e), i0 + e);
          }
        }
      }
    };
    // the tokens of the bins before `bin` into the list, those of it into `inside`
    auto gather = [&](int bin, bool before_too) {
      __syncthreads();
      if (t == 0) sh.above = sh.within = 0;
      __syncthreads();
      each_from(least_of(bin), [&](Raw raw, int i) {
        int k;
        scale.weigh((double)T::wide(raw), sh.steps, &k);
        const int b = bin_of(k);
        if (b == bin) {
          const uint32_t at = atomicAdd(&sh.within, 1u);
          if (at < kList) sh.inside[at] = code_of<T>(raw, i);
        } else if (b < bin && before_too && sh.above < kList) {
          const uint32_t at = atomicAdd(&sh.above, 1u);
          if (at < kList) sh.list[at] = code_of<T>(raw, i);
        }
      });
      __syncthreads();
    };
    auto raw_of = [&](uint64_t code) {  // the bits of a code's value
      const uint32_t key = ~(uint32_t)(code >> kIndexBits) & kKeyAll;
      constexpr uint32_t sign = 1u << (T::kKeyBits - 1);
      return (Raw)(key & sign ? key & (sign - 1) : ~key & kKeyAll);
    };
    // the border inside a bin: the code up to which its tokens' number or sum (in the
    // bin's unit) reaches `need`; after gather(bin, .)
    auto border_in = [&](int bin, bool weights, uint64_t need, uint64_t* before) {
      if (need < 1) need = 1;
      if (sh.within == 0) {  // a value between two bins was rounded into another: the largest alone
        *before = 0;
        uint32_t raw = __builtin_bit_cast(uint32_t, most);
        if constexpr (T::kKeyBits == 16) raw = T::one(most);
        return code_of<T>((Raw)raw, (1 << kIndexBits) - 1);
      }
      if (sh.within <= kList) {
        const int n = (int)sh.within;
        return select(sh, kCodeBits, need, before, [&](auto f) {
          for (int i = t; i < n; i += kThreads) {
            const uint64_t code = sh.inside[i];
            int k;
            const double m = scale.weigh((double)T::wide(raw_of(code)), sh.steps, &k);
            f(code, weights ? term_of(m) : 1);
          }
        });
      }
      const float least = least_of(bin);
      return select(sh, kCodeBits, need, before, [&](auto f) {
        each_from(least, [&](Raw raw, int i) {
          int k;
          const double m = scale.weigh((double)T::wide(raw), sh.steps, &k);
          if (bin_of(k) == bin) f(code_of<T>(raw, i), weights ? term_of(m) : 1);
        });
      });
    };

    uint64_t border = ~0ull;  // kept: codes up to it
    bool listed = false;      // the kept tokens are among the list's first `members`
    int members = 0;
    int last_bin = kBins - 1; // no kept token is behind this bin
    int chosen_bin = -1;      // the border is in this bin, of which `inside` has the tokens
    // puts `inside` behind the list, if both have room
    auto join_lists = [&] {
      const uint32_t n = sh.above + sh.within;
      const bool fits = sh.above <= kList && sh.within <= kList && n <= kList;
      if (fits) {
        for (uint32_t i = t; i < sh.within; i += kThreads) sh.list[sh.above + i] = sh.inside[i];
        members = (int)n;
      }
      __syncthreads();
      return fits;
    };
    uint64_t available = all_sum;  // what top_p takes its part of
    if (set.by_count) {
      int bin = bin_where(upto_count >= (uint32_t)set.top_k);
      if (bin == kBins && set.few()) bin = kBins - 1;  // fewer than top_k have weight: all of these
      if (bin < kBins) {
        last_bin = bin;
        if (t == bin) {
          sh.found_count = (int)(upto_count - count);
          sh.found_sum = upto - mine;
        }
        __syncthreads();
        const uint64_t rest = (uint64_t)(set.top_k - sh.found_count);
        const uint64_t ahead = sh.found_sum;
        gather(bin, set.few());
        listed = set.few() && join_lists();
        if (!listed) {
          uint64_t before;
          border = border_in(bin, false, rest, &before);
          chosen_bin = bin;
          if (set.few()) {  // of the bin only those up to the border
            __syncthreads();
            if (t == 0) sh.above = 0;
            __syncthreads();
            each_from(least_of(bin), [&](Raw raw, int i) {
              const uint64_t code = code_of<T>(raw, i);
              if (code > border) return;
              const uint32_t at = atomicAdd(&sh.above, 1u);
              if (at < kList) sh.list[at] = code;
            });
            __syncthreads();
            listed = true;
            members = (int)min(sh.above, (uint32_t)kList);
          } else {
            // the sum of what is kept: by weight up to the border's code
            uint64_t kept = 0;
            each_from(least_of(bin), [&](Raw raw, int i) {
              int k;
              const double m = scale.weigh((double)T::wide(raw), sh.steps, &k);
              if (bin_of(k) == bin && code_of<T>(raw, i) <= border) kept += term_of(m);
            });
            uint64_t all;
            block_scan(kept, sh.qwaves, &all);
            available = ahead + shifted(all, S - 40 + octave_of(bin));
          }
        } else {
          uint64_t before;
          const int n = members;
          border = select(sh, kCodeBits, (uint64_t)set.top_k, &before, [&](auto f) {
            for (int i = t; i < n; i += kThreads) f(sh.list[i], 1);
          });
        }
      }
    }
    if (set.by_weight && !listed && set.sums()) {
      uint64_t target = set.top_p > 0.f ? share(set.top_p, available, true) : 1;
      if (target < 1) target = 1;
      int bin = bin_where(mine && upto >= target);
      if (bin > last_bin) bin = last_bin;
      last_bin = bin;
      if (t == bin) sh.found_sum = upto - mine;
      __syncthreads();
      const uint64_t ahead = sh.found_sum;
      gather(bin, true);
      const int by = 40 - octave_of(bin) - S;  // from 2^S to the bin's unit
      const uint64_t missing = target > ahead ? target - ahead : 1;
      const uint64_t need = by >= 0 ? shifted(missing, by) : (missing + (1ull << -by) - 1) >> -by;
      uint64_t before;
      const uint64_t second = border_in(bin, true, need, &before);
      if (second < border) {
        border = second;
        chosen_bin = bin;
      }
      listed = join_lists();
    }
    const double floor_weight =  // of what min_p keeps
        set.by_least ? (double)(set.min_p < 1.f ? set.min_p : 1.f) : 0.0;
    int km;
    const double largest = scale.weigh(scale.ref, sh.steps, &km);
    const double least_weight = floor_weight * __builtin_ldexp(largest, km >> 10);
    float least = least_of(last_bin);
    if (set.by_least) {
      const double bins = 17.0 - 16.0 * log2(floor_weight);  // the top is less than an octave higher
      if (bins < (double)last_bin) least = least_of(bins);
      if (!listed && !set.by_count && !set.by_weight) {
        __syncthreads();
        if (t == 0) sh.above = sh.within = 0;
        __syncthreads();
        each_from(least, [&](Raw raw, int i) {
          int k;
          const double m = scale.weigh((double)T::wide(raw), sh.steps, &k);
          if (bin_of(k) >= kBins || __builtin_ldexp(m, k >> 10) < least_weight || sh.above > kList) return;
          const uint32_t at = atomicAdd(&sh.above, 1u);
          if (at < kList) sh.list[at] = code_of<T>(raw, i);
        });
        __syncthreads();
        listed = join_lists();
      }
    }
    auto kept_weight = [&](Raw raw, int i) -> uint64_t {
      if (code_of<T>(raw, i) > border) return 0;
      int k;
      const double m = scale.weigh((double)T::wide(raw), sh.steps, &k);
      if (bin_of(k) >= kBins || __builtin_ldexp(m, k >> 10) < least_weight) return 0;
      return place_of(m, k, S);
    };
    if (listed) {
      uint64_t code[kMine], weight[kMine], sum = 0;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const int i = t + j * kThreads;
        code[j] = i < members ? sh.list[i] : ~0ull;
        weight[j] = i < members
                        ? kept_weight(raw_of(code[j]), (int)(code[j] & ((1u << kIndexBits) - 1)))
                        : 0;
        sum += weight[j];
      }
      block_scan(sum, sh.qwaves, &total);
      uint64_t before;
      if (set.by_count && set.by_weight && set.few()) {
        // top_p of what top_k leaves, before min_p
        uint64_t plain[kMine], whole_sum = 0;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          plain[j] = 0;
          if (code[j] <= border && code[j] != ~0ull) {
            int k;
            const double m = scale.weigh((double)T::wide(raw_of(code[j])), sh.steps, &k);
            if (bin_of(k) < kBins) plain[j] = place_of(m, k, S);
          }
          whole_sum += plain[j];
        }
        uint64_t all;
        block_scan(whole_sum, sh.qwaves, &all);
        uint64_t target = set.top_p > 0.f ? share(set.top_p, all, true) : 1;
        if (target < 1) target = 1;
        border = select(sh, kCodeBits, target, &before, [&](auto f) {
#pragma unroll
          for (int j = 0; j < kMine; ++j)
            if (plain[j]) f(code[j], plain[j]);
        });
        sum = 0;
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          if (code[j] > border) weight[j] = 0;
          sum += weight[j];
        }
        block_scan(sum, sh.qwaves, &total);
      }
      const uint64_t goal = share(set.u, total, false) + 1;
      const uint64_t token = select(sh, kIndexBits, goal, &before, [&](auto f) {
#pragma unroll
        for (int j = 0; j < kMine; ++j)
          if (weight[j]) f(code[j] & ((1u << kIndexBits) - 1), weight[j]);
      });
      if (t == 0) {
        owner_token = (int)token;
        owner_value = T::wide(row.at[token]);
      }
    } else {
      // the piece in which the token lies, by the bins' sums; then its parts
      P piece = row;
      int offset = 0;
      uint64_t ahead = 0, goal = 0;
      const bool by_bins = chosen_bin >= 0 && set.sums() && !set.by_least;
      if (by_bins) {
        // of the border's bin, the kept tokens' sums by piece
        uint64_t* const edge = sh.sums;
        __syncthreads();
        if (t < kMostPieces) edge[t] = 0;
        __syncthreads();
        auto add = [&](Raw raw, int i) {
          int k;
          const double m = scale.weigh((double)T::wide(raw), sh.steps, &k);
          if (bin_of(k) == chosen_bin && code_of<T>(raw, i) <= border)
            atomicAdd((unsigned long long*)&edge[i / p.piece], (unsigned long long)term_of(m));
        };
        if (sh.within <= kList) {
          for (int i = t; i < (int)sh.within; i += kThreads)
            add(raw_of(sh.inside[i]), (int)(sh.inside[i] & ((1u << kIndexBits) - 1)));
        } else {
          each_from(least_of(chosen_bin), add);
        }
        __syncthreads();
        // all pieces' totals first, then the one that passes the goal
        for (int pass = 0; pass < 2; ++pass) {
          uint64_t cursor = 0;
          for (int c = 0; c < p.pieces; ++c) {
            const int by = __builtin_amdgcn_readlane(down, c);
            const int bin = t - 16 * by;
            uint64_t v = 0;
            if (by < 64 && bin >= 0 && t < chosen_bin)
              v = shifted(((const uint64_t*)(records + c * p.record + kSumsAt))[bin], S - 40 + octave);
            uint64_t sum_c;
            block_scan(v, sh.qwaves, &sum_c);
            sum_c += shifted(edge[c], S - 40 + octave_of(chosen_bin));
            if (pass == 1 && (cursor + sum_c >= goal || c + 1 == p.pieces)) {
              offset = c * p.piece;
              ahead = cursor;
              break;
            }
            cursor += sum_c;
          }
          if (pass == 0) {
            total = cursor;
            goal = share(set.u, total, false) + 1;
          }
        }
        piece.at = row.at + offset;
        piece.n = min(p.piece, p.vocab - offset);
      }
      __syncthreads();
      uint64_t* const parts = sh.list;  // list and inside: 2 kList
      const int stripes = piece.stripes(), all = stripes * kWaves;
      for (int s = 0; s < stripes; ++s) {
        const u4v w = piece.word(s);
        uint64_t sum_s = 0;
        const int i0 = piece.first(s);
        uint32_t some = 0;
#pragma unroll
        for (int e = 0; e < P::kPer; ++e) some |= (T::wide(P::element(w, e)) >= least) << e;
        for (; some; some &= some - 1) {
          const int e = __builtin_ctz(some);
          if (i0 + e < piece.n) sum_s += kept_weight(P::any(w, e), offset + i0 + e);
        }
        sum_s = wave_sum(sum_s);
        if (lane == 0) parts[s * kWaves + wave] = sum_s;
      }
      __syncthreads();
      const int each = (all + kThreads - 1) / kThreads;
      uint64_t sum_t = 0, here;
      for (int j = 0; j < each; ++j)
        if (t * each + j < all) sum_t += parts[t * each + j];
      const uint64_t up = block_scan(sum_t, sh.qwaves, &here);
      if (!by_bins) {
        total = here;
        goal = share(set.u, total, false) + 1;
      }
      uint64_t rest = goal - ahead;
      if (rest > here) rest = here;
      if (t == 0) sh.found = 0;
      __syncthreads();
      if (sum_t && up >= rest && up - sum_t < rest) {
        sh.found = t;
        sh.found_sum = up - sum_t;
      }
      __syncthreads();
      uint64_t before = sh.found_sum;
      int part = sh.found * each;
      for (; part + 1 < all; ++part) {
        const uint64_t v = parts[part];
        if (before + v >= rest) break;
        before += v;
      }
      pick(piece, part / kWaves, part % kWaves, rest - before, offset,
           [&](Raw raw, int i) { return kept_weight(raw, offset + i); });
    }
  }
  if (owner_token >= 0) {
    p.tokens[r] = owner_token;
    // log(w / total): the kept weights' total is measured from the top, as is the largest
    if (p.logprobs)
      p.logprobs[r] = (float)(((double)owner_value - scale.ref) / (double)set.temperature +
                              scale.shift * (0.69314718055994530942 / kSteps) -
                              (log((double)total) - S * 0.69314718055994530942));
  }
}

// ------------------------------------------------------------------ host side

int check_sample(const lutgemm_sample* s) {
  if (!s) return LUTGEMM_ERR_NULL;
  if (s->type != LUTGEMM_F16 && s->type != LUTGEMM_BF16 && s->type != LUTGEMM_F32)
    return LUTGEMM_ERR_SHAPE;
  if (s->rows < 0 || s->rows >= (1 << 22) || s->vocab < 1 || s->vocab > kMostTokens)
    return LUTGEMM_ERR_SHAPE;
  if (s->row_step < 0 || s->row_step >= ((int64_t)1 << 40)) return LUTGEMM_ERR_SHAPE;
  return LUTGEMM_OK;
}

struct SamplePlan {
  int pieces, piece, parts, slab;  // slab: rows of one launch
  size_t ws_bytes;
};

SamplePlan plan(const lutgemm_sample* s) {
  SamplePlan r{};
  const int vocab = s->vocab, per = s->type == LUTGEMM_F32 ? 4 : 8;
  const int full = kStripes * kThreads * per, least = (vocab + full - 1) / full;
  const int most = (vocab + kLeastPiece - 1) / kLeastPiece;
  int pieces = s->rows ? (512 + s->rows - 1) / s->rows : 1;
  pieces = pieces > most ? most : pieces;
  pieces = pieces < least ? least : pieces;
  pieces = pieces > kMostPieces ? kMostPieces : pieces;
  r.piece = ((vocab + pieces - 1) / pieces + 7) / 8 * 8;
  r.pieces = (vocab + r.piece - 1) / r.piece;
  r.parts = (r.piece + kThreads * per - 1) / (kThreads * per) * kWaves;
  r.slab = 4096 / r.pieces;
  if (r.slab > s->rows) r.slab = s->rows;
  r.ws_bytes = (size_t)r.slab * r.pieces * kRecord;
  return r;
}

template <class T>
int run_sample(SampleParams p, int slab, hipStream_t stream) {
  const int rows = p.rows;
  for (int r = 0; r < rows; r += slab) {
    p.rows = rows - r < slab ? rows - r : slab;
    int st = launch(chunk_kernel<T>, dim3((unsigned)(p.rows * p.pieces)), kThreads, p, stream);
    if (!st) st = launch(row_kernel<T>, dim3((unsigned)p.rows), kThreads, p, stream);
    if (st) return st;
    p.logits = (const typename T::Raw*)p.logits + slab * p.row_step;
    p.u += slab;
    if (p.temperature) p.temperature += slab;
    if (p.top_k) p.top_k += slab;
    if (p.top_p) p.top_p += slab;
    if (p.min_p) p.min_p += slab;
    p.tokens += slab;
    if (p.logprobs) p.logprobs += slab;
  }
  return LUTGEMM_OK;
}

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_sample_tokens_workspace(const lutgemm_sample* s, size_t* bytes) {
  const int st = check_sample(s);
  if (st) return st;
  if (!bytes) return LUTGEMM_ERR_NULL;
  *bytes = plan(s).ws_bytes;
  return LUTGEMM_OK;
}

extern "C" int lutgemm_sample_tokens(const lutgemm_sample* s, const void* d_logits, const float* d_u,
                                     const float* d_temperature, const int32_t* d_top_k,
                                     const float* d_top_p, const float* d_min_p, int64_t* d_tokens,
                                     float* d_logprobs, void* d_workspace, size_t workspace_bytes,
                                     void* stream) {
  try {
    int st = check_sample(s);
    if (st) return st;
    if (s->rows == 0) return LUTGEMM_OK;
    if (!d_logits || !d_u || !d_tokens || !d_workspace) return LUTGEMM_ERR_NULL;
    if (!aligned(d_logits, s->type == LUTGEMM_F32 ? 4 : 2) || !aligned(d_u, 4) ||
        !aligned(d_temperature, 4) || !aligned(d_top_k, 4) || !aligned(d_top_p, 4) ||
        !aligned(d_min_p, 4) || !aligned(d_tokens, 8) || !aligned(d_logprobs, 4) ||
        !aligned(d_workspace, 16))
      return LUTGEMM_ERR_ALIGN;
    const SamplePlan r = plan(s);
    if (workspace_bytes < r.ws_bytes) return LUTGEMM_ERR_BUFFER;
    const int64_t rows = s->rows, size = s->type == LUTGEMM_F32 ? 4 : 2;
    const Flat all[] = {{d_tokens, 8 * rows},
                        {d_logprobs, 4 * rows},
                        {d_workspace, (int64_t)r.ws_bytes},
                        {d_logits, size * ((rows - 1) * s->row_step + s->vocab)},
                        {d_u, 4 * rows},
                        {d_temperature, 4 * rows},
                        {d_top_k, 4 * rows},
                        {d_top_p, 4 * rows},
                        {d_min_p, 4 * rows}};
    if (clash(all, 3)) return LUTGEMM_ERR_SHAPE;
    int cus = 0;
    st = serve::check_device(&cus);
    if (st) return st;
    SampleParams p{};
    p.logits = d_logits;
    p.u = d_u;
    p.temperature = d_temperature;
    p.top_k = d_top_k;
    p.top_p = d_top_p;
    p.min_p = d_min_p;
    p.tokens = d_tokens;
    p.logprobs = d_logprobs;
    p.ws = (char*)d_workspace;
    p.row_step = s->row_step;
    p.record = kRecord;
    p.rows = s->rows;
    p.vocab = s->vocab;
    p.pieces = r.pieces;
    p.piece = r.piece;
    p.parts = r.parts;
    int bits = 0;
    while ((1 << bits) < s->vocab) ++bits;
    p.scale = 62 - bits < 50 ? 62 - bits : 50;
    hipStream_t strm = (hipStream_t)stream;
    if (s->type == LUTGEMM_F32) return run_sample<F32>(p, r.slab, strm);
    if (s->type == LUTGEMM_F16) return run_sample<Logit16<serve::F16>>(p, r.slab, strm);
    return run_sample<Logit16<serve::BF16>>(p, r.slab, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
