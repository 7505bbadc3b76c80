// sample.hip -- next tokens from logits by temperature, top-k, top-p and min-p and one
// given random number a row (lutgemm_sample_tokens; the definition is in lutgemm.h).
//
// All three filters keep the first tokens of one order (value falling, index rising), so
// a row's kept tokens are those before one border: a value, and among the tokens that
// have it an index. Borders and the drawn token follow from sums of weights, and one
// of 100000 tokens whose sums are off by 2^-24 is the wrong one in 1 of 100 rows:
// weights are computed in 64 bits (2^(i/1024) from a table and a cubic polynomial), and
// sums by value are integers, exact and so the same in any order: a weight m 2^e,
// m in [1, 2], adds m 2^40 to the sum of its bin of a sixteenth of an octave. Tokens
// below 2^-64 of the largest weight count as none.
//
// One workgroup to a row.
#include <type_traits>

#include "serve.h"

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kSteps = 1024;       // table entries of an octave
constexpr int kBins = 1024;        // sixteenths of octaves below the largest weight
constexpr int kBytes = 256;        // values of one byte of a key
constexpr int kMaxStripes = 256;   // stripes of a row
constexpr int64_t kMostTokens = 1 << 20;

struct SampleParams {
  const void* logits;
  const float* u;
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  int64_t* tokens;
  float* logprobs;
  int64_t row_step;
  int32_t rows, vocab;
};

struct F32 {
  typedef uint32_t Raw;
  static constexpr int kKeyBits = 32;
  static __device__ __forceinline__ float wide(uint32_t a) { return __builtin_bit_cast(float, a); }
};
template <class T>
struct Logit16 : T {
  typedef uint16_t Raw;
  static constexpr int kKeyBits = 16;
};

// An integer that rises with the value; the zeros are equal.
template <class T>
__device__ __forceinline__ uint32_t key_of(typename T::Raw raw) {
  constexpr uint32_t sign = 1u << (T::kKeyBits - 1);
  uint32_t b = raw;
  if (b == sign) b = 0;
  return b & sign ? ~b & (sign | (sign - 1)) : b | sign;
}

struct Shared {
  double steps[kSteps];
  double part[kMaxStripes * kWaves];  // sums or counts by stripe and wave, in order of the tokens
  uint64_t sums[kBins];
  uint32_t counts[kBins];
  double dwaves[kWaves];
  uint64_t qwaves[kWaves];
  uint32_t waves[kWaves];
  int32_t found;
  uint32_t found_rest;
  uint64_t found_sum, found_passed, found_all;
  double found_before;
};

// 16 bytes at any element's address: rows of odd lengths lie anywhere.
typedef uint32_t WordOf4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t WordOf2 __attribute__((ext_vector_type(4), aligned(2)));

// A row's tokens, kPer to a thread and stripe: stripe s, thread t has tokens
// (s kThreads + t) kPer ...
template <class T>
struct Row {
  typedef typename T::Raw Raw;
  static constexpr int kPer = 16 / sizeof(Raw);
  const Raw* at;
  int vocab, stripes;
  __device__ __forceinline__ int first(int stripe) const {
    return (stripe * kThreads + (int)threadIdx.x) * kPer;
  }
  // f(raw, token) of each of the thread's tokens of a stripe
  template <class F>
  __device__ __forceinline__ void each(int stripe, F f) const {
    typedef typename std::conditional<sizeof(Raw) == 4, WordOf4, WordOf2>::type word;
    const int i0 = first(stripe);
    if (i0 + kPer <= vocab) {
      const word w = *(const word*)(at + i0);
#pragma unroll
      for (int e = 0; e < kPer; ++e)
        f((Raw)(sizeof(Raw) == 4 ? w[e * sizeof(Raw) / 4] : w[e * sizeof(Raw) / 4] >> (16 * (e & 1))),
          i0 + e);
    } else {
      for (int i = i0; i < vocab; ++i) f(at[i], i);
    }
  }
};

// 2^(y/1024) = m 2^e with m in [1, 2] but for rounding; y at most 0.
struct Weigher {
  double largest, scale;  // scale: 1024 log2(e) / temperature
  const double* steps;
  __device__ __forceinline__ double operator()(double x, int* k) const {
    constexpr double kRound = 0x1.8p52, c = 0.69314718055994530942 / kSteps;
    double y = (x - largest) * scale;
    y = y < -1e6 ? -1e6 : y;
    const double s = y + kRound;
    *k = (int)(uint32_t)__builtin_bit_cast(uint64_t, s);
    const double f = y - (s - kRound);
    const double p = __builtin_fma(
        f, __builtin_fma(f, __builtin_fma(f, c * c * c / 6, c * c / 2), c), 1.0);
    return steps[*k & (kSteps - 1)] * p;
  }
};

__device__ __forceinline__ double times_power(double m, int e) { return __builtin_ldexp(m, e); }

// The weight's term of a bin's sum.
__device__ __forceinline__ uint64_t term_of(double m) {
  constexpr double kUnit = 0x1p12;  // the last place of 2^12 + m is 2^-40
  return __builtin_bit_cast(uint64_t, m + kUnit) - __builtin_bit_cast(uint64_t, kUnit);
}

__device__ __forceinline__ int bin_of(int k) { return -(k >> 6); }

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

// Kept: keys above `key`, and of those equal to it the tokens up to `last`.
struct Border {
  uint32_t key;
  int last;
};

// The border behind which `rest` tokens or (by weight) a sum of `part` of the whole is
// reached, and the sum of all before it. The bins' counts or sums are in LDS.
template <class T, bool kByWeight>
__device__ Border find_border(const Row<T>& row, const Weigher& weigh, Shared& sh, uint32_t rest,
                              double target, double* kept) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  // the bin
  const uint64_t sum = sh.sums[t];
  const double mine = times_power((double)sum, ((-t) >> 4) - 40);
  double total;
  uint32_t all = 0, upto_count = 0;
  const double upto = block_scan(mine, sh.dwaves, &total);
  if (!kByWeight) upto_count = block_scan(sh.counts[t], sh.waves, &all);
  if (t == 0) sh.found = INT32_MAX;
  __syncthreads();
  if (sum && (kByWeight ? upto >= target : upto_count >= rest)) atomicMin(&sh.found, t);
  __syncthreads();
  const int bin = sh.found;
  if (bin == INT32_MAX) {  // fewer tokens, or by rounding less, than asked for: all of them
    *kept = total;
    return {0u, INT32_MAX};
  }
  if (t == bin) {
    sh.found_before = upto - mine;
    if (!kByWeight) sh.found_rest = rest - (upto_count - sh.counts[t]);
  }
  __syncthreads();
  const double before = sh.found_before;
  const int power = ((-bin) >> 4) - 40;  // of the bin's sums' unit
  uint64_t need = 0;                     // what is still to be reached inside the bin
  if (kByWeight) {
    const double units = __builtin_ceil(times_power(target - before, -power));
    need = units < 1.0 ? 1 : (uint64_t)units;
  } else {
    need = sh.found_rest;
  }
  // the value's key, a byte at a time
  uint32_t key = 0;
  uint64_t passed = 0;  // sums in the bin before the border
  for (int shift = T::kKeyBits - 8; shift >= 0; shift -= 8) {
    __syncthreads();
    if (t < kBytes) {
      sh.sums[t] = 0;
      sh.counts[t] = 0;
    }
    __syncthreads();
    for (int s = 0; s < row.stripes; ++s)
      row.each(s, [&](typename T::Raw raw, int) {
        const uint32_t mykey = key_of<T>(raw);
        if (shift + 8 < 32 && (mykey >> (shift + 8)) != (key >> (shift + 8))) return;
        int k;
        const double m = weigh((double)T::wide(raw), &k);
        if (bin_of(k) != bin) return;
        atomicAdd((unsigned long long*)&sh.sums[(mykey >> shift) & 255], (unsigned long long)term_of(m));
        atomicAdd(&sh.counts[(mykey >> shift) & 255], 1u);
      });
    __syncthreads();
    const int byte = kBytes - 1 - t;  // from the largest down
    const uint64_t v = t < kBytes ? (kByWeight ? sh.sums[byte] : (uint64_t)sh.counts[byte]) : 0;
    const uint64_t w = t < kBytes ? sh.sums[byte] : 0;
    uint64_t all_v, all_w;
    const uint64_t up = block_scan(v, sh.qwaves, &all_v);
    const uint64_t up_w = block_scan(w, sh.qwaves, &all_w);
    // by rounding the sum may end just below what is asked for: then the last one
    const uint64_t want = need < all_v ? need : all_v;
    if (v && up >= want && up - v < want) {
      sh.found = byte;
      sh.found_sum = up - v;
      sh.found_passed = up_w - w;
      sh.found_rest = sh.counts[byte];
      sh.found_all = w;
    }
    __syncthreads();
    key |= (uint32_t)sh.found << shift;
    need = want - sh.found_sum;
    passed += sh.found_passed;
  }
  // all that are left have this value; of those the first `many` in order
  const uint32_t equal = sh.found_rest;
  const uint64_t one = sh.found_all / (equal ? equal : 1);
  uint64_t many = need;
  if (kByWeight) many = one ? (need + one - 1) / one : 1;
  if (many < 1) many = 1;
  if (many > equal) many = equal;
  *kept = before + times_power((double)(passed + many * one), power);
  __syncthreads();
  uint32_t* counts = (uint32_t*)sh.part;
  for (int s = 0; s < row.stripes; ++s) {
    uint32_t n = 0;
    row.each(s, [&](typename T::Raw raw, int) { n += key_of<T>(raw) == key; });
    n = wave_sum(n);
    if (lane == 0) counts[s * kWaves + wave] = n;
  }
  if (t == 0) sh.found = INT32_MAX;
  __syncthreads();
  // the stripe and wave in which the border's token lies: each thread has four of the parts
  const int parts = row.stripes * kWaves;
  uint32_t four[4], sum4 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    four[i] = 4 * t + i < parts ? counts[4 * t + i] : 0;
    sum4 += four[i];
  }
  uint32_t ignored;
  uint32_t ahead = block_scan(sum4, sh.waves, &ignored) - sum4;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (four[i] && ahead < many && ahead + four[i] >= many) {
      sh.found = 4 * t + i;
      sh.found_rest = (uint32_t)many - ahead;
    }
    ahead += four[i];
  }
  __syncthreads();
  const int part = sh.found;
  const uint32_t nth = sh.found_rest;
  __syncthreads();
  if (part != INT32_MAX && wave == part % kWaves) {
    uint32_t n = 0;
    row.each(part / kWaves, [&](typename T::Raw raw, int) { n += key_of<T>(raw) == key; });
    uint32_t up = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t o = __shfl_up(up, d, 64);
      if (lane >= d) up += o;
    }
    uint32_t seen = up - n;
    if (seen < nth && up >= nth)
      row.each(part / kWaves, [&](typename T::Raw raw, int i) {
        if (key_of<T>(raw) == key && ++seen == nth) sh.found = i;
      });
  }
  __syncthreads();
  const int last = sh.found;
  __syncthreads();
  return {key, last};
}

template <class T>
__global__ __launch_bounds__(kThreads) void sample_kernel(SampleParams p) {
  __shared__ Shared sh;
  fetch(p);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t r = blockIdx.x;
  Row<T> row;
  row.at = (const typename T::Raw*)p.logits + r * p.row_step;
  row.vocab = p.vocab;
  row.stripes = (p.vocab + kThreads * Row<T>::kPer - 1) / (kThreads * Row<T>::kPer);
  const float u = p.u[r];
  const float temperature = p.temperature ? p.temperature[r] : 1.f;
  const float top_p = p.top_p ? p.top_p[r] : 1.f, min_p = p.min_p ? p.min_p[r] : 0.f;
  const int top_k = p.top_k ? p.top_k[r] : 0;

  // the largest value, and whether any is +infinity or NaN
  float most = -INFINITY;
  bool bad = !(u >= 0.f && u < 1.f) || !(temperature >= 0.f && temperature < INFINITY) ||
             top_p != top_p || min_p != min_p;
  for (int s = 0; s < row.stripes; ++s)
    row.each(s, [&](typename T::Raw raw, int) {
      const float x = T::wide(raw);
      bad |= !(x < INFINITY);
      most = fmaxf(most, x);
    });
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
  float* waves = (float*)sh.waves;
  if (lane == 0) waves[wave] = most;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int w = 0; w < kWaves; ++w) most = fmaxf(most, waves[w]);
  if (bad || most == -INFINITY) {
    if (t == 0) {
      p.tokens[r] = -1;
      if (p.logprobs) p.logprobs[r] = __builtin_nanf("");
    }
    return;
  }
  if (temperature == 0.f) {
    if (t == 0) sh.found = INT32_MAX;
    __syncthreads();
    int least = INT32_MAX;
    for (int s = 0; s < row.stripes; ++s)
      row.each(s, [&](typename T::Raw raw, int i) {
        if (T::wide(raw) == most && i < least) least = i;
      });
    if (least < INT32_MAX) atomicMin(&sh.found, least);
    __syncthreads();
    if (t == 0) {
      p.tokens[r] = sh.found;
      if (p.logprobs) p.logprobs[r] = 0.f;
    }
    return;
  }
  sh.steps[t] = exp2((double)t / kSteps);
  const Weigher weigh = {(double)most, kSteps * 1.4426950408889634074 / (double)temperature, sh.steps};
  sh.sums[t] = 0;
  sh.counts[t] = 0;
  __syncthreads();

  Border border = {0u, INT32_MAX};
  const bool by_count = top_k > 0 && top_k < p.vocab, by_weight = top_p < 1.f;
  if (by_count || by_weight) {
    auto fill = [&] {
      for (int s = 0; s < row.stripes; ++s)
        row.each(s, [&](typename T::Raw raw, int) {
          int k;
          const double m = weigh((double)T::wide(raw), &k);
          const int bin = bin_of(k);
          if (bin >= kBins) return;
          atomicAdd((unsigned long long*)&sh.sums[bin], (unsigned long long)term_of(m));
          atomicAdd(&sh.counts[bin], 1u);
        });
      __syncthreads();
    };
    fill();
    double kept;
    if (by_count) border = find_border<T, false>(row, weigh, sh, (uint32_t)top_k, 0.0, &kept);
    if (by_weight) {
      if (by_count) {
        __syncthreads();
        sh.sums[t] = 0;
        sh.counts[t] = 0;
        __syncthreads();
        fill();
      } else {
        const double mine = times_power((double)sh.sums[t], ((-t) >> 4) - 40);
        block_scan(mine, sh.dwaves, &kept);
      }
      // the token that has the largest value is always kept
      double target = (double)top_p * kept;
      if (!(target > 0.0)) target = 0x1p-60;
      double ignored;
      const Border second = find_border<T, true>(row, weigh, sh, 0u, target, &ignored);
      if (second.key > border.key || (second.key == border.key && second.last < border.last))
        border = second;
    }
  }
  // the kept weights in order of the tokens
  const double least = min_p > 0.f ? (min_p < 1.f ? (double)min_p : 1.0) : 0.0;
  auto weight = [&](typename T::Raw raw, int i) -> double {
    const uint32_t key = key_of<T>(raw);
    if (key < border.key || (key == border.key && i > border.last)) return 0.0;
    int k;
    const double m = weigh((double)T::wide(raw), &k);
    if (bin_of(k) >= kBins) return 0.0;
    const double w = times_power(m, k >> 10);
    return w >= least ? w : 0.0;
  };
  __syncthreads();
  for (int s = 0; s < row.stripes; ++s) {
    double sum = 0.0;
    row.each(s, [&](typename T::Raw raw, int i) { sum += weight(raw, i); });
    sum = wave_sum(sum);
    if (lane == 0) sh.part[s * kWaves + wave] = sum;
  }
  if (t == 0) sh.found = -1;
  __syncthreads();
  const int parts = row.stripes * kWaves;
  double four[4], sum4 = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    four[i] = 4 * t + i < parts ? sh.part[4 * t + i] : 0.0;
    sum4 += four[i];
  }
  double total;
  double ahead = block_scan(sum4, sh.dwaves, &total) - sum4;
  const double goal = (double)u * total;
  // the first part that passes the goal; rounding may leave none: then the last that has weight
  int mine = -1, fallback = -1;
  double mine_ahead = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (four[i] > 0.0) fallback = 4 * t + i;
    if (mine < 0 && four[i] > 0.0 && ahead <= goal && ahead + four[i] > goal) {
      mine = 4 * t + i;
      mine_ahead = ahead;
    }
    ahead += four[i];
  }
  if (t == 0) sh.found_rest = 0;
  __syncthreads();
  if (fallback >= 0) atomicMax(&sh.found, fallback);
  if (mine >= 0) atomicMax(&sh.found_rest, (uint32_t)(0x7FFFFFFF - mine));
  __syncthreads();
  const bool passed = sh.found_rest != 0;
  const int part = passed ? 0x7FFFFFFF - (int)sh.found_rest : sh.found;
  if (mine == part) sh.found_before = mine_ahead;
  __syncthreads();
  const double before = passed ? sh.found_before : 0.0;
  if (wave != part % kWaves) return;
  // within the wave's tokens of the stripe
  double sum = 0.0;
  row.each(part / kWaves, [&](typename T::Raw raw, int i) { sum += weight(raw, i); });
  double up = sum;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double o = __shfl_up(up, d, 64);
    if (lane >= d) up += o;
  }
  double cursor = before + (up - sum);
  int token = -1, last = -1;
  double chosen = 0.0, last_weight = 0.0;
  row.each(part / kWaves, [&](typename T::Raw raw, int i) {
    const double w = weight(raw, i);
    cursor += w;
    if (w > 0.0) {
      last = i;
      last_weight = w;
      if (token < 0 && passed && cursor > goal) {
        token = i;
        chosen = w;
      }
    }
  });
  const uint64_t have = __ballot(token >= 0), some = __ballot(last >= 0);
  const int owner = have ? __builtin_ctzll(have) : 63 - __builtin_clzll(some);
  if (lane != owner) return;
  if (!have) {
    token = last;
    chosen = last_weight;
  }
  p.tokens[r] = token;
  if (p.logprobs) p.logprobs[r] = (float)(log(chosen) - log(total));
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

}  // namespace
}  // namespace lutgemm

using namespace lutgemm;

extern "C" int lutgemm_sample_tokens(const lutgemm_sample* s, const void* d_logits, const float* d_u,
                                     const float* d_temperature, const int32_t* d_top_k,
                                     const float* d_top_p, const float* d_min_p, int64_t* d_tokens,
                                     float* d_logprobs, void* stream) {
  try {
    int st = check_sample(s);
    if (st) return st;
    if (s->rows == 0) return LUTGEMM_OK;
    if (!d_logits || !d_u || !d_tokens) return LUTGEMM_ERR_NULL;
    if (!aligned(d_logits, s->type == LUTGEMM_F32 ? 4 : 2) || !aligned(d_u, 4) ||
        !aligned(d_temperature, 4) || !aligned(d_top_k, 4) || !aligned(d_top_p, 4) ||
        !aligned(d_min_p, 4) || !aligned(d_tokens, 8) || !aligned(d_logprobs, 4))
      return LUTGEMM_ERR_ALIGN;
    const int64_t rows = s->rows, size = s->type == LUTGEMM_F32 ? 4 : 2;
    const Flat all[] = {{d_tokens, 8 * rows},
                        {d_logprobs, 4 * rows},
                        {d_logits, size * ((rows - 1) * s->row_step + s->vocab)},
                        {d_u, 4 * rows},
                        {d_temperature, 4 * rows},
                        {d_top_k, 4 * rows},
                        {d_top_p, 4 * rows},
                        {d_min_p, 4 * rows}};
    if (clash(all, 2)) return LUTGEMM_ERR_SHAPE;
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
    p.row_step = s->row_step;
    p.rows = s->rows;
    p.vocab = s->vocab;
    const dim3 grid((unsigned)s->rows);
    hipStream_t strm = (hipStream_t)stream;
    if (s->type == LUTGEMM_F32) return launch(sample_kernel<F32>, grid, kThreads, p, strm);
    if (s->type == LUTGEMM_F16)
      return launch(sample_kernel<Logit16<serve::F16>>, grid, kThreads, p, strm);
    return launch(sample_kernel<Logit16<serve::BF16>>, grid, kThreads, p, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
