// sample.hip -- next tokens from logits by temperature, top-k, top-p and min-p and one
// given random number a row (lutgemm_sample_tokens; the definition is in lutgemm.h).
//
// All three filters keep the first tokens of one order (value falling, index rising), so
// a row's kept tokens are those before one border: a value, and among the tokens that
// have it an index. Borders and the drawn token follow from sums of weights, and of
// 100000 tokens whose sums are off by 2^-24 the wrong one is taken in 1 of 100 rows. So
// weights are computed in 64 bits, 2^y = m 2^e with m from a table of 2^(i/32), which lies across
// the LDS banks once, and a polynomial, and rounded once, to 41 bits. Their sums are
//   by value   m 2^40 as integers, in bins of a sixteenth of an octave, where the bin tells e:
//              exact, and the same in any order
//   by place   over the up to 512 tokens of a part (a wave's word of a stripe) in 64-bit
//              floating point, always in one order and exact where the weights are equal; parts
//              are summed as integers, 2^S of the largest weight, S = min(50, 62 - log2(vocab))
//   of a list  as integers, 2^50 of the largest weight
// Tokens below 2^-63 of the largest weight count as none.
//
// chunk_kernel takes a piece of a row to each workgroup and holds it in registers: its
// largest value, and relative to that (brought up to a whole octave, so that the
// pieces' bins and sums are each other's but for shifts) what the row's settings ask for:
// the sums of the bins (top_p, large top_k), the numbers of tokens in them (top_k), or the
// sums of the parts (no filter). row_kernel, a workgroup to each row, joins them, finds the bin
// of the border, reads the row once more for the tokens of this bin and the ones above, and
// ends on these in LDS where they are few (a radix select by weight, on codes of value
// and index, then on the index); where they are many, the bins' sums say in which piece the
// drawn token lies, and only that is weighed again.
//
// Measured (bf16, 256 rows of 131073, top_p; 67 MB, 10 us at a streaming read's rate): 80 us;
// fp16, 1 row of 50272 27 us, 48 rows of 32000 of all kinds 31; fp32, 61 rows of 128001
// without a filter 20. The kernels say what bounds each; their own times are a trace's, in which
// the two of a call sum to up to 4 us more than calls in a row take.
#include <algorithm>
#include <type_traits>

#include "serve.h"

// A weight has the same bits wherever it is computed, and Scale's two parts of a product are
// its parts: products and sums are joined only where this is written.
#pragma clang fp contract(off)

namespace lutgemm {
namespace {

using namespace serve;

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kSteps = 32;         // table entries of an octave
constexpr int kBins = 1024;        // sixteenths of octaves below a piece's top
constexpr int kOctaves = kBins / 16;
constexpr int kListUnit = 50;      // weights of a list: 2^50 m 2^e
constexpr int kList = 4096;        // tokens of a list
constexpr int kMine = kList / kThreads;
constexpr int kStripes = 5;        // words of 16 bytes of a piece that a thread holds at most
constexpr int kAhead = 4;          // words whose loads are under way
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
  int64_t row_step;
  int32_t vocab, pieces, piece, parts, scale;  // parts: of a piece; scale: S
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

// `n` tokens of a row: stripes of kThreads words of kPer tokens.
template <class T>
struct Piece {
  typedef typename T::Raw Raw;
  static constexpr int kPer = 16 / sizeof(Raw);
  __amdgpu_buffer_rsrc_t at;
  int n, lead;
  // Loads are of whole aligned words of 4 bytes, so a piece at an odd 2-byte address begins with
  // the element before it, `lead` of them, and one of an odd end ends with the element behind:
  // these lie in the aligned words of its own and count as -infinity, as does all
  // that is behind (buffer loads give zeros there).
  __device__ __forceinline__ Piece(const Raw* from, int count) {
    lead = sizeof(Raw) == 2 && ((uintptr_t)from & 2) ? 1 : 0;
    n = count + lead;
    at = __builtin_amdgcn_make_buffer_rsrc((void*)(from - lead), 0, (n * (int)sizeof(Raw) + 3) & ~3, 0x00027000);
  }
  __device__ __forceinline__ int stripes() const { return (n + kThreads * kPer - 1) / (kThreads * kPer); }
  // those in which the wave has tokens
  __device__ __forceinline__ int wave_stripes() const {
    const int at = __builtin_amdgcn_readfirstlane((int)threadIdx.x & ~63) * kPer;
    return n > at ? (n - at + kThreads * kPer - 1) / (kThreads * kPer) : 0;
  }
  __device__ __forceinline__ int first(int stripe) const {
    return (stripe * kThreads + (int)threadIdx.x) * kPer;
  }
  // the token of an element that is one: from 0 on
  __device__ __forceinline__ int token(int element) const { return element - lead; }
  __device__ __forceinline__ bool is_token(int element) const { return element >= lead && element < n; }
  // The thread's word of a stripe as it is loaded, and with -infinity for what is no token.
  __device__ __forceinline__ u4v load(int stripe) const {
    return __builtin_bit_cast(
        u4v, __builtin_amdgcn_raw_buffer_load_b128(at, first(stripe) * (int)sizeof(Raw), 0, 0));
  }
  __device__ __forceinline__ void place(u4v& w, int stripe) const {
    const int i = first(stripe);
    if (i + kPer <= n && i >= lead) return;
    constexpr int each = 4 / sizeof(Raw);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (each == 1) {
        w[j] = is_token(i + j) ? w[j] : T::kNone;
      } else {
        const uint32_t lo = is_token(i + 2 * j) ? w[j] & 0xFFFF : T::kNone;
        const uint32_t hi = is_token(i + 2 * j + 1) ? w[j] >> 16 : T::kNone;
        w[j] = hi << 16 | lo;
      }
    }
  }
  __device__ __forceinline__ u4v word(int stripe) const {
    u4v w = load(stripe);
    place(w, stripe);
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
// `ref`, whose own distance from it is `shift` in 32nds of an octave.
struct Scale {
  double ref, step, shift, top;
  float least;  // values below it have no weight: they are kOctaves + 1 octaves below the top
  __device__ __forceinline__ void set(float largest, float temperature) {
    const double octaves = 1.4426950408889634074 / (double)temperature;
    ref = (double)largest;
    step = octaves * kSteps;
    const double p = ref * octaves;  // below: p and what its rounding took
    if (__builtin_fabs(p) < 0x1p40) {
      top = __builtin_ceil(p);
      shift = ((p - top) + __builtin_fma(ref, octaves, -p)) * kSteps;
    } else {  // other values are more than 64 octaves away
      top = p;
      shift = 0.0;
    }
    const double x = ref + (-kSteps * (kOctaves + 1.0) - shift) / step;
    least = (float)x;
    if ((double)least < x) least = up(least);
  }
  static __device__ __forceinline__ float up(float x) {  // the next float
    const int32_t b = __builtin_bit_cast(int32_t, x);
    return x == 0.f ? 1e-45f : __builtin_bit_cast(float, b + (b >= 0 ? 1 : -1));
  }
  // The weight of a value from `least` to ref is m 2^(k >> 5), m in [1, 2] but for rounding, and
  // m = a b. 2^x by its Taylor polynomial with the fifth term, x^5 c^5 / 120, taken as the
  // nearest lower powers on |x| <= 1/2: off by 2^-43 at most.
  __device__ __forceinline__ void factors(double x, const double* steps, int* k, double* a,
                                          double* b) const {
    constexpr double kRound = 0x1.8p52, c = 0.69314718055994530942 / kSteps;
    constexpr double c5 = c * c * c * c * c / 120;
    const double y = __builtin_fma(x - ref, step, shift);
    const double s = y + kRound;
    *k = (int)(uint32_t)__builtin_bit_cast(uint64_t, s);
    const double f = y - (s - kRound);
    double p = __builtin_fma(f, c * c * c * c / 24, c * c * c / 6 + 0.3125 * c5);
    p = __builtin_fma(f, p, c * c / 2);
    p = __builtin_fma(f, p, c - 0.01953125 * c5);
    *a = __builtin_fma(f, p, 1.0);
    *b = steps[*k & (kSteps - 1)];
  }
  // In its bin's sum: m 2^40.
  static __device__ __forceinline__ uint64_t by_term(double a, double b) {
    constexpr double kUnit = 0x1p12;  // the last place of 2^12 + m is 2^-40
    return __builtin_bit_cast(uint64_t, __builtin_fma(a, b, kUnit)) - __builtin_bit_cast(uint64_t, kUnit);
  }
  __device__ __forceinline__ uint64_t term(double x, const double* steps, int* k) const {
    double a, b;
    factors(x, steps, k, &a, &b);
    return by_term(a, b);
  }
  // In the sum of a part: m 2^e, m of 41 bits, so that sums of equal weights are exact.
  static __device__ __forceinline__ double by_value(double a, double b, int k) {
    constexpr double kUnit = 0x1p12;
    return __builtin_ldexp(__builtin_fma(a, b, kUnit) - kUnit, k >> 5);
  }
  // In the unit of a list.
  __device__ __forceinline__ uint64_t listed(double x, const double* steps) const {
    constexpr double kOne = 0x1p52;
    double a, b;
    int k;
    factors(x, steps, &k, &a, &b);
    return __builtin_bit_cast(uint64_t, __builtin_ldexp(by_value(a, b, k), kListUnit) + kOne) -
           __builtin_bit_cast(uint64_t, kOne);
  }
  __device__ __forceinline__ double weight(double x, const double* steps, int* k) const {
    double a, b;
    factors(x, steps, k, &a, &b);
    return a * __builtin_ldexp(b, *k >> 5);
  }
};

// Sixteenths of octaves below the top, and the octave of such a bin.
__device__ __forceinline__ int bin_of(int k) { return -(k >> 1); }
__device__ __forceinline__ int octave_of(int bin) { return (-bin) >> 4; }

// v 2^by, without what falls below 1.
__device__ __forceinline__ uint64_t shifted(uint64_t v, int by) {
  return by >= 64 || by <= -64 ? 0 : by >= 0 ? v << by : v >> -by;
}

// The largest whole number of at most a * v, a in [0, 1) or -0; `up`: the smallest of at least.
__device__ __forceinline__ uint64_t share(float a, uint64_t v, bool up) {
  const uint32_t bits = __builtin_bit_cast(uint32_t, a) & 0x7FFFFFFF;
  const int e = (int)(bits >> 23);
  const uint64_t m = e ? (bits & 0x7FFFFF) | 0x800000 : bits & 0x7FFFFF;
  const int down = 150 - (e ? e : 1);  // a = m 2^-down
  const unsigned __int128 product = (unsigned __int128)v * m;
  if (down >= 100) return up && product ? 1 : 0;
  const unsigned __int128 rest = up ? (((unsigned __int128)1) << down) - 1 : 0;
  return (uint64_t)((product + rest) >> down);
}

// v of the lane that a DPP control names, 0 where there is none.
template <int Control, int Rows, class V>
__device__ __forceinline__ V from_lane(V v) {
  if constexpr (sizeof(V) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, Control, Rows, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), Control, Rows, 0xF, false);
    return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(
        V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), Control, Rows, 0xF, false));
  }
}

// Sums of the lanes up to this one: within rows of sixteen, then of the rows before.
template <class V>
__device__ __forceinline__ V wave_scan(V v) {
  v += from_lane<0x111, 0xF>(v);
  v += from_lane<0x112, 0xF>(v);
  v += from_lane<0x114, 0xF>(v);
  v += from_lane<0x118, 0xF>(v);
  v += from_lane<0x142, 0xA>(v);  // row 0's into 1, 2's into 3
  v += from_lane<0x143, 0xC>(v);  // row 1's into 2 and 3
  return v;
}

template <class V>
__device__ __forceinline__ V lane_of(V v, int lane) {  // the lane is the same for the wave
  if constexpr (sizeof(V) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)b, lane);
    const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), lane);
    return __builtin_bit_cast(V, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(V, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  }
}

// The bits that any lane has. (One atomic of each lane on one word instead: 5 us for 1024.)
__device__ __forceinline__ uint64_t wave_or(uint64_t v) {
  v |= from_lane<0x111, 0xF>(v);
  v |= from_lane<0x112, 0xF>(v);
  v |= from_lane<0x114, 0xF>(v);
  v |= from_lane<0x118, 0xF>(v);
  v |= from_lane<0x142, 0xA>(v);
  v |= from_lane<0x143, 0xC>(v);
  return lane_of(v, 63);
}

template <class V>
__device__ __forceinline__ V wave_sum(V v) {
  return lane_of(wave_scan(v), 63);
}

// A wave's part of block_scan, before and after its sums are in LDS.
template <class V>
__device__ __forceinline__ V scan_join(V v, const V* waves, V* total) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  V sums = lane < kWaves ? waves[lane] : V(0);
  sums = wave_scan(sums);
  *total = lane_of(sums, 63);
  return wave ? v + lane_of(sums, wave - 1) : v;
}

// Sums of the threads before this one and itself, in order; *total: of all.
template <class V>
__device__ __forceinline__ V block_scan(V v, V* waves, V* total) {
  v = wave_scan(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) waves[threadIdx.x >> 6] = v;
  __syncthreads();
  return scan_join(v, waves, total);
}

// Of two values at once.
template <class V, class W>
__device__ __forceinline__ void block_scan(V* v, V* v_waves, V* v_total, W* w, W* w_waves) {
  W ignored;
  *v = wave_scan(*v);
  *w = wave_scan(*w);
  __syncthreads();
  if ((threadIdx.x & 63) == 63) {
    v_waves[threadIdx.x >> 6] = *v;
    w_waves[threadIdx.x >> 6] = *w;
  }
  __syncthreads();
  *v = scan_join(*v, v_waves, v_total);
  *w = scan_join(*w, w_waves, &ignored);
}

// A row's settings, and what they make of it.
struct Settings {
  float u, temperature, top_p, min_p;
  int top_k;
  bool bad, by_count, by_weight, by_least;
  __device__ __forceinline__ Settings(const SampleParams& p, int64_t r) {
    // arrays that are not given are read as u: loads under a condition wait for one another
    auto or_u = [&](const float* a) { return a ? a : p.u; };
    const float t = or_u(p.temperature)[r], tp = or_u(p.top_p)[r], mp = or_u(p.min_p)[r];
    const int32_t tk = (p.top_k ? p.top_k : (const int32_t*)p.u)[r];
    u = p.u[r];
    temperature = p.temperature ? t : 1.f;
    top_p = p.top_p ? tp : 1.f;
    min_p = p.min_p ? mp : 0.f;
    top_k = p.top_k ? tk : 0;
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
  double top;     // of Scale::set(largest, temperature)
  float largest;
  int32_t bad, at, pad;  // at: greedy: the first token of the largest value
};
constexpr int kSumsAt = 64, kCountsAt = kSumsAt + kBins * 8, kPartsAt = kSumsAt;
constexpr int kRecord = kCountsAt + kBins * 4;

// Bound by instructions, for bins: 256 rows of 131073 37 us, of which 29 vector instructions a
// token, some of them in 64 bits, take 25; their LDS additions alone take 30 (4.7 M cycles of
// bank conflicts) and run beside them. Two or four tokens' table reads ahead of their additions: no
// faster; 6, 8 or 16 pieces to a row: 40, 44 and 60 us. Without a filter (61 rows of 128001 in 32
// bits) 15 us: 5 of reading, then 9 of 43 instructions a token, which cannot begin before the
// piece's largest value is known. A reference from the first tokens, raised where later ones pass it, in place of
// the piece in registers: 91.
template <class T>
__global__ __launch_bounds__(kThreads, 8) void chunk_kernel(SampleParams p) {
  typedef Piece<T> P;
  __shared__ __attribute__((aligned(256))) double steps[kSteps];
  // bin b is entry kLast - b; behind the bins there is room for values that have no weight
  constexpr int kLast = kBins + 31;
  __shared__ uint64_t sums[kLast + 1];
  __shared__ uint32_t counts[kLast + 1];
  __shared__ float waves[kWaves];
  __shared__ int32_t first;
  fetch(p);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t r = blockIdx.x / (unsigned)p.pieces;
  const int c = (int)(blockIdx.x % (unsigned)p.pieces);
  const int begin = c * p.piece;
  const P piece((const typename T::Raw*)p.logits + r * p.row_step + begin, min(p.piece, p.vocab - begin));
  const int stripes = piece.wave_stripes();
  u4v w[kStripes];
#pragma unroll
  for (int s = 0; s < kStripes; ++s)
    if (s < stripes) w[s] = piece.load(s);
  const Settings set(p, r);
  // while the loads are under way
  if (t < kSteps) steps[t] = exp2((double)t / kSteps);
  if (set.sums()) sums[kLast - t] = 0;
  if (set.counts()) counts[kLast - t] = 0;
  if (t == 0) first = INT32_MAX;
  float most = -INFINITY;
  bool bad = false;
#pragma unroll
  for (int s = 0; s < kStripes; ++s)
    if (s < stripes) {
      piece.place(w[s], s);
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) {
        const float x = T::wide(P::element(w[s], e));
        bad |= !(x < INFINITY);
        most = fmaxf(most, x);
      }
    }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) most = fmaxf(most, __shfl_xor(most, d, 64));
  if (lane == 0) waves[wave] = most;
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int v = 0; v < kWaves; ++v) most = fmaxf(most, waves[v]);
  char* const record = p.ws + (r * p.pieces + c) * kRecord;
  if (set.greedy()) {
    int least = INT32_MAX;
#pragma unroll
    for (int s = 0; s < kStripes; ++s)
      if (s < stripes)
#pragma unroll
        for (int e = 0; e < P::kPer; ++e) {
          const int i = piece.first(s) + e;
          if (T::wide(P::element(w[s], e)) == most && piece.is_token(i))
            least = min(least, piece.token(i));
        }
    if (least < INT32_MAX) atomicMin(&first, least);
    __syncthreads();
  }
  Scale scale;
  scale.set(most, set.temperature);
  if (t == 0) *(Head*)record = Head{scale.top, most, bad, begin + first, 0};
  if (set.bad || bad || set.greedy() || most == -INFINITY) return;
  if (set.places()) {
    double* const parts = (double*)(record + kPartsAt);
#pragma unroll
    for (int s = 0; s < kStripes; ++s) {
      if (s >= stripes) continue;
      double sum = 0.0;
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) {
        const float x = T::wide(P::element(w[s], e));
        double a, b;
        int k;
        scale.factors((double)x, steps, &k, &a, &b);
        sum += x >= scale.least ? Scale::by_value(a, b, k) : 0.0;
      }
      sum = wave_sum(sum);
      if (lane == 0) parts[s * kWaves + wave] = sum;
    }
    for (int s = stripes; s * kWaves < p.parts; ++s)
      if (lane == 0) parts[s * kWaves + wave] = 0.0;
    return;
  }
  auto fill = [&](auto with_sums, auto with_counts) {
#pragma unroll
    for (int s = 0; s < kStripes; ++s) {
      if (s >= stripes) continue;
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) {
        int k;
        const float x = T::wide(P::element(w[s], e));
        const uint64_t term = scale.term((double)x, steps, &k);
        const int at = x >= scale.least ? kLast - bin_of(k) : 0;
        if (with_sums) atomicAdd((unsigned long long*)&sums[at], (unsigned long long)term);
        if (with_counts) atomicAdd(&counts[at], 1u);
      }
    }
  };
  constexpr std::true_type yes;
  constexpr std::false_type no;
  if (set.sums() && set.counts())
    fill(yes, yes);
  else if (set.sums())
    fill(yes, no);
  else if (set.counts())
    fill(no, yes);
  __syncthreads();
  if (set.sums()) ((uint64_t*)(record + kSumsAt))[t] = sums[kLast - t];
  if (set.counts()) ((uint32_t*)(record + kCountsAt))[t] = counts[kLast - t];
}

// ------------------------------------------------------------------ rows

struct RowShared {
  double steps[kSteps];   // first: across the banks once
  uint64_t list[kList];   // indices, codes, the pieces' lanes' sums or the parts' sums
  uint64_t sums[2][256];
  uint64_t counts[2][256];
  uint64_t qwaves[kWaves];
  uint32_t waves[kWaves];
  uint64_t found_sum, found_code, found_rest, ones, zeros;
  int32_t found, found_count;
  uint32_t listed;        // tokens of the list
};

// The first code, of those that `members` hands to its argument with a value (at least 1)
// each, up to which the values sum to `target` (at least 1), in the order of the codes;
// *before: the sum ahead of it. If the sum is less, the last code. By eight bits at a time,
// from the highest in which codes differ, until one code is left: wave 0 finds the byte
// while the others clear the sums of the next eight bits.
template <class Members>
__device__ __forceinline__ uint64_t select(RowShared& sh, uint64_t target, uint64_t* before, Members members) {
  const int t = threadIdx.x, lane = t & 63;
  uint64_t ones = 0, zeros = 0;
  members([&](uint64_t code, uint64_t) {
    ones |= code;
    zeros |= ~code;
  });
  __syncthreads();
  if (t == 0) sh.ones = sh.zeros = 0;
  if (t < 256) sh.sums[0][t] = sh.counts[0][t] = 0;
  __syncthreads();
  ones = wave_or(ones);
  zeros = wave_or(zeros);
  if (lane == 0 && (ones | zeros)) {
    atomicOr((unsigned long long*)&sh.ones, (unsigned long long)ones);
    atomicOr((unsigned long long*)&sh.zeros, (unsigned long long)zeros);
  }
  __syncthreads();
  const uint64_t differ = sh.ones & sh.zeros;
  uint64_t prefix = sh.ones & sh.zeros ? 0 : sh.ones, passed = 0;
  if (!differ) {  // one code, or none
    __syncthreads();
    *before = 0;
    return prefix;
  }
  int shift = 64 - __builtin_clzll(differ);  // bits from here up are the same in all
  prefix = shift < 64 ? sh.ones >> shift : 0;
  int turn = 0;
  for (;;) {
    const int bits = min(shift, 8);
    shift -= bits;
    members([&](uint64_t code, uint64_t value) {
      const uint64_t high = code >> shift;
      if (high >> bits != prefix) return;
      const int byte = (int)high & ((1 << bits) - 1);
      atomicAdd((unsigned long long*)&sh.sums[turn][byte], (unsigned long long)value);
      atomicAdd((unsigned long long*)&sh.counts[turn][byte], 1ull);
    });
    __syncthreads();
    if (t >= 256 && t < 512) sh.sums[turn ^ 1][t - 256] = sh.counts[turn ^ 1][t - 256] = 0;
    if (t < 64) {
      uint64_t v[4], four = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = sh.sums[turn][4 * lane + i];
        four += v[i];
      }
      uint64_t up = wave_scan(four);
      const uint64_t all = lane_of(up, 63), want = target < all ? target : all;
      up -= four;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (v[i] && up < want && up + v[i] >= want) {
          sh.found = 4 * lane + i;
          sh.found_sum = up;
          sh.found_rest = want - up;
          sh.found_count = (int)sh.counts[turn][4 * lane + i];
        }
        up += v[i];
      }
    }
    __syncthreads();
    prefix = prefix << bits | (uint32_t)sh.found;
    passed += sh.found_sum;
    target = sh.found_rest;
    const bool one = sh.found_count == 1;
    if (shift == 0) break;
    if (one) {
      members([&](uint64_t code, uint64_t) {
        if (code >> shift == prefix) sh.found_code = code;
      });
      __syncthreads();
      prefix = sh.found_code;
      break;
    }
    turn ^= 1;
  }
  __syncthreads();
  *before = passed;
  return prefix;
}

// Bound by the latency of its steps, one row to a compute unit: 14 to 27 us for one row of 50272
// (heads and settings 1.8, bins 2.5, their sums 0.8, the border's bin 0.9, the list's tokens 5.4, their
// values 0.6, the select 2.8, the kept sums of the pieces 2.7, the parts of one 2.8, the token
// in one 2.9), 47 for 256 rows of 131073, whose second reading takes 7 to 13 (9 to 5 TB/s, by
// how many tokens it lists) and the weights of one piece 12. (A row in one workgroup from its
// first token on, one kernel: 185.) Scratch memory costs a launch of it: 240 bytes a lane 13 us,
// the 20 to 36 that are left none that shows.
template <class T>
__global__ __launch_bounds__(kThreads) void row_kernel(SampleParams p) {
  typedef Piece<T> P;
  typedef typename T::Raw Raw;
  constexpr uint32_t kKeyAll = T::kKeyBits == 32 ? ~0u : (1u << (T::kKeyBits & 31)) - 1;
  __shared__ __attribute__((aligned(256))) RowShared sh;
  fetch(p);
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t r = blockIdx.x;
  const char* const records = p.ws + r * p.pieces * kRecord;
  // the pieces' heads, one to a lane
  Head head = *(const Head*)(records + min(lane, p.pieces - 1) * kRecord);
  const Settings set(p, r);
  if (t < kSteps) sh.steps[t] = exp2((double)t / kSteps);  // while they are under way
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
  Scale scale;
  scale.set(most, set.temperature);
  // octaves of the pieces' tops below the row's, 64 for those without weight
  const double lower = scale.top - head.top;
  const int down = head.largest > -INFINITY && lower < 64.0 ? (int)lower : 64;
  const int S = p.scale;
  const Raw* const logits = (const Raw*)p.logits + r * p.row_step;
  const P row(logits, p.vocab);

  int owner_token = -1;   // of the thread that has found the token
  float owner_value = 0.f;
  uint64_t total = 0;     // of the kept weights, in units of 2^-unit
  int unit = S;

  // Of a part's tokens, by one wave: the first one up to which their weights sum to more than
  // `goal`; the last that has weight if rounding leaves none.
  auto pick = [&](const P& piece, int part, double goal, int offset, auto weight) {
    if (wave != part % kWaves) return;
    const u4v w = piece.word(part / kWaves);
    const int i0 = piece.first(part / kWaves);
    double v[P::kPer], sum = 0.0;
#pragma unroll
    for (int e = 0; e < P::kPer; ++e) {
      v[e] = piece.is_token(i0 + e) ? weight(P::element(w, e), piece.token(i0 + e)) : 0.0;
      sum += v[e];
    }
    double cursor = wave_scan(sum) - sum;
    int token = -1, last = -1;
    float value = 0.f, last_value = 0.f;
#pragma unroll
    for (int e = 0; e < P::kPer; ++e) {
      cursor += v[e];
      if (!(v[e] > 0.0)) continue;
      last = piece.token(i0 + e);
      last_value = T::wide(P::element(w, e));
      if (token < 0 && cursor > goal) {
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
  // A part's sum in the unit 2^-S of the row's top, `by` octaves above the piece's.
  auto in_units = [&](double v, int by) { return (uint64_t)__builtin_rint(__builtin_ldexp(v, S - by)); };

  if (set.places()) {
    // parts in order, a few to a thread
    const int all = p.pieces * p.parts, each = (all + kThreads - 1) / kThreads;
    auto part_at = [&](int i) -> uint64_t {
      const int at = min(i, all - 1), c = at / p.parts;
      const int by = __shfl(down, c, 64);  // by all lanes
      if (i >= all || by >= 64) return 0;
      return in_units(((const double*)(records + c * kRecord + kPartsAt))[at % p.parts], by);
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
    const P piece(logits + c * p.piece, min(p.piece, p.vocab - c * p.piece));
    pick(piece, part % p.parts, __builtin_ldexp((double)(goal - 1 - before), by - S), c * p.piece,
         [&](Raw raw, int) {
           const float x = T::wide(raw);
           if (!(x >= own.least)) return 0.0;
           double a, b;
           int k;
           own.factors((double)x, sh.steps, &k, &a, &b);
           return Scale::by_value(a, b, k);
         });
  } else {
    // the row's first words are under way while the bins are joined
    u4v first[kAhead];
    auto first_words = [&](u4v (&w)[kAhead]) __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) w[a] = row.load(a);
    };
    first_words(first);
    // the bins of all pieces: sums in their own octave's unit and in 2^S
    uint64_t sum = 0;
    uint32_t count = 0;
    constexpr int kPieces = 8;  // whose loads are under way together
    for (int c0 = 0; c0 < p.pieces; c0 += kPieces) {
      uint64_t v[kPieces];
      uint32_t n[kPieces];
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int c = min(c0 + j, p.pieces - 1);
        const int bin = max(t - 16 * __builtin_amdgcn_readlane(down, c), 0);
        v[j] = 0;
        n[j] = 0;
        if (set.sums()) v[j] = ((const uint64_t*)(records + c * kRecord + kSumsAt))[bin];
        if (set.counts()) n[j] = ((const uint32_t*)(records + c * kRecord + kCountsAt))[bin];
      }
#pragma unroll
      for (int j = 0; j < kPieces; ++j) {
        const int by = __builtin_amdgcn_readlane(down, min(c0 + j, p.pieces - 1));
        if (c0 + j < p.pieces && by < 64 && t >= 16 * by) {
          sum += v[j];
          count += n[j];
        }
      }
    }
    const int octave = octave_of(t);
    const uint64_t mine = shifted(sum, S - 40 + octave);
    uint64_t all_sum = 0, upto = 0;
    uint32_t all_count = 0, upto_count = 0;
    float upto_bound = 0.f;
    if (set.counts()) upto_count = block_scan(count, sh.waves, &all_count);
    if (set.sums()) {
      // a bin's terms are its lower edge's 2^40 m or up to a sixteenth of an octave more, so
      // their sum bounds their number
      upto = mine;
      upto_bound = (float)sum * __builtin_amdgcn_exp2f(-40.f - (float)(-t & 15) * 0.0625f) * 1.01f + 1.f;
      block_scan(&upto, sh.qwaves, &all_sum, &upto_bound, (float*)sh.waves);
    }

    // the bin of the thread that says so, which leaves what `then` writes; kBins if none does
    auto bin_where = [&](bool here, auto then) {
      __syncthreads();
      if (t == 0) sh.found = kBins;
      __syncthreads();
      if (here) {
        sh.found = t;
        then();
      }
      __syncthreads();
      return sh.found;
    };
    // a value that no token of the bins up to this one is below
    auto least_of = [&](double bin) {
      const double x = scale.ref + (-2.0 * bin - 0.5 - scale.shift) / scale.step;
      return fmaxf((float)(x - 1e-6 * (__builtin_fabs(x) + __builtin_fabs(scale.ref)) - 1e-30),
                   -__FLT_MAX__);  // never -infinity
    };
    // a value that no token of this bin or a later one is above
    auto most_of = [&](int bin) {
      const double x = scale.ref + (-2.0 * bin + 1.5 - scale.shift) / scale.step;
      return bin == 0 ? INFINITY
                      : (float)(x + 1e-6 * (__builtin_fabs(x) + __builtin_fabs(scale.ref)) + 1e-30);
    };
    // a value's bin, kBins and more for those without weight; and its term
    auto bin_at = [&](Raw raw, uint64_t* term) {
      const float x = T::wide(raw);
      if (!(x >= scale.least)) return kBins;
      int k;
      *term = scale.term((double)x, sh.steps, &k);
      return bin_of(k);
    };
    // f(word, in, first element) of every word of a wave that has tokens from `least` to
    // `limit`; in[e]: whether the lane's element e is one
    auto words_from = [&](u4v (&w)[kAhead], float least, float limit, auto f) __attribute__((always_inline)) {
      const int stripes = row.wave_stripes();
      for (int s0 = 0; s0 < stripes; s0 += kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) {
          // loads behind the row's end give zeros: under a condition each is waited for at once
          u4v now = w[a];
          w[a] = row.load(s0 + a + kAhead);
          if (s0 + a >= stripes) continue;
          row.place(now, s0 + a);
          bool in[P::kPer], some = false;
#pragma unroll
          for (int e = 0; e < P::kPer; ++e) {
            const float x = T::wide(P::element(now, e));
            in[e] = x >= least && x <= limit;
            some |= in[e];
          }
          if (__any(some)) f(now, in, row.first(s0 + a));
        }
      }
    };
    auto each_word = [&](float least, float limit, auto f) __attribute__((always_inline)) {
      u4v w[kAhead];
      first_words(w);
      words_from(w, least, limit, f);
    };
    // that as one word
    auto bits_of = [&](const bool (&in)[P::kPer]) {
      uint32_t bits = 0;
#pragma unroll
      for (int e = 0; e < P::kPer; ++e) bits |= in[e] ? 1u << e : 0;
      return bits;
    };
    // f(raw, index) of every token from `least` to `limit`
    auto each_from = [&](float least, float limit, auto f) __attribute__((always_inline)) {
      each_word(least, limit, [&](const u4v& w, const bool (&in)[P::kPer], int i0) {
        for (uint32_t bits = bits_of(in); bits; bits &= bits - 1) {
          const int e = __builtin_ctz(bits);
          f(P::any(w, e), row.token(i0 + e));
        }
      });
    };
    // The list's tokens, each thread's: their codes, ~0 for none, and bins; whole: all had room.
    uint64_t code[kMine];
    int code_bin[kMine];
    bool whole = false;
    // The tokens from `least` to `limit`: by their indices first, where the words are read.
    auto gather = [&](u4v (&first)[kAhead], float least, float limit) __attribute__((always_inline)) {
      uint32_t* const list = (uint32_t*)sh.list;
      __syncthreads();
      if (t == 0) sh.listed = 0;
      __syncthreads();
      words_from(first, least, limit, [&](const u4v&, const bool (&in)[P::kPer], int i0) {
        uint32_t count = 0, at = 0;
#pragma unroll
        for (int e = 0; e < P::kPer; ++e) count += __popcll(__ballot(in[e]));
        if (lane == 0) at = atomicAdd(&sh.listed, count);
        uint32_t bits = bits_of(in);
        at = __builtin_amdgcn_readfirstlane(at);
        if (at + count > kList) return;
        for (uint64_t some; (some = __ballot(bits != 0)) != 0; bits &= bits - 1) {
          const uint32_t before = __builtin_amdgcn_mbcnt_hi(
              (uint32_t)(some >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)some, 0));
          if (bits) list[at + before] = (uint32_t)row.token(i0 + __builtin_ctz(bits));
          at += __popcll(some);
        }
      });
      __syncthreads();
      const uint32_t n = sh.listed;
      whole = n <= kList;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const uint32_t i = t + j * kThreads;
        code[j] = ~0ull;
        code_bin[j] = kBins;
        if (i < n && whole) {  // read again: codes written by the collecting lanes 3 us more
          uint64_t ignored;
          const Raw raw = logits[list[i]];
          code[j] = code_of<T>(raw, (int)list[i]);
          code_bin[j] = bin_at(raw, &ignored);
        }
      }
    };
    auto raw_of = [&](uint64_t code) {  // the bits of a code's value
      const uint32_t key = ~(uint32_t)(code >> kIndexBits) & kKeyAll;
      constexpr uint32_t sign = 1u << (T::kKeyBits - 1);
      return (Raw)(key & sign ? key & (sign - 1) : ~key & kKeyAll);
    };
    // Of a list that was written as codes.
    auto take_list = [&]() __attribute__((always_inline)) {
      __syncthreads();
      const uint32_t n = sh.listed;
      whole = n <= kList;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        const uint32_t i = t + j * kThreads;
        code[j] = i < n && whole ? sh.list[i] : ~0ull;
      }
      return whole;
    };
    // the border inside a bin: the code up to which its tokens' number or sum (in the
    // bin's unit) reaches `need`; after its tokens were gathered
    auto border_in = [&](int bin, bool weights, uint64_t need, uint64_t* before) __attribute__((always_inline)) {
      if (need < 1) need = 1;
      // a value between two bins may be rounded into the other here: without any, the largest alone
      auto or_largest = [&](uint64_t code) {
        uint32_t raw = __builtin_bit_cast(uint32_t, most);
        if constexpr (T::kKeyBits == 16) raw = T::one(most);
        return code ? code : code_of<T>((Raw)raw, (1 << kIndexBits) - 1);
      };
      if (whole) {
        uint64_t value[kMine];
#pragma unroll
        for (int j = 0; j < kMine; ++j) {
          value[j] = 0;
          if (code_bin[j] != bin) continue;
          value[j] = 1;
          if (weights) bin_at(raw_of(code[j]), &value[j]);
        }
        return or_largest(select(sh, need, before, [&](auto f) {
#pragma unroll
          for (int j = 0; j < kMine; ++j)
            if (value[j]) f(code[j], value[j]);
        }));
      }
      // more than the list takes, of nearly equal logits: the row again for each byte (256 rows of
      // 131073: 320 us at a temperature of 20, 620 if all are equal)
      const float least = least_of(bin), limit = most_of(bin);
      return or_largest(select(sh, need, before, [&](auto f) {
        each_from(least, limit, [&](Raw raw, int i) {
          uint64_t term;
          if (bin_at(raw, &term) == bin) f(code_of<T>(raw, i), weights ? term : 1);
        });
      }));
    };

    if (set.by_least) __syncthreads();  // with min_p alone nothing has waited yet for the steps
    const double floor_weight =  // of what min_p keeps
        set.by_least ? (double)(set.min_p < 1.f ? set.min_p : 1.f) : 0.0;
    int k;
    const double least_weight = floor_weight * scale.weight(scale.ref, sh.steps, &k);
    // whether the value has weight, and at least so much
    auto counted = [&](float x, double at_least) {
      if (!(x >= scale.least)) return false;
      int k;
      const double w = scale.weight((double)x, sh.steps, &k);
      return bin_of(k) < kBins && w >= at_least;
    };
    // the tokens from `least` on that `takes` says into the list, as codes
    auto collect = [&](float least, auto takes) __attribute__((always_inline)) {
      __syncthreads();
      if (t == 0) sh.listed = 0;
      __syncthreads();
      each_from(least, INFINITY, [&](Raw raw, int i) {
        if (sh.listed > kList || !takes(raw, i)) return;
        const uint32_t at = atomicAdd(&sh.listed, 1u);
        if (at < kList) sh.list[at] = code_of<T>(raw, i);
      });
      return take_list();
    };
    auto collect_counted = [&](float least, double at_least) __attribute__((always_inline)) {
      return collect(least, [&](Raw raw, int) { return counted(T::wide(raw), at_least); });
    };
    uint64_t border = ~0ull;  // kept: codes up to it
    bool listed = false;      // the kept tokens are among the list's
    int last_bin = kBins - 1;  // no kept token is behind this bin
    int chosen_bin = -1;      // the border is in this bin, whose tokens were gathered
    uint64_t available = all_sum;  // what top_p takes its part of
    if (set.by_count) {
      const uint32_t k = (uint32_t)set.top_k;
      const int bin = bin_where(upto_count >= k && upto_count - count < k, [&] {
        sh.found_count = (int)(upto_count - count);
        sh.found_sum = upto - mine;
      });
      if (bin == kBins) {  // fewer have weight: all of these
        if (set.few()) listed = collect_counted(least_of(kBins - 1), 0.0);
      } else {
        last_bin = bin;
        const uint64_t rest = (uint64_t)(set.top_k - sh.found_count);
        const uint64_t ahead = sh.found_sum;
        gather(first, least_of(bin), set.few() ? INFINITY : most_of(bin));
        listed = set.few() && whole;
        if (!listed) {
          uint64_t before;
          border = border_in(bin, false, rest, &before);
          chosen_bin = bin;
          if (set.few()) {  // of the bin only those up to the border
            listed = collect(least_of(bin), [&](Raw raw, int i) { return code_of<T>(raw, i) <= border; });
          } else {
            // the sum of what is kept: by weight up to the border's code
            uint64_t kept = 0;
            each_from(least_of(bin), most_of(bin), [&](Raw raw, int i) {
              uint64_t term;
              if (bin_at(raw, &term) == bin && code_of<T>(raw, i) <= border) kept += term;
            });
            uint64_t all;
            block_scan(kept, sh.qwaves, &all);
            available = ahead + shifted(all, S - 40 + octave_of(bin));
          }
        } else {
          uint64_t before;
          border = select(sh, (uint64_t)set.top_k, &before, [&](auto f) {
#pragma unroll
            for (int j = 0; j < kMine; ++j)
              if (code_bin[j] <= bin) f(code[j], 1);
          });
        }
      }
    }
    if (set.by_weight && !listed && set.sums()) {
      uint64_t target = set.top_p > 0.f ? share(set.top_p, available, true) : 1;
      if (target < 1) target = 1;
      // in the last bin that top_k leaves, if not before
      const bool passes = mine && upto >= target && upto - mine < target;
      const int bin = bin_where(t < last_bin ? passes : t == last_bin && upto - mine < target, [&] {
        sh.found_sum = upto - mine;
        sh.found_count = upto_bound < (float)kList;
      });
      last_bin = bin;
      const uint64_t ahead = sh.found_sum;
      const bool small = sh.found_count;
      if (set.by_count) first_words(first);
      gather(first, least_of(bin), small ? INFINITY : most_of(bin));
      const int by = 40 - octave_of(bin) - S;  // from 2^S to the bin's unit
      const uint64_t missing = target > ahead ? target - ahead : 1;
      const uint64_t need = by >= 0 ? shifted(missing, by) : (missing + (1ull << -by) - 1) >> -by;
      uint64_t before;
      const uint64_t second = border_in(bin, true, need, &before);
      if (second < border) {
        border = second;
        chosen_bin = bin;
      }
      listed = small && whole;
    }
    float least = least_of(last_bin);
    if (set.by_least) {
      const double bins = 17.0 - 16.0 * log2(floor_weight);  // the top is less than an octave higher
      if (bins < (double)last_bin) least = least_of(bins);
      if (!listed && !set.by_count && !set.by_weight) {
        listed = collect_counted(least, least_weight);
      }
    }
    // the weight of a token of at least `least` if it is kept, as a part sums it
    const float edge = border == ~0ull ? least : T::wide(raw_of(border));
    const int edge_last = border == ~0ull ? INT32_MAX : (int)(border & ((1u << kIndexBits) - 1));
    auto kept_value = [&](float x, int i) __attribute__((always_inline)) {
      int k;
      double a, b;
      scale.factors((double)x, sh.steps, &k, &a, &b);
      bool kept = x > edge || (x == edge && i <= edge_last);
      if (border == ~0ull) kept = kept && x >= scale.least && bin_of(k) < kBins;
      if (set.by_least) kept = kept && a * __builtin_ldexp(b, k >> 5) >= least_weight;
      return kept ? Scale::by_value(a, b, k) : 0.0;
    };
    if (listed) {
      unit = kListUnit;
      uint64_t weight[kMine], sum = 0;
#pragma unroll
      for (int j = 0; j < kMine; ++j) {
        weight[j] = 0;
        if (code[j] <= border && code[j] != ~0ull && counted(T::wide(raw_of(code[j])), least_weight))
          weight[j] = scale.listed((double)T::wide(raw_of(code[j])), sh.steps);
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
            uint64_t term;
            if (bin_at(raw_of(code[j]), &term) < kBins)
              plain[j] = scale.listed((double)T::wide(raw_of(code[j])), sh.steps);
          }
          whole_sum += plain[j];
        }
        uint64_t all;
        block_scan(whole_sum, sh.qwaves, &all);
        uint64_t target = set.top_p > 0.f ? share(set.top_p, all, true) : 1;
        if (target < 1) target = 1;
        border = select(sh, target, &before, [&](auto f) {
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
      const uint64_t token = select(sh, goal, &before, [&](auto f) {
#pragma unroll
        for (int j = 0; j < kMine; ++j)
          if (weight[j]) f(code[j] & ((1u << kIndexBits) - 1), weight[j]);
      });
      if (t == 0) {
        owner_token = (int)token;
        owner_value = T::wide(logits[token]);
      }
    } else {
      // the piece in which the token lies, by the bins' sums; then its parts
      P piece = row;
      int offset = 0;
      uint64_t ahead = 0, goal = 0;
      bool by_bins = chosen_bin >= 0 && set.sums() && !set.by_least;
      if (by_bins) {
        // of each piece the sum of what is kept: the border's own tokens are added by themselves, each
        // lane to a word of its own (a wave's by piece 4 us more, all to one word 6), then
        // a wave adds a piece's bins before the border's
        uint64_t* const kept = sh.sums[0];
        uint64_t* const own = sh.list;  // [piece][lane]: of the border's bin
        static_assert(kMostPieces * 64 <= kList, "a word to each lane of each piece");
        __syncthreads();
        for (int i = t; i < 64 * p.pieces; i += kThreads) own[i] = 0;
        __syncthreads();
        auto add = [&](uint64_t term, int piece) {
          if (term) atomicAdd((unsigned long long*)&own[piece * 64 + lane], (unsigned long long)term);
        };
        auto kept_term = [&](uint64_t code) {
          uint64_t term = 0;
          return code <= border && bin_at(raw_of(code), &term) == chosen_bin ? term : 0ull;
        };
        if (whole) {
#pragma unroll
          for (int j = 0; j < kMine; ++j)
            if (code_bin[j] == chosen_bin)
              add(kept_term(code[j]), (int)(code[j] & ((1u << kIndexBits) - 1)) / p.piece);
        } else {
          each_word(least_of(chosen_bin), most_of(chosen_bin),
                    [&](const u4v& w, const bool (&in)[P::kPer], int i0) {
#pragma unroll
                      for (int e = 0; e < P::kPer; ++e) {
                        if (!in[e]) continue;
                        const int i = row.token(i0 + e);
                        add(kept_term(code_of<T>(P::element(w, e), i)), i / p.piece);
                      }
                    });
        }
        __syncthreads();
        for (int c = wave; c < p.pieces; c += kWaves) {
          const int by = __builtin_amdgcn_readlane(down, c);
          uint64_t v = 0;
          if (by < 64)
            for (int bin = lane + 16 * by; bin < chosen_bin; bin += 64)
              v += shifted(((const uint64_t*)(records + c * kRecord + kSumsAt))[bin - 16 * by],
                           S - 40 + octave_of(bin));
          v = wave_sum(v) + shifted(wave_sum(own[c * 64 + lane]), S - 40 + octave_of(chosen_bin));
          if (lane == 0) kept[c] = v;
        }
        __syncthreads();
        // the first piece that passes the goal
        uint64_t mine_c = 0;
        if (lane < p.pieces) mine_c = kept[lane];
        const uint64_t up = wave_scan(mine_c);
        total = lane_of(up, 63);
        goal = share(set.u, total, false) + 1;
        const uint64_t passes = __ballot(up >= goal && mine_c);
        const int c = passes ? __builtin_ctzll(passes) : p.pieces - 1;
        ahead = lane_of(up - mine_c, c);
        offset = c * p.piece;
        piece = P(logits + offset, min(p.piece, p.vocab - offset));
      }
      uint64_t* const parts = sh.list;
      static_assert(kMostTokens / (64 * 4) <= kList, "a word to each part of a row");
      // The parts' sums of the piece. Those of bins and of parts are rounded each by themselves: where
      // u is among the last places of the total, a piece can have a sum by its bins and none by its
      // parts. Then the parts of the whole row say, of which the largest token's has a sum.
      uint64_t sum_t, up, here;
      int all, each;
      for (;;) {
        __syncthreads();
        const int stripes = piece.wave_stripes();
        all = piece.stripes() * kWaves;
        if (lane == 0)  // of the last stripe, in which the wave may have no tokens
          parts[(piece.stripes() - 1) * kWaves + wave] = 0;
        for (int s0 = 0; s0 < stripes; s0 += kAhead) {
          u4v w[kAhead];
#pragma unroll
          for (int a = 0; a < kAhead; ++a) w[a] = piece.load(s0 + a);
#pragma unroll
          for (int a = 0; a < kAhead; ++a) {
            if (s0 + a >= stripes) continue;
            piece.place(w[a], s0 + a);
            const int i0 = piece.first(s0 + a);
            double sum_s = 0.0;
            uint32_t bits = 0;
#pragma unroll
            for (int e = 0; e < P::kPer; ++e)
              bits |= (uint32_t)(T::wide(P::element(w[a], e)) >= edge) << e;
            for (; bits; bits &= bits - 1) {
              const int e = __builtin_ctz(bits);
              sum_s += kept_value(T::wide(P::any(w[a], e)), offset + piece.token(i0 + e));
            }
            sum_s = wave_sum(sum_s);
            if (lane == 0) parts[(s0 + a) * kWaves + wave] = in_units(sum_s, 0);
          }
        }
        __syncthreads();
        each = (all + kThreads - 1) / kThreads;
        sum_t = 0;
        for (int j = 0; j < each; ++j)
          if (t * each + j < all) sum_t += parts[t * each + j];
        up = block_scan(sum_t, sh.qwaves, &here);
        if (here || !by_bins) break;
        by_bins = false;
        piece = row;
        offset = 0;
        ahead = 0;
      }
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
      pick(piece, part, __builtin_ldexp((double)(rest - 1 - before), -S), offset,
           [&](Raw raw, int i) { return kept_value(T::wide(raw), offset + i); });
    }
  }
  if (owner_token >= 0) {
    p.tokens[r] = owner_token;
    // log(w / total): the kept weights' total is measured from the top, as is the largest
    if (p.logprobs)
      p.logprobs[r] = fminf(0.f, (float)(((double)owner_value - scale.ref) / (double)set.temperature +
                              scale.shift * (0.69314718055994530942 / kSteps) -
                              (log((double)total) - unit * 0.69314718055994530942)));
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

// Two workgroups of chunk_kernel run on a compute unit at a time. Rows are cut so that
// their rounds take least time, where a piece costs as much as kFixed tokens besides its own (256
// rows of 131073: four pieces 38 us, five, in three rounds, 58).
SamplePlan plan(const lutgemm_sample* s) {
  constexpr int64_t kFixed = 12000, kSlots = 512;
  SamplePlan r{};
  const int vocab = s->vocab, per = kThreads * (s->type == LUTGEMM_F32 ? 4 : 8);
  const int full = kStripes * per - 8;  // a piece may begin with half a word
  int64_t best = INT64_MAX;
  for (int n = (vocab + full - 1) / full; n <= kMostPieces; ++n) {
    const int piece = ((vocab + n - 1) / n + 7) / 8 * 8, pieces = (vocab + piece - 1) / piece;
    if (n > 1 && piece < kLeastPiece && best < INT64_MAX) break;
    const int64_t time = ((int64_t)s->rows * pieces + kSlots - 1) / kSlots * (kFixed + piece);
    if (piece > full || time >= best) continue;
    best = time;
    r.piece = piece;
    r.pieces = pieces;
  }
  r.parts = (r.piece + 1 + per - 1) / per * kWaves;
  r.slab = std::max(1, std::min(s->rows, 4096 / r.pieces));
  r.ws_bytes = s->rows ? (size_t)r.slab * r.pieces * kRecord : 0;
  return r;
}

template <class T>
int run_sample(SampleParams p, int rows, int slab, hipStream_t stream) {
  for (int r = 0; r < rows; r += slab) {
    const int n = rows - r < slab ? rows - r : slab;
    int st = launch(chunk_kernel<T>, dim3((unsigned)(n * p.pieces)), kThreads, p, stream);
    if (!st) st = launch(row_kernel<T>, dim3((unsigned)n), kThreads, p, stream);
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
    p.vocab = s->vocab;
    p.pieces = r.pieces;
    p.piece = r.piece;
    p.parts = r.parts;
    int bits = 0;
    while ((1 << bits) < s->vocab) ++bits;
    p.scale = 62 - bits < 50 ? 62 - bits : 50;
    hipStream_t strm = (hipStream_t)stream;
    if (s->type == LUTGEMM_F32) return run_sample<F32>(p, s->rows, r.slab, strm);
    if (s->type == LUTGEMM_F16) return run_sample<Logit16<serve::F16>>(p, s->rows, r.slab, strm);
    return run_sample<Logit16<serve::BF16>>(p, s->rows, r.slab, strm);
  } catch (...) {
    return LUTGEMM_ERR_INTERNAL;
  }
}
