// Shared by the serving operators (heads.hip, attention.hip, adapters.hip): the
// element types with their matrix-core instructions, and the host's device check.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <atomic>

#include "lutgemm.h"

namespace lutgemm {
namespace serve {

typedef _Float16 h8 __attribute__((ext_vector_type(8)));
typedef _Float16 h2 __attribute__((ext_vector_type(2)));
typedef __bf16 b8 __attribute__((ext_vector_type(8)));
typedef __bf16 b2 __attribute__((ext_vector_type(2)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef uint32_t u2v __attribute__((ext_vector_type(2)));
typedef uint32_t u4v __attribute__((ext_vector_type(4)));
typedef float f2v __attribute__((ext_vector_type(2)));
typedef float f4v __attribute__((ext_vector_type(4)));
typedef uint16_t us2v __attribute__((ext_vector_type(2)));
typedef float f16v __attribute__((ext_vector_type(16)));

// An element type: operands of the matrix cores travel as 16-byte words of eight
// elements. Operand layouts (row or column i, eight consecutive k per lane):
//   32x32x16: i = lane % 32, k = 8 (lane / 32) + j; result entry r of a lane is row
//             8 (r / 4) + 4 (lane / 32) + r % 4, column lane % 32
//   16x16x32: i = lane % 16, k = 8 (lane / 16) + j; result entry r of a lane is row
//             4 (lane / 16) + r, column lane % 16
struct F16 {
  static constexpr bool kHalf = true;
  static constexpr uint32_t kExponent = 0x7C00;  // all ones: infinity or NaN
  static __device__ __forceinline__ f16v mfma32(u4v a, u4v b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a),
                                                  __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f4v mfma16(u4v a, u4v b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8, a),
                                                  __builtin_bit_cast(h8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {  // to nearest even
    const h2 v = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ f2v unpack(uint32_t w) {
    const h2 v = __builtin_bit_cast(h2, w);
    return f2v{(float)v.x, (float)v.y};
  }
  static __device__ __forceinline__ uint16_t one(float a) {
    return __builtin_bit_cast(uint16_t, (_Float16)a);
  }
  static __device__ __forceinline__ float wide(uint16_t a) {
    return (float)__builtin_bit_cast(_Float16, a);
  }
};

struct BF16 {
  static constexpr bool kHalf = false;
  static constexpr uint32_t kExponent = 0x7F80;
  static __device__ __forceinline__ f16v mfma32(u4v a, u4v b, f16v c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(b8, a),
                                                   __builtin_bit_cast(b8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f4v mfma16(u4v a, u4v b, f4v c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(b8, a),
                                                   __builtin_bit_cast(b8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const b2 v = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, v);
  }
  static __device__ __forceinline__ f2v unpack(uint32_t w) {
    return f2v{__builtin_bit_cast(float, w << 16), __builtin_bit_cast(float, w & 0xFFFF0000u)};
  }
  static __device__ __forceinline__ uint16_t one(float a) {
    return __builtin_bit_cast(uint16_t, (__bf16)a);
  }
  static __device__ __forceinline__ float wide(uint16_t a) {
    return __builtin_bit_cast(float, (uint32_t)a << 16);
  }
};

// Whether one of these words' elements, two to a word, is an infinity or NaN: their
// magnitudes are the largest.
template <class T, int N>
__device__ __forceinline__ bool any_non_finite(const u4v (&words)[N]) {
  us2v most = {0, 0};
#pragma unroll
  for (int j = 0; j < N; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      most = __builtin_elementwise_max(most, __builtin_bit_cast(us2v, words[j][e] & 0x7FFF7FFFu));
  return most.x >= T::kExponent || most.y >= T::kExponent;
}

// The words with zeros in place of infinities and NaN.
template <class T>
__device__ __forceinline__ u4v finite(u4v words) {
  constexpr uint32_t lo = T::kExponent, hi = T::kExponent << 16;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    words[e] &= ((words[e] & lo) == lo ? 0xFFFF0000u : ~0u) &
                ((words[e] & hi) == hi ? 0xFFFFu : ~0u);
  return words;
}

// `sum` with the infinity or NaN that an element may be.
template <class T>
__device__ __forceinline__ float with_non_finite(float sum, uint16_t element) {
  return (element & T::kExponent) == T::kExponent ? sum + T::wide(element) : sum;
}

// Four elements of a column of LDS: the sixteen lanes of a group give the addresses
// of a 4 x 16 block (lane i: row i / 4, columns 4 (i % 4) ..), and lane i receives
// column i, rows 0 .. 3.
__device__ __forceinline__ u2v read_column(const void* lds) {
  return __builtin_bit_cast(
      u2v, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(lds)));
}

// 16 bytes a lane from memory to LDS, in lane order from `to` on (the same for the
// wave). Buffer loads: while loads of the flat kind to LDS are under way the compiler
// lets no LDS read overtake another.
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, char* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (__attribute__((address_space(3))) void*)to, 16,
                                           offset, 0, 0, 0);
}

// This wave's loads have arrived, in LDS too.
__device__ __forceinline__ void wait_for_loads() { __builtin_amdgcn_s_waitcnt(0x0F70); }

// This wave's LDS reads have returned.
__device__ __forceinline__ void wait_for_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }

// A kernel's parameters, asked for together at its start: they lie in host memory, and
// fields first read where they are needed cost a trip there each.
template <class P>
__device__ __forceinline__ void fetch(const P& p) {
  constexpr int n = sizeof(P) / 4;
  const uint32_t* w = (const uint32_t*)&p;
#pragma unroll
  for (int i = 0; i < n; ++i) asm volatile("" ::"s"(w[i]));
}

// ------------------------------------------------------------------ host side

// The current device must be gfx950 (LUTGEMM_FAKE_ARCH, a debugging aid, replaces
// the reported name and bypasses the per-device cache). *cus: its compute units.
inline int check_device(int* cus) {
  static std::atomic<int> known_cus[64];  // > 0: gfx950 with so many; < 0: another
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return LUTGEMM_ERR_HIP;
  const char* fake = getenv("LUTGEMM_FAKE_ARCH");
  const bool cached = dev >= 0 && dev < 64 && !(fake && *fake);
  int n = cached ? known_cus[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return LUTGEMM_ERR_HIP;
    if (prop.multiProcessorCount <= 0) return LUTGEMM_ERR_HIP;
    const bool ours = strncmp((fake && *fake) ? fake : prop.gcnArchName, "gfx950", 6) == 0;
    n = ours ? prop.multiProcessorCount : -1;
    if (cached) known_cus[dev].store(n, std::memory_order_relaxed);
  }
  *cus = n;
  return n > 0 ? LUTGEMM_OK : LUTGEMM_ERR_UNSUPPORTED;
}

inline bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline bool stride_ok(int64_t s) { return s >= 0 && s % 8 == 0 && s < ((int64_t)1 << 40); }

// One axis of an output: its length (below 2^32) and its stride in elements.
struct Axis {
  int64_t n, stride;
};

// Whether rows of `width` elements, addressed along N axes, lie apart from each other:
// with the axes taken from the smallest stride up, each steps over all that is inside.
template <int N>
bool apart(Axis (&&axes)[N], int64_t width) {
  __int128 inside = width;
  for (int i = 0; i < N; ++i) {
    int least = -1;
    for (int j = 0; j < N; ++j)
      if (axes[j].n > 1 && (least < 0 || axes[j].stride < axes[least].stride)) least = j;
    if (least < 0) return true;
    if (axes[least].stride < inside) return false;
    inside += (__int128)(axes[least].n - 1) * axes[least].stride;
    axes[least].n = 1;
  }
  return true;
}

// n rows of `width` 2-byte elements, `step` elements apart.
struct Rows {
  const void* at;
  int64_t n, step, width;
};

// Whether two arrays of as many rows have memory in common. Rows of one fused buffer (the
// same step) may lie beside each other; arrays of other steps must lie apart as a whole.
inline bool overlap(const Rows& a, const Rows& b) {
  if (a.n < 1 || b.n < 1 || a.width < 1 || b.width < 1) return false;
  const __int128 a0 = (uintptr_t)a.at, b0 = (uintptr_t)b.at;
  const __int128 a1 = a0 + 2 * ((__int128)(a.n - 1) * a.step + a.width);
  const __int128 b1 = b0 + 2 * ((__int128)(b.n - 1) * b.step + b.width);
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.n == 1 || b.n == 1 || a.step != b.step || a.step == 0) return true;
  const __int128 step = 2 * (__int128)a.step;
  const __int128 after = ((b0 - a0) % step + step) % step;  // of b's rows behind a's
  return after < 2 * (__int128)a.width || after + 2 * (__int128)b.width > step;
}

template <class P>
int launch(void (*kernel)(P), dim3 grid, int threads, const P& p, hipStream_t stream) {
  P copy = p;
  void* args[] = {&copy};
  if (hipLaunchKernel((const void*)kernel, grid, dim3((unsigned)threads), args, 0, stream) ==
      hipSuccess)
    return LUTGEMM_OK;
  (void)hipGetLastError();  // it is reported here, not by a later call
  return LUTGEMM_ERR_HIP;
}

}  // namespace serve
}  // namespace lutgemm
