// lm_internal.h -- what the token-model operators (lm_*.hip) share: element
// types and their vector loads, cross-lane reductions, the workspace header,
// host-side argument helpers.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sgb_lm.h"

namespace sgb_lm {

// ---------------------------------------------------------------- workspace

// First bytes of every workspace.  The first error of the call with `epoch`
// is kept as epoch << 8 | code; a word from another epoch counts as none, so
// nothing needs clearing between calls.
struct Header {
  uint32_t status;
  uint32_t epoch;
};
constexpr size_t kHeaderBytes = 256;

// ---------------------------------------------------------------- elements

using bf16_t = __bf16;
using f16_t = _Float16;

template <typename T>
struct Vec {
  static constexpr int kWords = sizeof(T) * 2;
  typedef T type __attribute__((ext_vector_type(8)));
};

// Eight elements as loaded; an element's alignment is enough (the target's
// global loads and stores take any byte address).
template <typename T>
struct __attribute__((packed, aligned(sizeof(T)))) Raw8 {
  uint32_t w[Vec<T>::kWords];
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(bf16_t v) { return (float)v; }
__device__ __forceinline__ float widen(f16_t v) { return (float)v; }

// Loads p[0 .. n) (n <= 8; nothing for n <= 0); the others are zero.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, int n) {
  Raw8<T> r;
  if (n >= 8) {
    r = *reinterpret_cast<const Raw8<T>*>(p);
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::kWords; ++i) r.w[i] = 0;
    if (n > 0) {
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        if (i < n) {
          if constexpr (sizeof(T) == 4) {
            r.w[i] = __float_as_uint(p[i]);
          } else {
            const uint32_t u = reinterpret_cast<const uint16_t*>(p)[i];
            r.w[i >> 1] |= u << (16 * (i & 1));
          }
        }
      }
    }
  }
  return r;
}

// The same in two parts, for loads that are to be in flight while other work
// goes on: a branch around a load makes the compiler wait for it where the
// branch ends.  ask8() loads without one: from `at`, or the eight elements that
// end at `end` (>= 8) where fewer than eight are left; zeros where there is no
// row.  have8() then moves the n elements wanted to the front and clears the
// rest.  `row` is best uniform and `at` the lane's: one scalar base address.
static __device__ const uint32_t kNowhere[8] = {};

// *p, or `none` for a null pointer (uniform), without a branch.  The address
// space keeps a selected address out of the generic loads, which wait for LDS
// too.
template <typename U>
__device__ __forceinline__ U load_global(uintptr_t p, uint32_t bytes = 0) {
#ifdef __HIP_DEVICE_COMPILE__
  return *reinterpret_cast<const __attribute__((address_space(1))) U*>(
      reinterpret_cast<const __attribute__((address_space(1))) char*>(p) + bytes);
#else
  return *reinterpret_cast<const U*>(p + bytes);  // the host's pass has no such spaces
#endif
}
template <typename U>
__device__ __forceinline__ U value_or(const U* p, int64_t at, U none) {
  const U v = load_global<U>(p ? (uintptr_t)(p + at) : (uintptr_t)kNowhere);
  return p ? v : none;
}

template <typename T>
__device__ __forceinline__ Raw8<T> ask8(const T* row, uint32_t at, uint32_t end) {
  return load_global<Raw8<T>>(row ? (uintptr_t)row : (uintptr_t)kNowhere,
                              (row ? min(at, end - 8) : 0u) * (uint32_t)sizeof(T));
}

template <typename T>
__device__ __forceinline__ void have8(Raw8<T>& r, int n) {
  if (n < 8) {
    constexpr int W = Vec<T>::kWords, E = sizeof(T) / 2;  // words, half words an element
    const int by = 8 - n;
#pragma unroll
    for (int step = 4; step >= 1; step >>= 1) {
      const bool move = by & step;
      if (step * E >= 2) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t next = i + step * E / 2 < W ? r.w[i + step * E / 2] : 0u;
          r.w[i] = move ? next : r.w[i];
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const uint32_t next = i + 1 < W ? r.w[i + 1] : 0u;
          r.w[i] = move ? (r.w[i] >> 16 | next << 16) : r.w[i];
        }
      }
    }
    if (n <= 0) {
#pragma unroll
      for (int i = 0; i < W; ++i) r.w[i] = 0;
    }
  }
}

template <typename T>
__device__ __forceinline__ void widen8(const Raw8<T>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (sizeof(T) == 4) {
      v[i] = __uint_as_float(r.w[i]);
    } else if constexpr (__is_same(T, bf16_t)) {
      // the 16 bits are the high half of the fp32 word: exact
      v[i] = __uint_as_float((i & 1) ? (r.w[i >> 1] & 0xffff0000u) : (r.w[i >> 1] << 16));
    } else {
      v[i] = (float)__builtin_bit_cast(f16_t, (uint16_t)(r.w[i >> 1] >> (16 * (i & 1))));
    }
  }
}

// Stores v[0 .. n) rounded to T, to nearest even.  Whole vectors go past the
// caches' own copies (non-temporal): outputs as long as these would only push
// out what is still to be read.  With inputs that are in no cache yet, stored
// temporally and so: distillation of 4096 x 131072 bf16 491 and 450 us, of
// 1021 x 50021 fp16 (loss, then gradient) 89 and 76; block norms' backward on
// 32768 x 4096 bf16 328 and 323, but with fp32 residuals 474 and 505; block norms
// of 8192 x 4096 and penalties on 512 x 131072 the same within 2%.
template <typename U, typename V>
__device__ __forceinline__ void store_global(void* p, uint32_t bytes, V v) {
#ifdef __HIP_DEVICE_COMPILE__
  __builtin_nontemporal_store(
      v, reinterpret_cast<__attribute__((address_space(1))) U*>(
             reinterpret_cast<__attribute__((address_space(1))) char*>((uintptr_t)p) + bytes));
#endif
}

// (`row` is best uniform and `at` the lane's, as for loads.)
template <typename T>
__device__ __forceinline__ void store8(T* row, uint32_t at, const float (&v)[8], int n) {
  typename Vec<T>::type t;
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = (T)v[i];
  if (n >= 8) {
    typedef uint32_t Words __attribute__((ext_vector_type(4)));
    typedef Words Any __attribute__((aligned(2)));
    constexpr int W = sizeof(T) / 2;
    struct Quads {
      Words q[W];
    };
    const Quads r = __builtin_bit_cast(Quads, t);
#pragma unroll
    for (int i = 0; i < W; ++i) store_global<Any>(row, at * (uint32_t)sizeof(T) + 16 * i, r.q[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) row[at + i] = t[i];
  }
}

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8], int n) {
  store8(p, 0u, v, n);
}

// Eight elements of a type known at run time.
__device__ __forceinline__ void load8_as(const void* base, int dtype, int64_t at, int n,
                                         float (&v)[8]) {
  if (dtype == SGB_F32)
    widen8(load8(static_cast<const float*>(base) + at, n), v);
  else if (dtype == SGB_BF16)
    widen8(load8(static_cast<const bf16_t*>(base) + at, n), v);
  else
    widen8(load8(static_cast<const f16_t*>(base) + at, n), v);
}

// The same in two parts, as above (`width`
// >= 8, unless `tiny`: then all is left to have8_as).
struct RawAs {
  uint32_t w[8];
};
struct __attribute__((packed, aligned(2))) Four {
  uint32_t w[4];
};

template <bool TINY = false>
__device__ __forceinline__ RawAs ask8_as(const void* base, int dtype, int64_t col, int64_t width) {
  RawAs r{};
  if (TINY) return r;
  const uintptr_t p = base ? (uintptr_t)base + (dtype == SGB_F32 ? 4 : 2) * min(col, width - 8)
                           : (uintptr_t)kNowhere;
  const Four lo = load_global<Four>(p), hi = load_global<Four>(p + (dtype == SGB_F32 ? 16 : 0));
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = lo.w[i], r.w[4 + i] = hi.w[i];
  return r;
}

template <typename T>
__device__ __forceinline__ void widen_as(const RawAs& r, float (&v)[8]) {
  Raw8<T> x;
#pragma unroll
  for (int i = 0; i < Vec<T>::kWords; ++i) x.w[i] = r.w[i];
  widen8(x, v);
}

// `none` for all of them where there is no array.
template <bool TINY = false>
__device__ __forceinline__ void have8_as(const RawAs& r, const void* base, int dtype, int64_t col,
                                         int n, float none, float (&v)[8]) {
  if (!base) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = none;
    return;
  }
  if (TINY) {
    load8_as(base, dtype, col, n, v);
    return;
  }
  if (dtype == SGB_F32)
    widen_as<float>(r, v);
  else if (dtype == SGB_BF16)
    widen_as<bf16_t>(r, v);
  else
    widen_as<f16_t>(r, v);
  if (n < 8) {
#pragma unroll
    for (int step = 4; step >= 1; step >>= 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float next = i + step < 8 ? v[i + step] : 0.f;
        v[i] = (8 - n) & step ? next : v[i];
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = n > 0 ? v[i] : 0.f;
  }
}

// ---------------------------------------------------------------- wave64

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __uint_as_float(
      (uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xf, 0xf, true));
}

// Folds x over groups of `width` lanes (8, 16, 32 or 64, wave-uniform); every
// lane of a group gets the same bits.  Lane exchanges inside the vector unit
// (data-parallel primitives within a row of 16, then the row and half
// swaps): six dependent steps of a few cycles each, where a shuffle through
// LDS takes tens.
template <typename F>
__device__ __forceinline__ float wave_fold(float x, int width, F f) {
  x = f(x, dpp<0xB1>(x));   // lane ^ 1
  x = f(x, dpp<0x4E>(x));   // lane ^ 2
  x = f(x, dpp<0x141>(x));  // mirrored in 8
  if (width > 8) x = f(x, dpp<0x140>(x));  // mirrored in 16
  if (width > 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    x = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  if (width > 32) {
    const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false,
                                                    false);
    x = f(__uint_as_float(p[0]), __uint_as_float(p[1]));
  }
  return x;
}

__device__ __forceinline__ float wave_add(float x, int width = 64) {
  return wave_fold(x, width, [](float a, float b) { return a + b; });
}
__device__ __forceinline__ float wave_max(float x, int width = 64) {
  return wave_fold(x, width, [](float a, float b) { return fmaxf(a, b); });
}

// Records `code` as the call's error unless it already has one.
__device__ __forceinline__ void set_status(Header* h, uint32_t epoch, uint32_t code) {
  uint32_t old = __hip_atomic_load(&h->status, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  while ((old >> 8) != epoch) {
    const uint32_t seen = atomicCAS(&h->status, old, (epoch << 8) | code);
    if (seen == old) break;
    old = seen;
  }
}

// ---------------------------------------------------------------- host

uint32_t next_epoch();
int current_device();  // -1: none; a plan made then checks its calls' arguments, no more
int compute_units(int device);

struct DeviceGuard {
  int prev = -1;
  bool ok = false, changed = false;
  explicit DeviceGuard(int dev) {
    if (dev < 0 || hipGetDevice(&prev) != hipSuccess) return;
    if (prev == dev)
      ok = true;
    else
      ok = changed = hipSetDevice(dev) == hipSuccess;
  }
  ~DeviceGuard() {
    if (changed) (void)hipSetDevice(prev);
  }
};

inline size_t align_up(size_t n, size_t a) { return (n + a - 1) / a * a; }
inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline size_t elem_size(int dtype) { return dtype == SGB_F32 ? 4 : 2; }
inline bool float_dtype(int dtype) {
  return dtype == SGB_F32 || dtype == SGB_BF16 || dtype == SGB_F16;
}

// A matrix argument: there, aligned to its elements, rows that do not overlap.
inline bool matrix_ok(const void* p, int64_t width, int64_t stride, size_t elem) {
  return p && aligned(p, elem) && stride >= width && stride <= (1ll << 40);
}

// A launch of more threads is refused by the runtime.
constexpr int64_t kMostThreadsAtOnce = (1ll << 32) - 1;

inline bool workspace_ok(const void* ws) { return ws && aligned(ws, 256); }

// Do the bytes of two row-strided matrices (of `rows` rows, or rows_b the
// second) share a range?  (Interleaved rows of one buffer, e.g. the halves of
// wider rows, are told apart by `same stride, disjoint columns`; the stride of a
// single row says nothing and is taken for the other's.)
inline bool overlap(const void* a, int64_t wa, int64_t sa, size_t ea, const void* b, int64_t wb,
                    int64_t sb, size_t eb, int64_t rows, int64_t rows_b = -1) {
  if (rows_b < 0) rows_b = rows;
  if (!a || !b || rows <= 0 || rows_b <= 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  const uint64_t la = ((uint64_t)(rows - 1) * sa + wa) * ea,
                 lb = ((uint64_t)(rows_b - 1) * sb + wb) * eb;
  if (a0 + la <= b0 || b0 + lb <= a0) return false;
  if (rows < 2 && rows_b < 2) return true;
  const uint64_t pitch = rows < 2 ? (uint64_t)sb * eb : (uint64_t)sa * ea;
  if (rows >= 2 && rows_b >= 2 && pitch != (uint64_t)sb * eb) return true;
  const uint64_t d = (b0 >= a0 ? b0 - a0 : pitch - (a0 - b0) % pitch) % pitch;
  // b's columns start d bytes after a's in the shared pitch
  return !(d >= (uint64_t)wa * ea && d + (uint64_t)wb * eb <= pitch);
}

// An argument's elements: rows of `width` elements of `elem` bytes (a vector: one row).
struct Extent {
  const void* p;  // or null: not there
  int64_t rows, width, stride;
  size_t elem;
};
inline bool overlap(const Extent& a, const Extent& b) {
  return overlap(a.p, a.width, a.stride, a.elem, b.p, b.width, b.stride, b.elem, a.rows, b.rows);
}
inline Extent vector(const void* p, int64_t n, size_t elem) { return {p, 1, n, n, elem}; }

// Does any of `n` outputs share bytes with another, or with one of `m` inputs?
inline bool any_overlap(const Extent* out, int n, const Extent* in, int m) {
  for (int i = 0; i < n; ++i) {
    for (int j = 0; j < m; ++j)
      if (overlap(out[i], in[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

}  // namespace sgb_lm
