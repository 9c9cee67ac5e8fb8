// lm_vocab_ce.hip -- cross-entropy of the head's product over a large
// vocabulary, of libsgb_lm.so (formulas: include/sgb_lm_step.h).
//
// One product kernel, C = A B^T with both operands' rows along the summed
// dimension, and five epilogues:
//   logits   A = weight rows, B = hidden rows: each wave leaves the largest of
//            its logits and the sum of exponentials below it a token, and the
//            exponentials themselves where gradients are to follow;
//   d_hidden A = weight transposed, B = the logits' gradient;
//   d_weight A = hidden transposed, B = the logits' gradient transposed.
// The vocabulary, or the columns of the result, are A's rows: a lane holds four
// neighbours of them for one of B's rows, so the softmax's sums stay in the
// lane and the stores are of four elements.  The operands that have to be
// transposed are copied piece by piece (a piece of the weight: 128 MB written
// and read again from the last-level cache), and so are operands whose rows
// are not whole 128-byte lines.
//
// A chunk of tokens takes three products: its exponentials wait in 16 bits
// (32 for fp16 and fp32 operands) for the row sums, since computing the logits
// again would be a fourth.  They are relative to the largest of a wave's
// columns and scaled by 2^15, so fp16 holds 11 bits of all that matter, and the
// only rounding to the operands' type is that of the gradient itself.

#include <algorithm>
#include <cmath>
#include <new>

#include "lm_internal.h"
#include "sgb_lm_step.h"

using namespace sgb_lm;

namespace {

constexpr int kMaxD = 16384;
constexpr int64_t kMaxV = 1 << 23;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kUp = 32768.f;   // 2^15: see above; fp16 gradients are scaled by it too

typedef float Acc __attribute__((ext_vector_type(16)));
typedef float F4 __attribute__((ext_vector_type(4)));
typedef F4 F4Any __attribute__((aligned(4)));

__device__ __forceinline__ Acc mfma(Vec<bf16_t>::type a, Vec<bf16_t>::type b, Acc c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ Acc mfma(Vec<f16_t>::type a, Vec<f16_t>::type b, Acc c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// ---------------------------------------------------------------- the product

constexpr int kStep = 64;             // of the summed dimension a turn: 128 bytes a row
constexpr int kRowBytes = kStep * 2;

// A workgroup's tile of C (rows of A by rows of B), and a wave's.
struct Big {
  static constexpr int TM = 256, TN = 256, WM = 128, WN = 64;
};
struct Small {
  static constexpr int TM = 128, TN = 64, WM = 64, WN = 32;
};
template <typename C>
constexpr int kThreadsOf = C::TM / C::WM * (C::TN / C::WN) * 64;

enum Epilogue { kSums, kExps, kProbs, kAdd, kOut };

struct Product {
  const char *a, *b;
  int64_t lda, ldb;          // bytes from row to row; of 16
  int64_t plane_a, plane_b;  // bytes from one bf16 part of fp32 operands to the next
  int64_t M, N;              // rows of a, b
  int steps, split;          // of the summed dimension, over `split` workgroups
  int tm, tn;
  // logits
  float2* stats;             // [vocabulary / WM][tokens]
  int64_t tokens;
  const int64_t* labels;
  const float* lse;
  float* said;               // the label's logit
  void* exps;                // [tokens][ld_exps]
  int64_t ld_exps, v0, V;    // v0: the piece's first token of the vocabulary
  // sums
  float* sums;               // kAdd: [split][N][M]
  bool add;                  // to what is there
  // out
  void* out;                 // kOut: [N][ldo]
  int64_t ldo;
  int out_dtype;
  const float* add_from;     // [N][M] or null
  const float* most;         // times scale: what the sums are multiplied by
  float scale;
};

// Which bf16 parts (0: the highest) the products of fp32 operands are of, the
// smallest first; those left out are below 2^-25 of the whole.
constexpr uint32_t kPartsA = 0u << 0 | 2u << 2 | 1u << 4 | 0u << 6 | 1u << 8 | 0u << 10;
constexpr uint32_t kPartsB = 2u << 0 | 0u << 2 | 1u << 4 | 1u << 6 | 0u << 8 | 0u << 10;

// The workgroup's loads of R rows of 64 elements, straight to LDS, 16 bytes a
// lane.  A row is 128 bytes of LDS; its 16-byte parts are stored in an order
// of the row's own (exclusive or with row / 2), so that 16 lanes that read the
// same part of 16 rows touch all banks once.  LDS addresses of one load are
// consecutive over the lanes, so the order is made by what a lane loads.
template <int R, int WAVES>
struct Stage {
  static constexpr int J = R / (8 * WAVES);
  uint32_t off[J];
  __device__ __forceinline__ void init(int wave, int lane, int64_t left, int64_t ld) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = (wave * J + j) * 8 + (lane >> 3);
      const int part = (lane & 7) ^ ((row >> 1) & 7);
      // rows past the last are copies of it: nothing is read out of range
      off[j] = (uint32_t)min((int64_t)row, left - 1) * (uint32_t)ld + part * 16;
    }
  }
  __device__ __forceinline__ void load(const char* base, char* lds, int wave) const {
#ifdef __HIP_DEVICE_COMPILE__
#pragma unroll
    for (int j = 0; j < J; ++j)
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(base + off[j]),
          (__attribute__((address_space(3))) void*)(lds + (wave * J + j) * 1024), 16, 0, 0);
#endif
  }
};

__device__ __forceinline__ void all_loaded() {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ void store4(void* row, int64_t at, F4 v, int64_t n) {
  T* p = static_cast<T*>(row) + at;
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef T4 Any __attribute__((aligned(sizeof(T))));
  const T4 t = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  if (n >= 4) {
    *reinterpret_cast<Any*>(p) = t;
  } else {
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (i < n) p[i] = t[i];
  }
}
template <typename T>
__device__ __forceinline__ F4 load4(const void* row, int64_t at, int64_t n) {
  const T* p = static_cast<const T*>(row) + at;
  F4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < n) v[i] = widen(p[i]);
  return v;
}

template <typename E, int TERMS, int EPI, typename C>
__global__ __launch_bounds__(kThreadsOf<C>, 2) void k_product(Product p) {
  constexpr int TM = C::TM, TN = C::TN, WM = C::WM, WN = C::WN;
  constexpr int WAVES = kThreadsOf<C> / 64, FM = WM / 32, FN = WN / 32;
  constexpr int kBytes = (TM + TN) * kRowBytes;
  __shared__ __attribute__((aligned(1024))) char buf0[kBytes];
  __shared__ __attribute__((aligned(1024))) char buf1[kBytes];

  // Workgroups go round the eight dies; each die gets a run of tiles of its
  // own, eight tiles of A by some of B at a time, whose operands its L2 shares.
  const int total = p.tm * p.tn * p.split, per = (total + 7) >> 3;
  const int idx = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (idx >= total) return;
  const int tiles = p.tm * p.tn;
  const int part = idx / tiles, in_part = idx % tiles;
  const int group = in_part / (8 * p.tn), gm = min(8, p.tm - group * 8);
  const int in_group = in_part - group * 8 * p.tn;
  const int64_t m0 = (int64_t)(group * 8 + in_group % gm) * TM;
  const int64_t n0 = (int64_t)(in_group / gm) * TN;

  const int lane = (int)threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wm = wave % (TM / WM) * WM, wn = wave / (TM / WM) * WN;

  Stage<TM, WAVES> sa;
  Stage<TN, WAVES> sb;
  sa.init(wave, lane, p.M - m0, p.lda);
  sb.init(wave, lane, p.N - n0, p.ldb);
  const char* a = p.a + m0 * p.lda;
  const char* b = p.b + n0 * p.ldb;
  const int from = (int)((int64_t)p.steps * part / p.split);
  const int to = (int)((int64_t)p.steps * (part + 1) / p.split);
  const int turns = (to - from) * TERMS;
  int term = 0, step = from;
  const auto stage = [&](char* buf) {
    const int64_t at = (int64_t)step * kRowBytes;
    const char *pa = a + at, *pb = b + at;
    if (TERMS > 1) {
      pa += (kPartsA >> (2 * term) & 3) * p.plane_a;
      pb += (kPartsB >> (2 * term) & 3) * p.plane_b;
    }
    sa.load(pa, buf, wave);
    sb.load(pb, buf + TM * kRowBytes, wave);
    if (++step == to) {
      step = from;
      ++term;
    }
  };

  Acc acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int k = 0; k < 16; ++k) acc[i][j][k] = 0.f;

  const int key = (lane >> 1) & 7, row = (lane & 31) * kRowBytes;
  const auto compute = [&](const char* buf) {
    typedef typename Vec<E>::type V8;
    const char* la = buf + wm * kRowBytes + row;
    const char* lb = buf + (TM + wn) * kRowBytes + row;
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) {
      const int at = ((kk * 2 + (lane >> 5)) ^ key) * 16;
      V8 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i)
        fa[i] = *reinterpret_cast<const V8*>(la + at + i * 32 * kRowBytes);
#pragma unroll
      for (int j = 0; j < FN; ++j)
        fb[j] = *reinterpret_cast<const V8*>(lb + at + j * 32 * kRowBytes);
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) acc[i][j] = mfma(fa[i], fb[j], acc[i][j]);
    }
  };

  if (turns > 0) stage(buf0);
  int left = turns;
  for (; left >= 2; left -= 2) {
    all_loaded();
    stage(buf1);
    compute(buf0);
    all_loaded();
    if (left > 2) stage(buf0);
    compute(buf1);
  }
  if (left) {
    all_loaded();
    compute(buf0);
  }

  // acc[i][j][k]: C's row (of A) m0 + wm + 32 i + 8 (k / 4) + 4 (lane / 32) +
  // k % 4, its column (of B) n0 + wn + 32 j + lane % 32
  const int64_t mw = m0 + wm + 4 * (lane >> 5);
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int64_t n = n0 + wn + 32 * j + (lane & 31);
    const bool there = n < p.N;
    if (EPI == kSums || EPI == kExps) {
      typedef typename std::conditional<__is_same(E, bf16_t) && TERMS == 1, f16_t, float>::type X;
      if (m0 + wm + WM > p.M) {  // past the vocabulary
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (mw + 32 * i + 8 * (k >> 2) + (k & 3) >= p.M) acc[i][j][k] = -INFINITY;
      }
      const int64_t label = there ? p.labels[n] - (p.v0 + m0 + wm) : -1;
      if (label >= 0 && label < WM && label + m0 + wm < p.M) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int k = 0; k < 16; ++k)
            if (label == 32 * i + 8 * (k >> 2) + 4 * (lane >> 5) + (k & 3))
              p.said[n] = acc[i][j][k];
      }
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) top = fmaxf(top, acc[i][j][k]);
      const auto halves = [](float x, auto f) {
        const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x),
                                                        false, false);
        return f(__uint_as_float(s[0]), __uint_as_float(s[1]));
      };
      top = halves(top, [](float x, float y) { return fmaxf(x, y); });
      if (top == -INFINITY) top = 0.f;  // nothing but -inf: the sum is 0
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float e = exp2_((acc[i][j][k] - top) * kLog2e);
          acc[i][j][k] = e;
          sum += e;
        }
      sum = halves(sum, [](float x, float y) { return x + y; });
      if (there && lane < 32)
        p.stats[(p.v0 + m0 + wm) / WM * p.tokens + n] = make_float2(top, sum);
      if (EPI == kExps && there) {
        X* out = static_cast<X*>(p.exps) + n * p.ld_exps;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int k = 0; k < 16; k += 4) {
            constexpr float up = sizeof(X) == 2 ? kUp : 1.f;
            const F4 v = {acc[i][j][k] * up, acc[i][j][k + 1] * up, acc[i][j][k + 2] * up,
                          acc[i][j][k + 3] * up};
            store4<X>(out, p.v0 + mw + 32 * i + 2 * k, v, 4);
          }
      }
    } else if (EPI == kProbs) {
      typedef typename std::conditional<__is_same(E, bf16_t) && TERMS == 1, f16_t, float>::type X;
      if (!there) continue;
      const float lse = p.lse[n];
      constexpr float up = sizeof(X) == 2 ? kUp : 1.f;
      X* out = static_cast<X*>(p.exps) + n * p.ld_exps;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          F4 v;
#pragma unroll
          for (int u = 0; u < 4; ++u) v[u] = exp2_((acc[i][j][k + u] - lse) * kLog2e) * up;
          store4<X>(out, p.v0 + mw + 32 * i + 2 * k, v, 4);
        }
    } else if (EPI == kAdd) {
      if (!there) continue;
      float* out = p.sums + ((int64_t)part * p.N + n) * p.M;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const int64_t m = mw + 32 * i + 2 * k;
          if (m >= p.M) continue;
          F4 v = {acc[i][j][k], acc[i][j][k + 1], acc[i][j][k + 2], acc[i][j][k + 3]};
          if (p.add) v += load4<float>(out, m, p.M - m);
          store4<float>(out, m, v, p.M - m);
        }
    } else {
      if (!there) continue;
      const float by = p.scale * *p.most;
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const int64_t m = mw + 32 * i + 2 * k, n4 = p.M - m;
          if (n4 <= 0) continue;
          F4 v = {acc[i][j][k], acc[i][j][k + 1], acc[i][j][k + 2], acc[i][j][k + 3]};
          v *= by;
          if (p.add_from) v += load4<float>(p.add_from + n * p.M, m, n4);
          if (p.out_dtype == SGB_F32) {
            float* out = static_cast<float*>(p.out) + n * p.ldo;
            if (p.add) v += load4<float>(out, m, n4);
            store4<float>(out, m, v, n4);
          } else {
            E* out = static_cast<E*>(p.out) + n * p.ldo;
            if (p.add) v += load4<E>(out, m, n4);
            store4<E>(out, m, v, n4);
          }
        }
    }
  }
}

// ---------------------------------------------------------------- copies

// What an operand's element becomes: itself, or the three bf16 parts of an
// fp32 number, each what the ones before it leave (exact but for subnormals).
template <typename T>
struct Parts {
  static constexpr int kCount = 1;
  typedef T E;
  static __device__ __forceinline__ void split(T v, E (&out)[1]) { out[0] = v; }
};
template <>
struct Parts<float> {
  static constexpr int kCount = 3;
  typedef bf16_t E;
  static __device__ __forceinline__ void split(float v, E (&out)[3]) {
    bf16_t hi = (bf16_t)v;
    if (fabsf((float)hi) == INFINITY && fabsf(v) != INFINITY)  // the largest do not round up
      hi = __builtin_bit_cast(bf16_t, (uint16_t)(__float_as_uint(v) >> 16));
    const float r = v - (float)hi;
    out[0] = hi;
    out[1] = (bf16_t)r;
    out[2] = (bf16_t)(r - (float)out[1]);
  }
};

// [rows][D] to [rows][pitch], zeros past D.
template <typename T>
__global__ __launch_bounds__(256) void k_rows(const T* src, int64_t stride, int64_t rows, int D,
                                              typename Parts<T>::E* dst, int64_t pitch,
                                              int64_t plane) {
  typedef typename Parts<T>::E E;
  constexpr int P = Parts<T>::kCount;
  const int64_t groups = pitch / 8, all = rows * groups;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < all; g += (int64_t)gridDim.x * 256) {
    const int64_t r = g / groups;
    const int c = (int)(g % groups) * 8;
    E out[P][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      E e[P];
      Parts<T>::split(c + i < D ? src[r * stride + c + i] : (T)0.f, e);
#pragma unroll
      for (int k = 0; k < P; ++k) out[k][i] = e[k];
    }
#pragma unroll
    for (int k = 0; k < P; ++k)
      *reinterpret_cast<uint4*>(dst + k * plane + r * pitch + c) =
          *reinterpret_cast<const uint4*>(out[k]);
  }
}

constexpr int kTile = 64;

// [rows][D] to [D][pitch], zeros from `rows` to `pitch` and for rows whose
// factor is 0 (what they hold may be no number).
template <typename T>
__global__ __launch_bounds__(256) void k_transpose(const T* src, int64_t stride, int64_t rows,
                                                   int D, const float* factors,
                                                   typename Parts<T>::E* dst, int64_t pitch,
                                                   int64_t plane) {
  typedef typename Parts<T>::E E;
  constexpr int P = Parts<T>::kCount;
  __shared__ T tile[kTile][kTile + 4 / sizeof(T)];
  const int across = (D + kTile - 1) / kTile;
  const int64_t r0 = (int64_t)(blockIdx.x / across) * kTile;
  const int d0 = (int)(blockIdx.x % across) * kTile;
  const int t = (int)threadIdx.x;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (t >> 3) + 32 * u, c = (t & 7) * 8;
    const T* from = src + (r0 + r) * stride + d0 + c;
    const bool on = r0 + r < rows && (!factors || factors[r0 + r] != 0.f);
    const int n = on ? min(8, D - d0 - c) : 0;
    const Raw8<T> raw = load8(from, n);
    T v[8];
    __builtin_memcpy(v, &raw, sizeof v);
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[r][c + i] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int d = (t >> 3) + 32 * u, c = (t & 7) * 8;
    if (d0 + d >= D) continue;
    E out[P][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      E e[P];
      Parts<T>::split(tile[c + i][d], e);
#pragma unroll
      for (int k = 0; k < P; ++k) out[k][i] = e[k];
    }
#pragma unroll
    for (int k = 0; k < P; ++k)
      *reinterpret_cast<uint4*>(dst + k * plane + (int64_t)(d0 + d) * pitch + r0 + c) =
          *reinterpret_cast<const uint4*>(out[k]);
  }
}

// ---------------------------------------------------------------- row work

// A row's factor (0 where it does not count), and the largest magnitude of them
// all: d_weight's operand carries factor / largest, which no type's range can
// lose, d_hidden the factor itself at its end.
__global__ __launch_bounds__(1024) void k_factors(const int64_t* labels, const float* weights,
                                                  const float* above, int64_t rows, int64_t V,
                                                  float* factors, float* most, Header* hdr,
                                                  uint32_t epoch) {
  __shared__ float part[16];
  float top = 0.f;
  bool bad = false;
  for (int64_t r = threadIdx.x; r < rows; r += 1024) {
    const int64_t label = labels[r];
    const float w = value_or(weights, r, 1.f), g = value_or(above, r, 1.f);
    bad |= w != 0.f && label >= V;
    const float f = w == 0.f || label < 0 || label >= V ? 0.f : w * g;
    factors[r] = f;
    top = fmaxf(top, fabsf(f));
  }
  if (bad) set_status(hdr, epoch, SGB_ERR_INDEX_OUT_OF_RANGE);
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x < 64) {
    top = wave_max(threadIdx.x < 16 ? part[threadIdx.x] : 0.f);
    if (threadIdx.x == 0) {
      *most = top;
      hdr->epoch = epoch;
    }
  }
}

// The waves' sums of a row to its log-sum-exp and loss: 16 rows a workgroup.
__global__ __launch_bounds__(256) void k_lse(const float2* stats, int parts, int64_t tokens,
                                             const int64_t* labels, const float* weights,
                                             const float* said, int64_t V, float* loss, float* lse,
                                             Header* hdr, uint32_t epoch) {
  __shared__ float2 all[16][17];
  const int who = (int)threadIdx.x & 15, share = (int)threadIdx.x >> 4;
  const int64_t r = (int64_t)blockIdx.x * 16 + who;
  float m = -INFINITY, s = 0.f;
  const auto add = [&](float2 v) {
    if (v.y == 0.f) return;  // no mass, whatever its reference
    const float top = fmaxf(m, v.x);
    s = s * exp2_((m - top) * kLog2e) + v.y * exp2_((v.x - top) * kLog2e);
    m = top;
  };
  if (r < tokens) {
    int i = share;
    for (; i + 112 < parts; i += 128) {
      float2 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = stats[(int64_t)(i + 16 * u) * tokens + r];
#pragma unroll
      for (int u = 0; u < 8; ++u) add(v[u]);
    }
    for (; i < parts; i += 16) add(stats[(int64_t)i * tokens + r]);
  }
  all[share][who] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x < 16 && r < tokens) {
    m = -INFINITY;
    s = 0.f;
    for (int i = 0; i < 16; ++i) add(all[i][who]);
    const float l = m + logf(s);
    if (lse) lse[r] = l;
    const float w = value_or(weights, r, 1.f);
    const int64_t label = labels[r];
    if (w != 0.f && label >= V) set_status(hdr, epoch, SGB_ERR_INDEX_OUT_OF_RANGE);
    if (loss) loss[r] = w == 0.f || label < 0 || label >= V ? 0.f : w * (l - said[r]);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) hdr->epoch = epoch;
}

struct Grad {
  const void* exps;      // [tokens][ld_exps], the chunk's
  int64_t ld_exps, tokens;
  const float2* stats;   // null: relative to the row's lse already
  int wave_cols;
  const float* lse;
  const int64_t* labels;
  const float *factors, *most;
  int64_t v0, width, V;  // the piece
  void* g;               // [tokens][pitch] or null
  void* gt;              // [width][pitch_t] or null
  int64_t pitch, plane, pitch_t, plane_t;
};

// The gradient of a piece's logits from their exponentials: as it is (over the
// row's factor) and transposed (with it), in the operands' type, zeros past the
// vocabulary and past the last token.
template <typename T, typename X>
__global__ __launch_bounds__(256) void k_grad(Grad q) {
  typedef typename Parts<T>::E E;
  constexpr int P = Parts<T>::kCount;
  constexpr float kBy = __is_same(T, f16_t) ? kUp : 1.f;  // fp16 has no room below 2^-24
  __shared__ float tile[kTile][kTile + 1];
  const int across = (int)(q.pitch / kTile);
  const int64_t r0 = (int64_t)(blockIdx.x / across) * kTile;
  const int64_t c0 = (int64_t)(blockIdx.x % across) * kTile;
  const int t = (int)threadIdx.x;
  const float most = *q.most;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int lr = (t >> 3) + 32 * u, c = (t & 7) * 8;
    const int64_t r = r0 + lr;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    float share = 0.f;
    if (r < q.tokens) {
      const float f = q.factors[r];
      if (f != 0.f) {
        const int64_t at = q.v0 + c0 + c;
        const int n = (int)min((int64_t)8, q.v0 + q.width - at);
        share = f / most;
        float k = sizeof(X) == 2 ? 1.f / kUp : 1.f;
        if (q.stats)
          k *= exp2_((q.stats[at / q.wave_cols * q.tokens + r].x - q.lse[r]) * kLog2e);
        const int64_t label = q.labels[r] - at;
        float e[8];
        widen8(*reinterpret_cast<const Raw8<X>*>(static_cast<const X*>(q.exps) + r * q.ld_exps + at), e);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < n) v[i] = (e[i] * k - (label == i ? 1.f : 0.f)) * kBy;
      }
      if (q.g) {
        E out[P][8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          E e[P];
          Parts<T>::split((T)v[i], e);
#pragma unroll
          for (int k = 0; k < P; ++k) out[k][i] = e[k];
        }
#pragma unroll
        for (int k = 0; k < P; ++k)
          *reinterpret_cast<uint4*>(static_cast<E*>(q.g) + k * q.plane + r * q.pitch + c0 + c) =
              *reinterpret_cast<const uint4*>(out[k]);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[lr][c + i] = v[i] * share;
  }
  if (!q.gt) return;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int lv = (t >> 3) + 32 * u, c = (t & 7) * 8;
    if (c0 + lv >= q.width) continue;
    E out[P][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      E e[P];
      Parts<T>::split((T)tile[c + i][lv], e);
#pragma unroll
      for (int k = 0; k < P; ++k) out[k][i] = e[k];
    }
#pragma unroll
    for (int k = 0; k < P; ++k)
      *reinterpret_cast<uint4*>(static_cast<E*>(q.gt) + k * q.plane_t + (c0 + lv) * q.pitch_t + r0 + c) =
          *reinterpret_cast<const uint4*>(out[k]);
  }
}

// d_hidden: the parts' sums in their order, the row's factor, one rounding.
template <typename T>
__global__ __launch_bounds__(256) void k_join(const float* sums, int split, int64_t rows, int D,
                                              const float* factors, float scale, T* out,
                                              int64_t stride) {
  const int64_t groups = (D + 7) / 8, all = rows * groups;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < all; g += (int64_t)gridDim.x * 256) {
    const int64_t r = g / groups;
    const int c = (int)(g % groups) * 8, n = min(8, D - c);
    const float f = factors[r];
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (f != 0.f) {
      for (int s = 0; s < split; ++s) {
        float x[8];
        widen8(load8(sums + ((int64_t)s * rows + r) * D + c, n), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += x[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= f * scale;
    }
    store8(out + r * stride + c, v, n);
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_zero(T* out, int64_t stride, int64_t rows, int D) {
  const int64_t all = rows * D;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < all; g += (int64_t)gridDim.x * 256)
    out[g / D * stride + g % D] = (T)0.f;
}

}  // namespace

// ------------------------------------------------------------- host

struct sgb_vocab_ce_s {
  int device, cus;
  int D;
  int64_t V;
};

namespace {

constexpr int64_t kExpBytes = 1ll << 30;     // a chunk's exponentials
constexpr int64_t kStatBytes = 1ll << 28;    // their sums
constexpr int64_t kPieceElems = 1ll << 27;   // a piece's copies
constexpr int kMaxSplit = 16;

int64_t up(int64_t n, int64_t to) { return div_up(n, to) * to; }

// What a call lays out in its workspace.
struct Layout {
  int parts;           // of an element
  bool copy;           // fp32 operands are always copied (others where their rows ask for it)
  int64_t chunk, pad;  // rows a chunk, rounded up for the summed dimension
  int64_t piece;       // of the vocabulary
  int64_t pitch_d, ld_exps;
  size_t factors, lse, said, most, stats, x, w, exps, g, gt, xt, sums, dw, bytes;
};

template <typename C>
int64_t tiles_of(int64_t M, int64_t N) {
  return div_up(M, C::TM) * div_up(N, C::TN);
}
// 256 x 256 tiles where they give most compute units one.
bool big(int64_t M, int64_t N, int cus) { return tiles_of<Big>(M, N) * 4 >= 3 * (int64_t)cus; }

// d_hidden's summed dimension is shared out where it has few tiles.
int split_of(int64_t D, int64_t chunk, int cus) {
  if (big(D, chunk, cus)) return 1;
  return (int)std::clamp<int64_t>(2 * cus / tiles_of<Small>(D, chunk), 1, kMaxSplit);
}

Layout layout(const sgb_vocab_ce_s* p, int64_t rows, int dtype, bool gradient) {
  Layout l{};
  l.parts = dtype == SGB_F32 ? 3 : 1;
  const int64_t V = p->V, D = p->D, exp_size = dtype == SGB_BF16 ? 2 : 4;
  l.pitch_d = up(D, kStep);
  l.ld_exps = up(V, 256);
  int64_t most = kStatBytes / (div_up(l.ld_exps, Small::WM) * 8);
  if (gradient) most = std::min(most, kExpBytes / (l.ld_exps * exp_size));
  most = std::max<int64_t>(most / 256 * 256, 64);
  l.chunk = std::min(rows, most);
  l.pad = up(l.chunk, kStep);
  const int64_t room = kPieceElems / l.parts;
  l.piece = std::min(l.ld_exps,
                     std::max<int64_t>(256, std::min(room / l.pad, room / l.pitch_d) / 256 * 256));
  size_t at = kHeaderBytes;
  const auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += align_up((size_t)bytes, 256);
    return here;
  };
  const int64_t part = 2ll * l.parts;
  l.factors = take(4 * rows);
  l.lse = take(4 * rows);
  l.said = take(4 * rows);
  l.most = take(4);
  l.stats = take(div_up(l.ld_exps, Small::WM) * 8 * l.chunk);
  l.x = take(l.chunk * l.pitch_d * part);
  // a piece's weight rows, or their transpose
  const int64_t all = std::max(l.ld_exps * l.pitch_d, D * l.ld_exps);
  l.w = take(std::min(all, std::max(room, 256 * l.pitch_d)) * part);
  if (gradient) {
    l.exps = take(l.chunk * l.ld_exps * exp_size);
    const int64_t grads = std::min(l.pad * l.ld_exps, std::max(room, 256 * l.pad)) * part;
    l.g = take(grads);
    l.gt = take(grads);
    l.xt = take(D * l.pad * part);
    int64_t sums = 0;  // any fewer rows too
    for (int64_t c = std::min<int64_t>(l.chunk, 64);; c = std::min(c + 64, l.chunk)) {
      sums = std::max(sums, split_of(D, c, p->cus) * c);
      if (c == l.chunk) break;
    }
    l.sums = take(sums * D * 4);
    if (rows > l.chunk && dtype != SGB_F32) l.dw = take(V * D * 4);
  }
  l.bytes = at;
  return l;
}

struct Operand {
  const char* p;
  int64_t ld, plane;  // bytes
};

template <typename E, int TERMS, int EPI>
void product(Product& a, bool is_big, hipStream_t s) {
  a.tm = (int)div_up(a.M, is_big ? Big::TM : Small::TM);
  a.tn = (int)div_up(a.N, is_big ? Big::TN : Small::TN);
  const dim3 grid((unsigned)(div_up((int64_t)a.tm * a.tn * a.split, 8) * 8));
  if (is_big)
    hipLaunchKernelGGL((k_product<E, TERMS, EPI, Big>), grid, dim3(kThreadsOf<Big>), 0, s, a);
  else
    hipLaunchKernelGGL((k_product<E, TERMS, EPI, Small>), grid, dim3(kThreadsOf<Small>), 0, s, a);
}

unsigned blocks(int64_t threads, int cus) {
  return (unsigned)std::min<int64_t>(div_up(threads, 256), (int64_t)cus * 32);
}

enum Way { kForward, kBackward, kBoth };

template <typename T>
void enqueue(const sgb_vocab_ce_s* p, const sgb_vocab_ce_args* q, Way way, const Layout& l, char* ws,
             hipStream_t s) {
  typedef typename Parts<T>::E E;
  constexpr int TERMS = Parts<T>::kCount == 3 ? 6 : 1;
  typedef typename std::conditional<__is_same(T, bf16_t), f16_t, float>::type X;
  constexpr float kBy = __is_same(T, f16_t) ? kUp : 1.f;
  const int64_t R = q->rows, V = p->V;
  const int D = p->D;
  Header* hdr = reinterpret_cast<Header*>(ws);
  const uint32_t epoch = next_epoch();
  const auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  E* const xc = reinterpret_cast<E*>(ws + l.x);
  E* const wc = reinterpret_cast<E*>(ws + l.w);
  float *factors = at(l.factors), *most = at(l.most), *said = at(l.said);
  const float* lse_in = q->lse;
  float* lse_out = q->lse ? q->lse : at(l.lse);
  const float* lse = way == kBackward ? lse_in : lse_out;
  const T* hidden = static_cast<const T*>(q->hidden);
  const T* weight = static_cast<const T*>(q->weight);
  const bool grad = way != kForward;

  if (grad)
    hipLaunchKernelGGL(k_factors, dim3(1), dim3(1024), 0, s, q->labels, q->row_weights,
                       way == kBackward ? q->grad_loss : nullptr, R, V, factors, most, hdr, epoch);
  // Rows as the product reads them: whole 128-byte lines, 16-byte aligned.
  const auto fits = [&](const void* a, int64_t stride, int64_t rows) {
    return sizeof(T) == 2 && D % kStep == 0 && aligned(a, 16) && (rows < 2 || stride % 8 == 0);
  };
  const auto rows_of = [&](const T* src, int64_t stride, int64_t n, E* to) -> Operand {
    if (fits(src, stride, n)) return {reinterpret_cast<const char*>(src), stride * 2, 0};
    const int64_t plane = n * l.pitch_d;
    hipLaunchKernelGGL(k_rows<T>, dim3(blocks(plane / 8, p->cus)), dim3(256), 0, s, src, stride, n, D,
                       to, l.pitch_d, plane);
    return {reinterpret_cast<const char*>(to), l.pitch_d * 2, plane * 2};
  };
  const auto columns_of = [&](const T* src, int64_t stride, int64_t n, const float* only,
                              E* to) -> Operand {
    const int64_t pitch = up(n, kStep), plane = D * pitch;
    const unsigned grid = (unsigned)(pitch / kTile * div_up(D, kTile));
    hipLaunchKernelGGL(k_transpose<T>, dim3(grid), dim3(256), 0, s, src, stride, n, D, only, to, pitch,
                       plane);
    return {reinterpret_cast<const char*>(to), pitch * 2, plane * 2};
  };

  for (int64_t r0 = 0; r0 < R; r0 += l.chunk) {
    const int64_t n = std::min(l.chunk, R - r0);
    const T* x = hidden + r0 * q->hidden_stride;
    const Operand xo = rows_of(x, q->hidden_stride, n, xc);
    Product a{};
    a.b = xo.p;
    a.ldb = xo.ld;
    a.plane_b = xo.plane;
    a.N = a.tokens = n;
    a.steps = (int)(l.pitch_d / kStep);
    a.split = 1;
    a.stats = reinterpret_cast<float2*>(ws + l.stats);
    a.labels = q->labels + r0;
    a.lse = lse ? lse + r0 : nullptr;
    a.said = said + r0;
    a.exps = ws + l.exps;
    a.ld_exps = l.ld_exps;
    a.V = V;
    // the waves' width has to be one for all pieces
    const bool whole = fits(weight, q->weight_stride, V);
    const int64_t stride_v = whole ? V : l.piece;
    const bool is_big = big(std::min(stride_v, V), n, p->cus);
    const int wave_cols = is_big ? Big::WM : Small::WM;
    for (int64_t v0 = 0; v0 < V; v0 += stride_v) {
      const int64_t width = std::min(stride_v, V - v0);
      const Operand wo = rows_of(weight + v0 * q->weight_stride, q->weight_stride, width, wc);
      a.a = wo.p;
      a.lda = wo.ld;
      a.plane_a = wo.plane;
      a.M = width;
      a.v0 = v0;
      if (way == kForward)
        product<E, TERMS, kSums>(a, is_big, s);
      else if (way == kBoth)
        product<E, TERMS, kExps>(a, is_big, s);
      else
        product<E, TERMS, kProbs>(a, is_big, s);
    }
    if (way != kBackward)
      hipLaunchKernelGGL(k_lse, dim3((unsigned)div_up(n, 16)), dim3(256), 0, s, a.stats,
                         (int)div_up(V, wave_cols), n, a.labels,
                         q->row_weights ? q->row_weights + r0 : nullptr, a.said, V, q->loss + r0,
                         lse_out + r0, hdr, epoch);
    if (!grad) continue;

    Operand xt{};
    if (q->d_weight) xt = columns_of(x, q->hidden_stride, n, factors + r0, reinterpret_cast<E*>(ws + l.xt));
    const int split = split_of(D, n, p->cus);
    for (int64_t v0 = 0; v0 < V; v0 += l.piece) {
      const int64_t width = std::min(l.piece, V - v0);
      Grad g{};
      g.exps = a.exps;
      g.ld_exps = l.ld_exps;
      g.tokens = n;
      g.stats = way == kBoth ? a.stats : nullptr;
      g.wave_cols = wave_cols;
      g.lse = lse + r0;
      g.labels = a.labels;
      g.factors = factors + r0;
      g.most = most;
      g.v0 = v0;
      g.width = width;
      g.V = V;
      g.pitch = up(width, kStep);
      g.plane = n * g.pitch;
      g.pitch_t = up(n, kStep);
      g.plane_t = width * g.pitch_t;
      g.g = q->d_hidden ? ws + l.g : nullptr;
      g.gt = q->d_weight ? ws + l.gt : nullptr;
      hipLaunchKernelGGL((k_grad<T, X>), dim3((unsigned)(g.pitch / kTile * (g.pitch_t / kTile))),
                         dim3(256), 0, s, g);
      if (q->d_hidden) {
        const Operand wt = columns_of(weight + v0 * q->weight_stride, q->weight_stride, width, nullptr, wc);
        Product b{};
        b.a = wt.p;
        b.lda = wt.ld;
        b.plane_a = wt.plane;
        b.b = static_cast<const char*>(g.g);
        b.ldb = g.pitch * 2;
        b.plane_b = g.plane * 2;
        b.M = D;
        b.N = n;
        b.steps = (int)(g.pitch / kStep);
        b.split = split;
        b.sums = at(l.sums);
        b.add = v0 > 0;
        product<E, TERMS, kAdd>(b, big(D, n, p->cus), s);
      }
      if (q->d_weight) {
        const bool first = r0 == 0, last = r0 + n == R;
        const bool direct = (first && last) || q->d_weight_dtype == SGB_F32;
        Product b{};
        b.a = xt.p;
        b.lda = xt.ld;
        b.plane_a = xt.plane;
        b.b = static_cast<const char*>(g.gt);
        b.ldb = g.pitch_t * 2;
        b.plane_b = g.plane_t * 2;
        b.M = D;
        b.N = width;
        b.steps = (int)(g.pitch_t / kStep);
        b.split = 1;
        b.most = most;
        b.scale = q->grad_scale / kBy;
        if (direct || last) {
          const size_t e = elem_size(q->d_weight_dtype);
          b.out = static_cast<char*>(q->d_weight) + v0 * q->d_weight_stride * e;
          b.ldo = q->d_weight_stride;
          b.out_dtype = q->d_weight_dtype;
          b.add = q->accumulate || (direct && !first);
          b.add_from = direct ? nullptr : at(l.dw) + v0 * D;
        } else {
          b.out = at(l.dw) + v0 * D;
          b.ldo = D;
          b.out_dtype = SGB_F32;
          b.add = !first;
        }
        product<E, TERMS, kOut>(b, big(D, width, p->cus), s);
      }
    }
    if (q->d_hidden)
      hipLaunchKernelGGL(k_join<T>, dim3(blocks(n * div_up(D, 8), p->cus)), dim3(256), 0, s, at(l.sums),
                         split, n, D, factors + r0, q->grad_scale / kBy,
                         static_cast<T*>(q->d_hidden) + r0 * q->d_hidden_stride, q->d_hidden_stride);
  }
}

template <typename T>
void zero(const sgb_vocab_ce_s* p, const sgb_vocab_ce_args* q, hipStream_t s) {
  hipLaunchKernelGGL(k_zero<T>, dim3(blocks(p->V * p->D, p->cus)), dim3(256), 0, s,
                     static_cast<T*>(q->d_weight), q->d_weight_stride, p->V, p->D);
}

sgb_status call(sgb_vocab_ce p, const sgb_vocab_ce_args* q, Way way, void* ws, size_t ws_bytes,
                void* stream_) {
  if (!p || !q) return SGB_ERR_INVALID_ARGUMENT;
  const int64_t R = q->rows, V = p->V, D = p->D;
  const bool grad = way != kForward;
  if (!float_dtype(q->dtype) || R < 0 || R >= (1ll << 31)) return SGB_ERR_INVALID_ARGUMENT;
  const size_t e = elem_size(q->dtype);
  if (grad) {
    if (!std::isfinite(q->grad_scale) || (q->accumulate != 0 && q->accumulate != 1))
      return SGB_ERR_INVALID_ARGUMENT;
    if (q->d_weight && ((q->d_weight_dtype != SGB_F32 && q->d_weight_dtype != q->dtype) ||
                        !matrix_ok(q->d_weight, D, q->d_weight_stride, elem_size(q->d_weight_dtype))))
      return SGB_ERR_INVALID_ARGUMENT;
    if (way == kBackward && !q->d_hidden && !q->d_weight) return SGB_ERR_INVALID_ARGUMENT;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (R == 0 && (!grad || !q->d_weight || q->accumulate)) return SGB_OK;
  if (R > 0) {
    if (!matrix_ok(q->hidden, D, q->hidden_stride, e) || !matrix_ok(q->weight, D, q->weight_stride, e) ||
        !q->labels || !aligned(q->labels, 8) || !aligned(q->row_weights, 4) || !aligned(q->lse, 4))
      return SGB_ERR_INVALID_ARGUMENT;
    if (way != kBackward && (!q->loss || !aligned(q->loss, 4))) return SGB_ERR_INVALID_ARGUMENT;
    if (way == kBackward && (!q->lse || !aligned(q->grad_loss, 4))) return SGB_ERR_INVALID_ARGUMENT;
    if (grad && q->d_hidden && !matrix_ok(q->d_hidden, D, q->d_hidden_stride, e))
      return SGB_ERR_INVALID_ARGUMENT;
    if (grad) {
      const size_t ew = elem_size(q->d_weight_dtype);
      if (overlap(q->d_hidden, D, q->d_hidden_stride, e, q->hidden, D, q->hidden_stride, e, R) ||
          overlap(q->d_hidden, D, q->d_hidden_stride, e, q->weight, D, q->weight_stride, e, R, V) ||
          overlap(q->d_weight, D, q->d_weight_stride, ew, q->hidden, D, q->hidden_stride, e, V, R) ||
          overlap(q->d_weight, D, q->d_weight_stride, ew, q->weight, D, q->weight_stride, e, V) ||
          overlap(q->d_weight, D, q->d_weight_stride, ew, q->d_hidden, D, q->d_hidden_stride, e, V, R))
        return SGB_ERR_INVALID_ARGUMENT;
    }
    if (!workspace_ok(ws)) return SGB_ERR_INVALID_ARGUMENT;
  }
  const Layout l = layout(p, std::max<int64_t>(R, 1), q->dtype, grad);
  if (R > 0 && ws_bytes < l.bytes) return SGB_ERR_WORKSPACE_TOO_SMALL;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  if (R == 0) {
    q->d_weight_dtype == SGB_F32 ? zero<float>(p, q, s)
    : q->dtype == SGB_BF16       ? zero<bf16_t>(p, q, s)
                                 : zero<f16_t>(p, q, s);
  } else if (q->dtype == SGB_F32) {
    enqueue<float>(p, q, way, l, static_cast<char*>(ws), s);
  } else if (q->dtype == SGB_BF16) {
    enqueue<bf16_t>(p, q, way, l, static_cast<char*>(ws), s);
  } else {
    enqueue<f16_t>(p, q, way, l, static_cast<char*>(ws), s);
  }
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

}  // namespace

extern "C" {

sgb_status sgb_vocab_ce_create(sgb_vocab_ce* out, int32_t D, int64_t V) {
  if (!out) return SGB_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (D < 1 || V < 1) return SGB_ERR_INVALID_ARGUMENT;
  if (D > kMaxD || V > kMaxV) return SGB_ERR_UNSUPPORTED;
  sgb_vocab_ce_s* p = new (std::nothrow) sgb_vocab_ce_s();
  if (!p) return SGB_ERR_HIP;
  p->device = current_device();
  p->cus = compute_units(p->device);
  p->D = D;
  p->V = V;
  *out = p;
  return SGB_OK;
}

void sgb_vocab_ce_destroy(sgb_vocab_ce p) { delete p; }

sgb_status sgb_vocab_ce_workspace_bytes(sgb_vocab_ce p, int64_t rows, int32_t dtype,
                                        int32_t gradient, size_t* bytes) {
  if (!p || !bytes || rows < 0 || rows >= (1ll << 31) || !float_dtype(dtype))
    return SGB_ERR_INVALID_ARGUMENT;
  *bytes = layout(p, std::max<int64_t>(rows, 1), dtype, gradient != 0).bytes;
  return SGB_OK;
}

sgb_status sgb_vocab_ce_forward(sgb_vocab_ce p, const sgb_vocab_ce_args* q, void* ws,
                                size_t ws_bytes, void* stream) {
  return call(p, q, kForward, ws, ws_bytes, stream);
}
sgb_status sgb_vocab_ce_backward(sgb_vocab_ce p, const sgb_vocab_ce_args* q, void* ws,
                                 size_t ws_bytes, void* stream) {
  return call(p, q, kBackward, ws, ws_bytes, stream);
}
sgb_status sgb_vocab_ce_loss_grad(sgb_vocab_ce p, const sgb_vocab_ce_args* q, void* ws,
                                  size_t ws_bytes, void* stream) {
  return call(p, q, kBoth, ws, ws_bytes, stream);
}

}  // extern "C"
