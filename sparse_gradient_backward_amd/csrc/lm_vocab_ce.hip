// lm_vocab_ce.hip -- cross-entropy of the head's product over a large
// vocabulary, of libsgb_lm.so (formulas: include/sgb_lm_step.h).
//
// One product kernel, C = A B^T, and four epilogues:
//   logits   A = weight rows, B = hidden rows: each wave leaves the largest of
//            its logits and the sum of exponentials below it a token (kSums), and
//            the exponentials themselves where gradients are to follow (kExps;
//            kProbs, relative to a forward's lse);
//   d_hidden A = the weight, B = the logits' gradient, summed over the vocabulary;
//   d_weight A = hidden transposed, B = the logits' gradient, over the tokens
//            (both kGrads).
// The vocabulary, or the columns of the result, are A's rows: a lane holds four
// neighbours of them for one of B's rows, so the softmax's sums stay in the
// lane and the stores are of whole words.  An operand that is held the other way,
// the weight for d_hidden and the logits' gradient for d_weight, is read
// transposed from LDS by the instruction for it: a copy of it cost 105 us a
// piece of 128 M elements.  What is copied are hidden rows (transposed for
// d_weight, and where they end within a step) and weight rows that are no whole
// words of 16 bytes.
//
// A chunk of tokens takes three products: its exponentials wait in 16 bits
// (32 for fp16 and fp32 operands) for the row sums, since computing the logits
// again would be a fourth.  They are relative to the largest of a wave's
// columns (in a backward, the row's log-sum-exp) and scaled by 2^15, so fp16 holds 11
// bits of all that matter but the label's, whose gradient is computed from its
// logit, and the only rounding to the operands' type is that of the gradient itself.
// (Of few rows, or on demand, what it leaves goes into the products as well.)
//
// Bound by the matrix units where there are many tokens: 8192 tokens of 4096,
// 131072 in the vocabulary, bf16: 19.8 to 20.7 ms (cards differ) for the loss and
// both gradients, 1275 to 1335 TFLOP/s, where a library product of such sizes
// reaches 1500; the three products take 6.9, 6.5 and 6.4 ms, the rest 0.9.  Few
// tokens are bound by the weight's traffic: the loss of 8 takes 185 us, 5.8 TB/s.

#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "lm_internal.h"
#include "sgb_lm_step.h"

using namespace sgb_lm;

namespace {

constexpr int kMaxD = 16384;
constexpr int64_t kMaxV = 1 << 23;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
constexpr float kUp = 32768.f;   // 2^15: see above; fp16 gradients are scaled by it too

typedef float F4 __attribute__((ext_vector_type(4)));

// 16 bytes of an operand's row: a lane's part of a fragment.
template <typename E>
struct Frag {
  typedef E type __attribute__((ext_vector_type(16 / sizeof(E))));
};
__device__ __forceinline__ F4 mfma(Frag<bf16_t>::type a, Frag<bf16_t>::type b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma(Frag<f16_t>::type a, Frag<f16_t>::type b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ F4 mfma(float a, float b, F4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// ---------------------------------------------------------------- the product

constexpr int kRowBytes = 128;  // of the summed dimension a step
template <typename E>
constexpr int kStepOf = kRowBytes / (int)sizeof(E);
constexpr int kPad = 64;        // and what it is rounded up to

// A workgroup's tile of C (rows of A by rows of B), a wave's, and the steps that
// are loaded between two barriers.
struct Big {  // one workgroup a compute unit, for products that give each one
  static constexpr int TM = 256, TN = 256, WM = 128, WN = 64, kSteps = 1;
};
struct BigOther : Big {  // fewer fragments of the operand that is read transposed
  static constexpr int WM = 64, WN = 128;
};
struct Medium {  // two a compute unit, one at its start or end while the other multiplies
  static constexpr int TM = 128, TN = 128, WM = 64, WN = 64, kSteps = 1;
};
struct Tiny {  // for the time that loads take, not for how many there are
  static constexpr int TM = 64, TN = 64, WM = 32, WN = 32, kSteps = 4;
};
struct Thin {  // few of B's rows: what bounds it is A's being read
  static constexpr int TM = 256, TN = 16, WM = 64, WN = 16, kSteps = 1;
};
struct Brief {  // few steps: the result's being written; four a compute unit, one buffer each
  static constexpr int TM = 128, TN = 128, WM = 64, WN = 64, kSteps = 1;
};
template <typename C>
constexpr int kThreadsOf = C::TM / C::WM * (C::TN / C::WN) * 64;

template <typename C>
constexpr int kBufBytes = C::kSteps * (C::TM + C::TN) * kRowBytes;

enum Epilogue { kSums, kExps, kProbs, kGrads };
enum ByRow { kPlain, kKept, kScaled };

// What says how much a row counts.
struct Rows {
  const int64_t* labels;
  const float *weights, *above;  // null: ones
  int64_t V;
};
__device__ __forceinline__ float factor_of(const Rows& q, int64_t r) {
  const int64_t label = q.labels[r];
  const float w = value_or(q.weights, r, 1.f), g = value_or(q.above, r, 1.f);
  return w == 0.f || label < 0 || label >= q.V ? 0.f : w * g;
}

struct Product {
  const char *a, *b;
  int64_t lda, ldb;          // bytes from row to row; of 16
  int64_t plane_a, plane_b;  // bytes from one bf16 part of fp32 operands to the next
  int64_t M, N;              // rows of a, b; of an operand held the other way, columns,
  int64_t cols_a, cols_b;    // of which so many can be read
  int steps, split;          // of the summed dimension, over 1..steps workgroups
  int last;                  // elements of a's last step that are the operand's: rows
                             // that are no whole steps are read where they are
  const char* end_a;         // what can be read of it
  int tm, tn;
  Rows rows;
  // logits
  float2* stats;             // [vocabulary / WM][tokens]
  int64_t tokens;
  const float* lse;
  float* said;               // the label's logit
  void* exps;                // [tokens][ld_exps]
  int64_t ld_exps, v0, V;    // v0: the piece's first token of the vocabulary
  // gradients: sums for a later kernel, or out
  float* sums;               // [split][N][M] or null
  bool add;                  // to what is there
  void* out;                 // [N][ldo]
  int64_t ldo;
  int out_dtype;
  const float* add_from;     // [N][M] or null
  const float* most;         // (null: 1) times scale: what the sums are multiplied by
  float scale;
  int by_row;                // d_hidden, add_from with it: kScaled, or only kept (0 for
                             // a row that does not count)
};

// Which bf16 parts (0: the highest) the products of fp32 operands are of, the
// smallest first; those left out are below 2^-25 of the whole.
constexpr uint32_t kPartsA = 0u << 0 | 2u << 2 | 1u << 4 | 0u << 6 | 1u << 8 | 0u << 10;
constexpr uint32_t kPartsB = 2u << 0 | 0u << 2 | 1u << 4 | 1u << 6 | 0u << 8 | 0u << 10;

// 1 KB a wave and load to consecutive addresses of LDS, from `base`, the same for
// all lanes, and a lane's offset (a buffer's load: no addresses of 64 bits).
template <int J>
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t bytes, const uint32_t (&off)[J],
                                            char* lds) {
#ifdef __HIP_DEVICE_COMPILE__
  const __amdgpu_buffer_rsrc_t from =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, (int)bytes, 0x00027000);
#pragma unroll
  for (int j = 0; j < J; ++j)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        from, (__attribute__((address_space(3))) void*)(lds + j * 1024), 16, off[j], 0, 0, 0);
#endif
}

// The workgroup's loads of R rows of 64 elements, straight to LDS, 16 bytes a
// lane.  A row is 128 bytes of LDS; its 16-byte parts are stored in an order
// of the row's own (exclusive or with row / 2), so that 16 lanes that read the
// same part of 16 rows touch all banks once.  LDS addresses of one load are
// consecutive over the lanes, so the order is made by what a lane loads.
template <int R, int WAVES>
struct Stage {
  // (where there are fewer loads than waves, some waves make the same one)
  static constexpr int kLoads = R / 8, J = kLoads < WAVES ? 1 : kLoads / WAVES;
  uint32_t off[J];
  __device__ __forceinline__ void init(int wave, int lane, int64_t left, int64_t ld) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int row = (wave * J % kLoads + j) * 8 + (lane >> 3);
      const int part = (lane & 7) ^ ((row >> 1) & 7);
      // rows past the last are copies of it: nothing is read out of range
      off[j] = (uint32_t)min((int64_t)row, left - 1) * (uint32_t)ld + part * 16;
    }
  }
  __device__ __forceinline__ void load(const char* base, uint32_t bytes, char* lds, int wave) const {
    load_to_lds(base, bytes, off, lds + wave * J % kLoads * 1024);
  }
};

// The same of an operand held the other way, the summed dimension from row to
// row: a step's rows of R elements.  Elements of 16 bits are read from it
// transposed, 16 lanes at a time four rows of 32 bytes; of 32 bits one by one, 64
// bytes from each of four rows.  The rows' pieces of such sizes are stored in an
// order that puts those read at once into different banks.
template <int R, typename E>
struct Other {
  static constexpr int kRow = R * (int)sizeof(E), kPiece = 16 * (int)sizeof(E);
  static __device__ __forceinline__ int order(int row) {
    if (sizeof(E) == 4) return row >> 2 & 3;
    if (R > 64) return (row & 3) | (row >> 3 & 1) << 2;
    return (row >> 1 & 1) | (row >> 3 & 1) << 1;  // two rows to a round of banks
  }
  // A lane's first element of 16 columns from `col` on (of 16), in its first row;
  // those 16 i further are at ^ i * kPiece (col a multiple of as many as there are).
  static __device__ __forceinline__ uint32_t at(int lane, int col) {
    const int row = sizeof(E) == 4 ? 4 * (lane >> 4) : 8 * (lane >> 4) + (lane >> 2 & 3);
    const int in = sizeof(E) == 4 ? (lane & 15) * 4 : (lane & 3) * 8;
    return row * kRow + in + (col / 16 ^ order(row)) * kPiece;
  }
  static __device__ __forceinline__ typename Frag<E>::type read(const char* from) {
    typename Frag<E>::type v{};
#ifdef __HIP_DEVICE_COMPILE__
    if constexpr (sizeof(E) == 4) {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = *reinterpret_cast<const float*>(from + k * kRow);
    } else {
      typedef short H __attribute__((ext_vector_type(4)));
      typedef __attribute__((address_space(3))) H* P;
      struct {
        H lo, hi;
      } h = {__builtin_amdgcn_ds_read_tr16_b64_v4i16((P)from),
             __builtin_amdgcn_ds_read_tr16_b64_v4i16((P)(from + 4 * kRow))};
      v = __builtin_bit_cast(typename Frag<E>::type, h);
    }
#endif
    return v;
  }
};
template <int R, int WAVES, typename E>
struct StageOther {
  static constexpr int J = R / (8 * WAVES), kParts = R * (int)sizeof(E) / 16;
  uint32_t off[J];
  __device__ __forceinline__ void init(int wave, int lane, int64_t left, int64_t ld) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int at = (wave * J + j) * 64 + lane;  // 16 bytes each
      const int row = at / kParts;
      const int part = at % kParts ^ Other<R, E>::order(row) * (Other<R, E>::kPiece / 16);
      // columns past the last are copies of others
      off[j] = (uint32_t)row * (uint32_t)ld +
               (uint32_t)min((int64_t)part, left * (int)sizeof(E) / 16 - 1) * 16;
    }
  }
  __device__ __forceinline__ void load(const char* base, uint32_t bytes, char* lds, int wave) const {
    load_to_lds(base, bytes, off, lds + wave * (J * 1024));
  }
};

// Everything that this wave loads has arrived, and the others' too after the
// barrier.  (The builtin, since the compiler counts loads to LDS itself, and
// does not see a wait in assembly.)
__device__ __forceinline__ void all_loaded() {
  __builtin_amdgcn_s_waitcnt(7 << 4);  // vmcnt(0) lgkmcnt(0)
  __syncthreads();
}

// LAST: results, non-temporally: but for a d_weight or its sums that a later chunk
// adds to, no kernel here reads them again (both gradients of 8 rows of 4096, 131072
// tokens, bf16: 841 us so, 911 otherwise; of 300 1480 and 1522, of 8192 the same).
template <typename T, bool LAST = false>
__device__ __forceinline__ void store4(void* row, int64_t at, F4 v, int64_t n) {
  T* p = static_cast<T*>(row) + at;
  typedef T T4 __attribute__((ext_vector_type(4)));
  typedef T4 Any __attribute__((aligned(sizeof(T))));
  const T4 t = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
  if (n >= 4) {
    if (LAST)
      __builtin_nontemporal_store(t, reinterpret_cast<Any*>(p));
    else
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

// A wave's results on their way out, through LDS of its own: 16 of B's rows by
// FRAGS times 16 of A's, put in as the matrix instruction leaves them (four
// neighbours of a row a lane) and got as 16 bytes of whole rows, so that a store
// fills lines.  Exponentials of 8192 x 131072 logits of 4096, bf16: 7.5 ms with
// stores of what a lane holds, 7.3 so; of 1021 x 50021 of 1001, fp16: 175 and 163 us.
template <typename O, int FRAGS>
struct Rows16 {
  static constexpr int kFrags = FRAGS, kRow = FRAGS * 16 * (int)sizeof(O), kPitch = kRow + 16;
  static constexpr int kBytes = 16 * kPitch, kLanes = kRow / 16, kTurns = kLanes / 4;
  typedef O Words __attribute__((ext_vector_type(16 / sizeof(O))));
  static __device__ __forceinline__ void put(char* lds, int lane, int i, F4 v) {
    typedef O O4 __attribute__((ext_vector_type(4)));
    const O4 o = {(O)v[0], (O)v[1], (O)v[2], (O)v[3]};
    *reinterpret_cast<O4*>(lds + (lane & 15) * kPitch +
                           (16 * i + 4 * (lane >> 4)) * (int)sizeof(O)) = o;
  }
  static __device__ __forceinline__ int row(int lane, int turn) {
    return turn * (64 / kLanes) + lane / kLanes;
  }
  static __device__ __forceinline__ int col(int lane) {
    return lane % kLanes * (16 / (int)sizeof(O));
  }
  static __device__ __forceinline__ Words get(const char* lds, int lane, int turn) {
    return *reinterpret_cast<const Words*>(lds + row(lane, turn) * kPitch + lane % kLanes * 16);
  }
};

// f over the lanes 16 apart.
template <typename F>
__device__ __forceinline__ float quarters(float x, F f) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

// AO, BO: the operand is held the other way.
template <typename E, int TERMS, int EPI, typename C, bool AO, bool BO>
__device__ __forceinline__ void product_tile(const Product& p, int block, char* buf0, char* buf1) {
  constexpr int TM = C::TM, TN = C::TN, WM = C::WM, WN = C::WN;
  constexpr int WAVES = kThreadsOf<C> / 64, FM = WM / 16, FN = WN / 16;
  constexpr int kBytes = (TM + TN) * kRowBytes;
  constexpr bool kCut = TERMS == 1 && !BO;  // a may end within a step

  // Workgroups go round the eight dies; each die gets a run of tiles of its
  // own, eight tiles of A by some of B at a time, whose operands its L2 shares.
  const int total = p.tm * p.tn * p.split, per = (total + 7) >> 3;
  const int idx = (block & 7) * per + (block >> 3);
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

  typename std::conditional<AO, StageOther<TM, WAVES, E>, Stage<TM, WAVES>>::type sa;
  typename std::conditional<BO, StageOther<TN, WAVES, E>, Stage<TN, WAVES>>::type sb;
  sa.init(wave, lane, (AO ? p.cols_a : p.M) - m0, p.lda);
  sb.init(wave, lane, (BO ? p.cols_b : p.N) - n0, p.ldb);
  const char *a = p.a + m0 * (AO ? (int)sizeof(E) : p.lda);
  const char* b = p.b + n0 * (BO ? (int)sizeof(E) : p.ldb);
  const int from = (int)((int64_t)p.steps * part / p.split);
  const int to = (int)((int64_t)p.steps * (part + 1) / p.split);
  const int steps = (to - from) * TERMS, turns = (steps + C::kSteps - 1) / C::kSteps;
  int term = 0, step = from;
  const uint32_t last_bytes = (uint32_t)min(
      p.end_a - (a + (to - 1) * (AO ? kStepOf<E> * p.lda : (int64_t)kRowBytes)), (int64_t)UINT32_MAX);
  // The next steps' loads; past the last, that one's once more.  (A load that is
  // made only now and then makes the compiler wait for all of them.)
  const auto stage = [&](char* buf) {
#pragma unroll
    for (int s = 0; s < C::kSteps; ++s) {
      const char* pa = a + step * (AO ? kStepOf<E> * p.lda : kRowBytes);
      const char* pb = b + step * (BO ? kStepOf<E> * p.ldb : kRowBytes);
      if (TERMS > 1) {
        pa += (kPartsA >> (2 * term) & 3) * p.plane_a;
        pb += (kPartsB >> (2 * term) & 3) * p.plane_b;
      }
      const bool wrap = step + 1 == to, on = !wrap || term + 1 < TERMS;
      sa.load(pa, kCut && wrap ? last_bytes : UINT32_MAX, buf + s * kBytes, wave);
      sb.load(pb, UINT32_MAX, buf + s * kBytes + TM * kRowBytes, wave);
      term += wrap && on;
      step = wrap ? (on ? from : step) : step + 1;
    }
    __builtin_amdgcn_sched_barrier(0);  // (the compiler would put them off)
  };

  F4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = F4{0.f, 0.f, 0.f, 0.f};

  // A step is two halves, each with its fragments read while the one before
  // multiplies.  A turn's last products come after the barrier that frees its
  // buffer, and cover the next turn's first reads.
  typedef typename Frag<E>::type V;
  typedef Other<TM, E> OA;
  typedef Other<TN, E> OB;
  V fa[2][FM], fb[2][FN];
  const int key = (lane >> 1) & 7, row = (lane & 15) * kRowBytes;
  const uint32_t at_a = OA::at(lane, wm), at_b = OB::at(lane, wn);
  const auto read = [&](const char* buf, int kk) {
    const int at = row + ((kk * 4 + (lane >> 4)) ^ key) * 16;
    // (one address a fragment, made when it is needed: kept, they would spill)
    uint32_t oa = at_a, ob = at_b;
    if (AO) asm volatile("" : "+v"(oa));
    if (BO) asm volatile("" : "+v"(ob));
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (BO)
        fb[kk][j] = OB::read(buf + (TM * kRowBytes + kk * kStepOf<E> / 2 * OB::kRow + (ob ^ j * OB::kPiece)));
      else
        fb[kk][j] = *reinterpret_cast<const V*>(buf + (uint32_t)((TM + wn) * kRowBytes + at + j * 16 * kRowBytes));
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
      if constexpr (AO)
        fa[kk][i] = OA::read(buf + (kk * kStepOf<E> / 2 * OA::kRow + (oa ^ i * OA::kPiece)));
      else
        fa[kk][i] = *reinterpret_cast<const V*>(buf + (uint32_t)(wm * kRowBytes + at + i * 16 * kRowBytes));
    }
  };
  const auto multiply = [&](int kk) {
    // Products and reads in turn.  The first products come before any read: they
    // free their operands' registers for it.
    constexpr int kApart = sizeof(E) == 4 ? 4 : 2;  // reads of a fragment held the other way
    constexpr int kReads = FM * (AO ? kApart : 1) + FN * (BO ? kApart : 1);
    constexpr int kAll = FM * FN * (sizeof(E) == 4 ? 4 : 1);
    constexpr int kLead = kAll > kReads ? kAll - kReads < 8 ? kAll - kReads : 8 : 0;
    constexpr int kEach = kAll - kLead < kReads ? 1 : (kAll - kLead) / kReads;
    constexpr int kEvery = sizeof(E) == 4 ? 4 : 1;  // (fp32: four, far apart: each waits for the one before)
#pragma unroll
    for (int k = 0; k < kEvery; ++k)
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if constexpr (sizeof(E) == 4)
            acc[i][j] = mfma(fa[kk][i][k], fb[kk][j][k], acc[i][j]);
          else
            acc[i][j] = mfma(fa[kk][i], fb[kk][j], acc[i][j]);
        }
    if (kLead) __builtin_amdgcn_sched_group_barrier(0x008, kLead, 0);
#pragma unroll
    for (int i = 0; i < kReads && i < kAll; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
    }
    if (kAll > kLead + kEach * kReads)
      __builtin_amdgcn_sched_group_barrier(0x008, kAll - kLead - kEach * kReads, 0);
  };
  // What was read of a past its end (what follows it in memory, or nothing) is
  // made zero, as b's is there.
  const auto cut = [&](int kk, int s) {
    if constexpr (kCut) {
      const int most = from + s + 1 == p.steps ? p.last : kStepOf<E>;
      const int left = most - (kk * kStepOf<E> / 2 + (lane >> 4) * (16 / (int)sizeof(E)));
      typedef uint32_t U4 __attribute__((ext_vector_type(4)));
      U4 keep;
#pragma unroll
      for (int w = 0; w < 4; ++w)
        keep[w] = sizeof(E) == 4 ? (left > w ? ~0u : 0u)
                                 : (left > 2 * w + 1 ? ~0u : left > 2 * w ? 0xffffu : 0u);
#pragma unroll
      for (int i = 0; i < FM; ++i) fa[kk][i] = __builtin_bit_cast(V, __builtin_bit_cast(U4, fa[kk][i]) & keep);
    }
  };
  // a turn's steps but the last of their products
  const auto most = [&](const char* buf) {
    read(buf, 1);
    multiply(0);
  };
  const auto turn = [&](const char* buf) {
#pragma unroll
    for (int s = 0; s < C::kSteps; ++s) {
      most(buf + s * kBytes);
      if (s + 1 == C::kSteps) break;
      read(buf + (s + 1) * kBytes, 0);
      multiply(1);
    }
  };

  stage(buf0);
  if constexpr (__is_same(C, Brief)) {
    for (int s = 1;; ++s) {
      all_loaded();
      read(buf0, 0);
      cut(0, s - 1);
      multiply(0);
      read(buf0, 1);
      cut(1, s - 1);
      multiply(1);
      if (s >= turns) break;
      __syncthreads();
      stage(buf0);
    }
  } else {
    stage(buf1);
    all_loaded();
    read(buf0, 0);
    int left = turns;
    for (; left > 2; left -= 2) {
      turn(buf0);
      all_loaded();
      stage(buf0);
      read(buf1, 0);
      multiply(1);
      turn(buf1);
      all_loaded();
      stage(buf1);
      read(buf0, 0);
      multiply(1);
    }
    if (left > 1) {
      turn(buf0);
      all_loaded();
      read(buf1, 0);
      multiply(1);
    }
    const char* buf = left > 1 ? buf1 : buf0;
    int s = (turns - 1) * C::kSteps;
    cut(0, s);
    most(buf);
    for (++s; s < steps; ++s) {  // (none where a turn is one step)
      buf += kBytes;
      read(buf, 0);
      multiply(1);
      cut(0, s);
      most(buf);
    }
    cut(1, steps - 1);
    multiply(1);
  }
  all_loaded();  // LDS is free: no load to it is under way any more

  // acc[i][j][k]: C's row (of A) m0 + wm + 16 i + 4 (lane / 16) + k, its column
  // (of B) n0 + wn + 16 j + lane % 16
  const int64_t mw = m0 + wm + 4 * (lane >> 4);
  char* own = __is_same(C, Brief) ? buf0 + wave * Rows16<float, 4>::kBytes
                                  : (wave < WAVES / 2 ? buf0 : buf1) +
                                        wave % (WAVES / 2) * Rows16<float, 4>::kBytes;
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    __builtin_amdgcn_sched_barrier(0);  // (all at once would spill)
    const int64_t nw = n0 + wn + 16 * j, n = nw + (lane & 15);
    const bool there = n < p.N;
    if constexpr (EPI == kGrads) {
      float by = 1.f;
      if (!p.sums)
        by = p.scale * (p.by_row == kPlain ? value_or(p.most, 0, 1.f)
                        : !there           ? 0.f
                        : p.by_row == kKept ? (factor_of(p.rows, n) != 0.f ? 1.f : 0.f)
                                            : factor_of(p.rows, n));
      typedef Rows16<float, (FM < 4 ? FM : 4)> L;
#pragma unroll
      for (int i0 = 0; i0 < FM; i0 += L::kFrags) {
#pragma unroll
        for (int i = 0; i < L::kFrags; ++i) L::put(own, lane, i, acc[i0 + i][j]);
#pragma unroll
        for (int u = 0; u < L::kTurns; ++u) {
          const int r = L::row(lane, u);
          const float scale = __shfl(by, r);
          const int64_t at = nw + r, m = m0 + wm + 16 * i0 + L::col(lane), n4 = p.M - m;
          F4 v = L::get(own, lane, u);
          if (at >= p.N || n4 <= 0) continue;
          if (p.sums) {
            float* out = p.sums + ((int64_t)part * p.N + at) * p.M;
            if (p.add) v += load4<float>(out, m, n4);
            store4<float>(out, m, v, n4);
            continue;
          }
          F4 more = {0.f, 0.f, 0.f, 0.f};
          if (p.add_from) more = load4<float>(p.add_from + at * p.M, m, n4);
          if (p.by_row != kPlain)
            v = scale == 0.f ? F4{0.f, 0.f, 0.f, 0.f} : (v + more) * scale;
          else
            v = v * scale + more;
          if (p.out_dtype == SGB_F32) {
            float* out = static_cast<float*>(p.out) + at * p.ldo;
            if (p.add) v += load4<float>(out, m, n4);
            store4<float, true>(out, m, v, n4);
          } else {
            E* out = static_cast<E*>(p.out) + at * p.ldo;
            if (p.add) v += load4<E>(out, m, n4);
            store4<E, true>(out, m, v, n4);
          }
        }
      }
    } else {
      typedef typename std::conditional<__is_same(E, bf16_t) && TERMS == 1, f16_t, float>::type X;
      float top = 0.f, sum = 0.f;
      if constexpr (EPI != kProbs || sizeof(X) == 2) {  // (k_grad takes it from 16 bits)
        const int64_t label = there ? p.rows.labels[n] - (p.v0 + m0 + wm) : -1;
        if (label >= 0 && label < WM && label + m0 + wm < p.M) {
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (label == 16 * i + 4 * (lane >> 4) + k) p.said[n] = acc[i][j][k];
        }
      }
      if constexpr (EPI == kProbs) {
        if (there) top = p.lse[n];
      } else {
        if (m0 + wm + WM > p.M) {  // past the vocabulary
#pragma unroll
          for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (mw + 16 * i + k >= p.M) acc[i][j][k] = -INFINITY;
        }
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) top = fmaxf(top, acc[i][j][k]);
        top = quarters(top, [](float x, float y) { return fmaxf(x, y); });
        if (top == -INFINITY) top = 0.f;  // nothing but -inf: the sum is 0
      }
      typedef Rows16<X, (FM < 16 / (int)sizeof(X) ? FM : 16 / (int)sizeof(X))> L;
#pragma unroll
      for (int i0 = 0; i0 < FM; i0 += L::kFrags) {
#pragma unroll
        for (int i = 0; i < L::kFrags; ++i) {
          F4 v;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = exp2_((acc[i0 + i][j][k] - top) * kLog2e);
            sum += v[k];
          }
          if (EPI != kSums) L::put(own, lane, i, v * (sizeof(X) == 2 ? kUp : 1.f));
        }
        if constexpr (EPI != kSums) {
#pragma unroll
          for (int u = 0; u < L::kTurns; ++u) {
            const int64_t at = nw + L::row(lane, u);
            const auto v = L::get(own, lane, u);
            if (at >= p.N) continue;
            X* out = static_cast<X*>(p.exps) + at * p.ld_exps + (p.v0 + m0 + wm + 16 * i0 + L::col(lane));
            *reinterpret_cast<typename L::Words*>(out) = v;
          }
        }
      }
      if constexpr (EPI != kProbs) {
        sum = quarters(sum, [](float x, float y) { return x + y; });
        if (there && lane < 16)
          p.stats[(p.v0 + m0 + wm) / WM * p.tokens + n] = make_float2(top, sum);
      }
    }
  }
}

// (buf0, buf1: variables of their own, so that a read of one does not wait for
// loads to the other)
template <typename E, int TERMS, int EPI, typename C, bool AO, bool BO>
__global__ __launch_bounds__(kThreadsOf<C>, __is_same(C, Brief) ? 4 : 2) void k_product(Product p) {
  __shared__ __attribute__((aligned(1024))) char buf0[kBufBytes<C>];
  __shared__ __attribute__((aligned(1024))) char buf1[__is_same(C, Brief) ? 16 : kBufBytes<C>];
  product_tile<E, TERMS, EPI, C, AO, BO>(p, (int)blockIdx.x, buf0, buf1);
}

// d_hidden in the first workgroups, d_weight in the others.
template <typename E, int TERMS, typename C>
__global__ __launch_bounds__(kThreadsOf<C>, 2) void k_products(Product h, Product w, int first) {
  __shared__ __attribute__((aligned(1024))) char buf0[kBufBytes<C>], buf1[kBufBytes<C>];
  const int block = (int)blockIdx.x;
  if (block < first)
    product_tile<E, TERMS, kGrads, C, true, false>(h, block, buf0, buf1);
  else
    product_tile<E, TERMS, kGrads, C, false, true>(w, block - first, buf0, buf1);
}

// ---------------------------------------------------------------- copies

// What an operand's element becomes: itself, or (SPLIT) the three bf16 parts of an
// fp32 number, each what the ones before it leave (exact but for subnormals).
template <typename T, bool SPLIT>
struct Parts {
  static constexpr int kCount = 1;
  typedef T E;
  static __device__ __forceinline__ void split(T v, E (&out)[1]) { out[0] = v; }
};
template <>
struct Parts<float, true> {
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

template <typename T, bool SPLIT, typename V>
__device__ __forceinline__ void store_parts(const V (&v)[8], typename Parts<T, SPLIT>::E* to,
                                            int64_t plane) {
  typedef typename Parts<T, SPLIT>::E E;
  constexpr int P = Parts<T, SPLIT>::kCount;
  __attribute__((aligned(16))) E out[P][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    E e[P];
    Parts<T, SPLIT>::split((T)v[i], e);
#pragma unroll
    for (int k = 0; k < P; ++k) out[k][i] = e[k];
  }
#pragma unroll
  for (int k = 0; k < P; ++k)
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i)
      reinterpret_cast<uint4*>(to + k * plane)[i] = reinterpret_cast<const uint4*>(out[k])[i];
}

constexpr int kTile = 64;

// An operand's rows [rows][D] as the products read them: [up(rows)][pitch] with
// zeros past D and past the last row; transposed to [D][pitch_t] with zeros past
// the last row and in rows that do not count (what they hold may be no number);
// or both.
template <typename T, bool SPLIT>
struct Copy {
  typedef typename Parts<T, SPLIT>::E E;
  const T* src;
  int64_t stride, rows;
  int D;
  E *to, *to_t;  // or null
  int64_t pitch, plane, pitch_t, plane_t;
  Rows count;
};

// Tiles of 64 x 64, of `a` in the first workgroups and of `b` in the others.
template <typename T, bool SPLIT>
__global__ __launch_bounds__(256) void k_copy(Copy<T, SPLIT> a, Copy<T, SPLIT> b, unsigned first) {
  __shared__ __attribute__((aligned(16))) T tile[kTile][kTile + 4 / sizeof(T)];
  unsigned block = blockIdx.x;
  if (block >= first) {
    a = b;
    block -= first;
  }
  const unsigned across = (unsigned)((a.D + kTile - 1) / kTile);
  const int64_t r0 = (int64_t)(block / across) * kTile;
  const int d0 = (int)(block % across) * kTile;
  const int t = (int)threadIdx.x;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int r = (t >> 3) + 32 * u, c = (t & 7) * 8;
    const bool there = r0 + r < a.rows;
    Raw8<T> raw = load8(a.src + (r0 + r) * a.stride + d0 + c, there ? min(8, a.D - d0 - c) : 0);
    if (a.to) {
      T v[8];
      __builtin_memcpy(v, &raw, sizeof v);
      store_parts<T, SPLIT>(v, a.to + (r0 + r) * a.pitch + d0 + c, a.plane);
    }
    if (!a.to_t) continue;
    const bool on = there && factor_of(a.count, r0 + r) != 0.f;
    uint32_t* row = reinterpret_cast<uint32_t*>(&tile[r][c]);
#pragma unroll
    for (int i = 0; i < Vec<T>::kWords; ++i) row[i] = on ? raw.w[i] : 0u;
  }
  if (!a.to_t) return;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int d = (t >> 3) + 32 * u, c = (t & 7) * 8;
    if (d0 + d >= a.D) continue;
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = tile[c + i][d];
    store_parts<T, SPLIT>(v, a.to_t + (int64_t)(d0 + d) * a.pitch_t + r0 + c, a.plane_t);
  }
}

// ---------------------------------------------------------------- row work

// The largest magnitude of the rows' factors.  fp16 gradients for d_weight carry
// the factor over it, so that none leaves the type's range.
__global__ __launch_bounds__(1024) void k_most(Rows q, int64_t rows, float* most) {
  __shared__ float part[16];
  float top = 0.f;
  for (int64_t r = threadIdx.x; r < rows; r += 1024) top = fmaxf(top, fabsf(factor_of(q, r)));
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = top;
  __syncthreads();
  if (threadIdx.x < 64) {
    top = wave_max(threadIdx.x < 16 ? part[threadIdx.x] : 0.f);
    if (threadIdx.x == 0) *most = top;
  }
}

// A reference and a sum of exponentials relative to it.
struct Sum {
  float m = -INFINITY, s = 0.f;
  __device__ __forceinline__ void add(float2 v) {
    if (v.y == 0.f) return;  // no mass, whatever its reference
    const float top = fmaxf(m, v.x);
    s = s * exp2_((m - top) * kLog2e) + v.y * exp2_((v.x - top) * kLog2e);
    m = top;
  }
  // every `by`th of the waves' sums of a row, from `i` on
  __device__ __forceinline__ void add_all(const float2* stats, int parts, int64_t tokens, int64_t r,
                                          int i, int by) {
    for (; i + 7 * by < parts; i += 8 * by) {
      float2 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = stats[(int64_t)(i + by * u) * tokens + r];
#pragma unroll
      for (int u = 0; u < 8; ++u) add(v[u]);
    }
    for (; i < parts; i += by) add(stats[(int64_t)i * tokens + r]);
  }
  __device__ __forceinline__ float log() const { return m + logf(s); }
};

// Where a row's log-sum-exp and loss go.
struct Loss {
  const float2* stats;
  int parts;
  int64_t tokens;
  Rows rows;
  const float* said;
  float *loss, *lse;
  Header* hdr;
  uint32_t epoch;
};

__device__ __forceinline__ void mark(const Rows& q, int64_t r, Header* hdr, uint32_t epoch) {
  if (q.labels[r] >= q.V && value_or(q.weights, r, 1.f) != 0.f)
    set_status(hdr, epoch, SGB_ERR_INDEX_OUT_OF_RANGE);
}
__device__ __forceinline__ void finish_row(const Loss& q, int64_t r, float lse) {
  q.lse[r] = lse;
  const float f = factor_of(q.rows, r);
  q.loss[r] = f == 0.f ? 0.f : f * (lse - q.said[r]);
  mark(q.rows, r, q.hdr, q.epoch);
}

constexpr int kFewParts = 64;  // sums of a row that k_grad adds up itself
constexpr int kShares = 16;  // of a row's sums, each added up alone and then in turn

// 256 / SHARES rows a workgroup.  (One row of 2048 sums: 25 us with 16 shares, 13
// with 64.)
template <int SHARES>
__global__ __launch_bounds__(256) void k_lse(Loss q) {
  constexpr int kRows = 256 / SHARES;
  __shared__ float2 all[SHARES][kRows + 1];
  const int who = (int)threadIdx.x % kRows, share = (int)threadIdx.x / kRows;
  const int64_t r = (int64_t)blockIdx.x * kRows + who;
  Sum mine;
  if (r < q.tokens) mine.add_all(q.stats, q.parts, q.tokens, r, share, SHARES);
  all[share][who] = make_float2(mine.m, mine.s);
  __syncthreads();
  if (threadIdx.x < kRows && r < q.tokens) {
    Sum sum;
    for (int i = 0; i < SHARES; ++i) sum.add(all[i][who]);
    finish_row(q, r, sum.log());
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) q.hdr->epoch = q.epoch;
}

struct Grad {
  const void* exps;  // [tokens][ld_exps], the chunk's
  int64_t ld_exps;
  int wave_cols;     // of a wave's reference; 0: they are relative to the row's lse
  Loss rows;         // the chunk's; SUM: their lse and loss are found here
  const float* lse;
  const float* most;  // null: 1
  int64_t v0, width;  // the piece
  // over the row's factor, and with it (over the largest); or null
  void *plain, *scaled;  // [up(tokens)][pitch]
  int64_t pitch, plane;
  int64_t rest;      // elements to what the rounding left of each, or 0
};

// The gradient of a piece's logits from their exponentials, in the operands'
// type, zeros past the vocabulary and past the last token.  Of exponentials that
// waited in 16 bits the label's entry, p - 1, comes from its logit instead: where p
// is near one, the rounding (2^-12, the half step below one) may be all of it.  (In
// 32 bits it is 2^-25, less than the log-sum-exp's own.)
template <typename T, bool SPLIT, typename X, bool SUM>
__global__ __launch_bounds__(256) void k_grad(Grad q) {
  typedef typename Parts<T, SPLIT>::E E;
  constexpr float kBy = __is_same(T, f16_t) ? kUp : 1.f;  // fp16 has no room below 2^-24
  __shared__ float2 part[SUM ? kShares : 1][SUM ? kTile : 1];
  const unsigned across = (unsigned)(q.pitch / kTile);
  const int64_t r0 = (int64_t)(blockIdx.x / across) * kTile;
  const int64_t c0 = (int64_t)(blockIdx.x % across) * kTile;
  const int t = (int)threadIdx.x;
  const int64_t tokens = q.rows.tokens;
  // what this thread needs of its two rows, asked for at once
  const int c = (t & 7) * 8;
  const int64_t at = q.v0 + c0 + c;
  Raw8<X> raw[2];
  float f[2], top[2], lse[2];
  int64_t label[2];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int64_t r = min(r0 + (t >> 3) + 32 * u, tokens - 1);
    raw[u] = *reinterpret_cast<const Raw8<X>*>(static_cast<const X*>(q.exps) + r * q.ld_exps + at);
    top[u] = q.wave_cols ? q.rows.stats[at / q.wave_cols * tokens + r].x : 0.f;
    lse[u] = SUM ? 0.f : q.lse[r];
    f[u] = factor_of(q.rows.rows, r);
    label[u] = q.rows.rows.labels[r] - at;
  }
  const float most = value_or(q.most, 0, 1.f);
  if constexpr (SUM) {
    // (in k_lse's order: both give the same bits)
    const int64_t r = r0 + (t & 63);
    float2 v[kShares / 4][kFewParts / kShares];
#pragma unroll
    for (int u = 0; u < kShares / 4; ++u)
#pragma unroll
      for (int i = 0; i < kFewParts / kShares; ++i) {
        const int at = (t >> 6) + 4 * u + kShares * i;
        v[u][i] = r < tokens && at < q.rows.parts ? q.rows.stats[at * tokens + r] : float2{0.f, 0.f};
      }
#pragma unroll
    for (int u = 0; u < kShares / 4; ++u) {
      Sum mine;
#pragma unroll
      for (int i = 0; i < kFewParts / kShares; ++i) mine.add(v[u][i]);
      part[(t >> 6) + 4 * u][t & 63] = make_float2(mine.m, mine.s);
    }
    __syncthreads();
    if (t < 64) {
      Sum sum;
      for (int i = 0; i < kShares; ++i) sum.add(part[i][t]);
      const float lse = sum.log();
      part[0][t].x = lse;
      if (c0 == 0 && r < tokens) finish_row(q.rows, r, lse);
    }
    __syncthreads();
  } else if (q.wave_cols == 0 && q.v0 + c0 == 0 && t < 64 && r0 + t < tokens) {
    mark(q.rows.rows, r0 + t, q.rows.hdr, q.rows.epoch);
  }
  if (blockIdx.x == 0 && t == 0) q.rows.hdr->epoch = q.rows.epoch;
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const int lr = (t >> 3) + 32 * u;
    const bool there = r0 + lr < tokens;
    const int n = (int)min((int64_t)8, q.v0 + q.width - at);
    float k = sizeof(X) == 2 ? 1.f / kUp : 1.f;
    if (q.wave_cols) k *= exp2_((top[u] - (SUM ? part[0][lr].x : lse[u])) * kLog2e);
    const bool on = there && f[u] != 0.f;
    const float share = on ? f[u] / most : 0.f;
    float v[8], e[8];
    widen8(raw[u], e);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = on && i < n ? (e[i] * k - (sizeof(X) == 4 && label[u] == i ? 1.f : 0.f)) * kBy : 0.f;
    if (sizeof(X) == 2 && on && label[u] >= 0 && label[u] < n) {
      const float less =
          expm1f(q.rows.said[r0 + lr] - (SUM ? part[0][lr].x : lse[u])) * kBy;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (label[u] == i) v[i] = less;
    }
    const auto store = [&](void* out) {
      E* to = static_cast<E*>(out) + (r0 + lr) * q.pitch + c0 + c;
      store_parts<T, SPLIT>(v, to, q.plane);
      if (q.rest == 0) return;
      float left[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) left[i] = v[i] - (float)(E)v[i];
      store_parts<T, SPLIT>(left, to + q.rest, q.plane);
    };
    if (q.plain) store(q.plain);
    if (q.scaled) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= share;
      store(q.scaled);
    }
  }
}

// d_hidden: the parts' sums in their order, the row's factor, one rounding.
template <typename T>
__global__ __launch_bounds__(256) void k_join(const float* sums, int split, int64_t part_rows,
                                              int64_t rows, int D,
                                              Rows count, bool scaled, float scale, T* out,
                                              int64_t stride) {
  const int64_t groups = (D + 7) / 8, all = rows * groups;
  for (int64_t g = (int64_t)blockIdx.x * 256 + threadIdx.x; g < all; g += (int64_t)gridDim.x * 256) {
    const int64_t r = g / groups;
    const int c = (int)(g % groups) * 8, n = min(8, D - c);
    const float f = factor_of(count, r);
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (f != 0.f) {
#pragma unroll 4
      for (int s = 0; s < split; ++s) {
        float x[8];
        widen8(load8(sums + (s * part_rows + r) * D + c, n), x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += x[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] *= scaled ? f * scale : scale;
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

constexpr int64_t kExpBytes = 1ll << 31;     // a chunk's exponentials
constexpr int64_t kStatBytes = 1ll << 28;    // their sums
constexpr int64_t kPieceElems = 1ll << 27;   // a piece's gradients in the operands' type
constexpr int64_t kCopyElems = 1ll << 31;    // the weight's copy
constexpr int kMaxSplit = 32;

// So few rows have room in the products' tiles for what the rounding of the logits'
// gradient leaves, as further rows of d_hidden and a further stretch of d_weight's
// sum.  (Of many rows the roundings average out, to sqrt(2) times the output's own;
// of few one entry makes up a result, and it is up to twice.  More rows carry it if
// the call asks for it, as rows and a stretch of tiles of their own.  Errors of 80 rows of
// 2790, 2880 tokens, bf16: 0.0026 without, 0.0017 with; both gradients of 8 rows of
// 4096, 131072 tokens, 734 and 841 us, of 60 754 and 859, of 300 1480 and 1988, of
// 8192 20.5 and 34.8 ms.)
constexpr int64_t kFewRows = 128;

int64_t up(int64_t n, int64_t to) { return div_up(n, to) * to; }

template <typename C>
int64_t tiles_of(int64_t M, int64_t N) {
  return div_up(M, C::TM) * div_up(N, C::TN);
}

enum Tiles { kBig, kMedium, kTiny, kThin, kBrief };
int wave_cols_of(Tiles t) { return t == kBig ? Big::WM : t == kTiny ? Tiny::WM : Medium::WM; }

// The tiles of a product, and among how many workgroups each tile's summed
// dimension is shared out (their sums are then joined): what takes the least time
// by what a round of workgroups, as many as a compute unit holds at once, was
// measured to take, in us a step of 64 and beside the steps.  A gradient's tiles
// leave more behind than the logits'.  Both sides, in us:
//   loss, 512 tokens of 4096, 131072, bf16      Big 440, Medium 570
//   logits, 1021 of 1001, 50021, fp16           Big 130, Medium 117
//   logits, 512 of 256, 2000, fp32 in parts     Medium 24, Tiny 12
//   loss, 8 tokens of 4096, 131072              Thin 185 bf16, 373 fp32; others 194, 629
//   loss, 40 of the same, bf16                  Thin 281, Medium 198
//   both gradients, 8, 300 and 1000 of the same Brief for d_weight 841, 1480, 3000,
//     bf16                                      others 997, 1657, 2991
//   forward and backward, 6272 of 64, 13617     Brief 251, others 288
struct Choice {
  Tiles tiles;
  int split;
  double us;
};
// 16-bit operands, fp32 in parts (six products of 16 bits), fp32 as it is.
enum Rate { kHalf, kSplit, kWhole };
// For: the logits; a gradient; a gradient with B's rows held the other way.
enum Use { kLogits, kGradient, kOther };
Choice choose(int64_t M, int64_t N, int64_t K, Rate rate, int cus, Use use) {
  const double per64[3][5] = {  // Big, Medium, Tiny, Thin, Brief
      {1.65, 1.05, 0.39, 0.6, 2.3}, {9.9, 6.3, 2.34, 3.6, 0}, {14.0, 7.0, 1.0, 1.8, 15.0}};
  const double rest[3][5] = {{8, 2, 4, 3, 2.5}, {21, 8, 4.5, 3, 10}, {25, 9, 5, 3, 9}};
  const double* beside = rest[use == kLogits ? 0 : rate == kHalf ? 1 : 2];
  const int64_t tiles[5] = {tiles_of<Big>(M, N), tiles_of<Medium>(M, N), tiles_of<Tiny>(M, N),
                            tiles_of<Thin>(M, N), tiles_of<Brief>(M, N)};
  const int at_once[5] = {1, 2, 1, 2, 4};
  // (a round's time where a compute unit gets one workgroup)
  const double alone[5] = {1, rate == kWhole ? 0.6 : 0.75, 1, 0.6, 0.5};
  const int64_t steps = div_up(K, kPad);
  const int most = use == kGradient ? kMaxSplit : 1;
  Choice best{kBig, 1, 1e300};
  for (int t = 0; t < 5; ++t) {
    if (t == kThin && (use == kOther || N > Thin::TN)) continue;
    if (t == kBrief && rate == kSplit) continue;
    for (int split = 1; split <= most && split <= steps; ++split) {
      const int64_t all = tiles[t] * split;
      if (split > 1 && all > 2 * cus) break;
      double us = std::max((double)div_up(all, cus) / at_once[t], alone[t]) *
                  ((double)div_up(steps, split) * per64[rate][t] + beside[t]);
      if (split > 1) us += 4 + 2e-6 * (double)(M * N) * split;  // the sums written and read
      if (us < best.us) best = {(Tiles)t, split, us};
    }
  }
  return best;
}

// fp32 operands in parts take less of the matrix units and have to be copied, at
// 10 bytes an element and 4.5 TB/s: for few rows the copy costs more.  Both
// gradients, us in parts and as they are, tokens of 4096, 32000: 100 1293 and 848,
// 300 2236 and 2135, 1000 4425 and 5716.
bool in_parts(const sgb_vocab_ce_s* p, int64_t rows) {
  const double copy = (double)p->V * p->D * 10 / 4.5e6;
  return choose(p->V, rows, p->D, kSplit, p->cus, kLogits).us + copy <
         choose(p->V, rows, p->D, kWhole, p->cus, kLogits).us;
}

// What a call lays out in its workspace.
struct Layout {
  int parts;           // of an element
  int64_t chunk, pad;  // rows a chunk, rounded up for the summed dimension
  int64_t piece;       // of the vocabulary, whose gradients are held
  int64_t copied;      // and whose weight rows
  int64_t pitch_d, ld_exps;
  size_t lse, said, most, stats, x, xt, w, exps, plain, scaled, sums, dw, bytes;
};

Layout layout(const sgb_vocab_ce_s* p, int64_t rows, int dtype, bool gradient, bool exact) {
  Layout l{};
  l.parts = dtype == SGB_F32 ? 3 : 1;
  const int64_t V = p->V, D = p->D, exp_size = dtype == SGB_BF16 ? 2 : 4;
  l.pitch_d = up(D, kPad);
  l.ld_exps = up(V, 256);  // whole tiles
  int64_t most = kStatBytes / (l.ld_exps / Tiny::WM * 8);
  if (gradient) most = std::min(most, kExpBytes / (l.ld_exps * exp_size));
  most = std::min(most, kPieceElems / l.pitch_d);  // of their copies and sums
  most = std::max<int64_t>(most / 256 * 256, 64);
  l.chunk = std::min(rows, most);
  l.pad = up(l.chunk, kPad);
  // Whole tiles.  Rows that are no whole words of 16 bytes are always copied, as
  // parts are; others only if a stride or an address calls for it.
  const int64_t of_rows = l.parts > 1 ? l.pad
                          : exact     ? 2 * l.pad
                                      : std::max(l.pad, std::min(2 * l.pad, 2 * kFewRows));
  const int64_t room = kPieceElems / l.parts, size = dtype == SGB_F32 ? 4 : 2;
  const int64_t copy_room = l.parts > 1 || D * size % 16 != 0 ? kCopyElems / l.parts : room;
  l.piece = std::min(l.ld_exps, std::max<int64_t>(256, room / of_rows / 256 * 256));
  l.copied = std::min(l.ld_exps, std::max<int64_t>(256, copy_room / l.pitch_d / 256 * 256));
  size_t at = kHeaderBytes;
  const auto take = [&](int64_t bytes) {
    const size_t here = at;
    at += align_up((size_t)bytes, 256);
    return here;
  };
  const int64_t part = 2ll * l.parts;
  l.lse = take(4 * rows);
  l.said = take(4 * rows);
  l.most = take(4);
  l.stats = take(l.ld_exps / Tiny::WM * 8 * l.chunk);
  l.x = take(l.pad * l.pitch_d * part);
  l.w = take(l.copied * l.pitch_d * part);
  if (gradient) {
    l.xt = take(D * of_rows * part);
    l.exps = take(l.chunk * l.ld_exps * exp_size);
    const int64_t grads = std::min(l.ld_exps * of_rows, std::max(room, 256 * of_rows)) * part;
    l.scaled = take(grads);
    if (dtype == SGB_F16) l.plain = take(grads);
    // a split's sums for any fewer rows too: at most 2 cus tiles
    const int64_t shared = 2ll * p->cus * Big::TM * Big::TN / D + 1;
    l.sums = take(std::max(of_rows, std::min(kMaxSplit * of_rows, shared)) * D * 4);
    if (rows > l.chunk && dtype != SGB_F32) l.dw = take(V * D * 4);
  }
  l.bytes = at;
  return l;
}

template <typename C>
unsigned grid_of(Product& p) {
  p.tm = (int)div_up(p.M, C::TM);
  p.tn = (int)div_up(p.N, C::TN);
  return (unsigned)(div_up((int64_t)p.tm * p.tn * p.split, 8) * 8);
}

template <typename E, int TERMS, int EPI, bool AO = false, bool BO = false>
void product(Product p, Tiles tiles, hipStream_t s) {
  if (tiles == kBig)
    hipLaunchKernelGGL((k_product<E, TERMS, EPI, typename std::conditional<AO, BigOther, Big>::type, AO, BO>),
                       dim3(grid_of<Big>(p)), dim3(kThreadsOf<Big>), 0, s, p);
  else if (tiles == kMedium)
    hipLaunchKernelGGL((k_product<E, TERMS, EPI, Medium, AO, BO>), dim3(grid_of<Medium>(p)),
                       dim3(kThreadsOf<Medium>), 0, s, p);
  else if (tiles == kTiny)
    hipLaunchKernelGGL((k_product<E, TERMS, EPI, Tiny, AO, BO>), dim3(grid_of<Tiny>(p)),
                       dim3(kThreadsOf<Tiny>), 0, s, p);
  if constexpr (TERMS == 1)
    if (tiles == kBrief)
      hipLaunchKernelGGL((k_product<E, TERMS, EPI, Brief, AO, BO>), dim3(grid_of<Brief>(p)),
                         dim3(kThreadsOf<Brief>), 0, s, p);
  if constexpr (!BO)
    if (tiles == kThin)
      hipLaunchKernelGGL((k_product<E, TERMS, EPI, Thin, AO, BO>), dim3(grid_of<Thin>(p)),
                         dim3(kThreadsOf<Thin>), 0, s, p);
}

unsigned blocks(int64_t threads, int cus) {
  return (unsigned)std::min<int64_t>(div_up(threads, 256), (int64_t)cus * 32);
}

enum Way { kForward, kBackward, kBoth };

struct Operand {
  const char* p;
  int64_t ld, plane;  // bytes
  const char* end;    // null: rows are whole steps, and as many
  int64_t cols;
};

template <typename T, bool SPLIT>
struct Copies {  // asked for, to be launched together
  Copy<T, SPLIT> c[2];
  int n = 0;
  static unsigned tiles(const Copy<T, SPLIT>& c) {
    return (unsigned)(div_up(c.rows, kTile) * div_up(c.D, kTile));
  }
  void launch(hipStream_t s) {
    if (n == 0) return;
    const unsigned first = tiles(c[0]), second = n > 1 ? tiles(c[1]) : 0;
    hipLaunchKernelGGL((k_copy<T, SPLIT>), dim3(first + second), dim3(256), 0, s, c[0], c[n - 1], first);
    n = 0;
  }
};

template <typename T, bool SPLIT = false>
void enqueue(const sgb_vocab_ce_s* p, const sgb_vocab_ce_args* q, Way way, const Layout& l, char* ws,
             hipStream_t s) {
  typedef typename Parts<T, SPLIT>::E E;
  constexpr int TERMS = SPLIT ? 6 : 1, ES = sizeof(E);
  constexpr Rate RATE = SPLIT ? kSplit : ES == 4 ? kWhole : kHalf;
  typedef typename std::conditional<__is_same(T, bf16_t), f16_t, float>::type X;
  constexpr float kBy = __is_same(T, f16_t) ? kUp : 1.f;
  const int64_t R = q->rows, V = p->V;
  const int D = p->D;
  const bool grad = way != kForward, accumulate = q->accumulate & SGB_VOCAB_CE_ACCUMULATE;
  const bool rest = ES == 2 && !SPLIT && (R <= kFewRows || q->accumulate & SGB_VOCAB_CE_EXACT);
  const auto floats = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const auto elems = [&](size_t o) { return reinterpret_cast<E*>(ws + o); };
  float* most = __is_same(T, f16_t) && grad && q->d_weight ? floats(l.most) : nullptr;
  float* lse = q->lse ? q->lse : floats(l.lse);
  const float* above = way == kBackward ? q->grad_loss : nullptr;
  const T* weight = static_cast<const T*>(q->weight);
  const uint32_t epoch = next_epoch();
  const auto rows_at = [&](int64_t r) {
    return Rows{q->labels + r, q->row_weights ? q->row_weights + r : nullptr,
                above ? above + r : nullptr, V};
  };
  if (most) hipLaunchKernelGGL(k_most, dim3(1), dim3(1024), 0, s, rows_at(0), R, most);

  // Rows as the products read them: 16-byte aligned, a tile's within 32 bits; the
  // hidden rows, whose ends are not cut, of whole steps.
  const auto fits = [&](const void* a, int64_t stride, int64_t rows) {
    return !SPLIT && D * ES % 16 == 0 && aligned(a, 16) &&
           (rows < 2 || (stride * ES % 16 == 0 && stride * ES < (1 << 23)));
  };
  const bool weight_fits = fits(weight, q->weight_stride, V);
  const bool weight_copied = !weight_fits && l.copied >= V;  // as a whole
  Copies<T, SPLIT> copies;
  const auto copy_of = [&](const T* src, int64_t stride, int64_t n) {
    Copy<T, SPLIT> c{src, stride, n, D};
    c.pitch = l.pitch_d;
    c.plane = up(n, kPad) * c.pitch;
    c.pitch_t = up(n, kPad) * (rest ? 2 : 1);
    c.plane_t = D * c.pitch_t;
    return c;
  };
  const auto operand = [](const E* p, const Copy<T, SPLIT>& c) {
    return Operand{reinterpret_cast<const char*>(p), c.pitch * ES, c.plane * ES, nullptr, c.pitch};
  };
  Operand all{};
  if (weight_fits) {
    all = {reinterpret_cast<const char*>(weight), q->weight_stride * ES, 0,
           reinterpret_cast<const char*>(weight + (V - 1) * q->weight_stride + D), D};
  } else if (weight_copied) {
    Copy<T, SPLIT> c = copy_of(weight, q->weight_stride, V);
    c.to = elems(l.w);
    copies.c[copies.n++] = c;
    all = operand(c.to, c);
  }
  // a piece of the weight
  const auto weight_rows = [&](int64_t v0, int64_t width) {
    if (all.p) {
      Operand o = all;
      o.p += v0 * o.ld;
      return o;
    }
    Copy<T, SPLIT> c = copy_of(weight + v0 * q->weight_stride, q->weight_stride, width);
    c.to = elems(l.w);
    copies.c[copies.n++] = c;
    return operand(c.to, c);
  };
  const auto set_a = [&](Product& p, const Operand& o, int64_t K) {
    p.a = o.p;
    p.lda = o.ld;
    p.plane_a = o.plane;
    p.cols_a = o.cols;
    // (a copy's rows are whole steps; the difference to an address is signed)
    p.end_a = o.end ? o.end : reinterpret_cast<const char*>(INTPTR_MAX);
    p.steps = (int)div_up(K, kStepOf<E>);
    p.last = o.end ? (int)(K - (int64_t)(p.steps - 1) * kStepOf<E>) : kStepOf<E>;
  };

  // by pieces only where the weight's rows have to be copied so
  const int64_t logits_piece = all.p ? V : std::min(l.copied, l.piece);
  const int64_t piece = all.p ? l.piece : logits_piece;
  const bool one_piece = piece >= V;
  for (int64_t r0 = 0; r0 < R; r0 += l.chunk) {
    const int64_t n = std::min(l.chunk, R - r0);
    const Rows rows = rows_at(r0);
    const T* x = static_cast<const T*>(q->hidden) + r0 * q->hidden_stride;
    Copy<T, SPLIT> c = copy_of(x, q->hidden_stride, n);
    Operand xo{reinterpret_cast<const char*>(x), q->hidden_stride * ES, 0, nullptr, D}, xt{}, wo{};
    if (D % kPad != 0 || !fits(x, q->hidden_stride, n)) {
      c.to = elems(l.x);
      xo = operand(c.to, c);
    }
    if (grad && q->d_weight) {
      c.to_t = elems(l.xt);
      c.count = rows;
      xt = {reinterpret_cast<const char*>(c.to_t), c.pitch_t * ES, c.plane_t * ES, nullptr, c.pitch_t};
    }
    if (c.to || c.to_t) copies.c[copies.n++] = c;
    if (rest && c.to_t) {
      copies.launch(s);
      c.to = nullptr;
      c.to_t += up(n, kPad);
      copies.c[copies.n++] = c;
    }
    Product a{};
    a.b = xo.p;
    a.ldb = xo.ld;
    a.plane_b = xo.plane;
    a.N = a.tokens = n;
    a.split = 1;
    a.rows = rows;
    a.stats = reinterpret_cast<float2*>(ws + l.stats);
    a.lse = lse + r0;
    a.said = floats(l.said) + r0;
    a.exps = ws + l.exps;
    a.ld_exps = l.ld_exps;
    // (one kind of tile for all pieces: they share the rows of sums)
    const Tiles tiles = choose(std::min(logits_piece, V), n, D, RATE, p->cus, kLogits).tiles;
    for (int64_t v0 = 0; v0 < V; v0 += logits_piece) {
      const int64_t width = std::min(logits_piece, V - v0);
      wo = weight_rows(v0, width);
      copies.launch(s);
      set_a(a, wo, D);
      a.M = width;
      a.v0 = v0;
      if (way == kForward)
        product<E, TERMS, kSums>(a, tiles, s);
      else if (way == kBoth)
        product<E, TERMS, kExps>(a, tiles, s);
      else
        product<E, TERMS, kProbs>(a, tiles, s);
    }
    Loss loss{};
    loss.stats = a.stats;
    loss.parts = (int)div_up(V, wave_cols_of(tiles));
    loss.tokens = n;
    loss.rows = rows;
    loss.said = a.said;
    loss.loss = q->loss ? q->loss + r0 : nullptr;
    loss.lse = lse + r0;
    loss.hdr = reinterpret_cast<Header*>(ws);
    loss.epoch = epoch;
    const bool gradients = grad && (q->d_hidden || q->d_weight);
    const bool sum_later = way == kBoth && gradients && one_piece && loss.parts <= kFewParts;
    if (way != kBackward && !sum_later) {
      // few rows of many sums: more threads a row
      if (n < 1024 && loss.parts > kFewParts)
        hipLaunchKernelGGL(k_lse<64>, dim3((unsigned)div_up(n, 4)), dim3(256), 0, s, loss);
      else
        hipLaunchKernelGGL(k_lse<kShares>, dim3((unsigned)div_up(n, 256 / kShares)), dim3(256), 0, s, loss);
    }
    if (!gradients) continue;

    // (of the first piece, the longest, which writes every part's sums)
    const int64_t longest = std::min(piece, V);
    const int64_t of = rest ? 2 * up(n, kPad) : n;  // rows of the logits' gradient
    const Tiles tiles_w = choose(D, longest, of, RATE, p->cus, kOther).tiles;
    Choice for_h = choose(D, of, longest, RATE, p->cus, kGradient);
    // Two products that leave compute units idle run side by side, d_hidden's sum
    // shared out over those that d_weight leaves (512 tokens of 256, 2000, fp32: 16
    // us, 24 shared out over all, 20 one after the other).
    const bool together = q->d_hidden && q->d_weight && for_h.tiles == kTiny && tiles_w == kTiny;
    const int idle = p->cus - (int)std::min<int64_t>(p->cus, tiles_of<Tiny>(D, longest));
    if (together && idle > 0) {
      const Choice fewer = choose(D, of, longest, RATE, idle, kGradient);
      if (fewer.tiles == kTiny) for_h = fewer;
    }
    const int split = for_h.split;
    for (int64_t v0 = 0; v0 < V; v0 += piece) {
      const int64_t width = std::min(piece, V - v0);
      Grad g{};
      g.exps = a.exps;
      g.ld_exps = l.ld_exps;
      g.wave_cols = way == kBoth ? wave_cols_of(tiles) : 0;
      g.rows = loss;
      g.lse = lse + r0;
      g.most = most;
      g.v0 = v0;
      g.width = width;
      g.pitch = up(width, kPad);
      g.plane = up(n, kPad) * g.pitch;
      g.rest = rest ? g.plane : 0;
      // Both products take the gradient with the row's factor; but fp16 could not
      // hold that of a small one, and d_hidden takes it without.
      constexpr bool kTwo = __is_same(T, f16_t);
      if (q->d_weight || !kTwo) g.scaled = ws + l.scaled;
      if (q->d_hidden && kTwo) g.plain = ws + l.plain;
      const dim3 grid((unsigned)(g.pitch / kPad * (up(n, kPad) / kPad)));
      if (sum_later)
        hipLaunchKernelGGL((k_grad<T, SPLIT, X, true>), grid, dim3(256), 0, s, g);
      else
        hipLaunchKernelGGL((k_grad<T, SPLIT, X, false>), grid, dim3(256), 0, s, g);
      Product h{}, w{};
      if (q->d_hidden) {
        if (!one_piece) {  // (a single piece's is there)
          wo = weight_rows(v0, width);
          copies.launch(s);
        }
        set_a(h, wo, width);
        h.b = static_cast<const char*>(kTwo ? g.plain : g.scaled);
        h.ldb = g.pitch * ES;
        h.plane_b = g.plane * ES;
        h.M = D;
        h.N = of;
        h.split = std::min(split, h.steps);
        if (split == 1 && !rest && v0 + width == V) {
          h.rows = rows;
          h.by_row = kTwo ? kScaled : kKept;
          h.scale = q->grad_scale / kBy;
          h.add_from = v0 > 0 ? floats(l.sums) : nullptr;
          h.out = static_cast<T*>(q->d_hidden) + r0 * q->d_hidden_stride;
          h.ldo = q->d_hidden_stride;
          h.out_dtype = q->dtype;
        } else {
          h.sums = floats(l.sums);
          h.add = v0 > 0;
        }
      }
      if (q->d_weight) {
        const bool first = r0 == 0, last = r0 + n == R;
        const bool direct = (first && last) || q->d_weight_dtype == SGB_F32;
        set_a(w, xt, of);
        w.b = static_cast<const char*>(g.scaled);
        w.ldb = g.pitch * ES;
        w.plane_b = g.plane * ES;
        w.M = D;
        w.N = width;
        w.cols_b = g.pitch;
        w.split = 1;
        w.most = most;
        w.scale = q->grad_scale / kBy;
        if (direct || last) {
          w.out = static_cast<char*>(q->d_weight) +
                  v0 * q->d_weight_stride * elem_size(q->d_weight_dtype);
          w.ldo = q->d_weight_stride;
          w.out_dtype = q->d_weight_dtype;
          w.add = accumulate || (direct && !first);
          w.add_from = direct ? nullptr : floats(l.dw) + v0 * D;
        } else {
          w.out = floats(l.dw) + v0 * D;
          w.ldo = D;
          w.out_dtype = SGB_F32;
          w.add = !first;
        }
      }
      if (together) {
        const unsigned first = grid_of<Tiny>(h), second = grid_of<Tiny>(w);
        hipLaunchKernelGGL((k_products<E, TERMS, Tiny>), dim3(first + second), dim3(kThreadsOf<Tiny>),
                           0, s, h, w, (int)first);
      } else {
        if (q->d_hidden) product<E, TERMS, kGrads, true, false>(h, for_h.tiles, s);
        if (q->d_weight) product<E, TERMS, kGrads, false, true>(w, tiles_w, s);
      }
    }
    if (q->d_hidden && (split > 1 || rest))
      hipLaunchKernelGGL(k_join<T>, dim3(blocks(n * div_up(D, 8), p->cus)), dim3(256), 0, s,
                         floats(l.sums), rest ? 2 * split : split, rest ? up(n, kPad) : n, n, D, rows,
                         (bool)__is_same(T, f16_t), q->grad_scale / kBy,
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
    if (!std::isfinite(q->grad_scale) || q->accumulate < 0 ||
        q->accumulate > (SGB_VOCAB_CE_ACCUMULATE | SGB_VOCAB_CE_EXACT))
      return SGB_ERR_INVALID_ARGUMENT;
    if (q->d_weight && ((q->d_weight_dtype != SGB_F32 && q->d_weight_dtype != q->dtype) ||
                        !matrix_ok(q->d_weight, D, q->d_weight_stride, elem_size(q->d_weight_dtype))))
      return SGB_ERR_INVALID_ARGUMENT;
    if (way == kBackward && !q->d_hidden && !q->d_weight) return SGB_ERR_INVALID_ARGUMENT;
  }
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (R == 0 && (!grad || !q->d_weight || q->accumulate & SGB_VOCAB_CE_ACCUMULATE)) return SGB_OK;
  if (R > 0) {
    if (!matrix_ok(q->hidden, D, q->hidden_stride, e) || !matrix_ok(q->weight, D, q->weight_stride, e) ||
        !q->labels || !aligned(q->labels, 8) || !aligned(q->row_weights, 4) || !aligned(q->lse, 4))
      return SGB_ERR_INVALID_ARGUMENT;
    if (way != kBackward && (!q->loss || !aligned(q->loss, 4))) return SGB_ERR_INVALID_ARGUMENT;
    if (way == kBackward && (!q->lse || !aligned(q->grad_loss, 4))) return SGB_ERR_INVALID_ARGUMENT;
    if (grad && q->d_hidden && !matrix_ok(q->d_hidden, D, q->d_hidden_stride, e))
      return SGB_ERR_INVALID_ARGUMENT;
    if (!workspace_ok(ws)) return SGB_ERR_INVALID_ARGUMENT;
  }
  const Layout l = layout(p, std::max<int64_t>(R, 1), q->dtype, grad,
                          grad && q->accumulate & SGB_VOCAB_CE_EXACT);
  if (R > 0) {
    const bool back = way == kBackward;
    const Extent none{};
    const Extent lse = vector(q->lse, R, 4);
    const Extent in[] = {{q->hidden, R, D, q->hidden_stride, e},
                         {q->weight, V, D, q->weight_stride, e},
                         vector(q->labels, R, 8),
                         vector(q->row_weights, R, 4),
                         back ? lse : none,
                         back ? vector(q->grad_loss, R, 4) : none};
    const Extent out[] = {
        back ? none : vector(q->loss, R, 4),
        back ? none : lse,
        grad ? Extent{q->d_hidden, R, D, q->d_hidden_stride, e} : none,
        grad && q->d_weight ? Extent{q->d_weight, V, D, q->d_weight_stride, elem_size(q->d_weight_dtype)}
                            : none,
        vector(ws, (int64_t)std::min(l.bytes, ws_bytes), 1)};
    if (any_overlap(out, 5, in, 6)) return SGB_ERR_INVALID_ARGUMENT;
    if (ws_bytes < l.bytes) return SGB_ERR_WORKSPACE_TOO_SMALL;
  }
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  if (R == 0) {
    q->d_weight_dtype == SGB_F32 ? zero<float>(p, q, s)
    : q->dtype == SGB_BF16       ? zero<bf16_t>(p, q, s)
                                 : zero<f16_t>(p, q, s);
  } else if (q->dtype == SGB_F32) {
    if (in_parts(p, std::min(R, l.chunk)))
      enqueue<float, true>(p, q, way, l, static_cast<char*>(ws), s);
    else
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
  if (!p || !bytes || rows < 0 || rows >= (1ll << 31) || !float_dtype(dtype) || gradient < 0 ||
      gradient > 2)
    return SGB_ERR_INVALID_ARGUMENT;
  *bytes = layout(p, std::max<int64_t>(rows, 1), dtype, gradient != 0, gradient == 2).bytes;
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
