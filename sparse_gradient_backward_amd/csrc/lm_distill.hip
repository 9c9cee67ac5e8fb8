// lm_distill.hip -- distillation from a teacher's top logits, of libsgb_lm.so:
// loss and gradient of the student's logits (formulas: include/sgb_lm.h).
//
// With e_j = exp((x_j - m) / T), m the largest of the logits summed over:
//  - the loss needs sum e over the row (one pass, a running maximum and sum a
//    lane) and the K listed logits;
//  - the gradient of logit j is c e_j (c from the row's sums) but at the K
//    listed ids and the label, which are written over afterwards.
// With the teacher's tail mass the pass sums over the ids that are NOT listed
// (a bit each in LDS): the student's tail mass q' is a small difference that
// subtracting the listed ones from the whole would lose, and the listed ones
// are then added to it for the whole.  The K listed terms are taken in fp64:
// the loss is a difference of logarithms, the teacher's tail 1 - sum p.

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>

#include "lm_internal.h"

using namespace sgb_lm;

namespace {

constexpr int kThreads = 256;
constexpr int kStep = kThreads * 8;    // columns a workgroup takes at a time
constexpr int kMaxSpan = 131072;       // columns a workgroup takes in all (16 KB of bits)
constexpr int kMaxSplit = 64;          // workgroups a row
constexpr size_t kShortRow = 32768;    // bytes
constexpr int kMaxK = 1024;
constexpr int64_t kMaxV = (int64_t)kMaxSpan * kMaxSplit;

struct Args {
  const void* logits;
  const int64_t* ids;
  const float* values;
  const float* teacher_lse;
  const int64_t* labels;
  const float* weights;
  const float* grad_loss;
  float* loss;
  float* stats;
  void* grad;
  float4* part;  // [rows][split]: m, sum exp((x-m)/T), sum exp(x-m) (if asked for), 0
  Header* hdr;
  uint32_t epoch;
  int64_t sl, si, sv, sg;
  int64_t rows;
  int64_t V;
  int K, table;   // table: power of two >= 2 K
  int split, span;
  float T, c, kd, ce, scale;  // c = log2(e) / T
};

constexpr float kLog2e = 1.44269504088896341f;

// 2^x by the vector unit's own instruction (within 1 ulp; results below the
// normal range are zero, which in a sum relative to its largest term they are).
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float weight_of(const Args& a, int64_t row) {
  return a.weights ? a.weights[row] : 1.f;
}

// Running maximum and sums of a lane.  Starting from the lowest finite value
// keeps every difference below a number: -inf logits add exp2(-inf) = 0, and
// a row of the type's lowest value is a uniform row.
template <bool TWO>
struct Sums {
  float m = -FLT_MAX, s = 0.f, s1 = 0.f;

  // eight logits; -inf for those left out
  __device__ __forceinline__ void add(const float (&x)[8], float c) {
    float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])),
                      fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    top = fmaxf(top, m);
    const float d = m - top;
    s *= exp2_of(d * c);
    if (TWO) s1 *= exp2_of(d * kLog2e);
    m = top;
    float p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = exp2_of((x[i] - m) * c);
    s += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    if (TWO) {
#pragma unroll
      for (int i = 0; i < 8; ++i) p[i] = exp2_of((x[i] - m) * kLog2e);
      s1 += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    }
  }
  __device__ __forceinline__ void scale_to(float top, float c) {
    const float d = m - top;
    s *= exp2_of(d * c);
    if (TWO) s1 *= exp2_of(d * kLog2e);
    m = top;
  }
};

// ------------------------------------------------------------- streams

// f(eight logits as loaded, column) over columns [c0, c1) of a row, kAhead
// loads of a lane in flight.  Every lane makes every turn; f looks at the column.
constexpr int kAhead = 2;

template <int NT, typename T, typename F>
__device__ __forceinline__ void stream(const T* row, uint32_t c0, uint32_t c1, uint32_t V, F f) {
  constexpr uint32_t kStride = NT * 8;
  uint32_t col = c0 + threadIdx.x * 8;
  if (V < 8) {  // a load of eight does not fit
    const int n = (int)V - (int)col;
    f(load8(row + col, n), col, n);
    return;
  }
  Raw8<T> q[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) q[u] = ask8(row, col + u * kStride, c1);
  for (uint32_t base = c0; base < c1; base += kAhead * kStride) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      Raw8<T> r = q[u];
      q[u] = ask8(row, col + kAhead * kStride, c1);
      const int n = (int)c1 - (int)col;
      have8(r, n);
      f(r, col, n);
      col += kStride;
    }
  }
}

template <int NT, typename T>
__device__ __forceinline__ void write_zeros(T* grad, uint32_t c0, uint32_t c1) {
  const float zero[8] = {};
  for (uint32_t col = c0 + threadIdx.x * 8; col < c1; col += NT * 8)
    store8(grad, col, zero, (int)(c1 - col));
}

// Sets the bits of the row's listed ids in columns [c0, c1).
template <int NT>
__device__ __forceinline__ void mark_listed(const Args& a, int64_t row, int64_t c0, int64_t c1,
                                            uint32_t* bits) {
  for (int k = threadIdx.x; k < a.K; k += NT) {
    const int64_t id = a.ids[row * a.si + k];
    if (id >= c0 && id < c1) atomicOr(&bits[(id - c0) >> 5], 1u << ((id - c0) & 31));
  }
}

// The workgroup's sums over columns [c0, c1) (those without a bit), the same
// in every lane: the first NS lanes read the logits, the others do `aside`
// instead.
template <typename T, bool TAIL, bool TWO, int NT, int NS, typename G>
__device__ __forceinline__ float4 sums_of(const Args& a, const T* x, uint32_t c0, uint32_t c1,
                                          const uint32_t* bits, float (*red)[NT / 64], G aside) {
  Sums<TWO> sum;
  const bool streams = NS == NT || __builtin_amdgcn_readfirstlane(threadIdx.x) < NS;
  if (!streams) aside();
  auto add = [&](const Raw8<T>& r, uint32_t col, int n) {
    if (n <= 0) return;
    float v[8];
    widen8(r, v);
    uint32_t skip = n < 8 ? 0xffu << n & 0xffu : 0u;
    if (TAIL) skip |= reinterpret_cast<const uint8_t*>(bits)[(col - c0) >> 3];
    if (skip) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (skip >> i & 1) v[i] = -INFINITY;
    }
    sum.add(v, a.c);
  };
  if (streams) stream<NS>(x, c0, c1, (uint32_t)a.V, add);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float top = wave_max(sum.m);
  sum.scale_to(top, a.c);
  const float s = wave_add(sum.s), s1 = TWO ? wave_add(sum.s1) : 0.f;
  if (lane == 0) {
    red[0][wave] = top;
    red[1][wave] = s;
    red[2][wave] = s1;
  }
  __syncthreads();
  float m = red[0][0];
#pragma unroll
  for (int w = 1; w < NT / 64; ++w) m = fmaxf(m, red[0][w]);
  float4 o = make_float4(m, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    o.y += red[1][w] * exp2_of((red[0][w] - m) * a.c);
    if (TWO) o.z += red[2][w] * exp2_of((red[0][w] - m) * kLog2e);
  }
  return o;
}

template <typename T, bool TAIL, bool TWO>
__global__ __launch_bounds__(kThreads) void k_distill_sums(Args a) {
  extern __shared__ uint32_t bits[];  // TAIL: span / 32 words
  __shared__ float red[3][kThreads / 64];
  const int64_t row = blockIdx.x / (uint32_t)a.split;
  const int part = (int)(blockIdx.x % (uint32_t)a.split);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->epoch = a.epoch;
  if (weight_of(a, row) == 0.f) return;  // padding: not read
  const int64_t c0 = (int64_t)part * a.span, c1 = min(a.V, c0 + a.span);
  const T* x = static_cast<const T*>(a.logits) + row * a.sl;
  if (TAIL) {
    for (int i = threadIdx.x; i < a.span / 32; i += kThreads) bits[i] = 0;
    __syncthreads();
    mark_listed<kThreads>(a, row, c0, c1, bits);
    __syncthreads();
  }
  const float4 o = sums_of<T, TAIL, TWO, kThreads, kThreads>(a, x, (uint32_t)c0, (uint32_t)c1,
                                                             bits, red, [] {});
  if (threadIdx.x == 0) a.part[row * a.split + part] = o;
}

// ------------------------------------------------------------- listed terms

// The teacher's tail is 1 - sum p, a difference that the rounding of an fp32
// teacher_lse leaves above 0 in half of the rows whose listed ids are all the
// teacher gave mass to.  Against a student mass that is 0 (or so small that its
// logarithm is a mask's huge number) that rounding would make the loss infinite:
// up to 16 fp32 roundings of the log-sum-exp count as no tail where the logits
// outside are 2^-150 of the largest listed or less (2^23 of them 2^-127 of q).
constexpr float kLseRounding = 0x1p-20f;
constexpr float kNoMass = -150.f;

// What the row's gradient and loss need, by one wave.
struct Terms {
  double base;                // the largest logit; logarithms of sums are relative to it (a
                              // row may hold nothing but a huge negative number)
  double lse, lse1, lse_out;  // of x / T, of x, of x / T outside the listed (with a tail)
  double mass, tail;          // what q is multiplied by; the teacher's tail
  float m;                    // the sums' maximum
  float ca, cb;               // gradient: ca exp((x-m)/T) + cb exp(x-m)
  float above;                // row weight, scale and gradient from above
  int64_t label;              // -1: none
  float label_x;
  int repeated;               // some id is listed twice
};

struct Listed {  // in LDS, K of each
  float* x;
  float* p;
  int32_t* id;      // -1: not listed, or (as the owner of its id) another entry's
  int32_t* owner;   // 1: the entry that stands for its id
  int32_t* table;
};

__device__ __forceinline__ Listed listed_in(char* lds, int K) {
  Listed l;
  l.x = reinterpret_cast<float*>(lds);
  l.p = l.x + K;
  l.id = reinterpret_cast<int32_t*>(l.p + K);
  l.owner = l.id + K;
  l.table = l.owner + K;
  return l;
}

__host__ __device__ inline size_t listed_bytes(int K, int table) {
  return (size_t)(4 * K + table) * 4;
}

__device__ __forceinline__ double wave_add(double x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off, 64);
  return x;
}

// LDS written by the wave's own lanes is read by others of them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  __builtin_amdgcn_wave_barrier();
}

// What a row's terms need beside the sums over its logits (one wave): nothing
// here waits for them.
struct Known {
  double entropy;   // sum of p log p
  double reach;     // sum of p (x - top)
  double psum;      // sum of p
  double ls, ls1;   // sums of exp((x - top) / T), of exp(x - top), an id once
  float top;        // the largest listed logit
  float label_x, w, above;
  int64_t label;    // -1: none
  int tail, repeated;
};
// Known::tail: none, as nothing or every id of the vocabulary is listed; as it
// comes; no more than the rounding of teacher_lse
enum { kNoTail, kTail, kSlightTail };

template <typename T, bool TAIL, bool TWO>
__device__ __forceinline__ void gather(const Args& a, int64_t row, const Listed& l, Known& o) {
  const int lane = threadIdx.x & 63;
  const T* logits = static_cast<const T*>(a.logits) + row * a.sl;
  const double invT = 1.0 / (double)a.T;
  o.w = weight_of(a, row);
  o.above = o.w * a.scale * (a.grad_loss ? a.grad_loss[row] : 1.f);

  for (int i = lane; i < a.table; i += 64) l.table[i] = -1;
  wave_sync();
  bool bad = false, twice = false, some = false;
  float tmax = -FLT_MAX, top = -FLT_MAX;
  for (int k = lane; k < a.K; k += 64) {
    const int64_t id64 = a.ids[row * a.si + k];
    const bool there = id64 >= 0 && id64 < a.V;
    bad |= id64 >= a.V;
    const int32_t id = there ? (int32_t)id64 : -1;
    const float x = there ? widen(logits[id]) : 0.f;
    int own = 0;
    if (there) {
      some = true;
      tmax = fmaxf(tmax, a.values[row * a.sv + k]);
      top = fmaxf(top, x);
      uint32_t at = (uint32_t)id * 2654435761u >> 7;
      while (true) {  // at most K of the table's >= 2 K places are taken
        at &= (uint32_t)a.table - 1;
        const int32_t old = atomicCAS(&l.table[at], -1, id);
        if (old == -1) own = 1;
        if (old == -1 || old == id) break;
        ++at;
      }
      twice |= !own;
    }
    l.id[k] = id;
    l.owner[k] = own;
    l.x[k] = x;
  }
  const bool any = __ballot(some) != 0;
  o.repeated = __ballot(twice) != 0;
  o.tail = TAIL && any ? kTail : kNoTail;
  if (TAIL && a.V <= a.K) {  // can every id be listed?  (Counted apart from the loop above:
                             // in it, 4096 rows of 131072 took 497 us for 451.)
    float distinct = 0.f;
    for (int k = lane; k < a.K; k += 64) distinct += (float)l.owner[k];
    if (wave_add(distinct) == (float)a.V) o.tail = kNoTail;
  }
  tmax = wave_max(tmax);
  o.top = wave_max(top);

  // the teacher's log-sum-exp
  double tl;
  if (TAIL) {
    tl = (double)a.teacher_lse[row];
  } else {
    double z = 0.0;
    for (int k = lane; k < a.K; k += 64)
      if (l.id[k] >= 0) z += exp(((double)a.values[row * a.sv + k] - (double)tmax) * invT);
    z = wave_add(z);
    tl = z == 0.0 ? HUGE_VAL : (double)tmax * invT + log(z);  // nothing: every p is 0
  }
  double entropy = 0.0, reach = 0.0, psum = 0.0, ls = 0.0, ls1 = 0.0;
  for (int k = lane; k < a.K; k += 64) {
    double p = 0.0;
    const double d = (double)l.x[k] - (double)o.top;
    if (l.id[k] >= 0) {
      const double lp = (double)a.values[row * a.sv + k] * invT - tl;
      p = lp < -800.0 ? 0.0 : exp(lp);
      if (!(p <= 0.0)) {
        entropy += p * lp;
        reach += p * d;
      }
    }
    psum += p;
    l.p[k] = (float)p;
    if (TAIL && l.owner[k]) {
      ls += exp(d * invT);
      if (TWO) ls1 += exp(d);
    }
  }
  o.entropy = wave_add(entropy);
  o.reach = wave_add(reach);
  o.psum = wave_add(psum);
  if (TAIL && o.tail && (float)(1.0 - o.psum) <= kLseRounding * (1.f + fabsf((float)tl)))
    o.tail = kSlightTail;
  o.ls = TAIL ? wave_add(ls) : 0.0;
  o.ls1 = TAIL && TWO ? wave_add(ls1) : 0.0;

  o.label = -1;
  o.label_x = 0.f;
  if (a.labels) {
    const int64_t lab = a.labels[row];
    bad |= lab >= a.V;
    if (lab >= 0 && lab < a.V) {
      o.label = lab;
      o.label_x = widen(logits[lab]);
    }
  }
  if (__ballot(bad) && lane == 0) set_status(a.hdr, a.epoch, SGB_ERR_INDEX_OUT_OF_RANGE);
  wave_sync();
}

// The row's terms and loss from the sums over its logits (with a tail: over
// those not listed).
template <bool TAIL, bool TWO>
__device__ __forceinline__ void finish(const Args& a, const Known& n, float4 sums, Terms& o,
                                       double& loss) {
  const double invT = 1.0 / (double)a.T;
  double m = (double)sums.x, s = (double)sums.y, s1 = (double)sums.z;
  const double log_out = TAIL ? log(s) : 0.0;
  if (TAIL) {
    const double mm = fmax(m, (double)n.top), from = m - mm, listed = (double)n.top - mm;
    s = s * exp(from * invT) + n.ls * exp(listed * invT);
    if (TWO) s1 = s1 * exp(from) + n.ls1 * exp(listed);
    m = mm;
  }
  o.m = sums.x;
  o.above = n.above;
  o.repeated = n.repeated;
  o.label = n.label;
  o.label_x = n.label_x;
  o.base = m;
  o.lse = log(s);
  o.lse_out = TAIL ? ((double)sums.x - m) * invT + log_out : o.lse;
  o.lse1 = TWO ? log(s1) : o.lse;  // without a second sum T is 1 or there is no label

  double kl = 0.0;
  if (n.psum != 0.0)
    kl = n.entropy - (n.reach + ((double)n.top - m) * n.psum) * invT + o.lse * n.psum;
  o.tail = 0.0;
  o.mass = n.psum == 0.0 ? 0.0 : 1.0;
  if (TAIL) {
    o.tail = n.tail ? fmax(0.0, 1.0 - n.psum) : 0.0;
    if (n.tail == kSlightTail && (sums.y == 0.f || (sums.x - n.top) * a.c < kNoMass)) o.tail = 0.0;
    o.mass = n.psum + o.tail;
    if (o.tail > 0.0) kl += o.tail * (log(o.tail) - (o.lse_out - o.lse));
  }
  loss = (double)a.kd * (double)a.T * (double)a.T * kl;
  if (n.label >= 0) loss += (double)a.ce * (o.lse1 - ((double)n.label_x - m));
  loss *= (double)n.w;

  // ca, cb: relative to the pass's own maximum and sum
  const double kt = (double)o.above * (double)a.kd * (double)a.T;
  const double down = (double)sums.x - m;
  double ca;
  if (TAIL)
    ca = sums.y == 0.f ? 0.0
                       : kt * (o.mass * exp(o.lse_out - o.lse) - o.tail) / (double)sums.y;
  else
    ca = kt * o.mass * exp(down * invT - o.lse);
  double cb = 0.0;
  if (o.label >= 0) cb = (double)o.above * (double)a.ce * exp(down - o.lse1);
  if (!TWO) {
    ca += cb;
    cb = 0.0;
  }
  if (s == 0.0) loss = ca = o.mass = NAN;  // nothing but -inf: no distribution
  o.ca = (float)ca;
  o.cb = (float)cb;
}

template <typename T, bool TAIL, bool TWO>
__device__ void row_terms(const Args& a, int64_t row, float4 sums, Listed l, Terms& o,
                          double& loss) {
  Known n;
  gather<T, TAIL, TWO>(a, row, l, n);
  finish<TAIL, TWO>(a, n, sums, o, loss);
}

// The row's partial sums joined (one wave).
__device__ __forceinline__ float4 join_sums(const Args& a, const float4* part) {
  const int lane = threadIdx.x & 63;
  float4 q = lane < a.split ? part[lane] : make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
  const float m = wave_max(q.x);
  const float s = wave_add(q.y * exp2_of((q.x - m) * a.c));
  const float s1 = wave_add(q.z * exp2_of((q.x - m) * kLog2e));
  return make_float4(m, s, s1, 0.f);
}

// The loss alone (and the sums that a backward starts from): a wave a row.
template <typename T, bool TAIL, bool TWO>
__global__ __launch_bounds__(64) void k_distill_loss(Args a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int64_t row = blockIdx.x;
  float4* st = reinterpret_cast<float4*>(a.stats);
  if (weight_of(a, row) == 0.f) {
    if (threadIdx.x == 0) {
      a.loss[row] = 0.f;
      if (st) st[row] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const float4 sums = join_sums(a, a.part + row * a.split);
  Terms t;
  double loss;
  row_terms<T, TAIL, TWO>(a, row, sums, listed_in(lds, a.K), t, loss);
  if (threadIdx.x == 0) {
    a.loss[row] = (float)loss;
    if (st) st[row] = sums;
  }
}

// ------------------------------------------------------------- gradient

// Gradient at a listed id (of which this entry is the owner).
__device__ __forceinline__ float listed_grad(const Args& a, const Terms& t, const Listed& l, int k) {
  const double x = (double)l.x[k] - t.base, invT = 1.0 / (double)a.T;
  double p = (double)l.p[k];
  if (t.repeated) {
    p = 0.0;
    for (int j = 0; j < a.K; ++j)
      if (l.id[j] == l.id[k]) p += (double)l.p[j];
  }
  double g = (double)a.kd * (double)a.T * (t.mass * exp(x * invT - t.lse) - p);
  if (t.label >= 0)
    g += (double)a.ce * (exp(x - t.lse1) - (t.label == (int64_t)l.id[k] ? 1.0 : 0.0));
  return (float)(g * (double)t.above);
}

// Gradient at a label that is not listed.
template <bool TAIL>
__device__ __forceinline__ float label_grad(const Args& a, const Terms& t, float xl) {
  const double x = (double)xl - t.base, invT = 1.0 / (double)a.T;
  const double kd = TAIL ? (t.mass * exp(t.lse_out - t.lse) - t.tail) * exp(x * invT - t.lse_out)
                         : t.mass * exp(x * invT - t.lse);
  return (float)((double)t.above * ((double)a.kd * (double)a.T * kd +
                                    (double)a.ce * (exp(x - t.lse1) - 1.0)));
}

// What the stream cannot know of the gradient (one wave): the listed ids', left
// in place of their logits, and the label's.
template <bool TAIL>
__device__ __forceinline__ float listed_grads(const Args& a, const Terms& t, const Listed& l) {
  const int lane = threadIdx.x & 63;
  const float at_label = t.label >= 0 ? label_grad<TAIL>(a, t, t.label_x) : 0.f;
  for (int k = lane; k < a.K; k += 64)
    if (l.owner[k]) l.x[k] = listed_grad(a, t, l, k);
  return at_label;
}

// Writes it over columns [c0, c1), after the stream's stores.
template <typename T>
__device__ __forceinline__ void patch(const Args& a, int64_t row, int64_t c0, int64_t c1,
                                      const Terms& t, const Listed& l, float at_label) {
  const int lane = threadIdx.x & 63;
  T* grad = static_cast<T*>(a.grad) + row * a.sg;
  bool label_listed = false;
  for (int k = lane; k < a.K; k += 64) {
    if (!l.owner[k]) continue;
    const int64_t id = l.id[k];
    label_listed |= id == t.label;
    if (id >= c0 && id < c1) grad[id] = (T)l.x[k];
  }
  if (t.label >= c0 && t.label < c1 && !__ballot(label_listed) && lane == 0)
    grad[t.label] = (T)at_label;
}

template <typename T, bool TWO, int NT>
__device__ __forceinline__ void write_gradient(const Args& a, const T* x, T* grad, uint32_t c0,
                                               uint32_t c1, const Terms& t) {
  const float m = t.m, ca = t.ca, cb = t.cb;
  stream<NT>(x, c0, c1, (uint32_t)a.V, [&](const Raw8<T>& r, uint32_t col, int n) {
    if (n <= 0) return;
    float v[8];
    widen8(r, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float d = v[i] - m;
      float g = ca * exp2_of(d * a.c);
      if (TWO) g = fmaf(cb, exp2_of(d * kLog2e), g);
      v[i] = g;
    }
    store8(grad, col, v, n);
  });
}

template <typename T, bool TAIL, bool TWO>
__global__ __launch_bounds__(kThreads) void k_distill_grad(Args a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ Terms t;
  const int64_t row = blockIdx.x / (uint32_t)a.split;
  const int part = (int)(blockIdx.x % (uint32_t)a.split);
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->epoch = a.epoch;
  const int64_t c0 = (int64_t)part * a.span, c1 = min(a.V, c0 + a.span);
  const T* x = static_cast<const T*>(a.logits) + row * a.sl;
  T* grad = static_cast<T*>(a.grad) + row * a.sg;
  if (weight_of(a, row) == 0.f) {
    write_zeros<kThreads>(grad, (uint32_t)c0, (uint32_t)c1);
    if (a.loss && part == 0 && threadIdx.x == 0) a.loss[row] = 0.f;
    return;
  }
  const Listed l = listed_in(lds, a.K);
  if (threadIdx.x < 64) {
    // a backward starts from the sums its forward kept
    const float4 sums = a.stats ? reinterpret_cast<const float4*>(a.stats)[row]
                                : join_sums(a, a.part + row * a.split);
    Terms mine;
    double loss;
    row_terms<T, TAIL, TWO>(a, row, sums, l, mine, loss);
    if (threadIdx.x == 0) {
      t = mine;
      if (a.loss && part == 0) a.loss[row] = (float)loss;
    }
  }
  __syncthreads();
  write_gradient<T, TWO, kThreads>(a, x, grad, (uint32_t)c0, (uint32_t)c1, t);
  const float at_label = threadIdx.x < 64 ? listed_grads<TAIL>(a, t, l) : 0.f;
  __syncthreads();  // the stream's stores come before the patch's
  if (threadIdx.x < 64) patch<T>(a, row, c0, c1, t, l, at_label);
}

// ------------------------------------------------------------- a row a workgroup
//
// Where there are rows enough, a workgroup takes a whole row: the sums, the
// terms and (GRAD) the gradient.  The gradient's reading of the logits comes
// from the caches: at two workgroups of 1024 lanes a compute unit the rows in
// flight, 256 KB each, fit in the last level's 256 MB (of 4096 rows of 131072
// bf16, counters: 0.97 GB fetched and 1.08 GB written).
//
// Two share a compute unit at up to 64 registers a lane: so it is but for two
// sums (T other than 1, and labels), whose forms of 1024 lanes take 68 to 94
// (only the gradient without a tail 62) and run alone there: 585 us on those rows at
// T = 2.
//
// Measured on those at T = 1, with a tail and labels: 450 us (4.8 TB/s of the
// logits read and the gradient written; counters: the vector unit is busy for
// 64% of it), against 608 for the sums and the gradient in launches of
// their own and 534 for rows held in 256 registers a lane (read once, but a row
// a compute unit leaves nothing to do while its terms are found).  With every
// wave reading and the last one gathering besides, 1024 lanes took 454 us, 512
// 494, 256 598, and on 2048 rows of 8000 columns 52, 33 and 23 us.

template <typename T, bool TAIL, bool TWO, bool GRAD, int NT>
__global__ __launch_bounds__(NT) void k_distill_row(Args a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  __shared__ Terms terms;
  __shared__ Known known;
  __shared__ float red[3][NT / 64];
  const int t = (int)threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int64_t row = blockIdx.x;
  if (row == 0 && t == 0) a.hdr->epoch = a.epoch;
  T* grad = static_cast<T*>(a.grad) + row * a.sg;
  float4* stats = reinterpret_cast<float4*>(a.stats);
  const uint32_t V = (uint32_t)a.V;
  if (weight_of(a, row) == 0.f) {
    if (GRAD) write_zeros<NT>(grad, 0, V);
    if (t == 0) {
      a.loss[row] = 0.f;
      if (stats) stats[row] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    return;
  }
  const T* x = static_cast<const T*>(a.logits) + row * a.sl;
  uint32_t* bits = reinterpret_cast<uint32_t*>(lds);
  const Listed l = listed_in(lds + (TAIL ? a.span / 8 : 0), a.K);
  if (TAIL) {
    for (int i = t; i < a.span / 32; i += NT) bits[i] = 0;
    __syncthreads();
    mark_listed<NT>(a, row, 0, V, bits);
    __syncthreads();
  }
  // The last wave gathers what is listed while the others read, and finds the
  // listed ids' gradients while they write.
  constexpr int NS = NT - 64;
  auto aside = [&] {
    Known n;
    gather<T, TAIL, TWO>(a, row, l, n);
    if ((t & 63) == 0) known = n;
  };
  const float4 sums = sums_of<T, TAIL, TWO, NT, NS>(a, x, 0, V, bits, red, aside);
  if (wave == 0) {
    Terms mine;
    double loss;
    finish<TAIL, TWO>(a, known, sums, mine, loss);
    if (t == 0) {
      terms = mine;
      a.loss[row] = (float)loss;
      if (stats) stats[row] = sums;
    }
  }
  if (!GRAD) return;
  __syncthreads();
  float at_label = 0.f;
  if (wave == NT / 64 - 1)
    at_label = listed_grads<TAIL>(a, terms, l);
  else
    write_gradient<T, TWO, NS>(a, x, grad, 0, V, terms);
  __syncthreads();  // the stream's stores come before the patch's
  if (wave == NT / 64 - 1) patch<T>(a, row, 0, a.V, terms, l, at_label);
}

}  // namespace

// ------------------------------------------------------------- host

struct sgb_distill_s {
  int device, cus;
  int64_t V;
  int K, table;
  float T, kd, ce;
};

namespace {

// Workgroups a row: enough to give every compute unit four, as long as each
// keeps one step of columns; at least what the bits in LDS cover.
int split_of(const sgb_distill_s* p, int64_t rows) {
  const int64_t most = std::min<int64_t>(kMaxSplit, div_up(p->V, kStep));
  const int64_t least = div_up(p->V, kMaxSpan);
  const int64_t want = div_up(4 * (int64_t)p->cus, std::max<int64_t>(rows, 1));
  return (int)std::max(least, std::min(most, want));
}

// Parts of `rows` or fewer rows: split_of() falls in steps as rows grow, so that
// fewer rows can have more parts.  r rows have at most r * ceil(w / r) <= w + r - 1
// of the w workgroups wanted, and never fewer than `least` a row.
int64_t most_parts(const sgb_distill_s* p, int64_t rows) {
  const int64_t most = std::min<int64_t>(kMaxSplit, div_up(p->V, kStep));
  const int64_t least = div_up(p->V, kMaxSpan);
  const int64_t wanted = std::min(rows * most, 4 * (int64_t)p->cus + rows);
  return std::max(rows * least, wanted);
}

enum What { kLoss, kBackward, kBoth };

template <typename T, bool TAIL, bool TWO, bool GRAD, int NT>
void run_rows(Args a, hipStream_t s) {
  a.span = (int)align_up((size_t)a.V, 32);
  const size_t lds = (TAIL ? a.span / 8 : 0) + listed_bytes(a.K, a.table);
  hipLaunchKernelGGL((k_distill_row<T, TAIL, TWO, GRAD, NT>), dim3((unsigned)a.rows), dim3(NT), lds,
                     s, a);
}

// The longer the row, the more lanes: few rows in flight are long enough to
// keep the memory busy, and they have to fit in the caches.
int row_threads(size_t bytes) {
  return bytes <= kShortRow ? 256 : bytes <= 4 * kShortRow ? 512 : 1024;
}

template <typename T, bool TAIL, bool TWO, bool GRAD>
void run_rows(const Args& a, hipStream_t s) {
  const int threads = row_threads((size_t)a.V * sizeof(T));
  if (threads == 256)
    run_rows<T, TAIL, TWO, GRAD, 256>(a, s);
  else if (threads == 512)
    run_rows<T, TAIL, TWO, GRAD, 512>(a, s);
  else
    run_rows<T, TAIL, TWO, GRAD, 1024>(a, s);
}

// A row a workgroup, or several workgroups a row and the loss in a launch of
// its own?  (Loss and gradient: 64 rows of 131072 bf16 take 17 us in parts and
// 25 as rows, 128 take 26.5 and 26.8, 256 take 43 and 38; of 8000 columns 1 row
// takes 10.1 and 9.5.)  Past kMaxSpan columns a row's bits outgrow the 16 KB set
// aside for them; what a longer row in one workgroup would take, with or without
// a tail, was not measured (2048 rows of 131072 bf16 take 242 us as rows, of 151936
// 114 and 251 in parts).
bool rows_at_once(const Args& a, size_t elem, int cus) {
  return a.V <= kMaxSpan && (a.rows >= cus / 2 || (size_t)a.V * elem <= kShortRow);
}

// Threads of the call's largest launch.
int64_t threads_of(const Args& a, What what, size_t elem, int cus) {
  return what != kBackward && rows_at_once(a, elem, cus)
             ? a.rows * row_threads((size_t)a.V * elem)
             : a.rows * a.split * kThreads;
}

template <typename T, bool TAIL, bool TWO>
void run_as(const Args& a, What what, int cus, hipStream_t s) {
  if (what != kBackward && rows_at_once(a, sizeof(T), cus)) {
    if (what == kBoth)
      run_rows<T, TAIL, TWO, true>(a, s);
    else
      run_rows<T, TAIL, TWO, false>(a, s);
    return;
  }
  const dim3 grid((unsigned)(a.rows * a.split));
  const size_t terms = listed_bytes(a.K, a.table);
  if (what != kBackward)
    hipLaunchKernelGGL((k_distill_sums<T, TAIL, TWO>), grid, dim3(kThreads),
                       TAIL ? a.span / 8 : 0, s, a);
  if (what == kLoss)
    hipLaunchKernelGGL((k_distill_loss<T, TAIL, TWO>), dim3((unsigned)a.rows), dim3(64), terms, s,
                       a);
  else
    hipLaunchKernelGGL((k_distill_grad<T, TAIL, TWO>), grid, dim3(kThreads), terms, s, a);
}

template <typename T>
void run_typed(const Args& a, What what, int cus, hipStream_t s) {
  const bool tail = a.teacher_lse != nullptr, two = a.labels && a.T != 1.f;
  if (tail && two)
    run_as<T, true, true>(a, what, cus, s);
  else if (tail)
    run_as<T, true, false>(a, what, cus, s);
  else if (two)
    run_as<T, false, true>(a, what, cus, s);
  else
    run_as<T, false, false>(a, what, cus, s);
}

sgb_status run(sgb_distill p, const sgb_distill_args* q, void* ws, size_t ws_bytes, void* stream_,
               What what) {
  if (!p || !q) return SGB_ERR_INVALID_ARGUMENT;
  const int64_t R = q->rows;
  if (!float_dtype(q->dtype) || R < 0 || R >= (1ll << 25)) return SGB_ERR_INVALID_ARGUMENT;
  if ((p->ce != 0.f) != (q->labels != nullptr) && R > 0) return SGB_ERR_INVALID_ARGUMENT;
  if (R == 0) return SGB_OK;
  const size_t e = elem_size(q->dtype);
  if (!matrix_ok(q->logits, p->V, q->logits_stride, e) ||
      !matrix_ok(q->ids, p->K, q->ids_stride, 8) ||
      !matrix_ok(q->values, p->K, q->values_stride, 4) || !aligned(q->teacher_lse, 4) ||
      !aligned(q->labels, 8) || !aligned(q->row_weights, 4) || !aligned(q->grad_loss, 4))
    return SGB_ERR_INVALID_ARGUMENT;
  if (what != kBackward && (!q->loss || !aligned(q->loss, 4))) return SGB_ERR_INVALID_ARGUMENT;
  if (what == kBackward && !q->stats) return SGB_ERR_INVALID_ARGUMENT;
  if (what != kBoth && !aligned(q->stats, 16)) return SGB_ERR_INVALID_ARGUMENT;
  if (what != kLoss) {
    if (!matrix_ok(q->grad, p->V, q->grad_stride, e) || !std::isfinite(q->grad_scale))
      return SGB_ERR_INVALID_ARGUMENT;
    // the listed logits are read again after parts of the gradient are written
    if (overlap(q->logits, p->V, q->logits_stride, e, q->grad, p->V, q->grad_stride, e, R))
      return SGB_ERR_INVALID_ARGUMENT;
  }
  if (!workspace_ok(ws)) return SGB_ERR_INVALID_ARGUMENT;
  size_t need;
  const sgb_status st = sgb_distill_workspace_bytes(p, R, &need);
  if (st != SGB_OK) return st;
  if (ws_bytes < need) return SGB_ERR_WORKSPACE_TOO_SMALL;

  Args a{};
  a.logits = q->logits;
  a.ids = q->ids;
  a.values = q->values;
  a.teacher_lse = q->teacher_lse;
  a.labels = q->labels;
  a.weights = q->row_weights;
  a.grad_loss = what == kBackward ? q->grad_loss : nullptr;
  a.loss = what == kBackward ? nullptr : q->loss;
  a.stats = what == kBoth ? nullptr : q->stats;
  a.grad = q->grad;
  a.hdr = static_cast<Header*>(ws);
  a.part = reinterpret_cast<float4*>(static_cast<char*>(ws) + kHeaderBytes);
  a.epoch = next_epoch();
  a.sl = q->logits_stride;
  a.si = q->ids_stride;
  a.sv = q->values_stride;
  a.sg = q->grad_stride;
  a.rows = R;
  a.V = p->V;
  a.K = p->K;
  a.table = p->table;
  a.split = split_of(p, R);
  a.span = (int)(div_up(div_up(p->V, a.split), kStep) * kStep);
  a.split = (int)div_up(p->V, a.span);
  a.T = p->T;
  a.c = (float)(1.4426950408889634074 / (double)p->T);
  a.kd = p->kd;
  a.ce = p->ce;
  a.scale = what == kLoss ? 1.f : q->grad_scale;
  if (threads_of(a, what, e, p->cus) > kMostThreadsAtOnce) return SGB_ERR_UNSUPPORTED;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (q->dtype == SGB_F32)
    run_typed<float>(a, what, p->cus, s);
  else if (q->dtype == SGB_BF16)
    run_typed<bf16_t>(a, what, p->cus, s);
  else
    run_typed<f16_t>(a, what, p->cus, s);
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

}  // namespace

extern "C" {

sgb_status sgb_distill_create(sgb_distill* out, int64_t V, int32_t K, float T, float kd, float ce) {
  if (!out) return SGB_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (V < 1 || K < 1 || K > kMaxK || !(T > 0.f) || !std::isfinite(T) ||
      !std::isfinite((float)(1.4426950408889634074 / (double)T)) || !std::isfinite(kd) ||
      !std::isfinite(ce))
    return SGB_ERR_INVALID_ARGUMENT;
  if (V > kMaxV) return SGB_ERR_UNSUPPORTED;
  const int device = current_device();
  sgb_distill_s* p = new (std::nothrow) sgb_distill_s();
  if (!p) return SGB_ERR_HIP;
  p->device = device;
  p->cus = compute_units(device);
  p->V = V;
  p->K = K;
  p->table = 64;
  while (p->table < 2 * K) p->table *= 2;
  p->T = T;
  p->kd = kd;
  p->ce = ce;
  *out = p;
  return SGB_OK;
}

void sgb_distill_destroy(sgb_distill p) { delete p; }

sgb_status sgb_distill_workspace_bytes(sgb_distill p, int64_t rows, size_t* bytes) {
  if (!p || !bytes || rows < 0 || rows >= (1ll << 25)) return SGB_ERR_INVALID_ARGUMENT;
  *bytes = kHeaderBytes + align_up((size_t)most_parts(p, rows) * sizeof(float4), 256);
  return SGB_OK;
}

sgb_status sgb_distill_forward(sgb_distill p, const sgb_distill_args* q, void* ws, size_t n,
                               void* stream) {
  return run(p, q, ws, n, stream, kLoss);
}
sgb_status sgb_distill_backward(sgb_distill p, const sgb_distill_args* q, void* ws, size_t n,
                                void* stream) {
  return run(p, q, ws, n, stream, kBackward);
}
sgb_status sgb_distill_loss_grad(sgb_distill p, const sgb_distill_args* q, void* ws, size_t n,
                                 void* stream) {
  return run(p, q, ws, n, stream, kBoth);
}

}  // extern "C"
