// lm_penalty.hip -- logits penalties of libsgb_lm.so, before sampling
// (definition: include/sgb_lm.h).
//
// A workgroup takes a slice of one row's vocabulary.  It counts the row's
// tokens that fall into the slice in LDS, a word a vocabulary entry, and then
// reads, changes and writes each logit once.  Counting again in every slice
// costs a row's tokens from L2 a slice; counts in memory would cost two more
// passes as long as the logits.  The logits are loaded into registers before
// the counting, so that they arrive meanwhile.
//
// Measured: 512 rows of 131072 fp32 with 8192 tokens in 105 us a pass, 5.2 TB/s of
// the logits and tokens read and the logits written, bound by memory; 64 rows of
// bf16 with 4096 tokens 10.6 us, 9 rows of 50021 fp16 with 60001 tokens 13 to 15 us,
// both one round of workgroups whose time is the chain of loads, counting and
// streaming and the fetching of their code; one row of 32000 4.4 us in the
// kernel, little over an empty launch.

#include <algorithm>
#include <cmath>
#include <new>

#include "lm_internal.h"

using namespace sgb_lm;

namespace {

constexpr int kThreads = 512;        // twice as many where one round of loads cannot hold the tokens
constexpr int kMostThreads = 1024;
constexpr int kMinSlice = 1024;
// 32 KB of counts: four workgroups a compute unit, one counting while others
// stream (512 rows of 131072 fp32, 8192 tokens: 105 us; slices of 16384 116 us,
// of 4096, whose tokens are read twice as often, 124 us).
constexpr int kMaxSlice = 8192;
constexpr int kSteps = kMaxSlice / (8 * kThreads);   // eight logits a thread each
constexpr int kAhead = 4;                            // loads of four tokens in flight
constexpr int kBiasTurns = 1024 / kThreads;  // biases a thread
static_assert(kSteps >= 1 && kMaxSlice % (8 * kThreads) == 0, "a slice is held in registers");
// a count word: how often generated, seen in the prompt, which bias (+1)
constexpr uint32_t kCountBits = 21;
constexpr uint32_t kCountMask = (1u << kCountBits) - 1;
constexpr uint32_t kSeen = 1u << kCountBits;
constexpr uint32_t kBiasShift = kCountBits + 1;
constexpr int kMaxTokens = (int)kCountMask;
constexpr int kMaxBiases = (1 << (32 - kBiasShift)) - 1;

struct Args {
  const void* logits;
  void* out;
  const int32_t *tokens, *prompt, *lens;
  const float *rep, *freq, *pres;
  const int32_t* bias_ids;
  const float* bias;
  const uint32_t* mask;
  const int32_t* mask_index;
  Header* hdr;
  uint32_t epoch;
  int64_t sl, so, st, sbi, sb, sm;
  int64_t V;
  int L, biases, masks;
  int slices, slice;
};

struct __attribute__((packed, aligned(4))) Int4 {
  int32_t v[4];
};

template <typename T>
__global__ __launch_bounds__(kMostThreads) void k_penalty(Args a) {
  extern __shared__ __attribute__((aligned(16))) uint32_t word[];  // slice words
  __shared__ int twice;
  const int64_t row = blockIdx.x / a.slices;
  const int64_t v0 = (int64_t)(blockIdx.x % a.slices) * a.slice;
  const int size = (int)min((int64_t)a.slice, a.V - v0);
  const int nt = (int)blockDim.x, t = (int)threadIdx.x;
  int len = value_or(a.lens, row, a.L), prompt = value_or(a.prompt, row, 0);
  const float rep = value_or(a.rep, row, 1.f), freq = value_or(a.freq, row, 0.f),
              pres = value_or(a.pres, row, 0.f);
  int mask_row = a.mask ? value_or(a.mask_index, row, (int)row) : -1;
  uint32_t bad = 0;
  if (len < 0 || len > a.L || prompt < 0 || prompt > len) bad = SGB_ERR_BAD_OFFSETS;
  len = max(0, min(len, a.L));
  prompt = max(0, min(prompt, len));
  if (mask_row >= a.masks) {
    bad = SGB_ERR_INDEX_OUT_OF_RANGE;
    mask_row = -1;
  }

  // Loads return in order: first what is counted, then the slice's logits,
  // which are on their way meanwhile.
  const bool fours = a.L >= 4;
  const uintptr_t tokens = fours ? (uintptr_t)(a.tokens + row * a.st) : (uintptr_t)kNowhere;
  const int last = fours ? max(len - 4, 0) : 0;
  Int4 q[kAhead];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      q[u] = load_global<Int4>(tokens + 4 * (uintptr_t)min(i0 + u * nt * 4, last));
  };
  fetch(t * 4);
  const int32_t* bias_ids = a.bias_ids + row * a.sbi;
  int32_t bias_id[kBiasTurns];
#pragma unroll
  for (int u = 0; u < kBiasTurns; ++u) 
    bias_id[u] = load_global<int32_t>(
        a.biases ? (uintptr_t)(bias_ids + min(t + u * nt, a.biases - 1)) : (uintptr_t)kNowhere);
  const T* x = static_cast<const T*>(a.logits) + row * a.sl;
  // a last slice of fewer than eight has the elements before it loaded too
  const T* from = x + max(v0 - 8, (int64_t)0);
  const uint32_t off = v0 > 0 ? 8 : 0;
  Raw8<T> raw[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k)
    raw[k] = ask8(a.V < 8 ? nullptr : from, off + (k * nt + t) * 8, off + size);
  for (int i = t * 4; i < a.slice; i += nt * 4)
    *reinterpret_cast<uint4*>(word + i) = make_uint4(0, 0, 0, 0);
  if (t == 0) twice = 0;
  __syncthreads();

  int top = -1;  // the largest token or bias id
  auto count = [&](int32_t tok, int at_place) {
    const uint32_t at = (uint32_t)tok - (uint32_t)v0;  // a negative token is past any slice
    top = max(top, tok);
    if (at < (uint32_t)size) {
      if (at_place >= prompt)
        atomicAdd(&word[at], 1u);
      else
        atomicOr(&word[at], kSeen);
    }
  };
  if (fours) {
    auto count_all = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u * nt * 4, from = min(i, last);
        if (i >= len) break;  // (skipped code is not fetched either)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          // a load that ends with the row holds tokens of its neighbour's too
          const bool mine = from + j >= i && from + j < len;
          count(mine ? q[u].v[j] : -1, from + j);
        }
      }
    };
    count_all(t * 4);
    for (int i0 = t * 4 + kAhead * nt * 4; i0 < len; i0 += kAhead * nt * 4) {
      fetch(i0);
      count_all(i0);
    }
  } else if (t < len) {
    count(a.tokens[row * a.st + t], t);
  }
#pragma unroll
  for (int u = 0; u < kBiasTurns; ++u) {
    const int32_t id = t + u * nt < a.biases ? bias_id[u] : -1;
    const uint32_t at = (uint32_t)id - (uint32_t)v0;
    top = max(top, id);
    if (at < (uint32_t)size) {
      const uint32_t old = atomicOr(&word[at], (uint32_t)(t + u * nt + 1) << kBiasShift);
      if (old >> kBiasShift) twice = 1;
    }
  }
  if (top >= a.V) bad = SGB_ERR_INDEX_OUT_OF_RANGE;
  if (bad) set_status(a.hdr, a.epoch, bad);
  if (blockIdx.x == 0 && t == 0) a.hdr->epoch = a.epoch;
  __syncthreads();

  T* out = static_cast<T*>(a.out) + row * a.so + v0;
  const uint8_t* allowed =
      mask_row < 0 ? nullptr
                   : reinterpret_cast<const uint8_t*>(a.mask + mask_row * a.sm) + (v0 >> 3);
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int i = (k * nt + t) * 8;
    if (i >= size) break;
    const uint32_t ok = allowed ? allowed[i >> 3] : 0xffu;
    if (k == 0 && a.V < 8)
      raw[k] = load8(x + i, size - i);
    else
      have8(raw[k], size - i);
    float v[8];
    widen8(raw[k], v);
    const uint4 w0 = *reinterpret_cast<const uint4*>(word + i);
    const uint4 w1 = *reinterpret_cast<const uint4*>(word + i + 4);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    // Few of a sequence's tokens fall into one wave's 512 logits, but seldom
    // none: a turn of this loop takes one touched logit of each lane, where
    // the same for all eight cost the wave eight turns.
    uint32_t todo = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) todo |= w[j] ? 1u << j : 0u;
    todo &= ok;
    while (todo) {
      const int at = __builtin_ctz(todo);
      todo &= todo - 1;
      float y = v[0];
      uint32_t c = w[0];
#pragma unroll
      for (int j = 1; j < 8; ++j) {
        y = at == j ? v[j] : y;
        c = at == j ? w[j] : c;
      }
      const uint32_t n_said = c & kCountMask;
      if (c & (kSeen | kCountMask)) y = y > 0.f ? y / rep : y * rep;
      if (n_said) y = fmaf(-freq, (float)n_said, y) - pres;
      if (c >> kBiasShift) {
        if (!twice) {
          y += a.bias[row * a.sb + (c >> kBiasShift) - 1];
        } else {  // an id listed more than once: its biases in order
          float b = 0.f;
          for (int m = 0; m < a.biases; ++m)
            if (bias_ids[m] == v0 + i + at) b += a.bias[row * a.sb + m];
          y += b;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = at == j ? y : v[j];
    }
    if (allowed) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(ok >> j & 1)) v[j] = -INFINITY;
    }
    store8(out + i, v, size - i);
  }
}

}  // namespace

// ------------------------------------------------------------- host

struct sgb_penalty_s {
  int device, cus;
  int64_t V;
};

extern "C" {

sgb_status sgb_penalty_create(sgb_penalty* out, int64_t vocab) {
  if (!out) return SGB_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (vocab < 1 || vocab >= (1ll << 31)) return SGB_ERR_INVALID_ARGUMENT;
  const int device = current_device();
  sgb_penalty_s* p = new (std::nothrow) sgb_penalty_s();
  if (!p) return SGB_ERR_HIP;
  p->device = device;
  p->cus = compute_units(device);
  p->V = vocab;
  *out = p;
  return SGB_OK;
}

void sgb_penalty_destroy(sgb_penalty p) { delete p; }

sgb_status sgb_penalty_workspace_bytes(sgb_penalty p, int64_t rows, size_t* bytes) {
  if (!p || !bytes || rows < 0 || rows >= (1ll << 31)) return SGB_ERR_INVALID_ARGUMENT;
  *bytes = kHeaderBytes;
  return SGB_OK;
}

sgb_status sgb_penalty_apply(sgb_penalty p, const sgb_penalty_args* q, void* ws, size_t ws_bytes,
                             void* stream_) {
  if (!p || !q) return SGB_ERR_INVALID_ARGUMENT;
  const int64_t R = q->rows, V = p->V;
  if (!float_dtype(q->dtype) || R < 0 || R >= (1ll << 31) || q->max_tokens < 0 ||
      q->num_biases < 0 || q->num_masks < 0)
    return SGB_ERR_INVALID_ARGUMENT;
  if (q->max_tokens > kMaxTokens || q->num_biases > kMaxBiases) return SGB_ERR_UNSUPPORTED;
  if (R == 0) return SGB_OK;
  const size_t e = elem_size(q->dtype);
  if (!matrix_ok(q->logits, V, q->logits_stride, e) || !matrix_ok(q->out, V, q->out_stride, e))
    return SGB_ERR_INVALID_ARGUMENT;
  if (q->max_tokens > 0 && !matrix_ok(q->tokens, q->max_tokens, q->tokens_stride, 4))
    return SGB_ERR_INVALID_ARGUMENT;
  if (!aligned(q->prompt_lens, 4) || !aligned(q->lens, 4) || !aligned(q->repetition, 4) ||
      !aligned(q->frequency, 4) || !aligned(q->presence, 4) || !aligned(q->mask_index, 4))
    return SGB_ERR_INVALID_ARGUMENT;
  if ((q->bias_ids != nullptr) != (q->bias_values != nullptr)) return SGB_ERR_INVALID_ARGUMENT;
  const int biases = q->bias_ids ? q->num_biases : 0;
  if (biases > 0 && (!matrix_ok(q->bias_ids, biases, q->bias_ids_stride, 4) ||
                     !matrix_ok(q->bias_values, biases, q->bias_values_stride, 4)))
    return SGB_ERR_INVALID_ARGUMENT;
  if (q->mask && !matrix_ok(q->mask, div_up(V, 32), q->mask_stride, 4))
    return SGB_ERR_INVALID_ARGUMENT;
  if (q->mask && !q->mask_index && q->num_masks < R) return SGB_ERR_INVALID_ARGUMENT;
  const bool in_place = q->logits == q->out && q->logits_stride == q->out_stride;
  if (!in_place && overlap(q->logits, V, q->logits_stride, e, q->out, V, q->out_stride, e, R))
    return SGB_ERR_INVALID_ARGUMENT;
  if (!workspace_ok(ws)) return SGB_ERR_INVALID_ARGUMENT;
  if (ws_bytes < kHeaderBytes) return SGB_ERR_WORKSPACE_TOO_SMALL;

  Args a{};
  a.logits = q->logits;
  a.out = q->out;
  a.tokens = q->tokens;
  a.prompt = q->prompt_lens;
  a.lens = q->lens;
  a.rep = q->repetition;
  a.freq = q->frequency;
  a.pres = q->presence;
  a.bias_ids = q->bias_ids;
  a.bias = q->bias_values;
  a.mask = reinterpret_cast<const uint32_t*>(q->mask);
  a.mask_index = q->mask_index;
  a.hdr = static_cast<Header*>(ws);
  a.epoch = next_epoch();
  a.sl = q->logits_stride;
  a.so = q->out_stride;
  a.st = q->tokens_stride;
  a.sbi = q->bias_ids_stride;
  a.sb = q->bias_values_stride;
  a.sm = q->mask_stride;
  a.V = V;
  a.L = q->max_tokens;
  a.biases = biases;
  a.masks = q->num_masks;
  // the largest slice that still gives every compute unit two workgroups
  a.slice = kMinSlice;
  while (a.slice < kMaxSlice && R * div_up(V, a.slice * 2) >= 2 * p->cus) a.slice *= 2;
  a.slices = (int)div_up(V, a.slice);
  const int nt = a.L > kThreads * kAhead * 4 ? kMostThreads : kThreads;
  if (R * a.slices > kMostThreadsAtOnce / nt) return SGB_ERR_UNSUPPORTED;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  const dim3 grid((unsigned)(R * a.slices)), threads(nt);
  const size_t lds = (size_t)a.slice * 4;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (q->dtype == SGB_F32)
    hipLaunchKernelGGL(k_penalty<float>, grid, threads, lds, s, a);
  else if (q->dtype == SGB_BF16)
    hipLaunchKernelGGL(k_penalty<bf16_t>, grid, threads, lds, s, a);
  else
    hipLaunchKernelGGL(k_penalty<f16_t>, grid, threads, lds, s, a);
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

}  // extern "C"
