// lm_penalty.hip -- logits penalties of libsgb_lm.so, before sampling
// (definition: include/sgb_lm.h).
//
// A workgroup takes a slice of one row's vocabulary.  It counts the row's
// tokens that fall into the slice in LDS, a word a vocabulary entry, and then
// reads, changes and writes each logit once.  Counting again in every slice
// costs a row's tokens from L2 a slice; counts in memory would cost two more
// passes as long as the logits.

#include <algorithm>
#include <cmath>
#include <new>

#include "lm_internal.h"

using namespace sgb_lm;

namespace {

constexpr int kThreads = 512;
constexpr int kMinSlice = 1024;
constexpr int kMaxSlice = 16384;   // 64 KB of counts: two workgroups a compute unit
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
__global__ __launch_bounds__(kThreads) void k_penalty(Args a) {
  extern __shared__ uint32_t word[];  // slice words
  __shared__ int twice;
  const int64_t row = blockIdx.x / a.slices;
  const int64_t v0 = (int64_t)(blockIdx.x % a.slices) * a.slice;
  const int size = (int)min((int64_t)a.slice, a.V - v0);
  const int nt = (int)blockDim.x, t = (int)threadIdx.x;
  if (blockIdx.x == 0 && t == 0) a.hdr->epoch = a.epoch;

  for (int i = t * 4; i < a.slice; i += nt * 4)
    *reinterpret_cast<uint4*>(word + i) = make_uint4(0, 0, 0, 0);
  if (t == 0) twice = 0;
  int len = a.lens ? a.lens[row] : a.L;
  int prompt = a.prompt ? a.prompt[row] : 0;
  uint32_t bad = 0;
  if (len < 0 || len > a.L || prompt < 0 || prompt > len) bad = SGB_ERR_BAD_OFFSETS;
  len = max(0, min(len, a.L));
  prompt = max(0, min(prompt, len));
  int mask_row = -1;
  if (a.mask) {
    mask_row = a.mask_index ? a.mask_index[row] : (int)row;
    if (mask_row >= a.masks) {
      bad = SGB_ERR_INDEX_OUT_OF_RANGE;
      mask_row = -1;
    }
  }
  __syncthreads();

  for (int k = t; k < a.biases; k += nt) {
    const int64_t id = a.bias_ids[row * a.sbi + k];
    if (id >= a.V) bad = SGB_ERR_INDEX_OUT_OF_RANGE;
    if (id >= v0 && id < v0 + size) {
      const uint32_t old = atomicOr(&word[id - v0], (uint32_t)(k + 1) << kBiasShift);
      if (old >> kBiasShift) twice = 1;
    }
  }
  const int32_t* tokens = a.tokens + row * a.st;
  auto count = [&](int i, int32_t tok) {
    const int64_t at = (int64_t)tok - v0;
    if (tok >= a.V) bad = SGB_ERR_INDEX_OUT_OF_RANGE;
    if (at >= 0 && at < size) {
      if (i >= prompt)
        atomicAdd(&word[at], 1u);
      else
        atomicOr(&word[at], kSeen);
    }
  };
  for (int i = t * 4; i < len; i += nt * 4) {
    if (i + 4 <= len) {
      const Int4 q = *reinterpret_cast<const Int4*>(tokens + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) count(i + j, q.v[j]);
    } else {
      for (int j = i; j < len; ++j) count(j, tokens[j]);
    }
  }
  if (bad) set_status(a.hdr, a.epoch, bad);
  __syncthreads();

  const float rep = a.rep ? a.rep[row] : 1.f, freq = a.freq ? a.freq[row] : 0.f,
              pres = a.pres ? a.pres[row] : 0.f;
  const T* x = static_cast<const T*>(a.logits) + row * a.sl + v0;
  T* out = static_cast<T*>(a.out) + row * a.so + v0;
  const uint8_t* allowed =
      mask_row < 0 ? nullptr
                   : reinterpret_cast<const uint8_t*>(a.mask + mask_row * a.sm) + (v0 >> 3);
  for (int i = t * 8; i < size; i += nt * 8) {
    const int n = min(8, size - i);
    float v[8];
    widen8(load8(x + i, n), v);
    const uint4 w0 = *reinterpret_cast<const uint4*>(word + i);
    const uint4 w1 = *reinterpret_cast<const uint4*>(word + i + 4);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    if ((w[0] | w[1] | w[2] | w[3]) | (w[4] | w[5] | w[6] | w[7])) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t n_said = w[j] & kCountMask;
        if (w[j] & (kSeen | kCountMask)) v[j] = v[j] > 0.f ? v[j] / rep : v[j] * rep;
        if (n_said) v[j] = fmaf(-freq, (float)n_said, v[j]) - pres;
        if (w[j] >> kBiasShift) {
          if (!twice) {
            v[j] += a.bias[row * a.sb + (w[j] >> kBiasShift) - 1];
          } else {  // an id listed more than once: its biases in order
            float b = 0.f;
            for (int k = 0; k < a.biases; ++k)
              if (a.bias_ids[row * a.sbi + k] == v0 + i + j) b += a.bias[row * a.sb + k];
            v[j] += b;
          }
        }
      }
    }
    if (allowed) {
      const uint32_t ok = allowed[i >> 3];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(ok >> j & 1)) v[j] = -INFINITY;
    }
    store8(out + i, v, n);
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
  if (R * a.slices >= (1ll << 31)) return SGB_ERR_UNSUPPORTED;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  const dim3 grid((unsigned)(R * a.slices)), threads(std::min(kThreads, a.slice / 8));
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
