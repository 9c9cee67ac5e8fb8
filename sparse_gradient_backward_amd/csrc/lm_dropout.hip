// lm_dropout.hip -- dropout from a counter-based generator, of libsgb_lm.so
// (definition: include/sgb_lm_step.h).
//
// Eight columns a lane, the widest load of a 16-bit type, and one Philox4x32-10
// block (the published generator of Salmon, Moraes, Dror and Shaw, "Parallel
// Random Numbers: As Easy as 1, 2, 3", SC'11) for the eight: 16 bits an
// element.  32 bits an element would take two blocks, and the generator's ten
// rounds of quarter-rate products longer than the traffic.  The counter is
// the element's place, so a lane needs nothing from another and the mask is in
// no memory.
//
// Bound by memory: the generator runs while loads are in flight, four rows' at a
// time.  32768 x 4096 bf16 with the residual: 140 us, 5.75 TB/s, where a long
// elementwise product reaches 6.1; without it, the backward's form, 79 to 92 us;
// 512 x 256 fp32 3.6.  Rows of fewer than eight columns are loaded one element at a
// time (no load of eight lies within such a row).

#include <cmath>
#include <new>

#include "lm_internal.h"
#include "sgb_lm_step.h"

using namespace sgb_lm;

namespace {

constexpr int kThreads = 256;
constexpr int kMaxCols = 1 << 24;  // a row's bytes fit 32 bits
constexpr int kAhead = 4;  // row groups whose loads are in flight in a lane

struct Args {
  const void *x, *res;
  void* out;
  const uint64_t* state;
  int64_t sx, sr, so;
  int64_t rows, first;
  uint64_t seed, offset;
  int cols, blocks_a_row;  // workgroups side by side in a row
  int lanes;               // lanes a row has in a workgroup, a power of two
  uint32_t cut;
  float scale;
};

struct Bits {
  uint32_t w[4];
};

__device__ __forceinline__ Bits philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3,
                                       uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t p = (uint64_t)c0 * 0xD2511F53u, q = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(q >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)q;
    c2 = (uint32_t)(p >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)p;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Bits{{c0, c1, c2, c3}};
}

// TINY: rows of fewer than eight columns.
template <typename T, typename U, bool RES, bool TINY>
__global__ __launch_bounds__(kThreads) void k_dropout(Args a) {
  const int64_t block = blockIdx.x / a.blocks_a_row;
  const int across = (int)(blockIdx.x % a.blocks_a_row);
  const int t = (int)threadIdx.x;
  const int in_pass = kThreads / a.lanes;  // rows side by side
  const int64_t r0 = block * (int64_t)(in_pass * kAhead) + t / a.lanes;
  const int64_t c64 = ((int64_t)across * kThreads + t % a.lanes) * 8;
  if (c64 >= a.cols) return;
  const int col = (int)c64, n = min(8, a.cols - col);
  uint64_t seed = a.seed, offset = a.offset;
  if (a.state) {
    seed = a.state[0];
    offset += a.state[1];
  }
  Raw8<T> v[kAhead];
  Raw8<U> w[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t r = min(r0 + u * in_pass, a.rows - 1);  // past the last row: loaded, not used
    const T* x = static_cast<const T*>(a.x) + r * a.sx;
    if (TINY)
      v[u] = load8(x + col, n);
    else
      v[u] = ask8(x, (uint32_t)col, (uint32_t)a.cols);
    if (RES) {
      const U* y = static_cast<const U*>(a.res) + r * a.sr;
      if (TINY)
        w[u] = load8(y + col, n);
      else
        w[u] = ask8(y, (uint32_t)col, (uint32_t)a.cols);
    }
  }
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    const int64_t r = r0 + u * in_pass;
    if (r >= a.rows) break;
    const uint64_t R = (uint64_t)(a.first + r);
    const Bits b = philox((uint32_t)col >> 3, (uint32_t)R, 0x80000000u + (uint32_t)(R >> 32),
                          (uint32_t)offset, (uint32_t)seed, (uint32_t)(seed >> 32));
    if (!TINY) {
      have8(v[u], n);
      if (RES) have8(w[u], n);
    }
    float x[8], y[8];
    widen8(v[u], x);
    if (RES) widen8(w[u], y);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t bits = i & 1 ? b.w[i >> 1] >> 16 : b.w[i >> 1] & 0xffffu;
      if (RES)  // one rounding; what is dropped leaves the residual's bits
        x[i] = bits >= a.cut ? fmaf(x[i], a.scale, y[i]) : y[i];
      else
        x[i] = bits >= a.cut ? x[i] * a.scale : 0.f;
    }
    store8(static_cast<U*>(a.out) + r * a.so + col, x, n);
  }
}

template <typename T, typename U>
void launch(const Args& a, unsigned grid, hipStream_t s) {
  if (a.cols < 8) {
    if (a.res)
      hipLaunchKernelGGL((k_dropout<T, U, true, true>), dim3(grid), dim3(kThreads), 0, s, a);
    else
      hipLaunchKernelGGL((k_dropout<T, U, false, true>), dim3(grid), dim3(kThreads), 0, s, a);
  } else if (a.res) {
    hipLaunchKernelGGL((k_dropout<T, U, true, false>), dim3(grid), dim3(kThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_dropout<T, U, false, false>), dim3(grid), dim3(kThreads), 0, s, a);
  }
}

}  // namespace

struct sgb_dropout_s {
  int device;
  uint32_t cut;
  float scale;
};

extern "C" {

sgb_status sgb_dropout_create(sgb_dropout* out, double p) {
  if (!out) return SGB_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (!(p >= 0.0 && p <= 1.0)) return SGB_ERR_INVALID_ARGUMENT;
  sgb_dropout_s* d = new (std::nothrow) sgb_dropout_s();
  if (!d) return SGB_ERR_HIP;
  d->device = current_device();
  d->cut = (uint32_t)std::nearbyint(p * 65536.0);
  d->scale = d->cut == 65536 ? 0.f : (float)(65536.0 / (65536.0 - d->cut));
  *out = d;
  return SGB_OK;
}

void sgb_dropout_destroy(sgb_dropout p) { delete p; }

sgb_status sgb_dropout_apply(sgb_dropout p, const sgb_dropout_args* q, void* stream_) {
  if (!p || !q) return SGB_ERR_INVALID_ARGUMENT;
  const int64_t R = q->rows, D = q->cols;
  if (!float_dtype(q->dtype) || R < 0 || D < 1 || q->first_row < 0 || R >= (1ll << 62) ||
      q->first_row > (1ll << 62) - R || q->reserved != 0)
    return SGB_ERR_INVALID_ARGUMENT;
  if (q->out_dtype != q->dtype && (q->out_dtype != SGB_F32 || !q->residual))
    return SGB_ERR_INVALID_ARGUMENT;
  if (D > kMaxCols) return SGB_ERR_UNSUPPORTED;
  if (R == 0) return SGB_OK;
  const size_t e = elem_size(q->dtype), eo = elem_size(q->out_dtype);
  if (!matrix_ok(q->x, D, q->x_stride, e) || !matrix_ok(q->out, D, q->out_stride, eo) ||
      (q->residual && !matrix_ok(q->residual, D, q->residual_stride, eo)) || !aligned(q->state, 8))
    return SGB_ERR_INVALID_ARGUMENT;
  const bool on_x = q->out == q->x && q->out_dtype == q->dtype && (R < 2 || q->out_stride == q->x_stride);
  const bool on_res = q->out == q->residual && (R < 2 || q->out_stride == q->residual_stride);
  if (!on_x && overlap(q->out, D, q->out_stride, eo, q->x, D, q->x_stride, e, R))
    return SGB_ERR_INVALID_ARGUMENT;
  if (!on_res && overlap(q->out, D, q->out_stride, eo, q->residual, D, q->residual_stride, eo, R))
    return SGB_ERR_INVALID_ARGUMENT;
  if (overlap({q->out, R, D, q->out_stride, eo}, vector(q->state, 2, 8)))
    return SGB_ERR_INVALID_ARGUMENT;

  Args a{};
  a.x = q->x;
  a.res = q->residual;
  a.out = q->out;
  a.state = q->state;
  a.sx = q->x_stride;
  a.sr = q->residual_stride;
  a.so = q->out_stride;
  a.rows = R;
  a.first = q->first_row;
  a.seed = q->seed;
  a.offset = q->offset;
  a.cols = (int)D;
  a.cut = p->cut;
  a.scale = p->scale;
  const int64_t groups = div_up(D, 8);
  a.lanes = 1;
  while (a.lanes < kThreads && a.lanes < groups) a.lanes *= 2;
  a.blocks_a_row = (int)div_up(groups, a.lanes);
  const int64_t down = div_up(R, (int64_t)(kThreads / a.lanes) * kAhead);
  if (down > kMostThreadsAtOnce / kThreads / a.blocks_a_row) return SGB_ERR_UNSUPPORTED;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  const unsigned grid = (unsigned)(down * a.blocks_a_row);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (q->dtype == SGB_F32)
    launch<float, float>(a, grid, s);
  else if (q->dtype == SGB_BF16)
    q->out_dtype == SGB_F32 ? launch<bf16_t, float>(a, grid, s) : launch<bf16_t, bf16_t>(a, grid, s);
  else
    q->out_dtype == SGB_F32 ? launch<f16_t, float>(a, grid, s) : launch<f16_t, f16_t>(a, grid, s);
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

}  // extern "C"
