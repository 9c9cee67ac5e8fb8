// lm_quant.hip -- root-mean-square norm with the residual's addition and an
// output in 8 bits with scales, of libsgb_lm.so (definition:
// include/sgb_lm_step.h).
//
// A row is held by a team of lanes, eight columns a lane: the residual sum,
// its squares' sum, the largest magnitude and the codes come from registers,
// so each input is read once and each output written once.  The largest is taken
// of x_out * weight, before the norm's factor is known, so that a row's squares and
// its largest take one exchange between waves; the factor is then one division a
// scale.  The next row's loads are in flight while a row is worked on.  Squares,
// products and scales are fp32; the codes are the only rounding to fewer bits.
//
// Bound by memory: 8192 x 4096 bf16, fp32 residual, e4m3 in groups of 128: 65 us,
// 5.7 TB/s; with bf16 residual, int8 and a scale a row: 39; 32768 x 4096 bf16 without
// residual, e4m3, a scale a row: 74 to 83 us, 4.9 to 5.4 TB/s, 148 with two exchanges a
// row and one vector a lane.  One row of 4096: 4.1.

#include <algorithm>
#include <cmath>
#include <new>

#include "lm_internal.h"
#include "sgb_lm_step.h"

using namespace sgb_lm;

namespace {

constexpr int kMaxCols = 8192;
constexpr int kMaxWaves = 16;

struct Args {
  const void *h, *x;
  void* x_out;
  const void* weight;
  uint8_t* q;
  float* scales;
  float* stats;
  int64_t sh, sx, sxo, sq, ss;
  int64_t rows;
  int D, tpr, in_group;  // lanes a row, lanes a group
  int weight_dtype;
  float eps, inv_d;
};

// Largest of x over groups of `width` lanes (4, 8, .. 64): one that is no number
// wins.  Magnitudes as words compare like their values, and NaN above all.
__device__ __forceinline__ float fold_most(float v, int width) {
  const auto f = [](float a, float b) {
    return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
  };
  if (width == 4) {
    v = f(v, dpp<0xB1>(v));
    return f(v, dpp<0x4E>(v));
  }
  return wave_fold(v, width, f);
}

// Codes are p * by, p = v * weight and by = M / (the largest p): 1 / rms cancels.
// Every rounding on the way moves a few codes of those on the border between
// two, so p keeps its rest, by is two floats, and only their sum is rounded.
// Where the largest p is far from one, by or the rests would leave fp32's range:
// p is then taken of v * up, a power of two, which is exact.
struct Factor {
  float hi, lo, up;
  bool on;
};
__device__ __forceinline__ Factor factor_of(float most_p, float scale, float M) {
  Factor f{0.f, 0.f, 1.f, scale > 0.f && scale < INFINITY};  // nor NaN
  if (f.on) {  // most_p > 0
    // (from 2^90 on: weights end at 2^128, so a v that matters stays a normal number)
    f.up = most_p < 0x1p-64f ? 0x1p64f : most_p > 0x1p90f ? 0x1p-64f : 1.f;
    most_p *= f.up;
    float r = __builtin_amdgcn_rcpf(most_p);
    r = fmaf(r, fmaf(-most_p, r, 1.f), r);
    f.hi = M * r;
    f.lo = fmaf(-most_p, f.hi, M) * r;
  }
  return f;
}

// WIDE: a row is one or more whole waves'.  K: vectors of eight a lane.  RES:
// there is a residual.
template <typename T, typename U, int CODE, bool WIDE, int K, bool RES, bool TINY>
__global__ __launch_bounds__(WIDE ? 512 : 256) void k_quant(Args a) {
  __shared__ float2 parts[2][kMaxWaves];  // a wave's sum of squares, its largest p
  constexpr float M = CODE == SGB_CODE_INT8 ? 127.f : 448.f;
  const int t = (int)threadIdx.x, lane = t & 63, wave = t >> 6;
  const int teams = (int)blockDim.x / a.tpr, nw = WIDE ? a.tpr >> 6 : 1;
  const int team = WIDE ? __builtin_amdgcn_readfirstlane(t / a.tpr) : t / a.tpr;
  const int in_row = t % a.tpr, first = wave / nw * nw;
  int col[K], n[K];
  float w[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    col[k] = (in_row + k * a.tpr) * 8;
    n[k] = max(0, min(8, a.D - col[k]));
    const RawAs wr = ask8_as<TINY>(a.weight, a.weight_dtype, col[k], a.D);
    have8_as<TINY>(wr, a.weight, a.weight_dtype, col[k], n[k], 1.f, w[k]);
  }

  const int64_t step = (int64_t)gridDim.x * teams;
  int64_t r = (int64_t)blockIdx.x * teams + team;
  Raw8<T> h[K];
  Raw8<U> x[K];
  const auto ask = [&](int64_t row) {
    const int64_t at = min(row, a.rows - 1);  // past the last: loaded, not used
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const T* ph = static_cast<const T*>(a.h) + at * a.sh;
      const U* px = static_cast<const U*>(a.x) + at * a.sx;
      if (TINY) {
        h[k] = load8(ph + col[k], n[k]);
        if (RES) x[k] = load8(px + col[k], n[k]);
      } else {
        h[k] = ask8(ph, (uint32_t)col[k], (uint32_t)a.D);
        if (RES) x[k] = ask8(px, (uint32_t)col[k], (uint32_t)a.D);
      }
    }
  };
  ask(r);
  int phase = 0;
  // every team of a workgroup takes as many turns: barriers are the workgroup's
  const int64_t turns = (a.rows + step - 1) / step;
  for (int64_t turn = 0; turn < turns; ++turn, r += step) {
    const bool mine = r < a.rows;
    float v[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!TINY) have8(h[k], n[k]);
      widen8(h[k], v[k]);
      if (RES) {
        float y[8];
        if (!TINY) have8(x[k], n[k]);
        widen8(x[k], y);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] += y[i];
      }
    }
    if (turn + 1 < turns) ask(r + step);
    float s = 0.f, most[K], all = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (mine && a.x_out && n[k] > 0) store8(static_cast<U*>(a.x_out) + r * a.sxo + col[k], v[k], n[k]);
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // (columns past the row are zeros, and so is their weight)
        s = fmaf(v[k][i], v[k][i], s);
        top = max(top, __float_as_uint(v[k][i] * w[k][i]) & 0x7fffffffu);
      }
      most[k] = __uint_as_float(top);
      all = __uint_as_float(max(__float_as_uint(all), top));
    }
    // one exchange for the row's squares and its largest
    s = wave_add(s, WIDE ? 64 : a.tpr);
    if (a.in_group) {
#pragma unroll
      for (int k = 0; k < K; ++k) most[k] = fold_most(most[k], a.in_group);
    } else {
      all = fold_most(all, WIDE ? 64 : a.tpr);
    }
    if (WIDE && nw > 1) {
      if (lane == 0) parts[phase][wave] = make_float2(s, all);
      __syncthreads();
      const float2 part = lane < nw ? parts[phase][first + lane] : make_float2(0.f, 0.f);
      phase ^= 1;
      s = wave_add(part.x, 16);
      s = __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(s)));
      if (!a.in_group) {
        all = fold_most(part.y, 16);
        all = __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(all)));
      }
    }
    const float rs = 1.0f / sqrtf(fmaf(s, a.inv_d, a.eps));
    if (mine && a.stats && in_row == 0) {
      typedef float F4 __attribute__((ext_vector_type(4)));
      *reinterpret_cast<F4*>(a.stats + 4 * r) = F4{0.f, 1.f, 0.f, rs};
    }
    Factor by;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (a.in_group || k == 0) {
        const float top = a.in_group ? most[k] : all;
        float scale = top * rs / M;
        if (scale < 0x1p-126f) scale = 0.f;
        by = factor_of(top, scale, M);
        const int lanes = a.in_group ? a.in_group : a.tpr;
        if (mine && n[k] > 0 && in_row % lanes == 0)
          a.scales[r * a.ss + (a.in_group ? (in_row + k * a.tpr) / lanes : 0)] = scale;
      }
      if (!mine || n[k] <= 0) continue;
      if (by.up != 1.f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] *= by.up;
      }
      float c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float p = v[k][i] * w[k][i], rest = fmaf(v[k][i], w[k][i], -p);
        const float q = fmaf(p, by.hi, fmaf(p, by.lo, rest * by.hi));
        c[i] = by.on ? __builtin_amdgcn_fmed3f(q, -M, M) : 0.f;
      }
      uint32_t b[2] = {0, 0};
      if (CODE == SGB_CODE_INT8) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          b[i >> 2] |= ((uint32_t)(int)rintf(c[i]) & 0xffu) << (8 * (i & 3));
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i], c[4 * i + 1], 0, false);
          b[i] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c[4 * i + 2], c[4 * i + 3], p, true);
        }
      }
      uint8_t* out = a.q + r * a.sq + col[k];
      if (n[k] >= 8) {
        typedef uint32_t W2 __attribute__((ext_vector_type(2)));
        typedef W2 Any __attribute__((aligned(1)));
        store_global<Any>(out, 0, W2{b[0], b[1]});
      } else {
#pragma unroll
        for (int i = 0; i < 7; ++i)
          if (i < n[k]) out[i] = (uint8_t)(b[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
}

template <typename T, typename U, int CODE, bool RES>
void launch_as(const Args& a, unsigned grid, int threads, hipStream_t s) {
  const dim3 g(grid), b(threads);
  if (a.D < 8)
    hipLaunchKernelGGL((k_quant<T, U, CODE, false, 1, RES, true>), g, b, 0, s, a);
  else if (a.D > a.tpr * 8)
    hipLaunchKernelGGL((k_quant<T, U, CODE, true, 2, RES, false>), g, b, 0, s, a);
  else if (a.tpr >= 64)
    hipLaunchKernelGGL((k_quant<T, U, CODE, true, 1, RES, false>), g, b, 0, s, a);
  else
    hipLaunchKernelGGL((k_quant<T, U, CODE, false, 1, RES, false>), g, b, 0, s, a);
}

template <typename T, typename U, int CODE>
void launch(const Args& a, unsigned grid, int threads, hipStream_t s) {
  if (a.x)
    launch_as<T, U, CODE, true>(a, grid, threads, s);
  else
    launch_as<T, U, CODE, false>(a, grid, threads, s);
}

template <typename T, typename U>
void launch(const Args& a, int code, unsigned grid, int threads, hipStream_t s) {
  if (code == SGB_CODE_INT8)
    launch<T, U, SGB_CODE_INT8>(a, grid, threads, s);
  else
    launch<T, U, SGB_CODE_E4M3>(a, grid, threads, s);
}

}  // namespace

struct sgb_quant_norm_s {
  int device, cus;
  int D, code, group;
  float eps;
};

extern "C" {

sgb_status sgb_quant_norm_create(sgb_quant_norm* out, int32_t D, int32_t code, int32_t group,
                                 float eps) {
  if (!out) return SGB_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (D < 1 || D > kMaxCols || (code != SGB_CODE_INT8 && code != SGB_CODE_E4M3) ||
      (group != 0 && group != 32 && group != 64 && group != 128 && group != 256 && group != 512) ||
      !(eps >= 0.f) || std::isinf(eps))
    return SGB_ERR_INVALID_ARGUMENT;
  sgb_quant_norm_s* p = new (std::nothrow) sgb_quant_norm_s();
  if (!p) return SGB_ERR_HIP;
  p->device = current_device();
  p->cus = compute_units(p->device);
  p->D = D;
  p->code = code;
  p->group = group;
  p->eps = eps;
  *out = p;
  return SGB_OK;
}

void sgb_quant_norm_destroy(sgb_quant_norm p) { delete p; }

sgb_status sgb_quant_norm_forward(sgb_quant_norm p, const sgb_quant_norm_args* q, void* stream_) {
  if (!p || !q) return SGB_ERR_INVALID_ARGUMENT;
  const int64_t R = q->rows, D = p->D, groups = p->group ? div_up(D, p->group) : 1;
  if (!float_dtype(q->dtype) || !float_dtype(q->weight_dtype) || R < 0 || R >= (1ll << 31) ||
      (q->res_dtype != q->dtype && q->res_dtype != SGB_F32) || q->reserved != 0)
    return SGB_ERR_INVALID_ARGUMENT;
  if (R == 0) return SGB_OK;
  const size_t e = elem_size(q->dtype), er = elem_size(q->res_dtype);
  if (!matrix_ok(q->h, D, q->h_stride, e) || (q->x && !matrix_ok(q->x, D, q->x_stride, er)) ||
      (q->x_out && !matrix_ok(q->x_out, D, q->x_out_stride, er)) ||
      !matrix_ok(q->q, D, q->q_stride, 1) || !matrix_ok(q->scales, groups, q->scales_stride, 4) ||
      !q->weight || !aligned(q->weight, elem_size(q->weight_dtype)) || !aligned(q->stats, 16))
    return SGB_ERR_INVALID_ARGUMENT;
  const bool on_x = q->x_out == q->x && (R < 2 || q->x_out_stride == q->x_stride);
  const bool on_h = q->x_out == q->h && q->res_dtype == q->dtype &&
                    (R < 2 || q->x_out_stride == q->h_stride);
  // x_out may lie exactly on an input: the rest of what it may not touch
  const Extent x_out{q->x_out, R, D, q->x_out_stride, er}, h{q->h, R, D, q->h_stride, e},
      x{q->x, R, D, q->x_stride, er};
  const Extent others[] = {{q->q, R, D, q->q_stride, 1},
                           {q->scales, R, groups, q->scales_stride, 4},
                           vector(q->stats, 4 * R, 4)};
  const Extent read[] = {h, x, x_out, vector(q->weight, D, elem_size(q->weight_dtype))};
  if ((!on_x && overlap(x_out, x)) || (!on_h && overlap(x_out, h)) || overlap(x_out, read[3]) ||
      any_overlap(others, 3, read, 4))
    return SGB_ERR_INVALID_ARGUMENT;

  Args a{};
  a.h = q->h;
  a.x = q->x;
  a.x_out = q->x_out;
  a.weight = q->weight;
  a.q = q->q;
  a.scales = q->scales;
  a.stats = q->stats;
  a.sh = q->h_stride;
  a.sx = q->x_stride;
  a.sxo = q->x_out_stride;
  a.sq = q->q_stride;
  a.ss = q->scales_stride;
  a.rows = R;
  a.D = (int)D;
  a.weight_dtype = q->weight_dtype;
  a.eps = p->eps;
  a.inv_d = 1.f / (float)D;
  a.in_group = p->group < D ? p->group / 8 : 0;  // one group: the row's team may be narrower
  // Two vectors a lane from 1024 columns on: half the waves to fold over.
  a.tpr = 8;
  while (a.tpr * (D > 1024 ? 16 : 8) < D) a.tpr *= 2;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  const int threads = std::max(a.tpr, 256);
  const int64_t rows_a_block = threads / a.tpr;
  const int64_t most = (int64_t)p->cus * (2048 / threads);
  const unsigned grid = (unsigned)std::min(div_up(R, rows_a_block), most);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (q->dtype == SGB_F32)
    launch<float, float>(a, p->code, grid, threads, s);
  else if (q->dtype == SGB_BF16)
    q->res_dtype == SGB_F32 ? launch<bf16_t, float>(a, p->code, grid, threads, s)
                            : launch<bf16_t, bf16_t>(a, p->code, grid, threads, s);
  else
    q->res_dtype == SGB_F32 ? launch<f16_t, float>(a, p->code, grid, threads, s)
                            : launch<f16_t, f16_t>(a, p->code, grid, threads, s);
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

}  // extern "C"
