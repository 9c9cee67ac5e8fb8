// lm_norm.hip -- block norms of libsgb_lm.so: the norm after a block, its
// gate, the scaled residual and the norm before the next block, forward and
// backward (formulas: include/sgb_lm.h).
//
// A row is held by a team of TPR lanes, eight columns a lane (16 bytes of a
// 16-bit type, the widest load), so each input is read once and each output
// written once: both norms, their sums and the elementwise work happen
// between one load and one store.  Teams are 8 lanes to 16 waves wide (the
// power of two that covers the row); several teams share a workgroup.  A team
// walks over rows with the next row's loads in flight, and the parameters stay
// in its registers.
//
// Measured: forward, 8192 x 4096, fp32 residuals and bf16 blocks, layer norms:
// 83 us a pass, 4.9 TB/s of what it reads and writes once (72 us where the pass
// before left part of the inputs in the last-level cache); bound by memory.

#include <algorithm>
#include <new>

#include "lm_internal.h"

using namespace sgb_lm;

namespace {

constexpr int kMaxCols = 8192;
constexpr int kMaxWaves = 16;

// Team shapes: rows of fewer than eight columns (a load of eight does not fit
// in them); a team narrower than a wave; 1 to 8 waves; 16 waves (rows of more
// than 4096 columns, in workgroups of 1024).
enum Shape { kTiny, kNarrow, kWide, kWhole };
template <int S>
constexpr int kThreads = S == kWhole ? 1024 : 512;

// ------------------------------------------------------------- team sums

// Sums each of v[NV] over the team.  `lds` holds 2 * NV_MAX * kMaxWaves
// floats; successive calls use its halves in turn (`phase`), so that one
// barrier a call is enough: a half is written again only after the barrier of
// the call in between.  Contains a barrier if tpr > 64 (block-uniform).
template <int S, int NV>
__device__ __forceinline__ void team_sum(float (&v)[NV], int tpr, float* lds, int& phase) {
  const int in_wave = S <= kNarrow ? tpr : 64;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = wave_add(v[i], in_wave);
  if (S <= kNarrow || tpr == 64) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, nw = tpr >> 6;
  float* half = lds + phase * (2 * kMaxWaves);
  phase ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) half[i * kMaxWaves + wave] = v[i];
  }
  __syncthreads();
  const int first = wave / nw * nw;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float x = lane < nw ? half[i * kMaxWaves + first + lane] : 0.f;
    x = wave_add(x, 16);
    v[i] = __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(x)));
  }
}

// Mean and 1 / deviation of the team's row.  The layer norm's variance is the
// mean squared distance from the mean (a second sum over the registers):
// E[v^2] - E[v]^2 loses what matters when the mean is large.
template <int S>
__device__ __forceinline__ void row_stats(const float (&v)[8], int n, int kind, float inv_d,
                                          float eps, int tpr, float* lds, int& phase, float& mean,
                                          float& rs) {
  mean = 0.f;
  rs = 1.f;
  if (kind == SGB_NORM_NONE) return;
  float s[1];
  if (kind == SGB_NORM_LAYER) {
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s[0] += v[i];
    team_sum<S>(s, tpr, lds, phase);
    mean = s[0] * inv_d;
  }
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = i < n ? v[i] - mean : 0.f;
    s[0] = fmaf(d, d, s[0]);
  }
  team_sum<S>(s, tpr, lds, phase);
  rs = 1.0f / sqrtf(fmaf(s[0], inv_d, eps));
}

struct Params {  // of the two norms
  const void *post_w, *post_b, *pre_w, *pre_b;
  int dtype;
  int post, pre;
  float post_eps, pre_eps, scale;
};

// A row's loads, of which kTiny's are made when they are needed.
template <int S, typename T>
__device__ __forceinline__ Raw8<T> ask_row(const T* row, int64_t col, int64_t width) {
  if (S == kTiny) return Raw8<T>{};
  return ask8(row, col, width);
}
template <int S, typename T>
__device__ __forceinline__ void have_row(Raw8<T>& r, const T* row, int64_t col, int n) {
  if (S == kTiny)
    r = load8(row + col, row ? n : 0);
  else
    have8(r, n);
}

// This thread's team in the workgroup.  From a wave up it is the same for all
// lanes; saying so keeps row numbers and addresses in scalar registers.
template <int S>
__device__ __forceinline__ int team_in_block(int tpr) {
  const int t = (int)threadIdx.x / tpr;
  return S <= kNarrow ? t : __builtin_amdgcn_readfirstlane(t);
}

// ------------------------------------------------------------- forward

struct FwdArgs {
  Params p;
  const void *x, *h, *gate;
  void *x_out, *y;
  float* stats;
  int64_t sx, sh, sg, sxo, sy;
  int64_t rows, rpg, teams;  // teams in the grid
  int D, tpr;
};

template <typename T, typename R, int S>
__global__ __launch_bounds__(kThreads<S>) void k_norm_forward(FwdArgs a) {
  __shared__ float lds[4 * kMaxWaves];
  const int tpr = a.tpr, D = a.D;
  const int in_block = (int)blockDim.x / tpr;
  const int t = (int)threadIdx.x & (tpr - 1);
  const int64_t team = (int64_t)blockIdx.x * in_block + team_in_block<S>(tpr);
  const int col = t * 8, n = min(8, D - col);
  const float inv_d = 1.0f / (float)D;
  const T* h = static_cast<const T*>(a.h);
  const R* x = static_cast<const R*>(a.x);
  const T* gate = static_cast<const T*>(a.gate);

  Raw8<T> rh, rg;
  Raw8<R> rx;
  // without branches, so that nothing waits for these loads before the values
  // are used; rows past the last load it again
  auto fetch = [&](int64_t row) {
    const uint32_t r = (uint32_t)min(row, a.rows - 1);
    rh = ask_row<S>(h + r * a.sh, col, D);
    rx = ask_row<S>(x + r * a.sx, col, D);
    rg = ask_row<S>(gate ? gate + (int64_t)(r / (uint32_t)a.rpg) * a.sg : gate, col, D);
  };
  auto have = [&](int64_t row) {
    const uint32_t r = (uint32_t)min(row, a.rows - 1);
    have_row<S>(rh, h + r * a.sh, col, n);
    have_row<S>(rx, x + r * a.sx, col, n);
    have_row<S>(rg, gate ? gate + (int64_t)(r / (uint32_t)a.rpg) * a.sg : gate, col, n);
  };
  fetch(team);
  constexpr bool TINY = S == kTiny;
  float pw[8], pb[8], qw[8], qb[8];
  const int pt = a.p.dtype;
  const RawAs rpw = ask8_as<TINY>(a.p.post_w, pt, col, D), rpb = ask8_as<TINY>(a.p.post_b, pt, col, D),
              rqw = ask8_as<TINY>(a.p.pre_w, pt, col, D), rqb = ask8_as<TINY>(a.p.pre_b, pt, col, D);
  have8_as<TINY>(rpw, a.p.post_w, pt, col, n, 1.f, pw);
  have8_as<TINY>(rpb, a.p.post_b, pt, col, n, 0.f, pb);
  have8_as<TINY>(rqw, a.p.pre_w, pt, col, n, 1.f, qw);
  have8_as<TINY>(rqb, a.p.pre_b, pt, col, n, 0.f, qb);

  int phase = 0;
  // every team of the block makes the same number of turns: the sums' barriers
  const uint32_t turns =
      ((uint32_t)(a.rows - (int64_t)blockIdx.x * in_block) - 1) / (uint32_t)a.teams + 1;
  for (uint32_t k = 0; k < turns; ++k) {
    const int64_t row = team + k * a.teams;
    float v[8], xo[8], g[8];
    have(row);
    widen8(rh, v);
    widen8(rx, xo);
    widen8(rg, g);
    if (!gate) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = 1.f;
    }
    if (k + 1 < turns) fetch(row + a.teams);
    float mh, rsh, mx, rsx;
    row_stats<S>(v, n, a.p.post, inv_d, a.p.post_eps, tpr, lds, phase, mh, rsh);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float z = fmaf((v[i] - mh) * rsh, pw[i], pb[i]);
        // columns past the row hold zeros in every term but the bias's, which
        // loaded as zero there too
        xo[i] = fmaf(a.p.scale, xo[i], g[i] * z);
      }
    const bool on = row < a.rows;
      store8(static_cast<R*>(a.x_out) + row * a.sxo, (uint32_t)col, xo, on ? n : 0);
    row_stats<S>(xo, n, a.p.pre, inv_d, a.p.pre_eps, tpr, lds, phase, mx, rsx);
    if (a.y) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          y[i] = fmaf((xo[i] - mx) * rsx, qw[i], qb[i]);
        store8(static_cast<T*>(a.y) + row * a.sy, (uint32_t)col, y, on ? n : 0);
    }
    if (a.stats && on && t == 0) {
      float* s = a.stats + row * 4;
      s[0] = mh;
      s[1] = rsh;
      s[2] = mx;
      s[3] = rsx;
    }
  }
}

// ------------------------------------------------------------- backward
//
// With u, v the normalised x_out and h, means over the row's columns:
//   a  = dy * pre_weight          t  = dx_out + rs_x (a - u mean(a u) - mean(a))
//   dx = res_scale t              b  = t gate post_weight
//   dh = rs_h (b - v mean(b v) - mean(b))      (mean(a), mean(b): layer only)
//   d_pre_weight = sum dy u       d_pre_bias = sum dy
// The sums over rows that gate and post norm need are, for a gate's rows,
// A = sum t v and B = sum t:
//   d_gate = post_weight A + post_bias B,  d_post_weight = sum_g gate A,
//   d_post_bias = sum_g gate B,
// so two sums a column serve three outputs.
//
// Measured: 32768 x 4096 bf16, rms norms, one gate row: 315 us, 5.1 TB/s over
// four arrays read and two written, and 6 us for the join, and 500 us (4.8 TB/s)
// with fp32 residuals; 3001 x 1001 fp16 with a gate a row: 17 and 5 us, one round
// of workgroups whose time is their chain of loads, sums and barriers;
// 8192 x 4096 bf16, layer norms with biases, a gate for 1024 rows: 79 and 9 us.
//
// Each team sums over rows of its own in registers; a block's teams are added
// through LDS and one more launch adds the blocks' sums, column by column, in
// a fixed order.

// How the rows are dealt out.  `split`: rows sharing a gate row (all of them
// where there is none) are dealt to k teams of `rp` rows, a team has one gate
// row; else a team has rp rows, whole gates.
struct Deal {
  int64_t rp, k, teams, groups;
  int split;
};

struct BwdArgs {
  Params p;
  const void *dxo, *dy, *x, *h, *gate;
  const float* stats;
  void *dx, *dh, *dgate;
  float* par;   // [4][blocks][D]: sums of t v, t (times the gate unless `raw`), dy u, dy
  float* slot;  // [teams][D] d_gate of a team, where several share a gate
  Header* hdr;
  uint32_t epoch;
  int64_t sdxo, sdy, sx, sh, sg, sdx, sdh, sdg;
  int64_t rows, rpg;
  Deal d;
  int D, tpr, blocks;
  int raw;      // one gate row (or none): par holds A and B themselves
  int want;     // bits 0..3: par arrays that are wanted
  int use_h;
};

// FULL: a bias's gradient is wanted or a norm subtracts its mean (a layer norm);
// without it the two rms norms need neither the means nor half of the sums.
template <typename T, typename R, int S, bool GROUPED, bool FULL>
__global__ __launch_bounds__(kThreads<S>) void k_norm_backward(BwdArgs a) {
  __shared__ float lds[4 * kMaxWaves];
  constexpr int NT = kThreads<S>;
  __shared__ __attribute__((aligned(16))) float fold[S == kWhole ? 4 : NT * 8 * (FULL ? 4 : 2)];
  const int tpr = a.tpr, D = a.D;
  const int in_block = (int)blockDim.x / tpr;
  const int t = (int)threadIdx.x & (tpr - 1);
  const int64_t team = (int64_t)blockIdx.x * in_block + team_in_block<S>(tpr);
  const int col = t * 8, n = min(8, D - col);
  // no error to record, but an earlier call's is no longer the last one's
  if (blockIdx.x == 0 && threadIdx.x == 0) a.hdr->epoch = a.epoch;
  int64_t r0, r1, g0;  // the team's rows; its (first) gate row
  // (rows, teams and gates are below 2^31: 32-bit divisions)
  if (a.d.split) {
    const uint32_t group = (uint32_t)team / (uint32_t)a.d.k;
    g0 = group;
    r0 = g0 * a.rpg + ((uint32_t)team - group * (uint32_t)a.d.k) * a.d.rp;
    r1 = min(min(r0 + a.d.rp, (g0 + 1) * a.rpg), a.rows);
  } else {
    r0 = team * a.d.rp;
    r1 = min(r0 + a.d.rp, a.rows);
    g0 = a.gate ? (uint32_t)min(r0, a.rows) / (uint32_t)a.rpg : 0;
  }
  if (team >= a.d.teams) r1 = r0 = 0;
  const float inv_d = 1.0f / (float)D;
  const R* dxo = static_cast<const R*>(a.dxo);
  const R* x = static_cast<const R*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  const T* h = static_cast<const T*>(a.h);
  const T* gate = static_cast<const T*>(a.gate);

  Raw8<R> rdxo, rx;
  Raw8<T> rdy, rh, rg;
  float4 st;
  auto at_row = [&](int64_t row) { return min(row, a.rows - 1); };
  auto at_gate = [&](int64_t g) { return GROUPED ? gate + min(g, a.d.groups - 1) * a.sg : gate; };
  // without branches, as in the forward; rows past the team's are cleared, their
  // stats too: they may be another gate's rows, and what is not finite in them
  // would reach this team's sums through 0 * (1 / deviation)
  auto fetch = [&](int64_t row, int64_t g) {
    const int64_t r = at_row(row);
    st = load_global<float4>((uintptr_t)(a.stats + r * 4));
    rdxo = ask_row<S>(dxo + r * a.sdxo, col, D);
    rdy = ask_row<S>(dy ? dy + r * a.sdy : dy, col, D);
    rx = ask_row<S>(dy ? x + r * a.sx : (const R*)nullptr, col, D);
    rh = ask_row<S>(a.use_h ? h + r * a.sh : (const T*)nullptr, col, D);
    if (GROUPED) rg = ask_row<S>(at_gate(g), col, D);
  };
  auto have = [&](int64_t row, int64_t g) {
    const int64_t r = at_row(row);
    const int m = row < r1 ? n : 0;
    if (row >= r1) st = make_float4(0.f, 0.f, 0.f, 0.f);
    have_row<S>(rdxo, dxo + r * a.sdxo, col, m);
    have_row<S>(rdy, dy ? dy + r * a.sdy : dy, col, m);
    have_row<S>(rx, dy ? x + r * a.sx : (const R*)nullptr, col, m);
    have_row<S>(rh, a.use_h ? h + r * a.sh : (const T*)nullptr, col, m);
    if (GROUPED) have_row<S>(rg, at_gate(g), col, m);
  };
  fetch(r0, g0);
  constexpr bool TINY = S == kTiny;
  float pw[8], pb[8], qw[8], gt[8];
  const int pt = a.p.dtype;
  const void* post_b = FULL ? a.p.post_b : nullptr;
  const RawAs rpw = ask8_as<TINY>(a.p.post_w, pt, col, D), rpb = ask8_as<TINY>(post_b, pt, col, D),
              rqw = ask8_as<TINY>(a.p.pre_w, pt, col, D);
  if (gate && !GROUPED) {
    widen8(load8(gate + g0 * a.sg + col, r0 < r1 ? n : 0), gt);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) gt[i] = 1.f;
  }
  have8_as<TINY>(rpw, a.p.post_w, pt, col, n, 1.f, pw);
  have8_as<TINY>(rpb, post_b, pt, col, n, 0.f, pb);
  have8_as<TINY>(rqw, a.p.pre_w, pt, col, n, 1.f, qw);
  // A workgroup of 16 waves has 128 registers a lane: the parameters wait in
  // LDS there, each lane's own columns, and are read back where they are used
  // (in registers they cost over a hundred spills a lane).  That does not spare
  // all of them: GROUPED and FULL still spill 20 to 70 registers, two more forms
  // of fp32 elements 12 and 20; the others none.  8192 x 8192 bf16, layer norms
  // with biases, a gate a row: 435 us, 1.8 TB/s.
  constexpr bool IN_LDS = S == kWhole;
  __shared__ float4 held[IN_LDS ? 4 * 2 * NT : 1];
  auto put_by = [&](int which, const float (&v)[8]) {
    if constexpr (IN_LDS) {
      held[(2 * which) * NT + threadIdx.x] = make_float4(v[0], v[1], v[2], v[3]);
      held[(2 * which + 1) * NT + threadIdx.x] = make_float4(v[4], v[5], v[6], v[7]);
    }
  };
  auto get_by = [&](int which, float (&v)[8]) {
    if constexpr (IN_LDS) {
      const float4 x = held[(2 * which) * NT + threadIdx.x];
      const float4 y = held[(2 * which + 1) * NT + threadIdx.x];
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    }
  };
  put_by(0, qw);
  put_by(1, pw);
  if (!GROUPED) put_by(2, gt);
  if (FULL) put_by(3, pb);
  if (IN_LDS) __syncthreads();

  float A[8] = {}, B[8] = {}, P[8] = {}, Q[8] = {}, C[8] = {}, E[8] = {};
  int phase = 0;
  int64_t g = g0, left = GROUPED ? a.rpg : 0;  // rows to go in gate row g
  for (int64_t k = 0; k < a.d.rp; ++k) {
    const int64_t row = r0 + k;
    const bool on = row < r1;
    float dyv[8], u[8], v[8], tv[8];
    have(row, g);
    const float mh = FULL ? st.x : 0.f, rsh = st.y, mx = FULL ? st.z : 0.f, rsx = st.w;
      widen8(rdxo, tv);
      widen8(rdy, dyv);
      widen8(rx, u);
      widen8(rh, v);
      if (GROUPED) widen8(rg, gt);
    const bool last_of_gate = GROUPED && (left == 1 || row + 1 == r1);
    if (k + 1 < a.d.rp) fetch(row + 1, GROUPED && left == 1 ? g + 1 : g);

    if (dy) {
      float s[1 + FULL] = {};
      get_by(0, qw);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = (u[i] - mx) * rsx;
          const float d = dyv[i], w = d * qw[i];
          s[0] = fmaf(w, u[i], s[0]);
          if constexpr (FULL) s[1] += w;
          C[i] = fmaf(d, u[i], C[i]);
          if (FULL) E[i] += d;
        }
      team_sum<S>(s, tpr, lds, phase);
      const float m1 = s[0] * inv_d, m0 = FULL && a.p.pre == SGB_NORM_LAYER ? s[FULL] * inv_d : 0.f;
      get_by(0, qw);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          tv[i] = fmaf(rsx, fmaf(-u[i], m1, dyv[i] * qw[i]) - m0, tv[i]);
    }
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = tv[i] * a.p.scale;
      store8(static_cast<R*>(a.dx) + row * a.sdx, (uint32_t)col, o, on ? n : 0);
    float s[1 + FULL] = {};
    get_by(1, pw);
    if (!GROUPED) get_by(2, gt);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = (v[i] - mh) * rsh;
        A[i] = fmaf(tv[i], v[i], A[i]);
        if (FULL) B[i] += tv[i];
        tv[i] *= gt[i] * pw[i];  // now b
        s[0] = fmaf(tv[i], v[i], s[0]);
        if constexpr (FULL) s[1] += tv[i];
      }
    if (a.p.post != SGB_NORM_NONE) {
      team_sum<S>(s, tpr, lds, phase);
      const float m1 = s[0] * inv_d, m0 = FULL && a.p.post == SGB_NORM_LAYER ? s[FULL] * inv_d : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) tv[i] = (fmaf(-v[i], m1, tv[i]) - m0) * rsh;
    }
      store8(static_cast<T*>(a.dh) + row * a.sdh, (uint32_t)col, tv, on ? n : 0);

    if (GROUPED) {
      if (on && last_of_gate) {
          float o[8];
          get_by(1, pw);
          if (FULL) get_by(3, pb);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            o[i] = A[i] * pw[i];
            P[i] = fmaf(gt[i], A[i], P[i]);
            A[i] = 0.f;
            if (FULL) {
              o[i] = fmaf(B[i], pb[i], o[i]);
              Q[i] = fmaf(gt[i], B[i], Q[i]);
              B[i] = 0.f;
            }
          }
          if (a.dgate) store8(static_cast<T*>(a.dgate) + g * a.sdg, (uint32_t)col, o, n);
      }
      if (--left == 0) {
        left = a.rpg;
        ++g;
      }
    }
  }

  if (!GROUPED) {
    get_by(1, pw);
    get_by(2, gt);
    if (FULL) get_by(3, pb);
    if (a.slot && team < a.d.teams) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          o[i] = FULL ? fmaf(B[i], pb[i], A[i] * pw[i]) : A[i] * pw[i];
        store8(a.slot + team * D + col, o, n);
    }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        P[i] = a.raw ? A[i] : A[i] * gt[i];
        if (FULL) Q[i] = a.raw ? B[i] : B[i] * gt[i];
      }
  }
  // the block's teams, added in order
  if constexpr (S == kWhole) {
    float* out = a.par + (int64_t)blockIdx.x * D;
    const int64_t one = (int64_t)a.blocks * D;
    if (a.want & 1) store8(out + col, P, n);
    if (FULL && (a.want & 2)) store8(out + one + col, Q, n);
    if (a.want & 4) store8(out + 2 * one + col, C, n);
    if (FULL && (a.want & 8)) store8(out + 3 * one + col, E, n);
  } else {
    // One barrier for all of them, and every lane adds: short code, since a
    // workgroup with few rows waits for it to be fetched.
    constexpr int kSets = FULL ? 4 : 2;
    auto leave = [&](int set, const float (&v)[8]) {
      float4* f = reinterpret_cast<float4*>(fold + (set * NT + (int)threadIdx.x) * 8);
      f[0] = make_float4(v[0], v[1], v[2], v[3]);
      f[1] = make_float4(v[4], v[5], v[6], v[7]);
    };
    leave(0, P);
    leave(kSets / 2, C);
    if (FULL) leave(1, Q);
    if (FULL) leave(3, E);
    __syncthreads();
    const int width = tpr * 8, bits = __builtin_ctz(width);
#pragma unroll 1
    for (int e = (int)threadIdx.x; e < kSets * width; e += NT) {
      const int set = e >> bits, c = e & (width - 1);
      const int which = FULL ? set : 2 * set;
      if (!(a.want >> which & 1) || c >= D) continue;
      float x = 0.f;
#pragma unroll 4
      for (int m = 0; m < in_block; ++m) x += fold[set * NT * 8 + m * width + c];
      a.par[((int64_t)which * a.blocks + blockIdx.x) * D + c] = x;
    }
  }
}

// Adds up what the blocks (or a gate's teams) left, column by column: 16
// waves of 64 columns, each every 16th part, joined through LDS.
struct JoinArgs {
  const float *par, *slot;
  const void *post_w, *post_b, *gate;
  void* dgate;
  float* out[4];  // d_post_weight, d_post_bias, d_pre_weight, d_pre_bias
  int64_t sdg, k;
  int D, blocks, want, raw, pdtype, dtype;
};

__device__ __forceinline__ float elem_as(const void* p, int dtype, int64_t i) {
  return dtype == SGB_F32    ? static_cast<const float*>(p)[i]
         : dtype == SGB_BF16 ? (float)static_cast<const bf16_t*>(p)[i]
                             : (float)static_cast<const f16_t*>(p)[i];
}
__device__ __forceinline__ void put_as(void* p, int dtype, int64_t i, float v) {
  if (dtype == SGB_F32)
    static_cast<float*>(p)[i] = v;
  else if (dtype == SGB_BF16)
    static_cast<bf16_t*>(p)[i] = (bf16_t)v;
  else
    static_cast<f16_t*>(p)[i] = (f16_t)v;
}

__device__ __forceinline__ float join_column(const float* p, int64_t parts, int D, int col,
                                             float* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float s = 0.f;
  constexpr int N = 16;  // loads in flight
  for (int64_t k = wave; k < parts; k += 16 * N) {
    float v[N];
#pragma unroll
    for (int u = 0; u < N; ++u)
      v[u] = load_global<float>(
          (uintptr_t)(p + min(k + 16 * u, parts - 1) * D + min(col, D - 1)));
#pragma unroll
    for (int u = 0; u < N; ++u) s += k + 16 * u < parts ? v[u] : 0.f;
  }
  __syncthreads();
  lds[wave * 64 + lane] = s;
  __syncthreads();
  s = 0.f;
  if (wave == 0) {
#pragma unroll
    for (int w = 0; w < 16; ++w) s += lds[w * 64 + lane];
  }
  return s;  // whole in wave 0
}

__global__ __launch_bounds__(1024) void k_norm_join(JoinArgs a) {
  __shared__ float lds[1024];
  const int col = (int)blockIdx.x * 64 + (threadIdx.x & 63);
  const bool mine = threadIdx.x < 64 && col < a.D;
  if (blockIdx.y >= 3) {  // a gate shared by several teams
    const int64_t g = blockIdx.y - 3;
    const float s = join_column(a.slot + g * a.k * a.D, a.k, a.D, col, lds);
    if (mine) put_as(a.dgate, a.dtype, g * a.sdg + col, s);
    return;
  }
  if (blockIdx.y > 0) {  // the pre norm's two
    const int w = 1 + (int)blockIdx.y;
    if (!a.out[w]) return;
    const float s = (a.want >> w & 1) ? join_column(a.par + (int64_t)w * a.blocks * a.D, a.blocks,
                                                    a.D, col, lds)
                                      : 0.f;
    if (mine) a.out[w][col] = s;
    return;
  }
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (a.want >> i & 1)
      s[i] = join_column(a.par + (int64_t)i * a.blocks * a.D, a.blocks, a.D, col, lds);
  if (!mine) return;
  if (a.raw) {
    if (a.dgate) {
      float d = s[0] * (a.post_w ? elem_as(a.post_w, a.pdtype, col) : 1.f);
      if (a.post_b) d = fmaf(s[1], elem_as(a.post_b, a.pdtype, col), d);
      put_as(a.dgate, a.dtype, col, d);
    }
    const float gt = a.gate ? elem_as(a.gate, a.dtype, col) : 1.f;
    s[0] *= gt;
    s[1] *= gt;
  }
  if (a.out[0]) a.out[0][col] = s[0];
  if (a.out[1]) a.out[1][col] = s[1];
}

}  // namespace

// ------------------------------------------------------------- host

struct sgb_block_norm_s {
  int device, cus;
  int D, tpr;
  int post, pre;
  float post_eps, pre_eps, scale;
};

namespace {

int max_threads(const sgb_block_norm_s* p) { return p->tpr > 512 ? kThreads<kWhole> : kThreads<kWide>; }

// Most blocks of the backward: one or two fill a compute unit's registers.
int64_t backward_blocks(const sgb_block_norm_s* p, bool light) {
  return (int64_t)p->cus * (p->tpr > 512 || !light ? 1 : 2);
}

Deal deal_rows(const sgb_block_norm_s* p, int64_t rows, int64_t rpg, bool gate, bool light) {
  const int64_t target = backward_blocks(p, light) * (max_threads(p) / p->tpr);
  const int64_t rp = std::max<int64_t>(1, div_up(rows, target));
  Deal d{};
  d.groups = div_up(rows, rpg);
  if (!gate || rpg > 2 * rp) {
    d.split = 1;
    d.k = div_up(rpg, rp);
    d.rp = div_up(rpg, d.k);
    d.teams = d.groups * d.k;
  } else {
    d.rp = div_up(rp, rpg) * rpg;
    d.k = 1;
    d.teams = div_up(rows, d.rp);
  }
  return d;
}

sgb_status check(sgb_block_norm p, const sgb_norm_params* q, int dtype, int res_dtype, int64_t rows,
                 const void* gate, int64_t rpg) {
  if (!p || !q) return SGB_ERR_INVALID_ARGUMENT;
  if (!float_dtype(dtype) || !(res_dtype == SGB_F32 || res_dtype == dtype))
    return SGB_ERR_INVALID_ARGUMENT;
  if (rows < 0 || rows >= (1ll << 31) || (gate && rpg < 1)) return SGB_ERR_INVALID_ARGUMENT;
  if (!float_dtype(q->dtype)) return SGB_ERR_INVALID_ARGUMENT;
  const size_t e = elem_size(q->dtype);
  if ((p->post != SGB_NORM_NONE) != (q->post_weight != nullptr)) return SGB_ERR_INVALID_ARGUMENT;
  if ((p->pre != SGB_NORM_NONE) != (q->pre_weight != nullptr)) return SGB_ERR_INVALID_ARGUMENT;
  if ((q->post_bias && !q->post_weight) || (q->pre_bias && !q->pre_weight))
    return SGB_ERR_INVALID_ARGUMENT;
  if (!aligned(q->post_weight, e) || !aligned(q->post_bias, e) || !aligned(q->pre_weight, e) ||
      !aligned(q->pre_bias, e))
    return SGB_ERR_INVALID_ARGUMENT;
  return SGB_OK;
}

Params params_of(sgb_block_norm p, const sgb_norm_params* q) {
  return Params{q->post_weight, q->post_bias, q->pre_weight, q->pre_bias, q->dtype,
                p->post,        p->pre,       p->post_eps,   p->pre_eps,  p->scale};
}

template <typename T, typename R>
void forward_as(const sgb_block_norm_s* p, const FwdArgs& a, unsigned grid, unsigned threads,
                hipStream_t s) {
  const dim3 g(grid), n(threads);
  if (p->D < 8)
    hipLaunchKernelGGL((k_norm_forward<T, R, kTiny>), g, n, 0, s, a);
  else if (p->tpr < 64)
    hipLaunchKernelGGL((k_norm_forward<T, R, kNarrow>), g, n, 0, s, a);
  else if (p->tpr <= 512)
    hipLaunchKernelGGL((k_norm_forward<T, R, kWide>), g, n, 0, s, a);
  else
    hipLaunchKernelGGL((k_norm_forward<T, R, kWhole>), g, n, 0, s, a);
}

template <typename T, typename R, int S>
void backward_shaped(const BwdArgs& a, bool grouped, bool full, unsigned grid, hipStream_t s) {
  const dim3 g(grid), n(kThreads<S>);
  if (grouped && full)
    hipLaunchKernelGGL((k_norm_backward<T, R, S, true, true>), g, n, 0, s, a);
  else if (grouped)
    hipLaunchKernelGGL((k_norm_backward<T, R, S, true, false>), g, n, 0, s, a);
  else if (full)
    hipLaunchKernelGGL((k_norm_backward<T, R, S, false, true>), g, n, 0, s, a);
  else
    hipLaunchKernelGGL((k_norm_backward<T, R, S, false, false>), g, n, 0, s, a);
}

template <typename T, typename R>
void backward_as(const sgb_block_norm_s* p, const BwdArgs& a, bool grouped, bool full,
                 unsigned grid, hipStream_t s) {
  if (p->D < 8)
    backward_shaped<T, R, kTiny>(a, grouped, full, grid, s);
  else if (p->tpr < 64)
    backward_shaped<T, R, kNarrow>(a, grouped, full, grid, s);
  else if (p->tpr <= 512)
    backward_shaped<T, R, kWide>(a, grouped, full, grid, s);
  else
    backward_shaped<T, R, kWhole>(a, grouped, full, grid, s);
}

#define SGB_LM_NORM_DISPATCH(F, ...)                                         \
  do {                                                                       \
    if (dtype == SGB_F32)                                                    \
      F<float, float>(__VA_ARGS__);                                          \
    else if (dtype == SGB_BF16 && res_dtype == SGB_F32)                      \
      F<bf16_t, float>(__VA_ARGS__);                                         \
    else if (dtype == SGB_BF16)                                              \
      F<bf16_t, bf16_t>(__VA_ARGS__);                                        \
    else if (res_dtype == SGB_F32)                                           \
      F<f16_t, float>(__VA_ARGS__);                                          \
    else                                                                     \
      F<f16_t, f16_t>(__VA_ARGS__);                                          \
  } while (0)

}  // namespace

extern "C" {

sgb_status sgb_block_norm_create(sgb_block_norm* out, int32_t D, int32_t post, int32_t pre,
                                 float post_eps, float pre_eps, float res_scale) {
  if (!out) return SGB_ERR_INVALID_ARGUMENT;
  *out = nullptr;
  if (D < 1 || D > kMaxCols || post < SGB_NORM_NONE || post > SGB_NORM_LAYER ||
      pre < SGB_NORM_NONE || pre > SGB_NORM_LAYER)
    return SGB_ERR_INVALID_ARGUMENT;
  if (!(post_eps >= 0.f) || !(pre_eps >= 0.f)) return SGB_ERR_INVALID_ARGUMENT;
  const int device = current_device();
  sgb_block_norm_s* p = new (std::nothrow) sgb_block_norm_s();
  if (!p) return SGB_ERR_HIP;
  p->device = device;
  p->cus = compute_units(device);
  p->D = D;
  p->tpr = 8;
  while (p->tpr < 1024 && p->tpr * 8 < D) p->tpr *= 2;
  p->post = post;
  p->pre = pre;
  p->post_eps = post_eps;
  p->pre_eps = pre_eps;
  p->scale = res_scale;
  *out = p;
  return SGB_OK;
}

void sgb_block_norm_destroy(sgb_block_norm p) { delete p; }

sgb_status sgb_block_norm_workspace_bytes(sgb_block_norm p, int64_t rows, size_t* bytes) {
  if (!p || !bytes || rows < 0 || rows >= (1ll << 31)) return SGB_ERR_INVALID_ARGUMENT;
  // four sums a block and one d_gate a team, for any way of sharing gates.
  // Where n gates of more than 2 rp rows share rows / rp <= target teams' work,
  // each has at most target / (n - 1) + 1 teams (the last gate may have few
  // rows): the most, 2 target + 2, is with two; with rp = 1, 2 rows.
  const int64_t per_block = max_threads(p) / p->tpr;
  const int64_t target = backward_blocks(p, true) * per_block;
  const int64_t teams = std::min(2 * std::max<int64_t>(rows, 1), 2 * target + 2);
  const int64_t blocks = div_up(teams, per_block);
  *bytes = kHeaderBytes + align_up((size_t)(4 * blocks + teams) * p->D * sizeof(float), 256);
  return SGB_OK;
}

sgb_status sgb_block_norm_forward(sgb_block_norm p, const sgb_norm_params* q,
                                  const sgb_norm_forward_args* f, void* stream_) {
  if (!f) return SGB_ERR_INVALID_ARGUMENT;
  const int dtype = f->dtype, res_dtype = f->res_dtype;
  sgb_status st = check(p, q, dtype, res_dtype, f->rows, f->gate, f->rows_per_gate);
  if (st != SGB_OK) return st;
  if (f->rows == 0) return SGB_OK;
  if ((p->pre != SGB_NORM_NONE) != (f->y != nullptr)) return SGB_ERR_INVALID_ARGUMENT;
  const size_t e = elem_size(dtype), er = elem_size(res_dtype);
  const int D = p->D;
  const int64_t R = f->rows;
  if (!matrix_ok(f->x, D, f->x_stride, er) || !matrix_ok(f->h, D, f->h_stride, e) ||
      !matrix_ok(f->x_out, D, f->x_out_stride, er) ||
      (f->y && !matrix_ok(f->y, D, f->y_stride, e)) ||
      (f->gate && !matrix_ok(f->gate, D, f->gate_stride, e)) || !aligned(f->stats, 16))
    return SGB_ERR_INVALID_ARGUMENT;
  const int64_t G = f->gate ? div_up(R, f->rows_per_gate) : 0;
  const bool x_in_place = f->x_out == f->x && f->x_out_stride == f->x_stride;
  const bool h_in_place = f->y == f->h && f->y_stride == f->h_stride;
  if ((!x_in_place && overlap(f->x, D, f->x_stride, er, f->x_out, D, f->x_out_stride, er, R)) ||
      (!h_in_place && overlap(f->h, D, f->h_stride, e, f->y, D, f->y_stride, e, R)) ||
      overlap(f->h, D, f->h_stride, e, f->x_out, D, f->x_out_stride, er, R) ||
      overlap(f->x, D, f->x_stride, er, f->y, D, f->y_stride, e, R) ||
      overlap(f->x_out, D, f->x_out_stride, er, f->y, D, f->y_stride, e, R) ||
      (G && (overlap(f->gate, D, f->gate_stride, e, f->x_out, D, f->x_out_stride, er, G, R) ||
             overlap(f->gate, D, f->gate_stride, e, f->y, D, f->y_stride, e, G, R))))
    return SGB_ERR_INVALID_ARGUMENT;
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;

  FwdArgs a{};
  a.p = params_of(p, q);
  a.x = f->x;
  a.h = f->h;
  a.gate = f->gate;
  a.x_out = f->x_out;
  a.y = f->y;
  a.stats = f->stats;
  a.sx = f->x_stride;
  a.sh = f->h_stride;
  a.sg = f->gate_stride;
  a.sxo = f->x_out_stride;
  a.sy = f->y_stride;
  a.rows = R;
  a.rpg = f->gate ? std::min(f->rows_per_gate, R) : R;
  a.D = D;
  a.tpr = p->tpr;
  // one team a block until every compute unit has one, then fuller blocks
  int threads = std::max(64, p->tpr);
  while (threads < 512 && (int64_t)(threads / p->tpr) * p->cus < R) threads *= 2;
  const int per_block = threads / p->tpr;
  const int64_t resident = (int64_t)p->cus * (2048 / threads);
  const int64_t grid = std::min(div_up(R, per_block), resident);
  a.teams = grid * per_block;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  SGB_LM_NORM_DISPATCH(forward_as, p, a, (unsigned)grid, (unsigned)threads, s);
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

sgb_status sgb_block_norm_backward(sgb_block_norm p, const sgb_norm_params* q,
                                   const sgb_norm_backward_args* b, void* ws, size_t ws_bytes,
                                   void* stream_) {
  if (!b) return SGB_ERR_INVALID_ARGUMENT;
  const int dtype = b->dtype, res_dtype = b->res_dtype;
  sgb_status st = check(p, q, dtype, res_dtype, b->rows, b->gate, b->rows_per_gate);
  if (st != SGB_OK) return st;
  const int D = p->D;
  const int64_t R = b->rows;
  const bool pre = p->pre != SGB_NORM_NONE, post = p->post != SGB_NORM_NONE;
  if (b->d_gate && !b->gate) return SGB_ERR_INVALID_ARGUMENT;
  if (!post && (b->d_post_weight || b->d_post_bias)) return SGB_ERR_INVALID_ARGUMENT;
  if (!pre && (b->d_pre_weight || b->d_pre_bias)) return SGB_ERR_INVALID_ARGUMENT;
  if ((b->d_post_bias && !q->post_bias) || (b->d_pre_bias && !q->pre_bias))
    return SGB_ERR_INVALID_ARGUMENT;
  if (pre != (b->dy != nullptr) && R > 0) return SGB_ERR_INVALID_ARGUMENT;
  if (!aligned(b->d_post_weight, 4) || !aligned(b->d_post_bias, 4) || !aligned(b->d_pre_weight, 4) ||
      !aligned(b->d_pre_bias, 4))
    return SGB_ERR_INVALID_ARGUMENT;
  const size_t e = elem_size(dtype), er = elem_size(res_dtype);
  const bool use_h = post || b->d_gate;
  // rows past the last one belong to no gate
  const int64_t rpg = std::max<int64_t>(1, b->gate ? std::min(b->rows_per_gate, R) : R);
  size_t need = 0;
  if (R > 0) {
    if (!matrix_ok(b->dx_out, D, b->dx_out_stride, er) || !matrix_ok(b->dx, D, b->dx_stride, er) ||
        !matrix_ok(b->dh, D, b->dh_stride, e) ||
        (pre && (!matrix_ok(b->dy, D, b->dy_stride, e) ||
                 !matrix_ok(b->x_out, D, b->x_out_stride, er))) ||
        (use_h && !matrix_ok(b->h, D, b->h_stride, e)) ||
        (b->gate && !matrix_ok(b->gate, D, b->gate_stride, e)) ||
        (b->d_gate && !matrix_ok(b->d_gate, D, b->d_gate_stride, e)) || !b->stats ||
        !aligned(b->stats, 16))
      return SGB_ERR_INVALID_ARGUMENT;
    if (!workspace_ok(ws)) return SGB_ERR_INVALID_ARGUMENT;
    st = sgb_block_norm_workspace_bytes(p, R, &need);
    if (st != SGB_OK) return st;
    if (ws_bytes < need) return SGB_ERR_WORKSPACE_TOO_SMALL;
    // outputs against inputs and each other, but for the pairs that may be one
    struct M { const void* p; int64_t s; size_t e; } in[] = {
        {b->dx_out, b->dx_out_stride, er}, {b->dy, b->dy_stride, e},
        {pre ? b->x_out : nullptr, b->x_out_stride, er}, {use_h ? b->h : nullptr, b->h_stride, e}},
        out[] = {{b->dx, b->dx_stride, er}, {b->dh, b->dh_stride, e}};
    for (int o = 0; o < 2; ++o)
      for (int i = 0; i < 4; ++i) {
        const bool same = out[o].p == in[i].p && out[o].s == in[i].s;
        if (same && (o == 0 ? i == 0 : i == 1 || i == 3)) continue;
        if (overlap(out[o].p, D, out[o].s, out[o].e, in[i].p, D, in[i].s, in[i].e, R))
          return SGB_ERR_INVALID_ARGUMENT;
      }
    const int64_t G = b->gate ? div_up(R, b->rows_per_gate) : 0;
    // d_gate is written while other gates' rows are still read
    for (const M& m : in)
      if (overlap(b->d_gate, D, b->d_gate_stride, e, m.p, D, m.s, m.e, G, R))
        return SGB_ERR_INVALID_ARGUMENT;
    // the sums over rows against the other outputs and each other
    const void* sums[] = {b->d_post_weight, b->d_post_bias, b->d_pre_weight, b->d_pre_bias};
    for (const M& m : out)
      if (overlap(b->d_gate, D, b->d_gate_stride, e, m.p, D, m.s, m.e, G, R))
        return SGB_ERR_INVALID_ARGUMENT;
    for (int i = 0; i < 4; ++i) {
      if (overlap(sums[i], D, D, 4, b->d_gate, D, b->d_gate_stride, e, 1, G))
        return SGB_ERR_INVALID_ARGUMENT;
      for (const M& m : out)
        if (overlap(sums[i], D, D, 4, m.p, D, m.s, m.e, 1, R)) return SGB_ERR_INVALID_ARGUMENT;
      for (int j = 0; j < i; ++j)
        if (overlap(sums[i], D, D, 4, sums[j], D, D, 4, 1)) return SGB_ERR_INVALID_ARGUMENT;
    }
    if (overlap(b->dx, D, b->dx_stride, er, b->dh, D, b->dh_stride, e, R) ||
        overlap(b->gate, D, b->gate_stride, e, b->d_gate, D, b->d_gate_stride, e, G) ||
        overlap(b->gate, D, b->gate_stride, e, b->dx, D, b->dx_stride, er, G, R) ||
        overlap(b->gate, D, b->gate_stride, e, b->dh, D, b->dh_stride, e, G, R))
      return SGB_ERR_INVALID_ARGUMENT;
  }
  BwdArgs a{};
  a.p = params_of(p, q);
  a.dxo = b->dx_out;
  a.dy = b->dy;
  a.x = b->x_out;
  a.h = b->h;
  a.gate = b->gate;
  a.stats = b->stats;
  a.dx = b->dx;
  a.dh = b->dh;
  a.dgate = b->d_gate;
  a.sdxo = b->dx_out_stride;
  a.sdy = b->dy_stride;
  a.sx = b->x_out_stride;
  a.sh = b->h_stride;
  a.sg = b->gate_stride;
  a.sdx = b->dx_stride;
  a.sdh = b->dh_stride;
  a.sdg = b->d_gate_stride;
  a.rows = R;
  a.rpg = rpg;
  a.D = D;
  a.tpr = p->tpr;
  a.use_h = use_h;
  bool grouped = false, full = false;
  bool parts = false;  // does a gate's sum come from several teams?
  if (R > 0) {
    const bool gate_bias = q->post_bias && b->d_gate;
    full = b->d_post_bias || b->d_pre_bias || gate_bias || p->post == SGB_NORM_LAYER ||
           p->pre == SGB_NORM_LAYER;
    // Two workgroups share a compute unit only where a lane's values fit in 128
    // registers; else a second would wait for the first to end (3001 rows of
    // 1001 fp16 columns with a gate each: 26.4 us in two rounds, 19.7 in one).
    // 16-bit rms norms fit (two and one: 65536 x 1024 without a gate 153 and 161 us,
    // 32768 x 4096 with a gate each 380 and 419, with one or none 319 and 304), but
    // in teams narrower than a wave with gates they take 134.  fp32 residuals need
    // up to 160; with 16-bit blocks one form, ungrouped teams of waves, takes 127,
    // and two gain nothing there (3001 x 1024: 18.7 us and 16.1 as one; 32768 x 4096:
    // 507 to 510 and 452 to 498).
    a.d = deal_rows(p, R, rpg, b->gate != nullptr, true);
    if (full || er == 4 || (p->tpr < 64 && b->gate && !a.d.split))
      a.d = deal_rows(p, R, rpg, b->gate != nullptr, false);
    const int64_t per_block = max_threads(p) / p->tpr;
    a.blocks = (int)div_up(a.d.teams, per_block);
    a.raw = a.d.split && a.d.groups == 1;
    a.want = ((b->d_post_weight || (a.raw && b->d_gate)) ? 1 : 0) |
             ((b->d_post_bias || (a.raw && gate_bias)) ? 2 : 0) | (b->d_pre_weight ? 4 : 0) |
             (b->d_pre_bias ? 8 : 0);
    parts = a.d.split && !a.raw && b->d_gate;
    if (kHeaderBytes + (size_t)(4 * a.blocks + (parts ? a.d.teams : 0)) * D * sizeof(float) > need)
      return SGB_ERR_INTERNAL;
    a.hdr = static_cast<Header*>(ws);
    a.epoch = next_epoch();
    a.par = reinterpret_cast<float*>(static_cast<char*>(ws) + kHeaderBytes);
    a.slot = parts ? a.par + (int64_t)4 * a.blocks * D : nullptr;
    grouped = !a.d.split && b->gate;
  }
  DeviceGuard guard(p->device);
  if (!guard.ok) return SGB_ERR_HIP;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream_);
  if (R > 0) {
    SGB_LM_NORM_DISPATCH(backward_as, p, a, grouped, full, (unsigned)a.blocks, s);
  }
  if (a.want || parts ||
      (R == 0 && (b->d_post_weight || b->d_post_bias || b->d_pre_weight || b->d_pre_bias))) {
    JoinArgs j{};
    j.par = a.par;
    j.slot = a.slot;
    j.post_w = q->post_weight;
    j.post_b = q->post_bias;
    j.gate = R > 0 ? b->gate : nullptr;
    j.dgate = (a.raw || parts) ? b->d_gate : nullptr;
    j.out[0] = b->d_post_weight;
    j.out[1] = b->d_post_bias;
    j.out[2] = b->d_pre_weight;
    j.out[3] = b->d_pre_bias;
    j.sdg = b->d_gate_stride;
    j.k = a.d.k;
    j.D = D;
    j.blocks = a.blocks;
    j.want = a.want;
    j.raw = a.raw;
    j.pdtype = q->dtype;
    j.dtype = dtype;
    const unsigned ys = 3 + (parts ? (unsigned)a.d.groups : 0u);
    hipLaunchKernelGGL(k_norm_join, dim3((unsigned)div_up(D, 64), ys), dim3(1024), 0, s, j);
  }
  return hipGetLastError() == hipSuccess ? SGB_OK : SGB_ERR_HIP;
}

}  // extern "C"
