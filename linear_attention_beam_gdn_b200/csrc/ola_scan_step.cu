// One token of the selective state space scan for every beam.
//
//     S_b = exp(dt A) S_parent + dt v k^T,   o = S_b q + D v,   y = o * SiLU(z)
//
// Five operations per state element against 4 bytes read and 4 written: the bound is HBM, and the
// states are all of it. TPR lanes hold one row of the state as float4; a warp keeps kU rows per
// lane group in flight, and joins their kU output sums in one folding reduction. New states are
// written with streaming stores, which leave L2 to the parents that several beams share: 512 beams
// of 16 heads of 128 x 128 in 145 us (148 without; 89 % of the copy rate over the parents that are
// read). Heads go fastest over the grid: beams fastest took 167 us.
#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kStepThreads = 128;
constexpr int kU = 8;               // rows in flight per lane group

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p) {
  return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
}

// Sums v[0..7] over groups of TPR lanes; the lane keeps the sum of row fold_row(lane).
template <int TPR>
__device__ __forceinline__ float fold8(float (&v)[8], int lt) {
  static_assert(TPR >= 8, "one lane per row at least");
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int off = TPR >> (s + 1), n = 4 >> s;
    const bool up = lt & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = up ? v[i] : v[i + n];
      const float got = __shfl_xor_sync(kFull, send, off);
      v[i] = (up ? v[i + n] : v[i]) + got;
    }
  }
  float x = v[0];
#pragma unroll
  for (int off = TPR / 16; off > 0; off >>= 1) x += __shfl_xor_sync(kFull, x, off);
  return x;
}

template <typename T, int DK>
__global__ void __launch_bounds__(kStepThreads) scan_step_kernel(ScanArgs a) {
  constexpr int TPR = DK / 4 < 32 ? DK / 4 : 32;   // lanes per row
  constexpr int VPT = DK / (4 * TPR);              // float4 per lane and row
  constexpr int RPP = 32 / TPR;                    // rows a warp holds per register set
  constexpr int ROWS = RPP * kU;                   // rows per warp
  const int lane = threadIdx.x & 31, lt = lane % TPR, sub = lane / TPR;
  const int nrow = (a.d_v + ROWS - 1) / ROWS;
  const int64_t warp = (int64_t(blockIdx.x) * kStepThreads + threadIdx.x) >> 5;
  const int64_t i = warp / nrow;                   // (r, b, h), h fastest
  const int row0 = int(warp - i * nrow) * ROWS;
  if (i >= int64_t(a.R) * a.P * a.H) return;       // whole warps
  const int h = int(i % a.H);
  const int64_t rb = i / a.H;
  const int r = int(rb / a.P), b = int(rb - int64_t(r) * a.P);
  const int g = h / (a.H / a.G);
  const int p = parent_state(a.parent, r, b, a.P, a.Bp, a.err);
  const float* src = a.S_in + ((int64_t(r) * a.Bp + p) * a.H + h) * a.d_v * DK;
  float* dst = a.S_out + i * a.d_v * DK;

  float4 S[kU][VPT];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int row = row0 + u * RPP + sub;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
      S[u][j] = row < a.d_v ? *reinterpret_cast<const float4*>(src + int64_t(row) * DK +
                                                               (j * TPR + lt) * 4)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const T* kp = static_cast<const T*>(a.k) + int64_t(r) * a.k_seq + int64_t(b) * a.k_tok +
                int64_t(g) * DK;
  const T* qp = static_cast<const T*>(a.q) + int64_t(r) * a.q_seq + int64_t(b) * a.q_tok +
                int64_t(g) * DK;
  const T* vp = static_cast<const T*>(a.v) + int64_t(r) * a.v_seq + int64_t(b) * a.v_tok +
                int64_t(h) * a.d_v;
  float4 kk[VPT], qq[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    kk[j] = ld4<T>(kp + (j * TPR + lt) * 4);
    qq[j] = ld4<T>(qp + (j * TPR + lt) * 4);
  }
  float dt = a.dt[i] + (a.dt_bias ? a.dt_bias[h] : 0.f);
  if (a.softplus) dt = softplus_f(dt);
  const float al = expf(dt * a.A[h]);
  float o[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int row = row0 + u * RPP + sub;
    const float w = row < a.d_v ? dt * to_f32(vp[row]) : 0.f;
    o[u] = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float4& s = S[u][j];
      s.x = fmaf(al, s.x, w * kk[j].x);
      s.y = fmaf(al, s.y, w * kk[j].y);
      s.z = fmaf(al, s.z, w * kk[j].z);
      s.w = fmaf(al, s.w, w * kk[j].w);
      o[u] = fmaf(s.x, qq[j].x, fmaf(s.y, qq[j].y, fmaf(s.z, qq[j].z, fmaf(s.w, qq[j].w, o[u]))));
      if (row < a.d_v)
        __stcs(reinterpret_cast<float4*>(dst + int64_t(row) * DK + (j * TPR + lt) * 4), s);
    }
  }
  auto finish = [&](int u, float x) {
    const int row = row0 + u * RPP + sub;
    if (row >= a.d_v) return;
    if (a.D) x = fmaf(a.D[h], to_f32(vp[row]), x);
    if (a.z)
      x *= silu_f<T>(to_f32(static_cast<const T*>(a.z)[int64_t(r) * a.z_seq + int64_t(b) * a.z_tok +
                                                       int64_t(h) * a.d_v + row]));
    static_cast<T*>(a.y)[int64_t(r) * a.y_seq + int64_t(b) * a.y_tok + int64_t(h) * a.d_v + row] =
        from_f32<T>(x);
  };
  if constexpr (TPR >= 8) {
    const float x = fold8<TPR>(o, lt);
    const int u = (lt & (TPR / 2) ? 4 : 0) + (lt & (TPR / 4) ? 2 : 0) + (lt & (TPR / 8) ? 1 : 0);
    if ((lt & (TPR / 8 - 1)) == 0) finish(u, x);
  } else {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const float x = group_sum(o[u], TPR);
      if (lt == (u % TPR)) finish(u, x);
    }
  }
}

template <typename T, int DK>
cudaError_t run(const ScanArgs& a, cudaStream_t st) {
  constexpr int TPR = DK / 4 < 32 ? DK / 4 : 32;
  constexpr int ROWS = 32 / TPR * kU;
  const int64_t warps = int64_t(a.R) * a.P * a.H * ((a.d_v + ROWS - 1) / ROWS);
  const int64_t grid = (warps * 32 + kStepThreads - 1) / kStepThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  scan_step_kernel<T, DK><<<unsigned(grid), kStepThreads, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_width(const ScanArgs& a, cudaStream_t st) {
  switch (a.d_k) {
    case 16: return run<T, 16>(a, st);
    case 32: return run<T, 32>(a, st);
    case 64: return run<T, 64>(a, st);
    case 128: return run<T, 128>(a, st);
    default: return run<T, 256>(a, st);
  }
}

}  // namespace

cudaError_t launch_scan_step(const ScanArgs& a, int in_dtype, cudaStream_t st) {
  return in_dtype == OLA_BF16 ? by_width<__nv_bfloat16>(a, st) : by_width<float>(a, st);
}

}  // namespace ola
