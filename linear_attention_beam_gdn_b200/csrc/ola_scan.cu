// Selective state space scan, token by token: every width, fp32 and bf16, any alignment.
//
//     S <- exp(dt A) S + dt v k^T,   o = S q + D v,   y = o * SiLU(z)
//
// Rows of S (one per value column) never mix. Eight lanes share RV rows: each keeps d_k / 8 columns
// of them in registers for the whole piece of the sequence and the eight partial sums of o are
// joined by shuffles. Tokens are staged in shared memory 32 at a time as fp32.
//
// A long prompt of few sequences is cut into pieces: a first pass leaves each piece's own state
// (from zero) and decay, scan_join_kernel turns these into the state before each piece, and the
// second pass computes the outputs from there.
#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kTC = 32;             // tokens per tile
constexpr int kTPR = 8;             // lanes that share a row
constexpr int kScanThreads = 128;

template <int SEG>
__device__ __forceinline__ int seg_col(int lt, int i) {   // column of register i of lane lt
  return SEG == 2 ? lt * 2 + i : ((i >> 2) * kTPR + lt) * 4 + (i & 3);
}

template <int SEG>
__device__ __forceinline__ void load_seg(const float* row, int lt, float (&x)[SEG]) {
  if constexpr (SEG == 2) {
    const float2 t = *reinterpret_cast<const float2*>(row + lt * 2);
    x[0] = t.x;
    x[1] = t.y;
  } else {
#pragma unroll
    for (int i = 0; i < SEG / 4; ++i) {
      const float4 t = *reinterpret_cast<const float4*>(row + (i * kTPR + lt) * 4);
      x[4 * i] = t.x;
      x[4 * i + 1] = t.y;
      x[4 * i + 2] = t.z;
      x[4 * i + 3] = t.w;
    }
  }
}

// FULL: outputs too; otherwise only the piece's own state and decay.
template <typename T, int SEG, int RV, bool FULL>
__global__ void __launch_bounds__(kScanThreads) scan_tok_kernel(ScanArgs a) {
  constexpr int DK = SEG * kTPR;
  extern __shared__ __align__(16) float sm[];
  const int rows = (blockDim.x / kTPR) * RV;       // rows of this block
  float* ks = sm;                                  // [kTC][DK]
  float* qs = ks + kTC * DK;                       // [kTC][DK]
  float* vs = qs + (FULL ? kTC * DK : 0);          // [kTC][rows], times dt
  float* ys = vs + kTC * rows;                     // [kTC][rows]
  float* as = ys + (FULL ? kTC * rows : 0);        // [kTC] decay
  float* ds = as + kTC;                            // [kTC] dt
  const int nseg = FULL ? a.nseg : a.nseg - 1;
  const int seg = blockIdx.x % nseg;
  const int rh = blockIdx.x / nseg;
  const int r = rh / a.H, h = rh - r * a.H, g = h / (a.H / a.G);
  const int row0 = blockIdx.y * rows;
  const int tid = threadIdx.x, lt = tid % kTPR, rg = tid / kTPR;
  const int L = seq_len(a.lens, r, a.P);
  const int64_t p_begin = int64_t(seg) * a.seg_len;
  const int p0 = int(p_begin < L ? p_begin : L);
  const int p1 = int(p_begin + a.seg_len < L ? p_begin + a.seg_len : L);
  const T* vp = static_cast<const T*>(a.v) + int64_t(r) * a.v_seq + int64_t(h) * a.d_v;
  const T* kp = static_cast<const T*>(a.k) + int64_t(r) * a.k_seq + int64_t(g) * DK;
  const T* qp = static_cast<const T*>(a.q) + int64_t(r) * a.q_seq + int64_t(g) * DK;
  const float* dtp = a.dt + int64_t(r) * a.P * a.H + h;
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;

  const float* entering = nullptr;
  if (FULL)
    entering = a.nseg > 1 ? a.seg_S + (int64_t(rh) * a.nseg + seg) * a.d_v * DK
                          : (a.S_in ? a.S_in + int64_t(rh) * a.d_v * DK : nullptr);
  float S[RV][SEG];
#pragma unroll
  for (int j = 0; j < RV; ++j) {
    const int row = row0 + rg * RV + j;
#pragma unroll
    for (int i = 0; i < SEG; ++i)
      S[j][i] = entering && row < a.d_v ? entering[int64_t(row) * DK + seg_col<SEG>(lt, i)] : 0.f;
  }
  double logsum = 0.0;                             // thread 0: sum of dt A over the piece
  for (int pt = p0; pt < p1; pt += kTC) {
    const int np = min(kTC, p1 - pt);
    __syncthreads();
    if (tid < np) {
      float dt = dtp[int64_t(pt + tid) * a.H] + bias;
      if (a.softplus) dt = softplus_f(dt);
      ds[tid] = dt;
      as[tid] = expf(dt * A);
    }
    for (int i = tid; i < np * DK; i += blockDim.x) {
      const int t = i / DK, c = i % DK;
      ks[i] = to_f32(kp[int64_t(pt + t) * a.k_tok + c]);
      if (FULL) qs[i] = to_f32(qp[int64_t(pt + t) * a.q_tok + c]);
    }
    __syncthreads();
    for (int i = tid; i < np * rows; i += blockDim.x) {
      const int t = i / rows, c = row0 + i % rows;
      vs[i] = c < a.d_v ? ds[t] * to_f32(vp[int64_t(pt + t) * a.v_tok + c]) : 0.f;
    }
    if (!FULL && tid == 0)
      for (int t = 0; t < np; ++t) logsum += double(ds[t]) * double(A);
    __syncthreads();
    for (int t = 0; t < np; ++t) {
      float kk[SEG];
      load_seg<SEG>(ks + t * DK, lt, kk);
      const float al = as[t];
      const float* vrow = vs + t * rows + rg * RV;
      float o[RV];
      if (FULL) {
        float qq[SEG];
        load_seg<SEG>(qs + t * DK, lt, qq);
#pragma unroll
        for (int j = 0; j < RV; ++j) {
          const float w = vrow[j];
          o[j] = 0.f;
#pragma unroll
          for (int i = 0; i < SEG; ++i) {
            S[j][i] = fmaf(al, S[j][i], w * kk[i]);
            o[j] = fmaf(S[j][i], qq[i], o[j]);
          }
        }
#pragma unroll
        for (int j = 0; j < RV; ++j) {
          o[j] += __shfl_xor_sync(kFull, o[j], 1);
          o[j] += __shfl_xor_sync(kFull, o[j], 2);
          o[j] += __shfl_xor_sync(kFull, o[j], 4);
          if (lt == j) ys[t * rows + rg * RV + j] = o[j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < RV; ++j) {
          const float w = vrow[j];
#pragma unroll
          for (int i = 0; i < SEG; ++i) S[j][i] = fmaf(al, S[j][i], w * kk[i]);
        }
      }
    }
    if (FULL) {
      __syncthreads();
      for (int i = tid; i < np * rows; i += blockDim.x) {
        const int t = i / rows, c = row0 + i % rows;
        if (c >= a.d_v) continue;
        float o = ys[i];
        if (a.D) o = fmaf(D, to_f32(vp[int64_t(pt + t) * a.v_tok + c]), o);
        if (a.z)
          o *= silu_f<T>(to_f32(static_cast<const T*>(
              a.z)[int64_t(r) * a.z_seq + int64_t(pt + t) * a.z_tok + int64_t(h) * a.d_v + c]));
        static_cast<T*>(a.y)[int64_t(r) * a.y_seq + int64_t(pt + t) * a.y_tok +
                             int64_t(h) * a.d_v + c] = from_f32<T>(o);
      }
    }
  }
  float* out = nullptr;
  if (!FULL)
    out = a.seg_S + (int64_t(rh) * a.nseg + seg) * a.d_v * DK;
  else if (seg == nseg - 1 && a.S_out)
    out = a.S_out + int64_t(rh) * a.d_v * DK;
  if (out) {
#pragma unroll
    for (int j = 0; j < RV; ++j) {
      const int row = row0 + rg * RV + j;
      if (row >= a.d_v) continue;
#pragma unroll
      for (int i = 0; i < SEG; ++i) out[int64_t(row) * DK + seg_col<SEG>(lt, i)] = S[j][i];
    }
  }
  if (!FULL && tid == 0 && blockIdx.y == 0)
    a.seg_a[int64_t(rh) * a.nseg + seg] = float(exp(logsum));
}

// The state before each piece from the pieces' own states: e_0 = S_in, e_(s+1) = a_s e_s + S_s.
__global__ void __launch_bounds__(256) scan_join_kernel(ScanArgs a) {
  const int64_t n4 = int64_t(a.d_v) * a.d_k / 4;
  const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (at >= n4 * a.R * a.H) return;
  const int64_t rh = at / n4, e4 = at - rh * n4;
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.S_in) {
    const float* p = a.S_in + (rh * n4 + e4) * 4;  // any 4-byte alignment
    e = make_float4(p[0], p[1], p[2], p[3]);
  }
  float4* s = reinterpret_cast<float4*>(a.seg_S) + rh * a.nseg * n4 + e4;
  for (int i = 0; i < a.nseg; ++i, s += n4) {
    if (i + 1 == a.nseg) {
      *s = e;
      break;
    }
    const float4 own = *s;
    const float al = a.seg_a[rh * a.nseg + i];
    *s = e;
    e.x = fmaf(al, e.x, own.x);
    e.y = fmaf(al, e.y, own.y);
    e.z = fmaf(al, e.z, own.z);
    e.w = fmaf(al, e.w, own.w);
  }
}

template <typename T, int SEG, int RV>
cudaError_t run(const ScanArgs& a, cudaStream_t st) {
  constexpr int DK = SEG * kTPR;
  int threads = kTPR * ((a.d_v + RV - 1) / RV);
  threads = threads > kScanThreads ? kScanThreads : (threads + 31) / 32 * 32;
  const int rows = threads / kTPR * RV;
  const dim3 grid(unsigned(a.R * a.H * a.nseg), unsigned((a.d_v + rows - 1) / rows));
  const size_t full = sizeof(float) * (2 * kTC * DK + 2 * kTC * rows + 2 * kTC);
  const size_t own = sizeof(float) * (kTC * DK + kTC * rows + 2 * kTC);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [&] {
    cudaError_t x = cudaFuncSetAttribute(scan_tok_kernel<T, SEG, RV, true>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
    return x != cudaSuccess
               ? x
               : cudaFuncSetAttribute(scan_tok_kernel<T, SEG, RV, false>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, 100 * 1024);
  });
  if (e != cudaSuccess) return e;
  if (a.nseg > 1) {
    const dim3 g1(unsigned(a.R * a.H * (a.nseg - 1)), grid.y);
    scan_tok_kernel<T, SEG, RV, false><<<g1, threads, own, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_scan_join(a, st)) != cudaSuccess) return e;
  }
  scan_tok_kernel<T, SEG, RV, true><<<grid, threads, full, st>>>(a);
  return cudaGetLastError();
}

template <typename T>
cudaError_t by_width(const ScanArgs& a, cudaStream_t st) {
  switch (a.d_k) {
    case 16: return run<T, 2, 4>(a, st);
    case 32: return run<T, 4, 4>(a, st);
    case 64: return run<T, 8, 4>(a, st);
    case 128: return run<T, 16, 4>(a, st);
    default: return run<T, 32, 2>(a, st);
  }
}

}  // namespace

cudaError_t launch_scan_join(const ScanArgs& a, cudaStream_t st) {
  const int64_t n = int64_t(a.R) * a.H * a.d_v * a.d_k / 4;
  scan_join_kernel<<<unsigned((n + 255) / 256), 256, 0, st>>>(a);
  return cudaGetLastError();
}

// Pieces: while the sequences alone leave most of the machine idle (fewer than 4 blocks per SM),
// as many as fill it, of at least 64 tokens each.
void scan_tok_pieces(int R, int P, int H, int d_k, int d_v, int sms, int* nseg, int* seg_len) {
  const int64_t chains = int64_t(R) * H * ((d_v + 63) / 64);
  int64_t want = int64_t(4) * sms / chains;
  if (want > P / 64) want = P / 64;
  if (want < 2) want = 1;
  int64_t len = (int64_t(P) + want - 1) / want;
  len = (len + kTC - 1) / kTC * kTC;
  if (len < kTC) len = kTC;
  *seg_len = int(len);
  *nseg = int((int64_t(P) + len - 1) / len);
  if (*nseg < 1) *nseg = 1;
  (void)d_k;
}

cudaError_t launch_scan_tok(const ScanArgs& a, int in_dtype, cudaStream_t st) {
  return in_dtype == OLA_BF16 ? by_width<__nv_bfloat16>(a, st) : by_width<float>(a, st);
}

}  // namespace ola
