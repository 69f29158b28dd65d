// Selective state space scan, token by token: every width, fp32 and bf16, any alignment.
//
//     S <- exp(dt A) S + dt v k^T,   o = S q + D v,   y = o * SiLU(z)
//
// Rows of S (one per value column) never mix. Eight lanes share RV rows: each keeps d_k / 8 columns
// of them in registers for the whole piece of the sequence, two columns per instruction, and the
// eight partial sums of o are joined by shuffles, those of four tokens together. Tokens are staged
// in shared memory 16 at a time as they are, the next tile's copies in flight while one is worked
// on; what bounds it is the arithmetic, three packed operations per two state elements and token,
// and their latency where few blocks run (8 x 792 tokens of 16 heads of 64 x 128 in fp32: 200 us, the
// operations alone 69 us, the bytes 24).
//
// A long prompt of few sequences is cut into pieces: a first pass leaves each piece's own state
// (from zero) and decay, scan_join_kernel turns these into the state before each piece, and the
// second pass computes the outputs from there.
#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kTC = 16;             // tokens per tile
constexpr int kTPR = 8;             // lanes that share a row
constexpr int kScanThreads = 128;
constexpr int kGroups = kScanThreads / kTPR;
constexpr int kTok = 4;             // tokens whose output sums are joined together

// Lane lt of a row holds columns 4 (i kTPR + lt) .. + 3 (pairs 2 i, 2 i + 1), or 2 lt, 2 lt + 1 if
// there are only 16 columns.
template <int SEG>
__device__ __forceinline__ int seg_col(int lt, int pair) {
  return SEG == 2 ? lt * 2 : ((pair >> 1) * kTPR + lt) * 4 + (pair & 1) * 2;
}

template <typename T>
__device__ __forceinline__ void load_pairs4(const T* p, uint64_t& a, uint64_t& b) {
  if constexpr (sizeof(T) == 4) {
    const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(p);
    a = t.x;
    b = t.y;
  } else {
    const uint2 t = *reinterpret_cast<const uint2*>(p);
    a = u2(t.x << 16, t.x & 0xffff0000u);
    b = u2(t.y << 16, t.y & 0xffff0000u);
  }
}

template <typename T, int SEG>
__device__ __forceinline__ void load_seg(const T* row, int lt, uint64_t (&x)[SEG / 2]) {
  if constexpr (SEG == 2) {
    x[0] = f2(to_f32(row[lt * 2]), to_f32(row[lt * 2 + 1]));
  } else {
#pragma unroll
    for (int i = 0; i < SEG / 4; ++i) load_pairs4<T>(row + (i * kTPR + lt) * 4, x[2 * i], x[2 * i + 1]);
  }
}

// Copies `n` rows of `width` elements (source rows `stride` apart) to consecutive rows in shared
// memory: 16-byte asynchronous copies if `wide`, else element by element. Rows n .. kTC - 1 are set
// to zero, so that the arithmetic needs no bound.
template <typename T>
__device__ __forceinline__ void stage(T* dst, const T* src, int64_t stride, int n, int width,
                                      bool wide) {
  constexpr int E = 16 / int(sizeof(T));
  if (wide) {
    const int shift = __ffs(width / E) - 1;        // widths are powers of two
    for (int i = threadIdx.x; i < kTC << shift; i += kScanThreads) {
      const int t = i >> shift, c = (i - (t << shift)) * E;
      if (t < n)
        cp_async16(dst + t * width + c, src + int64_t(t) * stride + c);
      else
        *reinterpret_cast<uint4*>(dst + t * width + c) = make_uint4(0, 0, 0, 0);
    }
  } else {
    const int shift = __ffs(width) - 1;
    for (int i = threadIdx.x; i < kTC << shift; i += kScanThreads) {
      const int t = i >> shift, c = i - (t << shift);
      dst[i] = t < n ? src[int64_t(t) * stride + c] : from_f32<T>(0.f);
    }
  }
}

// FULL: outputs too; otherwise only the piece's own state and decay.
template <typename T, int SEG, int RV, bool FULL>
__global__ void __launch_bounds__(kScanThreads) scan_tok_kernel(ScanArgs a, int wide) {
  constexpr int DK = SEG * kTPR, ROWS = kGroups * RV;
  extern __shared__ __align__(16) unsigned char smem[];
  // two stages of k, q, v, z; then outputs, decays and steps of a tile
  constexpr int kStageElems = kTC * (DK * (FULL ? 2 : 1) + ROWS * (FULL ? 2 : 1));
  T* stages = reinterpret_cast<T*>(smem);
  float* ys = reinterpret_cast<float*>(smem + sizeof(T) * 2 * kStageElems);   // [kTC][ROWS]
  float* as = ys + (FULL ? kTC * ROWS : 0);        // [2][kTC] decay
  float* ds = as + 2 * kTC;                        // [2][kTC] dt
  const int nseg = FULL ? a.nseg : a.nseg - 1;
  const int seg = blockIdx.x % nseg;
  const int rh = blockIdx.x / nseg;
  const int r = rh / a.H, h = rh - r * a.H, g = h / (a.H / a.G);
  const int row0 = blockIdx.y * ROWS, nrow = min(ROWS, a.d_v - row0);
  const int tid = threadIdx.x, lt = tid % kTPR, rg = tid / kTPR;
  const int L = seq_len(a.lens, r, a.P);
  const int64_t p_begin = int64_t(seg) * a.seg_len;
  const int p0 = int(p_begin < L ? p_begin : L);
  const int p1 = int(p_begin + a.seg_len < L ? p_begin + a.seg_len : L);
  const int64_t col = int64_t(h) * a.d_v + row0;
  const T* vp = static_cast<const T*>(a.v) + int64_t(r) * a.v_seq + col;
  const T* kp = static_cast<const T*>(a.k) + int64_t(r) * a.k_seq + int64_t(g) * DK;
  const T* qp = static_cast<const T*>(a.q) + int64_t(r) * a.q_seq + int64_t(g) * DK;
  const T* zp = a.z ? static_cast<const T*>(a.z) + int64_t(r) * a.z_seq + col : nullptr;
  T* yp = static_cast<T*>(a.y) + int64_t(r) * a.y_seq + col;
  const float* dtp = a.dt + int64_t(r) * a.P * a.H + h;
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;

  auto k_of = [&](int b) { return stages + b * kStageElems; };
  auto v_of = [&](int b) { return stages + b * kStageElems + kTC * DK * (FULL ? 2 : 1); };
  auto load_dt = [&](int pt) -> float {            // one tile ahead of its use
    return tid < kTC && pt + tid < p1 ? dtp[int64_t(pt + tid) * a.H] : 0.f;
  };
  float raw = load_dt(p0);
  auto copy_tile = [&](int pt, int b) {
    const int np = min(kTC, p1 - pt);
    stage<T>(k_of(b), kp + int64_t(pt) * a.k_tok, a.k_tok, np, DK, wide);
    stage<T>(v_of(b), vp + int64_t(pt) * a.v_tok, a.v_tok, np, nrow, wide);
    if (FULL) {
      stage<T>(k_of(b) + kTC * DK, qp + int64_t(pt) * a.q_tok, a.q_tok, np, DK, wide);
      if (zp) stage<T>(v_of(b) + kTC * ROWS, zp + int64_t(pt) * a.z_tok, a.z_tok, np, nrow, wide);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (tid < kTC) {
      float dt = raw + bias;
      if (a.softplus) dt = softplus_f(dt);
      raw = load_dt(pt + kTC);
      // rows behind the end add nothing and decay nothing (0 * A is NaN for an infinite A)
      ds[b * kTC + tid] = tid < np ? dt : 0.f;
      as[b * kTC + tid] = tid < np ? expf(dt * A) : 1.f;
    }
  };
  double logsum = 0.0;                             // sum of dt A over the piece
  if (p0 < p1) copy_tile(p0, 0);
  const float* entering = nullptr;
  if (FULL && a.nseg > 1) wait_for_previous_kernel();
  if (!FULL) let_next_kernel_start();
  if (FULL)
    entering = a.nseg > 1 ? a.seg_S + (int64_t(rh) * a.nseg + seg) * a.d_v * DK
                          : (a.S_in ? a.S_in + int64_t(rh) * a.d_v * DK : nullptr);
  uint64_t S[RV][SEG / 2];
#pragma unroll
  for (int j = 0; j < RV; ++j) {
    const int row = rg * RV + j;
#pragma unroll
    for (int i = 0; i < SEG / 2; ++i) {
      const float* e = entering + int64_t(row0 + row) * DK + seg_col<SEG>(lt, i);
      S[j][i] = entering && row < nrow ? f2(e[0], e[1]) : f2(0.f, 0.f);
    }
  }
  int b = 0;
  for (int pt = p0; pt < p1; pt += kTC, b ^= 1) {
    const int np = min(kTC, p1 - pt);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                               // this tile is in; the other buffer was read
    if (pt + kTC < p1) copy_tile(pt + kTC, b ^ 1);
    const T* ks = k_of(b);
    const T* qs = ks + kTC * DK;
    const T* vs = v_of(b);
    const float* al = as + b * kTC;
    const float* dts = ds + b * kTC;
    if (!FULL && tid == 0)
      for (int t = 0; t < np; ++t) logsum += double(dts[t]);
#pragma unroll 1
    for (int t0 = 0; t0 < np; t0 += kTok) {
      float o[RV][kTok];
#pragma unroll
      for (int u = 0; u < kTok; ++u) {
        const int t = t0 + u;
#pragma unroll
        for (int j = 0; j < RV; ++j) o[j][u] = 0.f;
        uint64_t kk[SEG / 2], qq[FULL ? SEG / 2 : 1];
        load_seg<T, SEG>(ks + t * DK, lt, kk);
        if constexpr (FULL) load_seg<T, SEG>(qs + t * DK, lt, qq);
        const float dt = dts[t];
        const uint64_t a2 = f2(al[t], al[t]);
#pragma unroll
        for (int j = 0; j < RV; ++j) {
          const int row = rg * RV + j;
          const float w = row < nrow ? dt * to_f32(vs[t * nrow + row]) : 0.f;
          const uint64_t w2 = f2(w, w);
          uint64_t acc = f2(0.f, 0.f);
#pragma unroll
          for (int i = 0; i < SEG / 2; ++i) {
            S[j][i] = fma2(a2, S[j][i], mul2(w2, kk[i]));
            if constexpr (FULL) acc = fma2(S[j][i], qq[i], acc);
          }
          if (FULL) {
            const float2 h2 = un2(acc);
            o[j][u] = h2.x + h2.y;
          }
        }
      }
      if (FULL) {
        // sums over the eight lanes: lanes with bit 2 set take tokens 2, 3, with bit 1 the odd ones
#pragma unroll
        for (int j = 0; j < RV; ++j) {
          const bool up = lt & 4, odd = lt & 2;
          float s0 = up ? o[j][0] : o[j][2], s1 = up ? o[j][1] : o[j][3];
          float m0 = up ? o[j][2] : o[j][0], m1 = up ? o[j][3] : o[j][1];
          m0 += __shfl_xor_sync(kFull, s0, 4);
          m1 += __shfl_xor_sync(kFull, s1, 4);
          float m = odd ? m1 : m0;
          m += __shfl_xor_sync(kFull, odd ? m0 : m1, 2);
          m += __shfl_xor_sync(kFull, m, 1);
          const int t = t0 + (up ? 2 : 0) + (odd ? 1 : 0);
          if ((lt & 1) == 0 && t < np) ys[t * ROWS + rg * RV + j] = m;
        }
      }
    }
    if (FULL) {
      __syncthreads();
      const T* zs = vs + kTC * ROWS;
      auto value = [&](int t, int c) -> float {
        float o = ys[t * ROWS + c];
        if (a.D) o = fmaf(D, to_f32(vs[t * nrow + c]), o);
        if (zp) o *= silu_f<T>(to_f32(zs[t * nrow + c]));
        return o;
      };
      if (wide) {
        const int per = nrow / 4;                  // rows are 16-byte aligned: four values at a time
        for (int i = tid; i < np * per; i += kScanThreads) {
          const int t = i / per, c = (i - t * per) * 4;
          float f[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) f[e] = value(t, c + e);
          Pack<T, 4> o;
          o.pack(f);
          o.store(yp + int64_t(pt + t) * a.y_tok + c);
        }
      } else {
        for (int i = tid; i < np * nrow; i += kScanThreads) {
          const int t = i / nrow, c = i - t * nrow;
          yp[int64_t(pt + t) * a.y_tok + c] = from_f32<T>(value(t, c));
        }
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
      const int row = rg * RV + j;
      if (row >= nrow) continue;
#pragma unroll
      for (int i = 0; i < SEG / 2; ++i) {
        float* e = out + int64_t(row0 + row) * DK + seg_col<SEG>(lt, i);
        const float2 x = un2(S[j][i]);
        e[0] = x.x;
        e[1] = x.y;
      }
    }
  }
  if (!FULL && tid == 0 && blockIdx.y == 0)
    a.seg_a[int64_t(rh) * a.nseg + seg] = p0 < p1 ? float(exp(logsum * double(A))) : 1.f;
}

// The state before each piece from the pieces' own states: e_0 = S_in, e_(s+1) = a_s e_s + S_s.
__global__ void __launch_bounds__(256) scan_join_kernel(ScanArgs a) {
  const int64_t n4 = int64_t(a.d_v) * a.d_k / 4;
  const int64_t at = int64_t(blockIdx.x) * 256 + threadIdx.x;
  let_next_kernel_start();
  wait_for_previous_kernel();
  if (at >= n4 * a.R * a.H) return;
  const int64_t rh = at / n4, e4 = at - rh * n4;
  float4 e = make_float4(0.f, 0.f, 0.f, 0.f);
  if (a.S_in) {
    const float* p = a.S_in + (rh * n4 + e4) * 4;  // any 4-byte alignment
    e = make_float4(p[0], p[1], p[2], p[3]);
  }
  float4* s = reinterpret_cast<float4*>(a.seg_S) + rh * a.nseg * n4 + e4;
  const float* al = a.seg_a + rh * a.nseg;
  constexpr int kAhead = 8;                        // pieces loaded together
  for (int i0 = 0; i0 < a.nseg; i0 += kAhead) {
    float4 own[kAhead];
    float d[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i + 1 < a.nseg) {
        own[i] = s[i * n4];
        d[i] = al[i0 + i];
      }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= a.nseg) break;
      s[i * n4] = e;
      if (i0 + i + 1 == a.nseg) break;
      e.x = fmaf(d[i], e.x, own[i].x);
      e.y = fmaf(d[i], e.y, own[i].y);
      e.z = fmaf(d[i], e.z, own[i].z);
      e.w = fmaf(d[i], e.w, own[i].w);
    }
    s += kAhead * n4;
  }
}

template <typename T, int SEG, int RV>
cudaError_t run(const ScanArgs& a, int wide, cudaStream_t st) {
  constexpr int DK = SEG * kTPR, ROWS = kGroups * RV;
  const dim3 grid(unsigned(a.R * a.H * a.nseg), unsigned((a.d_v + ROWS - 1) / ROWS));
  constexpr size_t full =
      sizeof(T) * 4 * kTC * (DK + ROWS) + sizeof(float) * (kTC * ROWS + 4 * kTC);
  constexpr size_t own = sizeof(T) * 2 * kTC * (DK + ROWS) + sizeof(float) * 4 * kTC;
  static_assert(full <= 100 * 1024, "shared memory");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = once_per_device(done, [&] {
    cudaError_t x = cudaFuncSetAttribute(scan_tok_kernel<T, SEG, RV, true>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, full);
    return x != cudaSuccess
               ? x
               : cudaFuncSetAttribute(scan_tok_kernel<T, SEG, RV, false>,
                                      cudaFuncAttributeMaxDynamicSharedMemorySize, own);
  });
  if (e != cudaSuccess) return e;
  if (a.nseg > 1) {
    const dim3 g1(unsigned(a.R * a.H * (a.nseg - 1)), grid.y);
    scan_tok_kernel<T, SEG, RV, false><<<g1, kScanThreads, own, st>>>(a, wide);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_scan_join(a, st)) != cudaSuccess) return e;
  }
  // the outputs of a piece can start before its entering state is there
  if (a.nseg > 1)
    return launch_dependent(scan_tok_kernel<T, SEG, RV, true>, grid, kScanThreads, full, st, a,
                            wide);
  scan_tok_kernel<T, SEG, RV, true><<<grid, kScanThreads, full, st>>>(a, wide);
  return cudaGetLastError();
}

// Rows per block: 64, or what d_v needs; 32 where d_k = 256 would take too many registers. (32 rows
// where blocks of 64 leave fewer than four per SM measured 5 % slower: the loads of keys and queries
// are shared by half the rows.)
template <typename T, int SEG>
cudaError_t by_rows(const ScanArgs& a, int wide, cudaStream_t st) {
  if (a.d_v <= 16) return run<T, SEG, 1>(a, wide, st);
  if (a.d_v <= 32 || SEG == 32) return run<T, SEG, 2>(a, wide, st);
  if constexpr (SEG < 32) return run<T, SEG, 4>(a, wide, st);
  return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t by_width(const ScanArgs& a, int wide, cudaStream_t st) {
  switch (a.d_k) {
    case 16: return by_rows<T, 2>(a, wide, st);
    case 32: return by_rows<T, 4>(a, wide, st);
    case 64: return by_rows<T, 8>(a, wide, st);
    case 128: return by_rows<T, 16>(a, wide, st);
    default: return by_rows<T, 32>(a, wide, st);
  }
}

}  // namespace

cudaError_t launch_scan_join(const ScanArgs& a, cudaStream_t st) {
  const int64_t n = int64_t(a.R) * a.H * a.d_v * a.d_k / 4;
  return launch_dependent(scan_join_kernel, unsigned((n + 255) / 256), 256, 0, st, a);
}

// Pieces: while the sequences alone leave most of the machine idle (fewer than 4 blocks per SM),
// as many as fill it, of at least 16 tokens each (777 tokens of 18 chains of 64 x 32: 21.6 us, with
// at least 32 tokens 24.4 us, 64 tokens 29.0 us).
void scan_tok_pieces(int R, int P, int H, int d_v, int sms, int* nseg, int* seg_len) {
  const int64_t chains = int64_t(R) * H * ((d_v + 63) / 64);
  int64_t want = int64_t(4) * sms / chains;
  if (want > P / 16) want = P / 16;
  if (want < 4) want = 1;             // the first run costs two thirds of the second
  int64_t len = (int64_t(P) + want - 1) / want;
  len = (len + kTC - 1) / kTC * kTC;
  if (len < kTC) len = kTC;
  *seg_len = int(len);
  *nseg = int((int64_t(P) + len - 1) / len);
  if (*nseg < 1) *nseg = 1;
}

cudaError_t launch_scan_tok(const ScanArgs& a, int in_dtype, cudaStream_t st) {
  const int e = in_dtype == OLA_BF16 ? 2 : 4;
  auto on16 = [&](const void* p, int64_t tok, int64_t seq) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (tok * e) % 16 == 0 && (seq * e) % 16 == 0;
  };
  const int wide = on16(a.v, a.v_tok, a.v_seq) && on16(a.k, a.k_tok, a.k_seq) &&
                   on16(a.q, a.q_tok, a.q_seq) && on16(a.y, a.y_tok, a.y_seq) &&
                   (!a.z || on16(a.z, a.z_tok, a.z_seq));
  return in_dtype == OLA_BF16 ? by_width<__nv_bfloat16>(a, wide, st)
                              : by_width<float>(a, wide, st);
}

}  // namespace ola
