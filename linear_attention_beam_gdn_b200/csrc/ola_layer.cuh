// Shared by the operators around the recurrence (convolution, query/key norm, scan): argument
// blocks, the sticky error word's first-error rule, wide loads and the activation functions.
#pragma once

#include "ola_device.cuh"

namespace ola {

struct ConvArgs {
  int R, P, C, Bp;
  int silu, tt;                   // tt: tokens per thread
  int n_ctile, n_ttile;           // blocks along the channels, along the tokens
  int64_t x_tok, x_seq, y_tok, y_seq;
  const void* x;
  const float* w;                 // [C][W]
  const float* bias;              // [C] or null
  const void* state_in;
  const int* lens;
  const int* parent;
  void* y;
  void* state_out;
  int* err;
};

struct QkArgs {
  int64_t N;
  int Hq, Hk, d, rot, l2, hsplit;   // hsplit: warps that share one token's heads
  float eps;
  int64_t q_tok, k_tok, qo_tok, ko_tok;
  const void* q;
  const void* k;
  const float* wq;
  const float* wk;
  const int* pos;
  const float* inv_freq;
  void* q_out;
  void* k_out;
};

struct ScanArgs {
  int R, P, H, G, d_k, d_v, Bp;
  int softplus;
  int nseg, seg_len;              // pieces of a sequence, tokens in each (a multiple of the tile)
  int64_t v_tok, v_seq, k_tok, k_seq, q_tok, q_seq, z_tok, z_seq, y_tok, y_seq;
  const void* v;
  const float* dt;
  const float* A;
  const void* k;
  const void* q;
  const float* D;
  const float* dt_bias;
  const void* z;
  const float* S_in;
  const int* lens;
  const int* parent;
  void* y;
  float* S_out;
  float* seg_S;                   // [R][H][nseg][d_v][d_k]: a piece's own state, then the one before it
  float* seg_a;                   // [R][H][nseg] a piece's decay
  int* err;
};

// Programmatic dependent launch: a kernel launched with launch_dependent may start while the one
// before it on the stream still runs, and waits for its results only where it reads them.
__device__ __forceinline__ void wait_for_previous_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_kernel_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... Args, typename... Given>
cudaError_t launch_dependent(void (*kernel)(Args...), dim3 grid, dim3 block, size_t smem,
                             cudaStream_t st, const Given&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, Args(args)...);
}

// Tokens of sequence r.
__device__ __forceinline__ int seq_len(const int* lens, int r, int P) {
  return lens ? min(max(__ldg(lens + r), 0), P) : P;
}

// The parent state of beam b of request r among Bp.
__device__ __forceinline__ int parent_state(const int* parent, int r, int b, int B, int Bp,
                                            int* err) {
  if (!parent) return Bp == 1 ? 0 : b;
  int p = __ldg(parent + size_t(r) * B + b);
  if (p < 0 || p >= Bp) {
    report_error(err, OLA_ERR_BAD_PARENT, p, b);
    p = 0;
  }
  return p;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 at a time (fma.rn.f32x2): half the instructions of the scalar forms.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint64_t u2(uint32_t a, uint32_t b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 un2(uint64_t a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// u / (1 + e^-u). The bf16 form uses the approximate exponential and reciprocal (a few units of
// 2^-22, far below bf16's 2^-8; a denominator past 2^126 gives 0, the limit it has).
template <typename T>
__device__ __forceinline__ float silu_f(float u);
template <>
__device__ __forceinline__ float silu_f<float>(float u) {
  // the approximate reciprocal and one Newton step (within two units of 2^-23); the exponent's
  // limit keeps the denominator finite (SiLU below -88 is 0 to within 2^-118)
  const float d = 1.f + expf(fminf(-u, 88.f));
  const float r = rcp(d);
  return u * fmaf(r, fmaf(-d, r, 1.f), r);
}
template <>
__device__ __forceinline__ float silu_f<__nv_bfloat16>(float u) {
  return u * rcp(1.f + ex2(u * -1.4426950408889634f));
}
template <typename T>
__device__ __forceinline__ uint64_t silu2(uint64_t u) {
  const float2 x = un2(u);
  if constexpr (sizeof(T) == 4) {
    return f2(silu_f<float>(x.x), silu_f<float>(x.y));
  } else {
    const float2 e = un2(mul2(u, f2(-1.4426950408889634f, -1.4426950408889634f)));
    const float2 d = un2(add2(f2(ex2(e.x), ex2(e.y)), f2(1.f, 1.f)));
    return mul2(u, f2(rcp(d.x), rcp(d.y)));
  }
}

__device__ __forceinline__ float softplus_f(float x) { return x > 20.f ? x : log1pf(expf(x)); }

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) {
  return x;
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// VEC consecutive elements as they lie in memory: one 16- or 8-byte word or one element (VEC = 1).
template <typename T, int VEC>
struct Pack {
  uint4 raw;
  __device__ __forceinline__ void zero() { raw = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<uint4*>(p) = raw; }
  __device__ __forceinline__ void unpack(float (&f)[VEC]) const {
    const uint32_t wd[4] = {raw.x, raw.y, raw.z, raw.w};
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(wd[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(wd[i] << 16);
        f[2 * i + 1] = __uint_as_float(wd[i] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void pack(const float (&f)[VEC]) {
    if constexpr (sizeof(T) == 4) {
      raw = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                       __float_as_uint(f[3]));
    } else {
      uint32_t wd[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
        wd[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
      raw = make_uint4(wd[0], wd[1], wd[2], wd[3]);
    }
  }
};

template <>
struct Pack<__nv_bfloat16, 4> {
  uint2 raw;
  __device__ __forceinline__ void zero() { raw = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    raw = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const {
    *reinterpret_cast<uint2*>(p) = raw;
  }
  __device__ __forceinline__ void unpack(float (&f)[4]) const {
    f[0] = __uint_as_float(raw.x << 16);
    f[1] = __uint_as_float(raw.x & 0xffff0000u);
    f[2] = __uint_as_float(raw.y << 16);
    f[3] = __uint_as_float(raw.y & 0xffff0000u);
  }
  __device__ __forceinline__ void pack(const float (&f)[4]) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]);
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2], f[3]);
    raw = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                     *reinterpret_cast<const uint32_t*>(&b));
  }
};

template <typename T>
struct Pack<T, 1> {
  T raw;
  __device__ __forceinline__ void zero() { raw = from_f32<T>(0.f); }
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void store(T* p) const { *p = raw; }
  __device__ __forceinline__ void unpack(float (&f)[1]) const { f[0] = to_f32(raw); }
  __device__ __forceinline__ void pack(const float (&f)[1]) { raw = from_f32<T>(f[0]); }
};

cudaError_t launch_conv(ConvArgs a, int in_dtype, int W, bool wide, cudaStream_t stream);
cudaError_t launch_conv_step(ConvArgs a, int in_dtype, int W, bool wide, cudaStream_t stream);
cudaError_t launch_qk_norm(QkArgs a, int in_dtype, int pair, cudaStream_t stream);
cudaError_t launch_scan_tok(const ScanArgs& a, int in_dtype, cudaStream_t stream);
cudaError_t launch_scan_join(const ScanArgs& a, cudaStream_t stream);
cudaError_t launch_scan_step(const ScanArgs& a, int in_dtype, cudaStream_t stream);
void scan_tok_pieces(int R, int P, int H, int d_v, int sms, int* nseg, int* seg_len);

bool scan_chunk_supported(const ScanArgs& a, int in_dtype);
void scan_chunk_pieces(int R, int P, int H, int d_v, int sms, int* nseg, int* seg_len);
cudaError_t launch_scan_chunk(const ScanArgs& a, cudaStream_t stream);

}  // namespace ola
