// Short depthwise causal convolution, for prompts and for one token of every beam.
//
//     y[p][c] = act(bias[c] + sum_{i<W} w[c][i] u[p + i][c]),   u = (W-1 earlier tokens) ++ x
//
// 2W + a few operations per element against one read and one write of it: the bound is HBM. A
// thread owns 16 bytes of neighbouring channels and walks consecutive tokens with the window of
// the last W-1 inputs in registers, so an element is read once (plus the W-1 tokens before each
// thread's stretch, which its neighbour's reads leave in L2). The block brings its channels' taps
// in once, transposed through shared memory ([tap][channel], read 16 bytes at a time); sums run two
// channels per instruction. The window's values are moved, never recomputed: the state that leaves
// is the input's bits.
//
// Loads run through a ring in shared memory that each thread fills for itself (cp.async): deep
// prefetch without registers or barriers. Measured: 8 x 5120 tokens of 6144 bf16 channels in 167 us
// (1.0 GB, 92 % of the copy rate; before the ring 244 us, with 8-byte vectors 270); 8192 beams in
// 112 us (91 %; without the ring 135 us). One prompt of 1024 tokens takes 10.5 us from HBM (8.3 out
// of L2) where the copy rate gives 3.9: launch, taps and the ring's first fill. Rows whose start or
// stride is not a multiple of 16 bytes go one channel per thread, without the ring: 4 x 2000 tokens of
// 1001 bf16 channels in 19.3 us, where the copy rate gives 4.9.
#include <type_traits>

#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kConvThreads = 256;
constexpr int kConvUnroll = 4;      // tokens loaded together
constexpr int kAhead = 3;           // groups of them in flight
constexpr int kStepAhead = 3;       // beams in flight

// fp32 pairs of a pack: VEC elements as (VEC + 1) / 2 pairs.
template <typename T, int VEC>
struct Pairs {
  static constexpr int N = (VEC + 1) / 2;
  uint64_t p[N];
  __device__ __forceinline__ void from(const Pack<T, VEC>& k) {
    float f[VEC];
    k.unpack(f);
#pragma unroll
    for (int e = 0; e < N; ++e) p[e] = f2(f[2 * e], VEC > 1 ? f[VEC > 1 ? 2 * e + 1 : 0] : 0.f);
  }
  __device__ __forceinline__ void to(Pack<T, VEC>& k) const {
    float f[VEC];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float2 t = un2(p[e]);
      f[2 * e] = t.x;
      if (VEC > 1) f[VEC > 1 ? 2 * e + 1 : 0] = t.y;
    }
    k.pack(f);
  }
};

// Taps and biases of a thread's channels.
template <typename T, int VEC, int W>
struct Taps {
  static constexpr int N = (VEC + 1) / 2;
  uint64_t w[W][N], b[N];

  // Cooperative: the taps of the block's channels c0 .. c0 + nc - 1 go through shared memory.
  __device__ __forceinline__ void load(const ConvArgs& a, float* sm, int c0, int nc, int cl) {
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int have = min(nc, a.C - c0);
    for (int i = tid; i < have * W; i += kConvThreads)
      sm[(i % W) * nc + i / W] = __ldg(a.w + int64_t(c0) * W + i);
    for (int i = tid; i < have; i += kConvThreads)
      sm[W * nc + i] = a.bias ? __ldg(a.bias + c0 + i) : 0.f;
    __syncthreads();
    if (cl >= have) return;
#pragma unroll
    for (int i = 0; i <= W; ++i) {
      float f[VEC];
      const float* src = sm + i * nc + cl;
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int q = 0; q < VEC / 4; ++q) {
          const float4 t = reinterpret_cast<const float4*>(src)[q];
          f[4 * q] = t.x;
          f[4 * q + 1] = t.y;
          f[4 * q + 2] = t.z;
          f[4 * q + 3] = t.w;
        }
      } else {
        f[0] = src[0];
      }
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const uint64_t v = f2(f[2 * e], VEC > 1 ? f[VEC > 1 ? 2 * e + 1 : 0] : 0.f);
        if (i < W)
          w[i < W ? i : 0][e] = v;
        else
          b[e] = v;
      }
    }
  }
  // win[0..W-2] the earlier tokens, oldest first, x the newest
  __device__ __forceinline__ void apply(const Pairs<T, VEC>* win, const Pairs<T, VEC>& x,
                                        int silu, Pairs<T, VEC>& y) const {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      uint64_t u = b[e];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) u = fma2(w[i][e], win[i].p[e], u);
      u = fma2(w[W - 1][e], x.p[e], u);
      y.p[e] = silu ? silu2<T>(u) : u;
    }
  }
};

// blockDim = (channel vectors, token stretches); grid.x = channel blocks x token blocks x R.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) conv_kernel(ConvArgs a) {
  extern __shared__ __align__(16) float sm[];
  const int ct = blockIdx.x % a.n_ctile;
  const int rest = blockIdx.x / a.n_ctile;
  const int r = rest / a.n_ttile;
  const int64_t tile = int64_t(rest % a.n_ttile) * blockDim.y + threadIdx.y;
  const int nc = blockDim.x * VEC, c0 = ct * nc, cl = threadIdx.x * VEC, c = c0 + cl;
  const int64_t t0w = tile * a.tt;
  const bool active = c < a.C && (t0w < a.P || tile == 0);
  const int t0 = active ? int(t0w) : 0;
  const int L = seq_len(a.lens, r, a.P);
  const int t1 = active ? min(t0 + a.tt, L) : 0;
  const T* x = static_cast<const T*>(a.x) + int64_t(r) * a.x_seq + c;
  T* y = static_cast<T*>(a.y) + int64_t(r) * a.y_seq + c;
  // 16-byte vectors come through a ring of kAhead groups of tokens in shared memory, which every
  // thread fills for itself: deep prefetch without registers and without barriers
  constexpr bool ASYNC = VEC * sizeof(T) == 16;
  constexpr int kVecBytes = VEC * int(sizeof(T)), kSlot = kConvThreads * kVecBytes;
  unsigned char* ring = reinterpret_cast<unsigned char*>(sm + (W + 1) * nc) +
                        (threadIdx.y * blockDim.x + threadIdx.x) * kVecBytes;
  const int64_t xs = a.x_tok * int64_t(sizeof(T)), ys = a.y_tok * int64_t(sizeof(T));
  const char* xl = reinterpret_cast<const char*>(x + int64_t(t0) * a.x_tok);   // next to load
  int tl = t0, sl = 0;                                       // its token, its slot
  auto fetch_async = [&]() {
    if constexpr (ASYNC) {
      unsigned char* dst = ring + sl * (kConvUnroll * kSlot);
      if (tl + kConvUnroll <= t1) {
#pragma unroll
        for (int i = 0; i < kConvUnroll; ++i, xl += xs) cp_async16(dst + i * kSlot, xl);
      } else {
#pragma unroll
        for (int i = 0; i < kConvUnroll; ++i, xl += xs)
          if (tl + i < t1) cp_async16(dst + i * kSlot, xl);
      }
      tl += kConvUnroll;
      sl = sl + 1 < kAhead ? sl + 1 : 0;
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) fetch_async();
  Taps<T, VEC, W> taps;
  taps.load(a, sm, c0, nc, cl);
  if (!active) return;
  // the window before the stretch: earlier tokens, or the incoming state
  const T* si = a.state_in
                    ? static_cast<const T*>(a.state_in) + int64_t(r) * (W - 1) * a.C + c
                    : nullptr;
  Pairs<T, VEC> win[W - 1];
  if (t0 == 0) {
    Pack<T, VEC> keep[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      keep[j].zero();
      if (si) keep[j].load(si + int64_t(j) * a.C);
      win[j].from(keep[j]);
    }
    if (a.state_out) {
      // the last W-1 tokens of state ++ x[:L]; every read precedes the first write, so that
      // state_out may be state_in (no other thread touches these channels' states)
      Pack<T, VEC> out[W - 1];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const int t = L + j - (W - 1);
        if (t >= 0) {
          out[j].load(x + int64_t(t) * a.x_tok);
        } else {
#pragma unroll
          for (int i = 0; i < W - 1; ++i)
            if (i == t + W - 1) out[j] = keep[i];
        }
      }
      T* so = static_cast<T*>(a.state_out) + int64_t(r) * (W - 1) * a.C + c;
#pragma unroll
      for (int j = 0; j < W - 1; ++j) out[j].store(so + int64_t(j) * a.C);
    }
    if (t1 <= 0) return;
  } else {
    if (t0 >= t1) return;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {             // tt >= W - 1: these tokens exist
      Pack<T, VEC> p;
      p.load(x + int64_t(t0 + j - (W - 1)) * a.x_tok);
      win[j].from(p);
    }
  }
  int slot = 0;
  char* yl = reinterpret_cast<char*>(y + int64_t(t0) * a.y_tok);
  const char* xr = reinterpret_cast<const char*>(x + int64_t(t0) * a.x_tok);
  // kConvUnroll tokens from registers; ALL: every one of them exists
  auto group = [&](auto all, int t) {
    constexpr bool ALL = decltype(all)::value;
    Pack<T, VEC> in[kConvUnroll];
    if constexpr (ASYNC) asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
#pragma unroll
    for (int i = 0; i < kConvUnroll; ++i) {
      if constexpr (ASYNC) {
        in[i].load(reinterpret_cast<const T*>(ring + (slot * kConvUnroll + i) * kSlot));
      } else {
        in[i].zero();
        if (ALL || t + i < t1) in[i].load(reinterpret_cast<const T*>(xr));
        xr += xs;
      }
    }
    slot = slot + 1 < kAhead ? slot + 1 : 0;
    fetch_async();
    Pairs<T, VEC> u[W - 1 + kConvUnroll];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) u[j] = win[j];
#pragma unroll
    for (int i = 0; i < kConvUnroll; ++i) {
      u[W - 1 + i].from(in[i]);
      Pairs<T, VEC> yf;
      taps.apply(u + i, u[W - 1 + i], a.silu, yf);
      Pack<T, VEC> o;
      yf.to(o);
      if (ALL || t + i < t1) o.store(reinterpret_cast<T*>(yl));
      yl += ys;
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = u[kConvUnroll + j];
  };
  int t = t0;
#pragma unroll 1
  for (; t + kConvUnroll <= t1; t += kConvUnroll) group(std::true_type{}, t);
  if (t < t1) group(std::false_type{}, t);
}

// One token of every beam: thread = 16 bytes of channels x tt consecutive beams (of all requests).
// 16-byte vectors come through a thread-private ring of kStepAhead beams (window and token), the
// parent indices one beam further ahead.
template <typename T, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs a) {
  extern __shared__ __align__(16) float sm[];
  constexpr bool ASYNC = VEC * sizeof(T) == 16;
  constexpr int kVecBytes = VEC * int(sizeof(T)), kSlot = kConvThreads * kVecBytes;
  const int ct = blockIdx.x % a.n_ctile;
  const int64_t tile = int64_t(blockIdx.x / a.n_ctile) * blockDim.y + threadIdx.y;
  const int nc = blockDim.x * VEC, c0 = ct * nc, cl = threadIdx.x * VEC, c = c0 + cl;
  const int64_t n = int64_t(a.R) * a.P;
  const int64_t i0 = c < a.C ? tile * a.tt : n, i1 = min(i0 + a.tt, n);
  unsigned char* ring = reinterpret_cast<unsigned char*>(sm + (W + 1) * nc) +
                        (threadIdx.y * blockDim.x + threadIdx.x) * kVecBytes;
  // next beam to fetch: its request, beam and parent
  int64_t in = i0;
  int rn = int(i0 / a.P), bn = int(i0 - int64_t(rn) * a.P), slot_n = 0;
  int pn = i0 < i1 ? parent_state(a.parent, rn, bn, a.P, a.Bp, a.err) : 0;
  auto sources = [&](const T** si, const T** xp) {
    *si = static_cast<const T*>(a.state_in) + (int64_t(rn) * a.Bp + pn) * (W - 1) * a.C + c;
    *xp = static_cast<const T*>(a.x) + int64_t(rn) * a.x_seq + int64_t(bn) * a.x_tok + c;
  };
  auto advance = [&]() {
    ++in;
    if (++bn == a.P) {
      bn = 0;
      ++rn;
    }
    if (in < i1) pn = parent_state(a.parent, rn, bn, a.P, a.Bp, a.err);
  };
  auto fetch_async = [&]() {
    if constexpr (ASYNC) {
      if (in < i1) {
        const T *si, *xp;
        sources(&si, &xp);
        unsigned char* dst = ring + slot_n * (W * kSlot);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) cp_async16(dst + j * kSlot, si + int64_t(j) * a.C);
        cp_async16(dst + (W - 1) * kSlot, xp);
        advance();
      }
      slot_n = slot_n + 1 < kStepAhead ? slot_n + 1 : 0;
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
#pragma unroll
  for (int s = 0; s < kStepAhead; ++s) fetch_async();
  Taps<T, VEC, W> taps;
  taps.load(a, sm, c0, nc, cl);
  int r = int(i0 / a.P), b = int(i0 - int64_t(r) * a.P), slot = 0;
  T* so = static_cast<T*>(a.state_out) + i0 * (W - 1) * a.C + c;
#pragma unroll 1
  for (int64_t i = i0; i < i1; ++i) {
    Pack<T, VEC> s[W];
    if constexpr (ASYNC) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStepAhead - 1) : "memory");
      const unsigned char* src = ring + slot * (W * kSlot);
#pragma unroll
      for (int j = 0; j < W; ++j) s[j].load(reinterpret_cast<const T*>(src + j * kSlot));
      slot = slot + 1 < kStepAhead ? slot + 1 : 0;
      fetch_async();
    } else {
      const T *si, *xp;
      sources(&si, &xp);
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s[j].load(si + int64_t(j) * a.C);
      s[W - 1].load(xp);
      advance();
    }
    Pairs<T, VEC> u[W], yf;
#pragma unroll
    for (int j = 0; j < W; ++j) u[j].from(s[j]);
    taps.apply(u, u[W - 1], a.silu, yf);
    Pack<T, VEC> o;
    yf.to(o);
    o.store(static_cast<T*>(a.y) + int64_t(r) * a.y_seq + int64_t(b) * a.y_tok + c);
#pragma unroll
    for (int j = 0; j < W - 1; ++j, so += a.C) s[j + 1].store(so);
    if (++b == a.P) {
      b = 0;
      ++r;
    }
  }
}

template <typename T, int VEC, int W>
cudaError_t run(const ConvArgs& a, bool step, dim3 block, unsigned grid, cudaStream_t st) {
  const size_t smem = sizeof(float) * (W + 1) * block.x * VEC;
  constexpr bool ASYNC = VEC * sizeof(T) == 16;
  constexpr size_t slot = size_t(kConvThreads) * 16;
  const size_t ring = ASYNC ? slot * (step ? kStepAhead * W : kAhead * kConvUnroll) : 0;
  auto kernel = step ? conv_step_kernel<T, VEC, W> : conv_kernel<T, VEC, W>;
  if (smem + ring > 48 * 1024) {
    static std::atomic<uint64_t> done[2] = {};
    cudaError_t e = once_per_device(done[step], [&] {
      return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 80 * 1024);
    });
    if (e != cudaSuccess) return e;
  }
  kernel<<<grid, block, smem + ring, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t by_taps(const ConvArgs& a, int W, bool step, dim3 block, unsigned grid,
                    cudaStream_t st) {
  if (W == 2) return run<T, VEC, 2>(a, step, block, grid, st);
  if (W == 3) return run<T, VEC, 3>(a, step, block, grid, st);
  return run<T, VEC, 4>(a, step, block, grid, st);
}

cudaError_t launch(ConvArgs a, int in_dtype, int W, bool wide, bool step, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int vec = wide ? (in_dtype == OLA_BF16 ? 8 : 4) : 1;
  const int64_t nvec = (int64_t(a.C) + vec - 1) / vec;
  // a warp's width of channel vectors (512 bytes of a row): wider blocks would bring in more taps
  // for the same tokens
  int bx = 8;
  while (bx < 32 && bx < nvec) bx *= 2;
  const int by = kConvThreads / bx;
  a.n_ctile = int((nvec + bx - 1) / bx);
  const int64_t rows = step ? int64_t(a.R) * a.P : a.P;
  const int64_t seqs = step ? 1 : a.R;
  auto blocks = [&](int tt) {
    const int64_t n = (rows + int64_t(tt) * by - 1) / (int64_t(tt) * by);
    return (n < 1 ? 1 : n) * seqs * a.n_ctile;
  };
  // Tokens (beams) per thread: the count whose waves of blocks, two per SM, end first. A wave takes
  // its count and a start (taps, window, the ring's first fill) worth 8 tokens, or a beam. Against
  // powers of two that leave 1 (prompts) or 8 blocks for every SM: 1 x 1024 tokens of 6144 channels
  // 8.3 us and 9.7 (out of L2), 4 x 1024 22 and 25, 8 x 5120 167 and 177, 1024 beams 18 and 26, 8192
  // beams 112 both. Longer stretches: prompts up to 256 173 us (of 167), beams up to 16 114 (of 112).
  // Two per SM is what the 16-byte kernels' registers and ring leave room for; the single-channel
  // kernels would hold more and follow the same rule unmeasured. Stretches do not span sequences:
  // many sequences of a few tokens leave most thread rows idle (1024 x 4 tokens of 6144: 273 us, floor
  // 21).
  const int64_t slots = 2 * int64_t(sms);
  int64_t least = 0;
  for (int tt = step ? 2 : 4; tt <= (step ? 12 : 64); tt += step ? 1 : 4) {
    const int64_t cost = (blocks(tt) + slots - 1) / slots * (tt + (step ? 1 : 8));
    if (!least || cost < least) {
      least = cost;
      a.tt = tt;
    }
  }
  const int64_t grid = blocks(a.tt);
  a.n_ttile = int(grid / seqs / a.n_ctile);
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const dim3 block(bx, by);
  if (in_dtype == OLA_BF16)
    return wide ? by_taps<__nv_bfloat16, 8>(a, W, step, block, unsigned(grid), st)
                : by_taps<__nv_bfloat16, 1>(a, W, step, block, unsigned(grid), st);
  return wide ? by_taps<float, 4>(a, W, step, block, unsigned(grid), st)
              : by_taps<float, 1>(a, W, step, block, unsigned(grid), st);
}

}  // namespace

cudaError_t launch_conv(ConvArgs a, int in_dtype, int W, bool wide, cudaStream_t stream) {
  return launch(a, in_dtype, W, wide, false, stream);
}

cudaError_t launch_conv_step(ConvArgs a, int in_dtype, int W, bool wide, cudaStream_t stream) {
  return launch(a, in_dtype, W, wide, true, stream);
}

}  // namespace ola
