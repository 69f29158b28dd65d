// Norm of every query and key head with the position rotation in the same pass.
//
//     n = x * rsqrt(m + eps) * w,  m = mean or sum of x^2 over the head; then, on pairs (a, b) of
//     the first `rot` dims,  (a cos - b sin, b cos + a sin),  angle = position * inv_freq.
//
// A head is read once and written once: the bound is HBM. A group of GL lanes owns a head: each
// lane holds items of two 16-byte chunks. An item is one rotation pair of chunks (j, j + rot/2)
// or two neighbouring chunks, so a rotation never leaves its lane; the sum of squares is joined by
// shuffles. A warp takes one token's heads 32 / GL at a time; the token's angles are worked out
// once, each by one of the groups, and handed round by shuffles. Angles are reduced in fp64:
// position * inv_freq in fp32 would be off by 2^-24 of up to 10^5 radians.
#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kQkThreads = 128;

// GL lanes per head, NI items per lane (items past the head's end are idle).
template <typename T, int GL, int NI, bool PAIR>
__global__ void __launch_bounds__(kQkThreads) qk_norm_kernel(QkArgs a) {
  constexpr int E = 16 / int(sizeof(T));          // elements per chunk
  constexpr int NG = 32 / GL;                     // heads a warp takes together
  const int lane = threadIdx.x & 31, gl = lane % GL, grp = lane / GL;
  const int64_t warp = (int64_t(blockIdx.x) * kQkThreads + threadIdx.x) >> 5;
  const int64_t tok = warp / a.hsplit;
  const int part = int(warp % a.hsplit);
  if (tok >= a.N) return;                         // whole warps
  const int nch = a.d / E, half = a.rot / (2 * E), nitem = (nch + 1) / 2;
  // chunks of this lane's items; -1: none
  int c0[NI], c1[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int j = gl + i * GL;
    if (!PAIR && j < half) {
      c0[i] = j;
      c1[i] = j + half;
    } else {
      c0[i] = 2 * j;                              // 2 half + 2 (j - half)
      c1[i] = 2 * j + 1;
    }
    if (j >= nitem) c0[i] = c1[i] = -1;
    if (c1[i] >= nch) c1[i] = -1;
  }
  // cos and sin of the E angles of each item: E pairs of chunks (j, j + half), or E / 2 pairs
  // inside each of the two chunks. Group g works out the angles e = g, g + NG, ...
  float cs[NI][E], sn[NI][E];
  if (a.rot) {
    const double pos = double(__ldg(a.pos + tok));
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int j = gl + i * GL;
      float mc[(E + NG - 1) / NG], ms[(E + NG - 1) / NG];
#pragma unroll
      for (int m = 0; m < (E + NG - 1) / NG; ++m) {
        const int f = j * E + m * NG + grp;       // the same index in both pairings
        mc[m] = 1.f;
        ms[m] = 0.f;
        if (f < a.rot / 2 && m * NG + grp < E) {
          double turns = pos * double(__ldg(a.inv_freq + f)) * 0.15915494309189533577;
          turns -= rint(turns);
          sincospif(float(2.0 * turns), &ms[m], &mc[m]);
        }
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        cs[i][e] = __shfl_sync(kFull, mc[e / NG], (e % NG) * GL + gl);
        sn[i][e] = __shfl_sync(kFull, ms[e / NG], (e % NG) * GL + gl);
      }
    }
  }
  const int heads = a.Hq + a.Hk;
  const int per = ((heads + a.hsplit - 1) / a.hsplit + NG - 1) / NG * NG;
  const int h1 = min(heads, (part + 1) * per);
  for (int hb = part * per; hb < h1; hb += NG) {
    const int h = hb + grp;
    const bool on = h < h1;
    const bool isq = h < a.Hq;
    const T* src = isq ? static_cast<const T*>(a.q) + tok * a.q_tok + int64_t(h) * a.d
                       : static_cast<const T*>(a.k) + tok * a.k_tok + int64_t(h - a.Hq) * a.d;
    T* dst = isq ? static_cast<T*>(a.q_out) + tok * a.qo_tok + int64_t(h) * a.d
                 : static_cast<T*>(a.k_out) + tok * a.ko_tok + int64_t(h - a.Hq) * a.d;
    const float* w = isq ? a.wq : a.wk;
    Pack<T, E> r0[NI], r1[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      r0[i].zero();
      r1[i].zero();
      if (on && c0[i] >= 0) r0[i].load(src + c0[i] * E);
      if (on && c1[i] >= 0) r1[i].load(src + c1[i] * E);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      float x0[E], x1[E];
      r0[i].unpack(x0);
      r1[i].unpack(x1);
#pragma unroll
      for (int e = 0; e < E; ++e) s = fmaf(x0[e], x0[e], fmaf(x1[e], x1[e], s));
    }
#pragma unroll
    for (int o = GL / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
    const float rs = rsqrtf((a.l2 ? s : s / float(a.d)) + a.eps);
    if (!on) continue;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (c0[i] < 0) continue;
      float x0[E], x1[E];
      r0[i].unpack(x0);
      r1[i].unpack(x1);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        x0[e] *= rs;
        x1[e] *= rs;
      }
      if (w) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x0[e] *= __ldg(w + c0[i] * E + e);
          if (c1[i] >= 0) x1[e] *= __ldg(w + c1[i] * E + e);
        }
      }
      if (a.rot) {
        if (!PAIR) {
          if (c0[i] < half) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float p = x0[e], q = x1[e];
              x0[e] = p * cs[i][e] - q * sn[i][e];
              x1[e] = q * cs[i][e] + p * sn[i][e];
            }
          }
        } else {
          // rot is a multiple of 16, so a chunk is rotated as a whole or not at all
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            if (c0[i] * E < a.rot) {
              const float p = x0[2 * e], q = x0[2 * e + 1];
              x0[2 * e] = p * cs[i][e] - q * sn[i][e];
              x0[2 * e + 1] = q * cs[i][e] + p * sn[i][e];
            }
            if (c1[i] * E < a.rot) {
              const float p = x1[2 * e], q = x1[2 * e + 1];
              x1[2 * e] = p * cs[i][E / 2 + e] - q * sn[i][E / 2 + e];
              x1[2 * e + 1] = q * cs[i][E / 2 + e] + p * sn[i][E / 2 + e];
            }
          }
        }
      }
      Pack<T, E> o;
      o.pack(x0);
      o.store(dst + c0[i] * E);
      if (c1[i] >= 0) {
        o.pack(x1);
        o.store(dst + c1[i] * E);
      }
    }
  }
}

template <typename T, int GL, int NI>
cudaError_t run(const QkArgs& a, int pair, unsigned grid, cudaStream_t st) {
  if (pair)
    qk_norm_kernel<T, GL, NI, true><<<grid, kQkThreads, 0, st>>>(a);
  else
    qk_norm_kernel<T, GL, NI, false><<<grid, kQkThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_norm(QkArgs a, int in_dtype, int pair, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = device_sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int E = in_dtype == OLA_BF16 ? 8 : 4;
  const int nitem = (a.d / E + 1) / 2;
  int gl = 1;
  while (gl < 32 && gl < nitem) gl *= 2;
  const int ng = 32 / gl;
  // few tokens: their heads are shared out over more warps, down to one head group each
  const int groups = (a.Hq + a.Hk + ng - 1) / ng;
  a.hsplit = 1;
  while (a.hsplit < groups && a.N * a.hsplit < int64_t(16) * sms) a.hsplit *= 2;
  const int64_t warps = a.N * a.hsplit;
  const int64_t grid = (warps * 32 + kQkThreads - 1) / kQkThreads;
  if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned g = unsigned(grid);
  if (in_dtype == OLA_BF16) {
    if (gl == 1) return run<__nv_bfloat16, 1, 1>(a, pair, g, st);
    if (gl == 2) return run<__nv_bfloat16, 2, 1>(a, pair, g, st);
    if (gl == 4) return run<__nv_bfloat16, 4, 1>(a, pair, g, st);
    if (gl == 8) return run<__nv_bfloat16, 8, 1>(a, pair, g, st);
    if (gl == 16) return run<__nv_bfloat16, 16, 1>(a, pair, g, st);
    return run<__nv_bfloat16, 32, 1>(a, pair, g, st);
  }
  if (nitem > 32) return run<float, 32, 2>(a, pair, g, st);
  if (gl == 1) return run<float, 1, 1>(a, pair, g, st);
  if (gl == 2) return run<float, 2, 1>(a, pair, g, st);
  if (gl == 4) return run<float, 4, 1>(a, pair, g, st);
  if (gl == 8) return run<float, 8, 1>(a, pair, g, st);
  if (gl == 16) return run<float, 16, 1>(a, pair, g, st);
  return run<float, 32, 1>(a, pair, g, st);
}

}  // namespace ola
