// Norm of every query and key head with the position rotation in the same pass.
//
//     n = x * rsqrt(m + eps) * w,  m = mean or sum of x^2 over the head; then, on pairs (a, b) of
//     the first `rot` dims,  (a cos - b sin, b cos + a sin),  angle = position * inv_freq.
//
// A head is read once and written once: the bound is HBM. A group of GL lanes owns a head: each
// lane holds items of two 16-byte chunks. An item is one rotation pair of chunks (j, j + rot/2)
// or two neighbouring chunks, so a rotation never leaves its lane; the sum of squares is joined by
// shuffles. A warp takes one token's heads 32 / GL at a time, the next ones' loads ahead of the
// arithmetic, and walks over tokens; weights lie in shared memory in the items' order, so that
// neighbouring lanes read neighbouring 16 bytes. The token's angles are worked out once, one per
// lane, and handed round through shared memory. Angles are reduced in fp64: position * inv_freq in
// fp32 would be off by 2^-24 of up to 10^5 radians.
//
// Measured, bf16: 40960 tokens of 32 heads of 128 in 105 us (97 % of the copy rate); 20480 tokens of
// 18 heads of 256, weighted, 64 dims rotated, in 72 us (80 %: the weights' reads and the shuffles
// share the load-store pipe; with weights in channel order, where lanes met in the banks, it was 85 %
// busy and took 78 us). Worse: weights in registers (81), loads two groups ahead (81).
#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kQkThreads = 128;
// Resident blocks per SM (the launch bounds): the grid is one such wave, each warp walks on. The
// rotated form takes 71.8 us at 6, 74.2 at 5, 74.9 at 7 and 83 at 8.
constexpr int qk_blocks(int ni, int rot) { return ni > 1 ? 4 : rot ? 6 : 8; }

// GL lanes per head, NI items per lane (items past the head's end are idle).
// ROT: 0 no rotation, 1 pairs (i, i + rot/2), 2 pairs (2i, 2i + 1).
template <typename T, int GL, int NI, int ROT>
__global__ void __launch_bounds__(kQkThreads, qk_blocks(NI, ROT)) qk_norm_kernel(QkArgs a) {
  constexpr int E = 16 / int(sizeof(T));          // elements per chunk
  constexpr int H2 = E / 2;                       // fp32 pairs per chunk
  constexpr int NG = 32 / GL;                     // heads a warp takes together
  extern __shared__ __align__(16) float sm[];     // wq, wk [d] each; per warp: cos, sin
  const int lane = threadIdx.x & 31, gl = lane % GL, grp = lane / GL;
  const int nwarp = gridDim.x * (kQkThreads / 32);
  const int64_t w0 = int64_t(blockIdx.x) * (kQkThreads / 32) + (threadIdx.x >> 5);
  const int nang = ROT ? (a.rot / 2 + 31) / 32 * 32 : 0;   // table entries, filled up
  const int nch = a.d / E, half = a.rot / (2 * E), nitem = (nch + 1) / 2;
  const int nwt = nitem * 2 * E;                  // weights of one kind, filled up
  float* ct = sm + 2 * nwt + (threadIdx.x >> 5) * 2 * nang;
  float* st = ct + nang;
  // the two chunks of item j; the second may lie past the head's end
  auto chunk0 = [&](int j) { return ROT == 1 && j >= half ? j + half : j; };
  auto chunk1 = [&](int j) { return ROT == 1 && j < half ? j + half : j + nitem; };
  const bool weighted = a.wq || a.wk;
  if (weighted) {
    // [four elements of an item][item][4]: neighbouring lanes read neighbouring 16 bytes
    for (int i = threadIdx.x; i < nwt; i += kQkThreads) {
      const int four = i / (4 * nitem), j = i / 4 % nitem;
      const int c = four < E / 4 ? chunk0(j) : chunk1(j);
      const int ch = c * E + four % (E / 4) * 4 + i % 4;
      sm[i] = a.wq && c < nch ? __ldg(a.wq + ch) : 1.f;
      sm[nwt + i] = a.wk && c < nch ? __ldg(a.wk + ch) : 1.f;
    }
    __syncthreads();
  }
  // chunks of this lane's items; -1: none
  int c0[NI], c1[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int j = gl + i * GL;
    c0[i] = j < nitem ? chunk0(j) : -1;
    c1[i] = j < nitem && chunk1(j) < nch ? chunk1(j) : -1;
  }
  const int uq = (a.Hq + NG - 1) / NG, uk = (a.Hk + NG - 1) / NG;   // head groups
  const int per = (uq + uk + a.hsplit - 1) / a.hsplit;
  const float inv_d = 1.f / float(a.d);
  auto freq = [&](int f) -> double {              // turns per position
    return double(__ldg(a.inv_freq + f)) * 0.15915494309189533577;
  };
  const double first = ROT && lane < a.rot / 2 ? freq(lane) : 0.0;
  for (int64_t w = w0; w < a.N * a.hsplit; w += nwarp) {
    const int64_t tok = w / a.hsplit;
    const int part = int(w - tok * a.hsplit);
    const int u0 = part * per, u1 = min(uq + uk, u0 + per);
    // this lane group's head in q's and k's rows, and the step to the next one
    const int64_t step = int64_t(NG) * a.d;
    const T* qs = static_cast<const T*>(a.q) + tok * a.q_tok + (int64_t(u0) * NG + grp) * a.d;
    T* qd = static_cast<T*>(a.q_out) + tok * a.qo_tok + (int64_t(u0) * NG + grp) * a.d;
    const int uk0 = u0 > uq ? u0 - uq : 0;
    const T* ks = static_cast<const T*>(a.k) + tok * a.k_tok + (int64_t(uk0) * NG + grp) * a.d;
    T* kd = static_cast<T*>(a.k_out) + tok * a.ko_tok + (int64_t(uk0) * NG + grp) * a.d;
    Pack<T, E> n0[NI], n1[NI];
    auto fetch = [&](int u) {                     // called for u0, u0 + 1, ... in turn
      const bool isq = u < uq;
      const T* src = isq ? qs : ks;
      const bool on = u < u1 && (isq ? u * NG + grp < a.Hq : (u - uq) * NG + grp < a.Hk);
      if (isq) qs += step; else ks += step;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        n0[i].zero();
        n1[i].zero();
        if (on && c0[i] >= 0) n0[i].load(src + c0[i] * E);
        if (on && c1[i] >= 0) n1[i].load(src + c1[i] * E);
      }
    };
    fetch(u0);
    // cos, sin of an item's E angles: of the pairs of chunks (j, j + half), or of E / 2 pairs
    // inside each of its two chunks
    uint64_t cs[NI][H2], sn[NI][H2];
    if (ROT) {
      __syncwarp();
      const double pos = double(__ldg(a.pos + tok));
      for (int f = lane; f < nang; f += 32) {
        float c = 1.f, s = 0.f;
        if (f < a.rot / 2) {
          double turns = pos * (f < 32 ? first : freq(f));
          turns -= rint(turns);
          if constexpr (sizeof(T) == 2) {
            // within 2^-20 in -pi .. pi, far below bf16's 2^-8
            const float x = float(turns) * 6.283185307179586f;
            s = __sinf(x);
            c = __cosf(x);
          } else {
            sincospif(float(2.0 * turns), &s, &c);
          }
        }
        ct[f] = c;
        st[f] = s;
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int j = gl + i * GL;
#pragma unroll
        for (int e = 0; e < H2; ++e) {
          // ROT 2: pairs 0 .. H2 / 2 - 1 belong to chunk j, the others to chunk j + nitem
          const int f = ROT == 1          ? j * E + 2 * e
                        : 2 * e < H2      ? j * H2 + 2 * e
                                          : (j + nitem) * H2 + 2 * e - H2;
          cs[i][e] = f < nang ? *reinterpret_cast<const uint64_t*>(ct + f) : 0;
          sn[i][e] = f < nang ? *reinterpret_cast<const uint64_t*>(st + f) : 0;
        }
      }
    }
#pragma unroll 1
    for (int u = u0; u < u1; ++u) {
      const bool isq = u < uq;
      const bool on = isq ? u * NG + grp < a.Hq : (u - uq) * NG + grp < a.Hk;
      T* dst = isq ? qd : kd;
      if (isq) qd += step; else kd += step;
      uint64_t x0[NI][H2], x1[NI][H2], s2 = f2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float f0[E], f1[E];
        n0[i].unpack(f0);
        n1[i].unpack(f1);
#pragma unroll
        for (int e = 0; e < H2; ++e) {
          x0[i][e] = f2(f0[2 * e], f0[2 * e + 1]);
          x1[i][e] = f2(f1[2 * e], f1[2 * e + 1]);
          s2 = fma2(x0[i][e], x0[i][e], fma2(x1[i][e], x1[i][e], s2));
        }
      }
      fetch(u + 1);
      const float2 st2 = un2(s2);
      float s = st2.x + st2.y;
#pragma unroll
      for (int o = GL / 2; o > 0; o >>= 1) s += __shfl_xor_sync(kFull, s, o);
      const float rs = rsqrtf((a.l2 ? s : s * inv_d) + a.eps);
      if (!on) continue;
      const uint64_t rs2 = f2(rs, rs);
      const float* wt = sm + (isq ? 0 : nwt) + 4 * gl;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        if (c0[i] < 0) continue;
#pragma unroll
        for (int e = 0; e < H2; ++e) {
          x0[i][e] = mul2(x0[i][e], rs2);
          x1[i][e] = mul2(x1[i][e], rs2);
        }
        if (weighted) {
#pragma unroll
          for (int e = 0; e < H2; e += 2) {
            const float* p = wt + 4 * (i * GL + e / 2 * nitem);
            const ulonglong2 a2 = *reinterpret_cast<const ulonglong2*>(p);
            const ulonglong2 b2 = *reinterpret_cast<const ulonglong2*>(p + nwt / 2);
            x0[i][e] = mul2(x0[i][e], a2.x);
            x0[i][e + 1] = mul2(x0[i][e + 1], a2.y);
            x1[i][e] = mul2(x1[i][e], b2.x);
            x1[i][e + 1] = mul2(x1[i][e + 1], b2.y);
          }
        }
        if (ROT == 1) {
          if (c0[i] < half) {
            const uint64_t neg = f2(-1.f, -1.f);
#pragma unroll
            for (int e = 0; e < H2; ++e) {
              const uint64_t p = x0[i][e], q = x1[i][e];
              x0[i][e] = fma2(p, cs[i][e], mul2(mul2(q, sn[i][e]), neg));
              x1[i][e] = fma2(q, cs[i][e], mul2(p, sn[i][e]));
            }
          }
        } else if (ROT == 2) {
          // rot is a multiple of 16, so a chunk is rotated as a whole or not at all
          const bool one = c0[i] * E < a.rot, both = c1[i] * E < a.rot;
#pragma unroll
          for (int e = 0; e < H2; ++e) {
            // pair e of chunk 0 has angle e, of chunk 1 angle E / 2 + e
            auto turn = [&](uint64_t v, int k) {
              const float2 c2 = un2(cs[i][k / 2]), t2 = un2(sn[i][k / 2]), xy = un2(v);
              const float c = k & 1 ? c2.y : c2.x, t = k & 1 ? t2.y : t2.x;
              return f2(xy.x * c - xy.y * t, xy.y * c + xy.x * t);
            };
            if (one) x0[i][e] = turn(x0[i][e], e);
            if (one && both) x1[i][e] = turn(x1[i][e], H2 + e);
          }
        }
        float f[E];
        Pack<T, E> o;
#pragma unroll
        for (int e = 0; e < H2; ++e) {
          const float2 t = un2(x0[i][e]);
          f[2 * e] = t.x;
          f[2 * e + 1] = t.y;
        }
        o.pack(f);
        o.store(dst + c0[i] * E);
        if (c1[i] >= 0) {
#pragma unroll
          for (int e = 0; e < H2; ++e) {
            const float2 t = un2(x1[i][e]);
            f[2 * e] = t.x;
            f[2 * e + 1] = t.y;
          }
          o.pack(f);
          o.store(dst + c1[i] * E);
        }
      }
    }
  }
}

template <typename T, int GL, int NI>
cudaError_t run(const QkArgs& a, int pair, unsigned grid, cudaStream_t st) {
  const int nang = a.rot ? (a.rot / 2 + 31) / 32 * 32 : 0;
  constexpr int E = 16 / int(sizeof(T));
  const int nwt = (a.d / E + 1) / 2 * 2 * E;
  const size_t smem = sizeof(float) * 2 * (nwt + nang * (kQkThreads / 32));
  if (!a.rot)
    qk_norm_kernel<T, GL, NI, 0><<<grid, kQkThreads, smem, st>>>(a);
  else if (pair)
    qk_norm_kernel<T, GL, NI, 2><<<grid, kQkThreads, smem, st>>>(a);
  else
    qk_norm_kernel<T, GL, NI, 1><<<grid, kQkThreads, smem, st>>>(a);
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
  const int groups = (a.Hq + ng - 1) / ng + (a.Hk + ng - 1) / ng;
  a.hsplit = 1;
  while (a.hsplit < groups && a.N * a.hsplit < int64_t(16) * sms) a.hsplit *= 2;
  int64_t grid = (a.N * a.hsplit * 32 + kQkThreads - 1) / kQkThreads;
  const int64_t most = int64_t(sms) * qk_blocks(nitem > 32 ? 2 : 1, a.rot);
  if (grid > most) grid = most;
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
