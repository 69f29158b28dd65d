// Selective state space scan of bf16 prompts in chunks of 128 tokens on tensor cores, d_k <= 128.
//
//     S <- exp(dt A) S + dt v k^T,   o = S q + D v,   y = o * SiLU(z)
//
// Over a chunk entered with state S0, with c_t = sum_{i<=t} dt_i A (a log decay, <= 0):
//     o_t = e^{c_t} S0 q_t + sum_{s<=t} e^{c_t - c_s} dt_s (q_t . k_s) v_s
//     S_C = e^{c_C} S0 + sum_s (e^{c_C - c_s} dt_s v_s) k_s^T
// as four products per chunk, each with fp32 accumulation in tensor memory:
//     G  = Q K^T              128 x 128 x d_k     (exact bf16 operands)
//     Y1 = P V                128 x 64 x 128      P = G * decay * dt below the diagonal, as bf16
//     Y2 = Q S0^T             128 x 64 x d_k      S0 as bf16; o = Y1 + e^{c_t} Y2
//     dS = K^T (W V)          d_k x 64 x 128      W V in three bf16 parts (24 bits)
// The state itself stays in fp32 (tensor memory) and never meets a rounded operand: S_C is as exact
// as an fp32 sum, which is why W V is cut into three bf16 parts and not rounded to one. P and the
// copy of S0 are rounded to bf16 on the way to y alone, which is bf16 itself.
//
// No exponent is ever positive: inside a block of 32 tokens P takes exp2 of the difference of two
// running sums, between blocks s < t it is (e^{c_t - end of s's block}) (e^{end - c_s} dt_s), a
// factor per row and one per column.
//
// One block per (sequence, head, 64 value columns, piece), one per SM:
//   warps 0-7    G -> P (thread = token t, half of the columns; P into tensor memory as the A
//                operand of Y1); warps 0-3 also the next chunk's scalars (dt, running sums)
//   warps 8-15   outputs (thread = token t, half of the columns): Y1 + e^{c_t} Y2, D, gate; y staged
//                over v (rows of 32 scattered 16-byte stores would take half of the data pipe)
//   warps 16-23  W V (thread = token s, half of the columns)
//   warps 24-27  state rows (thread = key column, S^T in tensor memory): S = e^{c_C} S + dS and its
//                bf16 copy. In the first run of a piece, which has no outputs: warps 8-15
//   warp 28      tcgen05.mma: dS;   warp 29  tcgen05.mma: Y1, the next chunk's G, Y2
//   warp 30      TMA loads of v, stores of y
//   warp 31      TMA loads of keys and queries
// Two issuing warps, so that neither chain (G -> P -> Y1 and W V -> dS -> S -> Y2) waits behind the
// other's operands; nothing but Y2 waits for the state. A piece of a cut sequence runs twice: dS
// alone first (FULL = false), then, once scan_join_kernel has made the state before every piece,
// the outputs.
//
// What bounds it: not HBM (64 prompts of 5120 tokens, 16 heads of 128 x 128: 5.5 GB in 1.60 ms of
// short runs, 52 % of the copy rate; 1.91-1.96 ms in long ones, where the clock falls), not the matrix
// pipe (32 % busy) and not shared memory alone, though every chunk passes 16 KB of v, y, three parts
// of W V and the keys and queries through it, most of it twice (60 % of its data pipe): the chains
// above stand in front of two stages (64 KB of keys and queries each, three would not fit). The wait
// of G for the read of P is part of them: 1.60 ms with it, 1.57 in the order of issue alone, which
// nothing guarantees. Measured before that wait, and worse than 1.54-1.57 ms: y stored straight from
// registers (1.74 ms), y staged over the queries (1.90), P in place of G behind barriers of 64 threads
// (1.74), 16 state columns at a time (1.63), four W V or four output warps (1.85 against 1.79 in long
// runs).
#include "ola_layer.cuh"

namespace ola {

namespace {

constexpr int kQ = 128;                 // tokens per chunk
constexpr int kNV = 64;                 // value columns per block
constexpr int kThr = 1024;
constexpr uint32_t kBlk = kQ * 128;     // 16 KB: 128 rows of 64 bf16 columns

// tensor memory columns
constexpr uint32_t kTG = 0;             // G, 128; then P, 8 columns of bf16 pairs for each 16 of G
constexpr uint32_t kTD = 128;           // dS of the three parts of W V, 64 each
constexpr uint32_t kTS = 320;           // S^T fp32, 64
constexpr uint32_t kTY1 = 384;
constexpr uint32_t kTY2 = 448;

constexpr int kScFloats = 356;          // suf[128], dt[128], colf[96], block sums[4]

template <int KB>                       // 64-column blocks of d_k
struct Lay {
  static constexpr int NST = KB == 2 ? 2 : 3;              // stages
  static constexpr uint32_t kQr = KB * kBlk;               // keys, then queries
  static constexpr uint32_t kKQ = 2 * KB * kBlk;           // one stage of both
  static constexpr uint32_t kV = NST * kKQ;                // values, then y
  static constexpr uint32_t kXw = kV + NST * kBlk;         // W V: three parts
  static constexpr uint32_t kS = kXw + 3 * kBlk;           // state copy [64 KB rows][64 columns]
  static constexpr uint32_t kSc = kS + KB * 8192;          // scalars per stage
  static constexpr uint32_t kBar = kSc + NST * kScFloats * 4;
  static constexpr int kNBar = 7 * NST + 13;
  static constexpr uint32_t kBad = kBar + kNBar * 8;       // flag
  // the tensor-memory address is handed over in the scalars' place, before they are written
  static constexpr uint32_t kBytes = kBad + 8;
};
static_assert(Lay<1>::kBar % 8 == 0 && Lay<2>::kBar % 8 == 0, "mbarriers");
static_assert(Lay<1>::kBytes <= 232448 && Lay<2>::kBytes <= 232448, "shared memory per block");
static_assert((kScFloats * 4) % 16 == 0, "float4 rows of scalars");

struct ChunkScan {
  CUtensorMap mv, mk, mq, my;           // [R][P][heads][d] bf16, boxes of 64 x 1 x 128 x 1
  ScanArgs a;
  int ntile;                            // blocks of 64 value columns
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t pack2(uint64_t a) {
  const float2 f = un2(a);
  return pack2(f.x, f.y);
}

// Two loads of 16 columns of this thread's tensor-memory lane, one wait.
__device__ __forceinline__ void tmem_ld16x2(uint32_t ta, uint32_t tb, uint32_t (&x)[16],
                                            uint32_t (&y)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%33];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]), "=r"(x[6]), "=r"(x[7]), "=r"(x[8]), "=r"(x[9]), "=r"(x[10]), "=r"(x[11]), "=r"(x[12]), "=r"(x[13]), "=r"(x[14]), "=r"(x[15]),
        "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3]), "=r"(y[4]), "=r"(y[5]), "=r"(y[6]), "=r"(y[7]), "=r"(y[8]), "=r"(y[9]), "=r"(y[10]), "=r"(y[11]), "=r"(y[12]), "=r"(y[13]), "=r"(y[14]), "=r"(y[15])
      : "r"(ta), "r"(tb)
      : "memory");
}

// 8 columns each of the three parts of dS (64 columns apart) and of S, one wait.
__device__ __forceinline__ void tmem_ld8x4(uint32_t td, uint32_t (&a)[8], uint32_t (&b)[8],
                                           uint32_t (&c)[8], uint32_t ts, uint32_t (&s)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%32];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%33];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%16, %17, %18, %19, %20, %21, %22, %23}, [%34];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%24, %25, %26, %27, %28, %29, %30, %31}, [%35];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3]), "=r"(a[4]), "=r"(a[5]), "=r"(a[6]), "=r"(a[7]), "=r"(b[0]), "=r"(b[1]), "=r"(b[2]), "=r"(b[3]), "=r"(b[4]), "=r"(b[5]), "=r"(b[6]), "=r"(b[7]),
        "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3]), "=r"(c[4]), "=r"(c[5]), "=r"(c[6]), "=r"(c[7]), "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]), "=r"(s[4]), "=r"(s[5]), "=r"(s[6]), "=r"(s[7])
      : "r"(td), "r"(td + 64), "r"(td + 128), "r"(ts)
      : "memory");
}

// 8 consecutive columns of this thread's lane.
__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int c0,
                                             int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::
          "l"(reinterpret_cast<uint64_t>(map)),
      "r"(smem_u32(src)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}


__device__ __forceinline__ bool warp_wait(uint64_t* bar, int phase) {
  return __all_sync(kFull, mbar_wait_bounded(bar, uint32_t(phase) & 1u));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// A value that is not finite makes NaN of its products with the masked weights too, so of its
// column's outputs earlier in its chunk. They are taken again: the recurrence in fp32 from the
// piece's start to the last such value, by the whole block over tiles staged in shared memory, where
// a thread holds 8 key columns of one value column and warps without an affected column only stage.
// From the value on the column's outputs and state are not finite anyway. Such values in one column at
// token 5000 of 5120 (40 heads of 128 x 128) take a call of 125 us to 380 us, in 64 columns to 910
// (two value columns per thread in half of the warps: 524 and 850; a warp per column that walks the
// tokens in global memory: 7900 and 16400).
__device__ __noinline__ void second_look(const ScanArgs& a, const float* entering,
                                         unsigned char* sm, int r, int h, int g, int v0, int nv,
                                         int p0, int p1) {
  using bf16 = __nv_bfloat16;
  constexpr int kRow = 128;                        // key columns of a staged row, filled up
  bf16* ks = reinterpret_cast<bf16*>(sm);          // [kQ][kRow], then the same of q
  bf16* qs = ks + kQ * kRow;
  bf16* vs = qs + kQ * kRow;                       // [kQ][kNV]
  float2* al = reinterpret_cast<float2*>(vs + kQ * kNV);   // [kQ] decay, dt
  int* first = reinterpret_cast<int*>(al + kQ);    // [kNV] a column's first bad token
  int* last = first + kNV;                         // behind the last output to be taken
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bf16* v = static_cast<const bf16*>(a.v) + int64_t(r) * a.v_seq + int64_t(h) * a.d_v + v0;
  const bf16* k = static_cast<const bf16*>(a.k) + int64_t(r) * a.k_seq + int64_t(g) * a.d_k;
  const bf16* q = static_cast<const bf16*>(a.q) + int64_t(r) * a.q_seq + int64_t(g) * a.d_k;
  __syncthreads();                                 // every role is done with shared memory
  if (tid < kNV) first[tid] = p1;
  if (tid == kNV) *last = p0;
  __syncthreads();
  if (2 * lane < nv) {
#pragma unroll 4
    for (int p = p0 + warp; p < p1; p += kThr / 32) {
      const uint32_t x = __ldg(reinterpret_cast<const uint32_t*>(v + int64_t(p) * a.v_tok) + lane);
      if ((x & 0x7f80u) == 0x7f80u) atomicMin(first + 2 * lane, p);
      if ((x & 0x7f800000u) == 0x7f800000u) atomicMin(first + 2 * lane + 1, p);
    }
  }
  __syncthreads();
  // this thread's value column, its outputs [from, to) and 8 key columns
  const int c = tid >> 4, kg = tid & 15;
  const int to = c < nv ? first[c] : p1, from = p0 + (to - p0) / kQ * kQ;
  const bool mine = to < p1 && from < to;
  if (mine && kg == 0) atomicMax(last, to);
  __syncthreads();
  const int end = *last;
  uint64_t S[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 8 * kg + 2 * j;
    const float* s = entering + int64_t(v0 + c) * a.d_k + e;
    S[j] = entering && mine && e < a.d_k ? f2(s[0], s[1]) : f2(0.f, 0.f);
  }
  const float A = a.A[h], bias = a.dt_bias ? a.dt_bias[h] : 0.f, D = a.D ? a.D[h] : 0.f;
  auto pairs = [](const bf16* p, uint64_t (&x)[4]) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    x[0] = u2(w.x << 16, w.x & 0xffff0000u);
    x[1] = u2(w.y << 16, w.y & 0xffff0000u);
    x[2] = u2(w.z << 16, w.z & 0xffff0000u);
    x[3] = u2(w.w << 16, w.w & 0xffff0000u);
  };
  auto step = [&](int t) {
    const float2 ad = al[t];
    const float w1 = ad.y * to_f32(vs[t * kNV + c]);
    const uint64_t w = f2(w1, w1), d = f2(ad.x, ad.x);
    uint64_t kk[4];
    pairs(ks + t * kRow + 8 * kg, kk);
#pragma unroll
    for (int j = 0; j < 4; ++j) S[j] = fma2(d, S[j], mul2(w, kk[j]));
  };
  for (int pt = p0; pt < end; pt += kQ) {
    const int n = min(kQ, end - pt);
    const bool here = mine && from == pt;
    const bool outputs = __syncthreads_or(here);   // and: the tile before was read
    const uint4 z4 = make_uint4(0, 0, 0, 0);
    for (int i = tid; i < n * (kRow / 8); i += kThr) {
      const int t = i / (kRow / 8), e = i % (kRow / 8) * 8;
      const bool in = e < a.d_k;
      const int64_t p = pt + t;
      *reinterpret_cast<uint4*>(ks + t * kRow + e) =
          in ? __ldg(reinterpret_cast<const uint4*>(k + p * a.k_tok + e)) : z4;
      if (outputs)
        *reinterpret_cast<uint4*>(qs + t * kRow + e) =
            in ? __ldg(reinterpret_cast<const uint4*>(q + p * a.q_tok + e)) : z4;
    }
    for (int i = tid; i < n * (kNV / 8); i += kThr) {
      const int t = i / (kNV / 8), e = i % (kNV / 8) * 8;
      *reinterpret_cast<uint4*>(vs + t * kNV + e) =
          e < nv ? __ldg(reinterpret_cast<const uint4*>(v + int64_t(pt + t) * a.v_tok + e)) : z4;
    }
    if (tid < n) {
      float dt = __ldg(a.dt + (int64_t(r) * a.P + pt + tid) * a.H + h) + bias;
      if (a.softplus) dt = softplus_f(dt);
      al[tid] = make_float2(expf(dt * A), dt);
    }
    __syncthreads();
    if (!__any_sync(kFull, mine && pt < to)) continue;
    if (!__any_sync(kFull, here)) {
#pragma unroll 4
      for (int t = 0; t < n; ++t) step(t);
      continue;
    }
    for (int t = 0; t < n; ++t) {
      step(t);
      uint64_t qq[4], acc = f2(0.f, 0.f);
      pairs(qs + t * kRow + 8 * kg, qq);
#pragma unroll
      for (int j = 0; j < 4; ++j) acc = fma2(S[j], qq[j], acc);
      const float2 h2 = un2(acc);
      float o = group_sum(h2.x + h2.y, 16);
      const int64_t p = pt + t;
      if (!here || kg != 0 || p >= to) continue;
      if (a.D) o = fmaf(D, to_f32(vs[t * kNV + c]), o);
      const int64_t col = int64_t(h) * a.d_v + v0 + c;
      if (a.z)
        o *= silu_f<bf16>(to_f32(
            static_cast<const bf16*>(a.z)[int64_t(r) * a.z_seq + p * a.z_tok + col]));
      static_cast<bf16*>(a.y)[int64_t(r) * a.y_seq + p * a.y_tok + col] = from_f32<bf16>(o);
    }
  }
}

template <int KB, bool FULL, bool GATE>
__global__ void __launch_bounds__(kThr, 1) scan_chunk_kernel(const __grid_constant__ ChunkScan c) {
  using Y = Lay<KB>;
  constexpr int NST = Y::NST;
  extern __shared__ __align__(1024) unsigned char sm[];
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + Y::kBar);
  uint64_t* kq_full = bar;               // [NST] keys and queries landed (TMA bytes)
  uint64_t* kq_free = bar + NST;         // [NST] ... read by the products (one commit per issuer)
  uint64_t* v_full = bar + 2 * NST;      // [NST] values landed (TMA bytes)
  uint64_t* v_done = bar + 3 * NST;      // [NST] y written over the values (NY warps); dS done if !FULL
  uint64_t* sc_full = bar + 4 * NST;     // [NST] scalars written (4 warps)
  uint64_t* sc_free = bar + 5 * NST;     // [NST] scalars read (commits, state and output warps)
  uint64_t* x_done = bar + 6 * NST;      // [NST] values read by the W V warps (8 warps)
  uint64_t* one = bar + 7 * NST;
  uint64_t* xw_full = one + 0;           // [2] W V of 64 tokens written (4 warps)
  uint64_t* xw_free = one + 2;           // [2] ... read by dS (commit)
  uint64_t* ds_full = one + 4;           // dS done
  uint64_t* ds_free = one + 5;           // dS read (NS warps)
  uint64_t* g_full = one + 6;            // G done, and Y1 of the chunk before
  uint64_t* p_full = one + 7;            // G read and P written (8 warps)
  uint64_t* s_full = one + 8;            // state copy written (NS warps)
  uint64_t* y_full = one + 9;            // Y1 and Y2 done
  uint64_t* y_free = one + 10;           // Y1 and Y2 read (NY warps)
  uint64_t* done = one + 11;             // every MMA completed (both issuers)
  uint64_t* p_read = one + 12;           // P read by Y1 (commit)
  volatile uint32_t* bad = reinterpret_cast<uint32_t*>(sm + Y::kBad);   // a state is not finite
  uint32_t* holder = reinterpret_cast<uint32_t*>(sm + Y::kSc);
  const ScanArgs& a = c.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int NY = FULL ? 8 : 4, NS = 12 - NY;       // output and state warps

  // block -> (sequence, head, value columns, piece); neighbours share keys and queries
  const int nseg = FULL ? a.nseg : a.nseg - 1;
  const int tile = blockIdx.x % c.ntile;
  const int rest = blockIdx.x / c.ntile;
  const int rh = rest % (a.R * a.H), seg = rest / (a.R * a.H);
  const int r = rh / a.H, h = rh - r * a.H, g = h / (a.H / a.G);
  const int L = seq_len(a.lens, r, a.P);
  const int64_t pb = int64_t(seg) * a.seg_len;
  const int p0 = int(pb < L ? pb : L), p1 = int(pb + a.seg_len < L ? pb + a.seg_len : L);
  const int nch = (p1 - p0 + kQ - 1) / kQ;
  const int v0 = kNV * tile, nv = min(kNV, a.d_v - v0);
  float* out =                             // the state behind it
      !FULL                           ? a.seg_S + (int64_t(rh) * a.nseg + seg) * a.d_v * a.d_k
      : seg == nseg - 1 && a.S_out ? a.S_out + int64_t(rh) * a.d_v * a.d_k
                                   : nullptr;
  // S_out takes S_in's place: written last, since the second look below reads S_in again
  const bool late = FULL && a.nseg == 1 && a.S_in == a.S_out;
  const float* entering =                  // the state before the piece
      !FULL        ? nullptr
      : a.nseg > 1 ? a.seg_S + (int64_t(rh) * a.nseg + seg) * a.d_v * a.d_k
      : a.S_in     ? a.S_in + int64_t(rh) * a.d_v * a.d_k
                   : nullptr;

  if (smem_u32(sm) & 1023u) {              // the swizzled tiles' alignment; the whole block leaves
    if (tid == 0) report_error(a.err, OLA_ERR_CUDA, 59, 0);
    return;
  }
  if (tid == 0) {
    for (int s = 0; s < NST; ++s) {
      mbar_init(&kq_full[s], 1);
      mbar_init(&kq_free[s], FULL ? 2 : 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&v_done[s], FULL ? NY : 1);
      mbar_init(&x_done[s], 8);
      mbar_init(&sc_full[s], 4);
      mbar_init(&sc_free[s], FULL ? 2 + NY + NS : 1 + NS);
    }
    for (int u = 0; u < 2; ++u) {
      mbar_init(&xw_full[u], 4);
      mbar_init(&xw_free[u], 1);
    }
    mbar_init(ds_full, 1);
    mbar_init(ds_free, NS);
    mbar_init(g_full, 1);
    mbar_init(p_full, 8);
    mbar_init(s_full, NS);
    mbar_init(y_full, 1);
    mbar_init(y_free, NY);
    mbar_init(done, 2);
    mbar_init(p_read, 1);
    *bad = 0;
    fence_barrier_init();
  }
  if (warp == 29) tmem_alloc(holder, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (!FULL) let_next_kernel_start();
  const uint32_t tmem = *holder;
  __syncthreads();                         // read by all before the first scalars take its place
  const uint32_t base = smem_u32(sm);
  const float* scal = reinterpret_cast<const float*>(sm + Y::kSc);

  if (warp >= 28) {
    if (warp == 28) {
      // ---------------------------------------------------------------- product dS
      // A = keys read MN-major (key columns along M; for d_k <= 64 the upper 64 rows read the next
      // tile and are not used), B = the three parts of W V side by side: the keys are read once
      const uint32_t id_d = idesc_bf16_f32_amn(128, 3 * kNV) | (1u << 16);       // A, B MN-major
      bool ok = true;
      for (int i = 0; i < nch; ++i) {
        const int s = i % NST;
        ok = warp_wait(&kq_full[s], i / NST) && (i == 0 || warp_wait(ds_free, i - 1));
#pragma unroll 1
        for (int u = 0; u < 2 && ok; ++u) {              // 64 tokens each
          ok = warp_wait(&xw_full[u], i);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t dk = sw128_mnmajor_desc(base + s * Y::kKQ + u * 8192, kBlk, 1024);
            const uint64_t dx = sw128_mnmajor_desc(base + Y::kXw + u * 8192, kBlk, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16(tmem + kTD, dk + k * 128, dx + k * 128, id_d, u != 0 || k != 0);
            umma_commit(&xw_free[u]);
            if (u == 1) {
              umma_commit(ds_full);
              umma_commit(&kq_free[s]);
              umma_commit(&sc_free[s]);
              if (!FULL) umma_commit(&v_done[s]);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
      }
      if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 60, 0);
      if (elect_one()) umma_commit(done);
      __syncwarp();
    } else if (warp == 29) {
      // ---------------------------------------------------------------- products Y1, G, Y2
      if (FULL) {
        const uint32_t id_g = idesc_bf16_f32(128, 128);
        const uint32_t id_y = idesc_bf16_f32(128, kNV) | (1u << 16);             // B MN-major
        bool ok = true;
#pragma unroll 1
        for (int i = -1; i < nch && ok; ++i) {
          const int s = i < 0 ? 0 : i % NST;
          if (i >= 0) {
            // Y1: A = P in tensor memory, B = the values (rows = tokens)
            ok = warp_wait(p_full, i) && warp_wait(&v_full[s], i / NST) &&
                 (i == 0 || warp_wait(y_free, i - 1));
            // (the values' rows behind the end of a padded sequence are cleared by then)
            if (ok && p1 - (p0 + i * kQ) < kQ) ok = warp_wait(&xw_full[0], i) && warp_wait(&xw_full[1], i);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dv = sw128_mnmajor_desc(base + Y::kV + s * kBlk, kBlk, 1024);
#pragma unroll
              for (int k = 0; k < 8; ++k)
                umma_bf16_ts(tmem + kTY1, tmem + kTG + k * 16, dv + k * 128, id_y, k != 0);
              umma_commit(p_read);
            }
            __syncwarp();
          }
          if (i + 1 < nch) {
            // G of the next chunk: queries x keys. It takes P's place, and products of different
            // shape and accumulator are not ordered by their issue: Y1 has to have read P
            const int s1 = (i + 1) % NST;
            ok = warp_wait(&kq_full[s1], (i + 1) / NST) && (i < 0 || warp_wait(p_read, i));
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dk = sw128_kmajor_desc(base + s1 * Y::kKQ);
              const uint64_t dq = sw128_kmajor_desc(base + s1 * Y::kKQ + Y::kQr);
#pragma unroll
              for (int k = 0; k < 4 * KB; ++k) {
                const uint64_t off = (k >> 2) * (kBlk >> 4) + (k & 3) * 2;
                umma_bf16(tmem + kTG, dq + off, dk + off, id_g, k != 0);
              }
              umma_commit(g_full);
            }
            __syncwarp();
          }
          if (i >= 0) {
            // Y2: A = queries, B = the state copy (rows = key columns)
            ok = warp_wait(s_full, i);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              const uint64_t dq = sw128_kmajor_desc(base + s * Y::kKQ + Y::kQr);
              const uint64_t dsd = sw128_mnmajor_desc(base + Y::kS, kBlk, 1024);
#pragma unroll
              for (int k = 0; k < 4 * KB; ++k)
                umma_bf16(tmem + kTY2, dq + (k >> 2) * (kBlk >> 4) + (k & 3) * 2, dsd + k * 128,
                          id_y, k != 0);
              umma_commit(y_full);
              umma_commit(&kq_free[s]);
              umma_commit(&sc_free[s]);
            }
            __syncwarp();
          }
        }
        if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 61, 0);
      }
      if (elect_one()) umma_commit(done);
      __syncwarp();
      mbar_wait_bounded(done, 0);              // both issuers, before tensor memory is released
      __syncwarp();
    } else if (warp == 30) {
      // ---------------------------------------------------------------- values in, y out
      if (lane == 0) {
        prefetch_tmap(&c.mv);
        auto load = [&](int i) {
          const int s = i % NST;
          mbar_arrive_expect_tx(&v_full[s], kBlk);
          tma_load_4d(sm + Y::kV + s * kBlk, &c.mv, &v_full[s], kNV * tile, h, p0 + i * kQ, r);
        };
        int issued = 0;
        for (; issued < nch && issued < NST; ++issued) load(issued);
        for (int i = 0; i < nch; ++i) {
          const int s = i % NST;
          if (!mbar_wait_bounded(&v_done[s], (i / NST) & 1)) {
            report_error(a.err, OLA_ERR_TIMEOUT, 66, i);
            break;
          }
          // rows past P are clipped; a sequence that ends inside the chunk but before P was
          // stored row by row
          if (FULL && (p0 + (i + 1) * kQ <= p1 || p1 == a.P)) {
            tma_store_4d(&c.my, sm + Y::kV + s * kBlk, kNV * tile, h, p0 + i * kQ, r);
            bulk_commit();
            bulk_wait_read();
          }
          if (issued < nch) load(issued++);
        }
        for (int i = issued > NST ? issued - NST : 0; i < issued; ++i)
          mbar_wait_bounded(&v_full[i % NST], (i / NST) & 1);
        if (FULL) bulk_wait_all();
      }
      __syncwarp();
    } else {
      // ---------------------------------------------------------------- keys, queries
      if (lane == 0) {
        prefetch_tmap(&c.mk);
        if (FULL) prefetch_tmap(&c.mq);
        int issued = 0;
        for (int i = 0; i < nch; ++i) {
          const int s = i % NST, n = i / NST;
          if (n > 0 && !mbar_wait_bounded(&kq_free[s], (n - 1) & 1)) {
            report_error(a.err, OLA_ERR_TIMEOUT, 68, i);
            break;
          }
          mbar_arrive_expect_tx(&kq_full[s], (FULL ? 2 : 1) * KB * kBlk);
          unsigned char* st = sm + s * Y::kKQ;
          const int p = p0 + i * kQ;
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            tma_load_4d(st + b * kBlk, &c.mk, &kq_full[s], 64 * b, g, p, r);
            if (FULL) tma_load_4d(st + Y::kQr + b * kBlk, &c.mq, &kq_full[s], 64 * b, g, p, r);
          }
          issued = i + 1;
        }
        // the copies still in flight land before the block exits
        for (int i = issued > NST ? issued - NST : 0; i < issued; ++i)
          mbar_wait_bounded(&kq_full[i % NST], (i / NST) & 1);
      }
      __syncwarp();
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------------ G -> P
    const int w4 = warp & 3, t = 32 * w4 + lane, c0 = 16 * (warp >> 2);   // columns of a block
    const uint32_t tl = tmem + (uint32_t(32 * w4) << 16);
    // the scalars of chunk i (thread = token): every sum runs over the tokens behind the token, in
    // its block of 32
    const float A2 = a.A[h] * 1.4426950408889634f;
    const float bias = a.dt_bias ? a.dt_bias[h] : 0.f;
    const float* dtp = a.dt + int64_t(r) * a.P * a.H + h;
    auto load_dt = [&](int i) -> float {
      const int p = p0 + i * kQ + t;
      return i < nch && p < p1 ? __ldg(dtp + int64_t(p) * a.H) : 0.f;
    };
    float raw = c0 == 0 ? load_dt(0) : 0.f;
    auto scalars = [&](int i) -> bool {
      const int s = i % NST, n = i / NST;
      // tokens behind the end take no part: dt = 0, no decay
      float dt = raw + bias;
      if (a.softplus) dt = softplus_f(dt);
      // a decay below 2^-256 is 0; the clamp keeps sums of resets finite. It would hide a decay that
      // is not a number (A NaN, or 0 * inf): the token's weight becomes one then
      const float e = dt * A2;
      if (e != e) dt = e;
      float sum = fmaxf(e, -256.f);
      if (t >= p1 - (p0 + i * kQ)) dt = sum = 0.f;   // both: 0 * A is NaN for an infinite A
      raw = load_dt(i + 1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float d = __shfl_down_sync(kFull, sum, o);
        if (lane + o < 32) sum += d;
      }
      float suf = __shfl_down_sync(kFull, sum, 1);
      if (lane == 31) suf = 0.f;
      if (n > 0 && !warp_wait(&sc_free[s], n - 1)) return false;
      float* out = reinterpret_cast<float*>(sm + Y::kSc) + s * kScFloats;
      out[t] = suf;
      out[128 + t] = dt;
      if (w4 < 3) out[256 + t] = dt * ex2(suf);
      if (lane == 0) out[352 + w4] = sum;
      warp_arrive(&sc_full[s]);
      return true;
    };
    bool ok = c0 != 0 || nch == 0 || scalars(0);
    if (!FULL) {
      for (int i = 1; i < nch && ok && c0 == 0; ++i) ok = scalars(i);
      if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 67, 0);
    } else {
      // s <= t within t's own block, as bits of the packed pairs
      uint32_t keep[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        keep[e] = (c0 + 2 * e <= lane ? 0xffffu : 0u) | (c0 + 2 * e + 1 <= lane ? 0xffff0000u : 0u);
      for (int i = 0; i < nch && ok; ++i) {
        const int s = i % NST;
        ok = warp_wait(&sc_full[s], i / NST);
        if (!ok) break;
        const float* suf = scal + s * kScFloats;
        const float* bs = suf + 352;
        const float mine = suf[t];
        ok = warp_wait(g_full, i);
        if (!ok) break;
        tc_fence_after();
        {
          // t's own block of 32 tokens
          const int col = 32 * w4 + c0;
          float x[16];
          tmem_ld16(tl + kTG + col, x);
          const uint64_t neg = f2(-mine, -mine);
          uint32_t p[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const ulonglong2 l2 = *reinterpret_cast<const ulonglong2*>(suf + col + 4 * q);
            const ulonglong2 d2 = *reinterpret_cast<const ulonglong2*>(suf + 128 + col + 4 * q);
            const float2 a0 = un2(add2(l2.x, neg)), a1 = un2(add2(l2.y, neg));
            const uint64_t w0 = mul2(f2(ex2(a0.x), ex2(a0.y)), d2.x);
            const uint64_t w1 = mul2(f2(ex2(a1.x), ex2(a1.y)), d2.y);
            p[2 * q] = pack2(mul2(f2(x[4 * q], x[4 * q + 1]), w0)) & keep[2 * q];
            p[2 * q + 1] = pack2(mul2(f2(x[4 * q + 2], x[4 * q + 3]), w1)) & keep[2 * q + 1];
          }
          tmem_st8(tl + kTG + col, p);
        }
        {
          const uint32_t z[8] = {};
#pragma unroll 1
          for (int j = w4 + 1; j < 4; ++j) tmem_st8(tl + kTG + 32 * j + c0, z);   // s > t
        }
        float mid = bs[w4] - mine;           // log2 decay from the end of block j to t
#pragma unroll 1
        for (int j = w4 - 1; j >= 0; --j) {
          const int col = 32 * j + c0;
          const float rf1 = ex2(mid);
          const uint64_t rf = f2(rf1, rf1);
          mid += bs[j];
          float x[16];
          tmem_ld16(tl + kTG + col, x);
          uint32_t p[8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const ulonglong2 c2 = *reinterpret_cast<const ulonglong2*>(suf + 256 + col + 4 * q);
            p[2 * q] = pack2(mul2(f2(x[4 * q], x[4 * q + 1]), mul2(rf, c2.x)));
            p[2 * q + 1] = pack2(mul2(f2(x[4 * q + 2], x[4 * q + 3]), mul2(rf, c2.y)));
          }
          tmem_st8(tl + kTG + col, p);
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(p_full);
        if (c0 == 0 && i + 1 < nch) ok = scalars(i + 1);
      }
      if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 62, 0);
    }
  } else if (warp >= 16 && warp < 24) {
    // ------------------------------------------------------------------ W V
    const int w4 = warp & 3, t = 32 * w4 + lane, q0 = 4 * ((warp - 16) >> 2);
    bool ok = true;
    for (int i = 0; i < nch; ++i) {
      const int s = i % NST, n = i / NST;
      const bool live = t < p1 - (p0 + i * kQ);
      ok = warp_wait(&sc_full[s], n);
      if (!ok) break;
      const float* suf = scal + s * kScFloats;
      float after = suf[t];
      for (int j = w4 + 1; j < 4; ++j) after += suf[352 + j];
      const float w1 = suf[128 + t] * exp2f(after);
      const uint64_t w = f2(w1, w1);
      ok = warp_wait(&v_full[s], n) && (i == 0 || warp_wait(&xw_free[w4 >> 1], i - 1));
      if (!ok) break;
      unsigned char* vrow = sm + Y::kV + s * kBlk + t * 128;
      unsigned char* xrow = sm + Y::kXw + t * 128;
      if (p1 - (p0 + i * kQ) < kQ) {
        // padding may hold anything, also NaN: its key and value rows are cleared
        ok = warp_wait(&kq_full[s], n);
        if (!ok) break;
        if (!live) {
          const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll 1
          for (int q = q0; q < q0 + 4; ++q) {
            const uint32_t off = uint32_t((q ^ (t & 7)) << 4);
            *reinterpret_cast<uint4*>(vrow + off) = z;
#pragma unroll
            for (int b = 0; b < KB; ++b)
              *reinterpret_cast<uint4*>(sm + s * Y::kKQ + b * kBlk + t * 128 + off) = z;
          }
        }
      }
      // a product of 24 bits is its upper 8 bits, the next 8 and the rest, each cut off exactly
      uint4 nx = *reinterpret_cast<const uint4*>(vrow + ((q0 ^ (t & 7)) << 4));
#pragma unroll 1
      for (int q = q0; q < q0 + 4; ++q) {
        const uint32_t off = uint32_t((q ^ (t & 7)) << 4);
        const uint32_t vw[4] = {nx.x, nx.y, nx.z, nx.w};
        if (q + 1 < q0 + 4) nx = *reinterpret_cast<const uint4*>(vrow + (((q + 1) ^ (t & 7)) << 4));
        uint32_t h1[4], h2[4], h3[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t sign = 0x80000000u;
          const uint64_t f = mul2(u2(vw[e] << 16, vw[e] & 0xffff0000u), w);
          const float2 ff = un2(f);
          const uint32_t a0 = __float_as_uint(ff.x), a1 = __float_as_uint(ff.y);
          h1[e] = __byte_perm(a0, a1, 0x7632);
          const uint64_t r =
              add2(f, u2((a0 & 0xffff0000u) ^ sign, (a1 & 0xffff0000u) ^ sign));
          const float2 rr = un2(r);
          const uint32_t b0 = __float_as_uint(rr.x), b1 = __float_as_uint(rr.y);
          h2[e] = __byte_perm(b0, b1, 0x7632);
          const float2 uu = un2(
              add2(r, u2((b0 & 0xffff0000u) ^ sign, (b1 & 0xffff0000u) ^ sign)));
          h3[e] = __byte_perm(__float_as_uint(uu.x), __float_as_uint(uu.y), 0x7632);
        }
        *reinterpret_cast<uint4*>(xrow + off) = make_uint4(h1[0], h1[1], h1[2], h1[3]);
        *reinterpret_cast<uint4*>(xrow + kBlk + off) = make_uint4(h2[0], h2[1], h2[2], h2[3]);
        *reinterpret_cast<uint4*>(xrow + 2 * kBlk + off) = make_uint4(h3[0], h3[1], h3[2], h3[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&xw_full[w4 >> 1]);
        if (FULL) mbar_arrive(&x_done[s]);
      }
    }
    if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 63, 0);
  } else if (FULL ? warp >= 24 : warp < 16) {
    // ------------------------------------------------------------------ state rows
    const int w4 = warp & 3, k = 32 * w4 + lane;
    // 8-column pieces of this warp
    constexpr int kPer = NS == 8 ? 4 : 8;
    const int qb = NS == 8 ? 4 * ((warp - 8) >> 2) : 0;
    const uint32_t tl = tmem + (uint32_t(32 * w4) << 16);
    const bool mine = k < a.d_k, holds = k < 64 * KB;    // a key column, a row of the copy
    if (FULL && a.nseg > 1) wait_for_previous_kernel();    // the state before this piece
    unsigned char* row = sm + Y::kS + k * 128;             // the copy: 64 columns, 128-byte swizzle
    auto copy8 = [&](int q, const uint32_t (&x)[8]) {
      if (holds)
        *reinterpret_cast<uint4*>(row + ((q ^ (k & 7)) << 4)) =
            make_uint4(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                       pack2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                       pack2(__uint_as_float(x[4]), __uint_as_float(x[5])),
                       pack2(__uint_as_float(x[6]), __uint_as_float(x[7])));
    };
#pragma unroll 1
    for (int q = qb; q < qb + kPer; ++q) {
      uint32_t x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = entering && mine && 8 * q + e < nv
                   ? __float_as_uint(entering[int64_t(v0 + 8 * q + e) * a.d_k + k])
                   : 0u;
      tmem_st8(tl + kTS + 8 * q, x);
      if (FULL) copy8(q, x);
    }
    tmem_st_wait();
    tc_fence_before();
    if (FULL) fence_proxy_async_smem();
    warp_arrive(s_full);
    double logsum = 0.0;
    bool ok = true;
    for (int i = 0; i < nch; ++i) {
      const int s = i % NST;
      ok = warp_wait(&sc_full[s], i / NST);
      if (!ok) break;
      const float4 b4 = *reinterpret_cast<const float4*>(scal + s * kScFloats + 352);
      const float total = (b4.x + b4.y) + (b4.z + b4.w);
      warp_arrive(&sc_free[s]);
      if (!FULL) logsum += double(total);
      // e^{c_C} S as S + (e^{c_C} - 1) S where the decay is slow, so that it is not rounded chunk
      // after chunk; a fast decay would cancel in that form and is taken as it is
      const float ex = total * 0.69314718055994531f;
      const bool slow = ex > -0.5f;
      const float mul1 = slow ? expm1f(ex) : expf(ex), keep1 = slow ? 1.f : 0.f;
      const uint64_t mul = f2(mul1, mul1), keep = f2(keep1, keep1);
      ok = warp_wait(ds_full, i) && (!FULL || warp_wait(y_full, i));
      if (!ok) break;
      tc_fence_after();
#pragma unroll 1
      for (int q = qb; q < qb + kPer; ++q) {
        uint32_t d0[8], d1[8], d2[8], old[8], x[8];
        tmem_ld8x4(tl + kTD + 8 * q, d0, d1, d2, tl + kTS + 8 * q, old);
        if (q + 1 == qb + kPer) {
          tc_fence_before();
          warp_arrive(ds_free);
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          const uint64_t own = add2(u2(d0[e], d0[e + 1]),
                                    add2(u2(d1[e], d1[e + 1]), u2(d2[e], d2[e + 1])));
          const uint64_t o = u2(old[e], old[e + 1]);
          const float2 n2 = un2(fma2(mul, o, fma2(keep, o, own)));
          x[e] = __float_as_uint(n2.x);
          x[e + 1] = __float_as_uint(n2.y);
        }
        tmem_st8(tl + kTS + 8 * q, x);
        if (FULL) copy8(q, x);
      }
      tmem_st_wait();
      tc_fence_before();
      if (FULL) fence_proxy_async_smem();
      warp_arrive(s_full);
    }
    if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 64, 0);
    if (out || FULL) {
      uint64_t odd = f2(0.f, 0.f);           // NaN once an element is not finite
#pragma unroll 1
      for (int q = qb / 2; q < (qb + kPer) / 2; ++q) {
        float x[16];
        tmem_ld16(tl + kTS + 16 * q, x);
        if (out && !late) {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (mine && 16 * q + e < nv) out[int64_t(v0 + 16 * q + e) * a.d_k + k] = x[e];
        }
        if (FULL) {
#pragma unroll
          for (int e = 0; e < 16; e += 2) odd = fma2(f2(x[e], x[e + 1]), f2(0.f, 0.f), odd);
        }
      }
      const float2 o2 = un2(odd);
      if (FULL && mine && o2.x + o2.y != 0.f) *bad = 1;
      __syncwarp();
    }
    if (!FULL && tile == 0 && k == 0 && qb == 0)
      a.seg_a[int64_t(rh) * a.nseg + seg] = float(exp2(logsum));
  } else {
    // ------------------------------------------------------------------ outputs
    if (FULL) {
      const int w4 = warp & 3, t = 32 * w4 + lane;
      constexpr int kPer = NY == 8 ? 2 : 4;             // 16-column pieces of this warp
      const int hb = NY == 8 ? 2 * ((warp - 8) >> 2) : 0;
      const uint32_t tl = tmem + (uint32_t(32 * w4) << 16);
      const bool skip = a.D != nullptr;
      const float D = skip ? a.D[h] : 0.f;
      const uint64_t D2 = f2(D, D);
      const __nv_bfloat16* zp =
          GATE ? static_cast<const __nv_bfloat16*>(a.z) + int64_t(r) * a.z_seq +
                     int64_t(h) * a.d_v + v0
               : nullptr;
      __nv_bfloat16* yp = static_cast<__nv_bfloat16*>(a.y) + int64_t(r) * a.y_seq +
                          int64_t(h) * a.d_v + v0;
      bool ok = true;
      for (int i = 0; i < nch; ++i) {
        const int s = i % NST;
        const int p = p0 + i * kQ + t;
        const bool live = p < p1;
        const uint4* zrow = reinterpret_cast<const uint4*>(GATE ? zp + int64_t(p) * a.z_tok : nullptr);
        if (GATE && live) {
          // the row's four sectors on their way to L1 while the products run
#pragma unroll
          for (int q = hb; q < hb + kPer; ++q)
            if (16 * q < nv) asm volatile("prefetch.global.L1 [%0];" ::"l"(zrow + 2 * q));
        }
        ok = warp_wait(&sc_full[s], i / NST);
        if (!ok) break;
        const float* suf = scal + s * kScFloats;
        float cum = suf[352 + w4] - suf[t];
        for (int j = 0; j < w4; ++j) cum += suf[352 + j];
        const float ec = ex2(cum);
        const uint64_t ec2 = f2(ec, ec);
        warp_arrive(&sc_free[s]);
        unsigned char* vrow = sm + Y::kV + s * kBlk + t * 128;
        const bool by_tma = p0 + (i + 1) * kQ <= p1 || p1 == a.P;
        ok = warp_wait(y_full, i) && warp_wait(&x_done[s], i / NST);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int hq = hb; hq < hb + kPer; ++hq) {   // 16 columns, two 16-byte pieces of a row
          uint4 z4[2], v4[2];
          unsigned char* at[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int q = 2 * hq + u;
            at[u] = vrow + ((q ^ (t & 7)) << 4);
            z4[u] = v4[u] = make_uint4(0, 0, 0, 0);
            if (GATE && live && 8 * q < nv) z4[u] = __ldg(zrow + q);
            if (skip) v4[u] = *reinterpret_cast<const uint4*>(at[u]);
          }
          uint32_t x1[16], x2[16];
          tmem_ld16x2(tl + kTY1 + 16 * hq, tl + kTY2 + 16 * hq, x1, x2);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t vw[4] = {v4[u].x, v4[u].y, v4[u].z, v4[u].w};
            const uint32_t zw[4] = {z4[u].x, z4[u].y, z4[u].z, z4[u].w};
            uint32_t ow[4];
            uint64_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int b = 8 * u + 2 * e;
              o[e] = fma2(ec2, u2(x2[b], x2[b + 1]), u2(x1[b], x1[b + 1]));
            }
            if (skip) {
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = fma2(D2, u2(vw[e] << 16, vw[e] & 0xffff0000u), o[e]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (GATE)
                o[e] = mul2(o[e], silu2<__nv_bfloat16>(u2(zw[e] << 16, zw[e] & 0xffff0000u)));
              ow[e] = pack2(o[e]);
            }
            const uint4 o4 = make_uint4(ow[0], ow[1], ow[2], ow[3]);
            if (by_tma)
              *reinterpret_cast<uint4*>(at[u]) = o4;
            else if (live && 8 * (2 * hq + u) < nv)
              *(reinterpret_cast<uint4*>(yp + int64_t(p) * a.y_tok) + 2 * hq + u) = o4;
          }
        }
        tc_fence_before();
        warp_arrive(y_free);
        fence_proxy_async_smem();
        warp_arrive(&v_done[s]);
      }
      if (!ok && lane == 0) report_error(a.err, OLA_ERR_TIMEOUT, 65, 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (FULL && *bad) {
    // every output has been stored by now
    second_look(a, entering, sm, r, h, g, v0, nv, p0, p1);
    __syncthreads();
  }
  if (late && out && warp >= 24 && warp < 28) {
    const int w4 = warp & 3, k = 32 * w4 + lane;
#pragma unroll 1
    for (int q = 0; q < kNV / 16; ++q) {
      float x[16];
      tmem_ld16(tmem + (uint32_t(32 * w4) << 16) + kTS + 16 * q, x);
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (k < a.d_k && 16 * q + e < nv) out[int64_t(v0 + 16 * q + e) * a.d_k + k] = x[e];
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 29) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------- host side

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                             const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                             const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn map_encoder() {
  static std::atomic<EncodeFn> fn{nullptr};
  EncodeFn f = fn.load(std::memory_order_acquire);
  if (!f) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess) {
      f = reinterpret_cast<EncodeFn>(p);
      fn.store(f, std::memory_order_release);
    }
  }
  return f;
}

// [R][P][heads][d] bf16 with the given strides as a 4-D map (column, head, token, sequence) of
// 64 x 1 x 128 x 1 boxes, 128-byte swizzle. Columns past d and tokens past P read 0 and are not
// written.
bool rows_map(CUtensorMap* map, const void* base, int d, int heads, int P, int R, int64_t tok,
              int64_t seq) {
  EncodeFn fn = map_encoder();
  if (!fn) return false;
  cuuint64_t dims[4] = {cuuint64_t(d), cuuint64_t(heads), cuuint64_t(P), cuuint64_t(R)};
  cuuint64_t strides[3] = {cuuint64_t(d) * 2, cuuint64_t(tok) * 2, cuuint64_t(seq) * 2};
  cuuint32_t box[4] = {64, 1, kQ, 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int KB>
cudaError_t run(const ChunkScan& c, cudaStream_t st) {
  constexpr uint32_t bytes = Lay<KB>::kBytes;
  static std::atomic<uint64_t> set{0};
  cudaError_t e = once_per_device(set, [&] {
    cudaError_t x = cudaSuccess;
    for (auto f : {scan_chunk_kernel<KB, true, true>, scan_chunk_kernel<KB, true, false>,
                   scan_chunk_kernel<KB, false, false>})
      if (x == cudaSuccess)
        x = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    return x;
  });
  if (e != cudaSuccess) return e;
  const int64_t chains = int64_t(c.a.R) * c.a.H * c.ntile;
  if (c.a.nseg > 1) {
    scan_chunk_kernel<KB, false, false>
        <<<unsigned(chains * (c.a.nseg - 1)), kThr, bytes, st>>>(c);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if ((e = launch_scan_join(c.a, st)) != cudaSuccess) return e;
  }
  const unsigned grid = unsigned(chains * c.a.nseg);
  auto full = c.a.z ? scan_chunk_kernel<KB, true, true> : scan_chunk_kernel<KB, true, false>;
  // the outputs of a piece can start before its entering state is there
  if (c.a.nseg > 1) return launch_dependent(full, grid, kThr, bytes, st, c);
  full<<<grid, kThr, bytes, st>>>(c);
  return cudaGetLastError();
}

}  // namespace

bool scan_chunk_supported(const ScanArgs& a, int in_dtype) {
  if (in_dtype != OLA_BF16 || a.d_k > 128 || a.P < 1) return false;
  // 16-byte rows, strides within the tensor map's 2^40 bytes
  auto ok = [&](const void* p, int64_t tok, int64_t seq) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && tok % 8 == 0 && seq % 8 == 0 &&
           tok < (int64_t(1) << 39) && seq < (int64_t(1) << 39);
  };
  return ok(a.v, a.v_tok, a.v_seq) && ok(a.k, a.k_tok, a.k_seq) && ok(a.q, a.q_tok, a.q_seq) &&
         ok(a.y, a.y_tok, a.y_seq) && (!a.z || ok(a.z, a.z_tok, a.z_seq));
}

// Pieces: one block runs per SM, so a batch that leaves at least half of them idle is cut into as
// many pieces as fill them.
void scan_chunk_pieces(int R, int P, int H, int d_v, int sms, int* nseg, int* seg_len) {
  const int64_t chains = int64_t(R) * H * ((d_v + kNV - 1) / kNV);
  const int64_t chunks = (int64_t(P) + kQ - 1) / kQ;
  int64_t want = sms / chains;
  if (want > chunks) want = chunks;
  if (want < 2) want = 1;
  const int64_t per = want > 0 ? (chunks + want - 1) / want : 1;
  *seg_len = int((per < 1 ? 1 : per) * kQ);
  *nseg = int((int64_t(P) + *seg_len - 1) / *seg_len);
  if (*nseg < 1) *nseg = 1;
}

cudaError_t launch_scan_chunk(const ScanArgs& a, cudaStream_t st) {
  ChunkScan c;
  c.a = a;
  c.ntile = (a.d_v + kNV - 1) / kNV;
  if (!rows_map(&c.mv, a.v, a.d_v, a.H, a.P, a.R, a.v_tok, a.v_seq) ||
      !rows_map(&c.mk, a.k, a.d_k, a.G, a.P, a.R, a.k_tok, a.k_seq) ||
      !rows_map(&c.mq, a.q, a.d_k, a.G, a.P, a.R, a.q_tok, a.q_seq) ||
      !rows_map(&c.my, a.y, a.d_v, a.H, a.P, a.R, a.y_tok, a.y_seq))
    return cudaErrorInvalidValue;
  return a.d_k <= 64 ? run<1>(c, st) : run<2>(c, st);
}

}  // namespace ola
