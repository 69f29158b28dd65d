// Host side of the operators around the recurrence declared in include/ola.h: argument checks,
// dispatch, and the per-device error word that their kernels report to.
#include <atomic>
#include <initializer_list>
#include <mutex>

#include "ola_layer.cuh"
#include "ola_rows.h"

using namespace ola;

// The code of the first error recorded since it was last read, which ola_layer_status returns; its
// detail and index (see report_error) lie beside it for a debugger.
static __device__ int g_layer_err[4];
// what status calls took from it, a slot for each call under way
constexpr int kTaken = 1024;
static __device__ int g_layer_taken[kTaken];

namespace {

constexpr int kMaxDevices = 64;

ola_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return OLA_OK;
  cudaGetLastError();
  if (e == cudaErrorMemoryAllocation) return OLA_ERR_OOM;
  return e == cudaErrorInvalidConfiguration ? OLA_ERR_UNSUPPORTED : OLA_ERR_CUDA;
}

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool width_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128 || d == 256; }

// Reads and clears the error code in one step, so that each recorded error goes to one caller.
__global__ void take_error_kernel(int slot) { g_layer_taken[slot] = atomicExch(g_layer_err, 0); }

// Device address of the error word, resolved once per device; refuses devices the library was
// not built for.
ola_status error_word(int** out) {
  static std::mutex mu;
  static int* addr[kMaxDevices] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return from_cuda(e);
  if (dev < 0 || dev >= kMaxDevices) return OLA_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(mu);
  if (!addr[dev]) {
    int major = 0;
    e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (e != cudaSuccess) return from_cuda(e);
    if (major != 10) return OLA_ERR_UNSUPPORTED;
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_layer_err);
    if (e != cudaSuccess) return from_cuda(e);
    addr[dev] = static_cast<int*>(p);
  }
  *out = addr[dev];
  return OLA_OK;
}

bool on16(const Rows& t) {
  return !t.p || (aligned(t.p, 16) && (t.tok * t.e) % 16 == 0 && (t.seq * t.e) % 16 == 0);
}

bool dtype_ok(int t) { return t == OLA_F32 || t == OLA_BF16; }

// Checks shared by the two convolutions; fills `a` (without the state) and says whether every row
// is 16-byte aligned.
ola_status conv_args(const ola_conv_desc* d, const void* x, const float* w, const float* bias,
                     void* y, ConvArgs* a, Rows* rx, Rows* ry) {
  if (!d || !w) return OLA_ERR_INVALID_ARG;
  if (d->R < 1 || d->P < 0 || d->C < 1 || !dtype_ok(d->in_dtype) || (d->silu & ~1))
    return OLA_ERR_INVALID_ARG;
  // token indices, and those of a tile past the end, are 32-bit
  if (d->W < 2 || d->W > 4 || d->P > (1 << 30)) return OLA_ERR_UNSUPPORTED;
  if (d->P > 0 && (!x || !y)) return OLA_ERR_INVALID_ARG;
  const int e = d->in_dtype == OLA_BF16 ? 2 : 4;
  *rx = Rows{x, d->R, d->P, d->x_tok, d->x_seq, d->C, e};
  *ry = Rows{y, d->R, d->P, d->y_tok, d->y_seq, d->C, e};
  if (!strides(rx, false) || !strides(ry, true)) return OLA_ERR_INVALID_ARG;
  if (!aligned(x, e) || !aligned(y, e) || !aligned(w, 4) || !aligned(bias, 4))
    return OLA_ERR_INVALID_ARG;
  if (overlap(*rx, *ry)) return OLA_ERR_INVALID_ARG;
  if (overlap(*ry, flat(w, int64_t(d->C) * d->W, 4)) || (bias && overlap(*ry, flat(bias, d->C, 4))))
    return OLA_ERR_INVALID_ARG;
  *a = ConvArgs{};
  a->R = d->R;
  a->P = d->P;
  a->C = d->C;
  a->silu = d->silu;
  a->x_tok = rx->tok;
  a->x_seq = rx->seq;
  a->y_tok = ry->tok;
  a->y_seq = ry->seq;
  a->x = x;
  a->w = w;
  a->bias = bias;
  a->y = y;
  return OLA_OK;
}

// Checks shared by the two scans; fills `a` without the states.
ola_status scan_shape(const ola_scan_desc* d) {
  if (!d) return OLA_ERR_INVALID_ARG;
  if (d->R < 1 || d->P < 0 || d->H < 1 || d->G < 1 || d->H % d->G || !dtype_ok(d->in_dtype) ||
      (d->softplus & ~1))
    return OLA_ERR_INVALID_ARG;
  if (!width_ok(d->d_k) || !width_ok(d->d_v)) return OLA_ERR_UNSUPPORTED;
  // blocks and (sequence, head, piece) indices are 32-bit
  if (int64_t(d->R) * d->H > (int64_t(1) << 24) || d->P > (1 << 30)) return OLA_ERR_UNSUPPORTED;
  return OLA_OK;
}

struct ScanRows {
  Rows v, k, q, z, y;
};

ola_status scan_args(const ola_scan_desc* d, const void* v, const float* dt, const float* A,
                     const void* k, const void* q, const float* D, const float* dt_bias,
                     const void* z, void* y, ScanArgs* a, ScanRows* t) {
  ola_status s = scan_shape(d);
  if (s != OLA_OK) return s;
  if (!A) return OLA_ERR_INVALID_ARG;
  if (d->P > 0 && (!v || !dt || !k || !q || !y)) return OLA_ERR_INVALID_ARG;
  const int e = d->in_dtype == OLA_BF16 ? 2 : 4;
  const int64_t wv = int64_t(d->H) * d->d_v, wk = int64_t(d->G) * d->d_k;
  t->v = Rows{v, d->R, d->P, d->v_tok, d->v_seq, wv, e};
  t->k = Rows{k, d->R, d->P, d->k_tok, d->k_seq, wk, e};
  t->q = Rows{q, d->R, d->P, d->q_tok, d->q_seq, wk, e};
  t->z = Rows{z, d->R, d->P, d->z_tok, d->z_seq, wv, e};
  t->y = Rows{y, d->R, d->P, d->y_tok, d->y_seq, wv, e};
  for (Rows* x : {&t->v, &t->k, &t->q, &t->z, &t->y}) {
    if (!strides(x, x == &t->y) || !aligned(x->p, e)) return OLA_ERR_INVALID_ARG;
    if (x != &t->y && overlap(*x, t->y)) return OLA_ERR_INVALID_ARG;
  }
  for (const float* x : {dt, A, D, dt_bias})
    if (!aligned(x, 4)) return OLA_ERR_INVALID_ARG;
  if (d->P > 0 && overlap(t->y, flat(dt, int64_t(d->R) * d->P * d->H, 4)))
    return OLA_ERR_INVALID_ARG;
  *a = ScanArgs{};
  a->R = d->R;
  a->P = d->P;
  a->H = d->H;
  a->G = d->G;
  a->d_k = d->d_k;
  a->d_v = d->d_v;
  a->softplus = d->softplus;
  a->nseg = 1;
  a->seg_len = d->P > 0 ? d->P : 1;
  a->v_tok = t->v.tok, a->v_seq = t->v.seq;
  a->k_tok = t->k.tok, a->k_seq = t->k.seq;
  a->q_tok = t->q.tok, a->q_seq = t->q.seq;
  a->z_tok = t->z.tok, a->z_seq = t->z.seq;
  a->y_tok = t->y.tok, a->y_seq = t->y.seq;
  a->v = v;
  a->dt = dt;
  a->A = A;
  a->k = k;
  a->q = q;
  a->D = D;
  a->dt_bias = dt_bias;
  a->z = z;
  a->y = y;
  return OLA_OK;
}

// Scratch layout: the pieces' states, then their decays.
uint64_t ws_bytes_for(const ola_scan_desc* d, int nseg) {
  if (nseg < 2) return 0;
  const uint64_t rh = uint64_t(d->R) * d->H * nseg;
  return rh * d->d_v * d->d_k * 4 + (rh * 4 + 15) / 16 * 16;
}

// SM count for the choice of pieces; without a device (host-only queries) a B200's.
int sm_count() {
  int n = 0;
  if (device_sm_count(&n) != cudaSuccess) {
    cudaGetLastError();
    return 148;
  }
  return n;
}

}  // namespace

extern "C" {

ola_status ola_layer_status(void* stream) {
  int* err = nullptr;
  ola_status s = error_word(&err);
  if (s != OLA_OK) return s;
  static std::atomic<unsigned> calls{0};
  const int slot = int(calls.fetch_add(1, std::memory_order_relaxed) % kTaken);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int code = 0;
  take_error_kernel<<<1, 1, 0, st>>>(slot);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = cudaMemcpyFromSymbolAsync(&code, g_layer_taken, sizeof(int), slot * sizeof(int),
                                  cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return from_cuda(e);
  return static_cast<ola_status>(code);
}

ola_status ola_conv(const ola_conv_desc* d, const void* x, const float* w, const float* bias,
                    const void* state_in, const int32_t* lens, void* y, void* state_out,
                    void* stream) {
  ConvArgs a;
  Rows rx, ry;
  ola_status s = conv_args(d, x, w, bias, y, &a, &rx, &ry);
  if (s != OLA_OK) return s;
  int64_t n;
  if (!elements({d->R, d->W - 1, d->C}, &n)) return OLA_ERR_UNSUPPORTED;
  const Rows si = flat(state_in, n, rx.e), so = flat(state_out, n, rx.e);
  if (!aligned(state_in, rx.e) || !aligned(state_out, rx.e) || !aligned(lens, 4))
    return OLA_ERR_INVALID_ARG;
  if (overlap(rx, so) || overlap(ry, si) || overlap(ry, so)) return OLA_ERR_INVALID_ARG;
  if (state_in != state_out && overlap(si, so)) return OLA_ERR_INVALID_ARG;
  if (d->P == 0 && !state_out) return OLA_OK;
  s = error_word(&a.err);
  if (s != OLA_OK) return s;
  a.state_in = state_in;
  a.lens = lens;
  a.state_out = state_out;
  const bool wide = on16(rx) && on16(ry) && (int64_t(d->C) * rx.e) % 16 == 0 &&
                    aligned(state_in, 16) && aligned(state_out, 16);
  return from_cuda(launch_conv(a, d->in_dtype, d->W, wide, static_cast<cudaStream_t>(stream)));
}

ola_status ola_conv_step(const ola_conv_desc* d, int32_t Bp, const void* x, const float* w,
                         const float* bias, const void* state_in, const int32_t* parent_idx,
                         void* y, void* state_out, void* stream) {
  ConvArgs a;
  Rows rx, ry;
  ola_status s = conv_args(d, x, w, bias, y, &a, &rx, &ry);
  if (s != OLA_OK) return s;
  if (d->P < 1 || Bp < 1 || !state_in || !state_out) return OLA_ERR_INVALID_ARG;
  if (!parent_idx && Bp != 1 && Bp != d->P) return OLA_ERR_INVALID_ARG;
  int64_t ni, no;
  if (!elements({d->R, Bp, d->W - 1, d->C}, &ni) || !elements({d->R, d->P, d->W - 1, d->C}, &no))
    return OLA_ERR_UNSUPPORTED;
  const Rows si = flat(state_in, ni, rx.e), so = flat(state_out, no, rx.e);
  if (!aligned(state_in, rx.e) || !aligned(state_out, rx.e) || !aligned(parent_idx, 4))
    return OLA_ERR_INVALID_ARG;
  if (overlap(rx, so) || overlap(ry, si) || overlap(ry, so)) return OLA_ERR_INVALID_ARG;
  const bool in_place = state_in == state_out && !parent_idx && Bp == d->P;
  if (!in_place && overlap(si, so)) return OLA_ERR_INVALID_ARG;
  s = error_word(&a.err);
  if (s != OLA_OK) return s;
  a.Bp = Bp;
  a.state_in = state_in;
  a.parent = parent_idx;
  a.state_out = state_out;
  const bool wide = on16(rx) && on16(ry) && (int64_t(d->C) * rx.e) % 16 == 0 &&
                    aligned(state_in, 16) && aligned(state_out, 16);
  return from_cuda(
      launch_conv_step(a, d->in_dtype, d->W, wide, static_cast<cudaStream_t>(stream)));
}

ola_status ola_qk_norm(const ola_qk_desc* d, const void* q, const void* k, const float* wq,
                       const float* wk, const int32_t* positions, const float* inv_freq,
                       void* q_out, void* k_out, void* stream) {
  if (!d) return OLA_ERR_INVALID_ARG;
  if (d->N < 0 || d->Hq < 0 || d->Hk < 0 || d->d < 1 || !dtype_ok(d->in_dtype) || (d->l2 & ~1) ||
      (d->pair & ~1) || !(d->eps >= 0.f))
    return OLA_ERR_INVALID_ARG;
  if (d->d % 8 || d->d > 512 || d->rot < 0 || d->rot % 16 || d->rot > d->d)
    return OLA_ERR_UNSUPPORTED;
  if (int64_t(d->Hq) + d->Hk > (1 << 20)) return OLA_ERR_UNSUPPORTED;
  const int e = d->in_dtype == OLA_BF16 ? 2 : 4;
  Rows rq{q, 1, d->N, d->q_tok, 0, int64_t(d->Hq) * d->d, e};
  Rows rk{k, 1, d->N, d->k_tok, 0, int64_t(d->Hk) * d->d, e};
  Rows oq{q_out, 1, d->N, d->qo_tok, 0, rq.width, e};
  Rows ok{k_out, 1, d->N, d->ko_tok, 0, rk.width, e};
  for (Rows* x : {&rq, &rk, &oq, &ok}) {
    if (x->width == 0) x->p = nullptr;
    if (x->width > 0 && d->N > 0 && !x->p) return OLA_ERR_INVALID_ARG;
    if (!strides(x, x == &oq || x == &ok)) return OLA_ERR_INVALID_ARG;
    // one sequence: its stride is not used
    if (x->p && (!aligned(x->p, 16) || (x->tok * e) % 16)) return OLA_ERR_INVALID_ARG;
  }
  for (const float* x : {wq, wk, inv_freq})
    if (!aligned(x, 4)) return OLA_ERR_INVALID_ARG;
  if (!aligned(positions, 4)) return OLA_ERR_INVALID_ARG;
  if (d->rot && d->N > 0 && (!positions || !inv_freq)) return OLA_ERR_INVALID_ARG;
  // a head may be replaced in place; any other sharing is refused
  const bool same_q = q == q_out && rq.tok == oq.tok, same_k = k == k_out && rk.tok == ok.tok;
  if ((!same_q && overlap(rq, oq)) || (!same_k && overlap(rk, ok)) || overlap(rq, ok) ||
      overlap(rk, oq) || overlap(oq, ok))
    return OLA_ERR_INVALID_ARG;
  if (d->N == 0 || d->Hq + d->Hk == 0) return OLA_OK;
  int* err = nullptr;
  ola_status s = error_word(&err);
  if (s != OLA_OK) return s;
  QkArgs a{};
  a.N = d->N;
  a.Hq = d->Hq;
  a.Hk = d->Hk;
  a.d = d->d;
  a.rot = d->rot;
  a.l2 = d->l2;
  a.eps = d->eps;
  a.q_tok = rq.tok;
  a.k_tok = rk.tok;
  a.qo_tok = oq.tok;
  a.ko_tok = ok.tok;
  a.q = rq.p;
  a.k = rk.p;
  a.wq = wq;
  a.wk = wk;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.k_out = k_out;
  return from_cuda(launch_qk_norm(a, d->in_dtype, d->pair, static_cast<cudaStream_t>(stream)));
}

ola_status ola_scan_workspace_bytes(const ola_scan_desc* d, uint64_t* out_bytes) {
  if (!out_bytes) return OLA_ERR_INVALID_ARG;
  ola_status s = scan_shape(d);
  if (s != OLA_OK) return s;
  // enough for either form, so that it does not hang on the pointers' alignment
  int n = 1, len = 0;
  const int sms = sm_count();
  scan_tok_pieces(d->R, d->P, d->H, d->d_v, sms, &n, &len);
  if (d->in_dtype == OLA_BF16) {
    int n2 = 1;
    scan_chunk_pieces(d->R, d->P, d->H, d->d_v, sms, &n2, &len);
    n = n2 > n ? n2 : n;
  }
  *out_bytes = ws_bytes_for(d, n);
  return OLA_OK;
}

ola_status ola_scan(const ola_scan_desc* d, const void* v, const float* dt, const float* A,
                    const void* k, const void* q, const float* D, const float* dt_bias,
                    const void* z, const float* S_in, const int32_t* lens, void* y, float* S_out,
                    void* ws, uint64_t ws_bytes, void* stream) {
  ScanArgs a;
  ScanRows t;
  ola_status s = scan_args(d, v, dt, A, k, q, D, dt_bias, z, y, &a, &t);
  if (s != OLA_OK) return s;
  const int64_t n = int64_t(d->R) * d->H * d->d_v * d->d_k;
  const Rows si = flat(S_in, n, 4), so = flat(S_out, n, 4);
  if (!aligned(S_in, 4) || !aligned(S_out, 4) || !aligned(lens, 4)) return OLA_ERR_INVALID_ARG;
  if (S_in != S_out && overlap(si, so)) return OLA_ERR_INVALID_ARG;
  for (const Rows* x : {&t.v, &t.k, &t.q, &t.z, &t.y})
    if (overlap(*x, so)) return OLA_ERR_INVALID_ARG;
  if (overlap(t.y, si)) return OLA_ERR_INVALID_ARG;
  const bool chunked = scan_chunk_supported(a, d->in_dtype);
  if (chunked)
    scan_chunk_pieces(d->R, d->P, d->H, d->d_v, sm_count(), &a.nseg, &a.seg_len);
  else
    scan_tok_pieces(d->R, d->P, d->H, d->d_v, sm_count(), &a.nseg, &a.seg_len);
  const uint64_t need = ws_bytes_for(d, a.nseg);
  if (need) {
    if (!ws || ws_bytes < need || !aligned(ws, 16)) return OLA_ERR_INVALID_ARG;
    const Rows w = flat(ws, int64_t(need), 1);
    for (const Rows* x : std::initializer_list<const Rows*>{&t.v, &t.k, &t.q, &t.z, &t.y, &si, &so})
      if (overlap(*x, w)) return OLA_ERR_INVALID_ARG;
    a.seg_S = static_cast<float*>(ws);
    a.seg_a = a.seg_S + int64_t(d->R) * d->H * a.nseg * d->d_v * d->d_k;
  }
  s = error_word(&a.err);
  if (s != OLA_OK) return s;
  a.S_in = S_in;
  a.lens = lens;
  a.S_out = S_out;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return from_cuda(chunked ? launch_scan_chunk(a, st) : launch_scan_tok(a, d->in_dtype, st));
}

ola_status ola_scan_step(const ola_scan_desc* d, int32_t Bp, const void* v, const float* dt,
                         const float* A, const void* k, const void* q, const float* D,
                         const float* dt_bias, const void* z, const float* state_in,
                         const int32_t* parent_idx, void* y, float* state_out, void* stream) {
  ScanArgs a;
  ScanRows t;
  ola_status s = scan_args(d, v, dt, A, k, q, D, dt_bias, z, y, &a, &t);
  if (s != OLA_OK) return s;
  if (d->P < 1 || Bp < 1 || !state_in || !state_out) return OLA_ERR_INVALID_ARG;
  if (!parent_idx && Bp != 1 && Bp != d->P) return OLA_ERR_INVALID_ARG;
  if (!aligned(state_in, 16) || !aligned(state_out, 16) || !aligned(parent_idx, 4))
    return OLA_ERR_INVALID_ARG;
  int64_t ni, no;
  if (!elements({d->R, Bp, d->H, d->d_v, d->d_k}, &ni) ||
      !elements({d->R, d->P, d->H, d->d_v, d->d_k}, &no))
    return OLA_ERR_UNSUPPORTED;
  const Rows si = flat(state_in, ni, 4), so = flat(state_out, no, 4);
  const bool in_place = state_in == state_out && !parent_idx && Bp == d->P;
  if (!in_place && overlap(si, so)) return OLA_ERR_INVALID_ARG;
  for (const Rows* x : {&t.v, &t.k, &t.q, &t.z, &t.y})
    if (overlap(*x, so)) return OLA_ERR_INVALID_ARG;
  if (overlap(t.y, si)) return OLA_ERR_INVALID_ARG;
  s = error_word(&a.err);
  if (s != OLA_OK) return s;
  a.Bp = Bp;
  a.S_in = state_in;
  a.parent = parent_idx;
  a.S_out = state_out;
  return from_cuda(launch_scan_step(a, d->in_dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
