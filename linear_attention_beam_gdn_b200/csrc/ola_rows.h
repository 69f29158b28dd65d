// Extents, strides and overlaps of the row tensors that the operators around the recurrence are
// given (host only, no CUDA).
#pragma once

#include <cstdint>
#include <initializer_list>

namespace ola {

// A tensor of R sequences x P rows of `width` contiguous elements of `e` bytes.
struct Rows {
  const void* p;
  int64_t R, P, tok, seq, width;
  int e;
  bool empty() const { return !p || R == 0 || P == 0 || width == 0; }
  int64_t extent() const { return ((R - 1) * seq + (P - 1) * tok + width) * e; }
};

constexpr int64_t kMostElements = int64_t(1) << 46;   // byte offsets stay far inside 64 bits

// Fills in default strides; false if they cannot be what the rows need. Every bound is tested before
// the product that it bounds.
inline bool strides(Rows* t, bool output) {
  const int64_t most = kMostElements;
  if (t->tok == 0) t->tok = t->width;
  if (t->tok < t->width || t->tok >= most || (t->P > 1 && t->tok > most / t->P)) return false;
  if (t->seq == 0) t->seq = t->P * t->tok;
  if (t->seq < 0 || t->seq >= most || (t->R > 1 && t->seq > most / t->R)) return false;
  return !(output && t->R > 1 && t->P > 0 && t->seq < (t->P - 1) * t->tok + t->width);
}

// Product of sizes; false if it is above kMostElements.
inline bool elements(std::initializer_list<int64_t> sizes, int64_t* n) {
  *n = 1;
  for (int64_t s : sizes)
    if (s == 0) {
      *n = 0;
      return true;
    }
  for (int64_t s : sizes) {
    if (s < 0 || *n > kMostElements / s) return false;
    *n *= s;
  }
  return true;
}

// Whether two row sets share bytes. Column slices of one wide buffer (equal token strides, sequence
// strides that are whole tokens) are told apart; otherwise overlapping extents count as shared.
inline bool overlap(Rows a, Rows b) {
  if (a.empty() || b.empty()) return false;
  const int64_t pa = int64_t(reinterpret_cast<uintptr_t>(a.p));
  const int64_t pb = int64_t(reinterpret_cast<uintptr_t>(b.p));
  if (pa + a.extent() <= pb || pb + b.extent() <= pa) return false;
  // one token per sequence: the token stride means nothing, the sequences are the rows
  for (Rows* t : {&a, &b})
    if (t->P == 1) *t = Rows{t->p, 1, t->R, t->seq, t->R * t->seq, t->width, t->e};
  const int64_t ta = a.tok * a.e, tb = b.tok * b.e;
  if (ta == tb && (a.R == 1 || a.seq % a.tok == 0) && (b.R == 1 || b.seq % b.tok == 0)) {
    const int64_t off = ((pb - pa) % ta + ta) % ta;
    return !(off >= a.width * a.e && off + b.width * b.e <= ta);
  }
  return true;
}

inline Rows flat(const void* p, int64_t n, int e) { return Rows{p, 1, 1, n, n, n, e}; }

}  // namespace ola
