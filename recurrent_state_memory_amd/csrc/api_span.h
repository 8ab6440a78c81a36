// api_span.h -- host-side checks shared by the C ABI layers of the channelwise
// operators: alignment, and that a call's outputs keep off its inputs and each
// other.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace gdr {

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A buffer of a call; absent ones (p == NULL) are skipped everywhere.
struct Span {
  const void* p;
  size_t bytes;
  size_t align;   // the element's size
};

inline bool spans_clash(const Span& a, const Span& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

template <int NI, int NO>
inline bool spans_aligned(const Span (&ins)[NI], const Span (&outs)[NO]) {
  for (const Span& s : ins)
    if (s.p && !aligned_to(s.p, s.align)) return false;
  for (const Span& s : outs)
    if (s.p && !aligned_to(s.p, s.align)) return false;
  return true;
}

// Whether every output is apart from every input and every other output;
// (same_in, same_out) is the one pair that may be the same buffer.
template <int NI, int NO>
inline bool spans_apart(const Span (&ins)[NI], const Span (&outs)[NO], int same_in = -1, int same_out = -1) {
  for (int o = 0; o < NO; ++o) {
    for (int i = 0; i < NI; ++i)
      if (!(o == same_out && i == same_in && outs[o].p == ins[i].p) && spans_clash(outs[o], ins[i])) return false;
    for (int k = 0; k < o; ++k)
      if (spans_clash(outs[o], outs[k])) return false;
  }
  return true;
}

}  // namespace gdr
