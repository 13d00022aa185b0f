// gb_overlap.h — the overlap check of the C-ABI layer (gb_api.cpp and
// gb_optim_api.cpp; each compiles its own copy).  Host only.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <cstdio>
#include <vector>

#include "gb_internal.h"

namespace gb {
namespace {

// ---------------------------------------------------------------------------
// Overlapping buffers.  Every buffer a call writes (outputs, and the buffers
// it reads and rewrites: residuals, workspaces, staging buffers) must share
// no byte with any other buffer of the call, except where the ABI lets one
// output be one input exactly (out == srcs[0]: same address, same length);
// inputs may overlap one another.  A partial overlap would let one lane's
// store reach the values another lane has still to read.  The spans are
// sorted, so a batch of thousands of buckets costs O(N log N); a call with
// few buffers keeps them in fixed storage and allocates nothing.
// ---------------------------------------------------------------------------
struct Span {
  uintptr_t lo = 0, hi = 0;  // bytes [lo, hi)
  const char* name = "";
  long i = -1, j = -1;  // indices shown with the name, -1 if none
};

class Spans {
 public:
  void add(const void* p, size_t bytes, const char* name, long i = -1, long j = -1) {
    if (p == nullptr || bytes == 0) return;
    Span s;
    s.lo = reinterpret_cast<uintptr_t>(p);
    s.hi = s.lo + bytes;
    s.name = name;
    s.i = i;
    s.j = j;
    if (n_ < kInline) {
      inline_[n_] = s;
    } else {
      if (n_ == kInline) heap_.assign(inline_, inline_ + kInline);
      heap_.push_back(s);
    }
    n_++;
  }
  // An input, left out when it is exactly the output `alias` may be.
  void add_input(const void* p, size_t bytes, const void* alias, const char* name, long i = -1, long j = -1) {
    if (p != nullptr && p == alias) return;
    add(p, bytes, name, i, j);
  }
  Span* data() { return n_ <= kInline ? inline_ : heap_.data(); }
  size_t size() const { return n_; }

 private:
  static constexpr size_t kInline = 48;
  Span inline_[kInline];
  std::vector<Span> heap_;
  size_t n_ = 0;
};

void span_label(const Span& s, char* buf, size_t size) {
  if (s.j >= 0) std::snprintf(buf, size, "%s[%ld * k + %ld]", s.name, s.i, s.j);
  else if (s.i >= 0) std::snprintf(buf, size, "%s[%ld]", s.name, s.i);
  else std::snprintf(buf, size, "%s", s.name);
}

gb_status overlap_error(const char* fn, const Span& a, const Span& b) {
  char la[64], lb[64];
  span_label(a, la, sizeof la);
  span_label(b, lb, sizeof lb);
  char msg[384];
  std::snprintf(msg, sizeof msg, "%s: %s overlaps %s (bytes %#zx..%#zx and %#zx..%#zx)", fn, la, lb, (size_t)a.lo,
                (size_t)a.hi, (size_t)b.lo, (size_t)b.hi);
  return fail_status(GB_ERR_INVALID_ARG, msg);
}

bool by_start(const Span& a, const Span& b) { return a.lo < b.lo; }

// outs: every buffer the call writes; ins: the buffers it only reads, the
// exactly aliased input already left out.
gb_status check_disjoint(const char* fn, Spans& outs, Spans& ins) {
  Span* o = outs.data();
  Span* in = ins.data();
  const size_t no = outs.size(), ni = ins.size();
  std::sort(o, o + no, by_start);
  size_t far = 0;  // the output reaching furthest so far
  for (size_t a = 1; a < no; a++) {
    if (o[a].lo < o[far].hi) return overlap_error(fn, o[far], o[a]);
    if (o[a].hi > o[far].hi) far = a;
  }
  // the outputs are now disjoint and in order, so their ends increase too:
  // the inputs starting before an output's end only grow from one output to
  // the next, and the one of them reaching furthest decides
  std::sort(in, in + ni, by_start);
  size_t q = 0;
  long reach = -1;
  for (size_t a = 0; a < no; a++) {
    for (; q < ni && in[q].lo < o[a].hi; q++) {
      if (reach < 0 || in[q].hi > in[reach].hi) reach = (long)q;
    }
    if (reach >= 0 && in[reach].hi > o[a].lo) return overlap_error(fn, o[a], in[reach]);
  }
  return GB_OK;
}

}  // namespace
}  // namespace gb
