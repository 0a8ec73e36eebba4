// Index arithmetic of the page fork, shared by the kernel and the host (and run on the host by
// the CPU tests).  Every function takes what comes from device memory as it is.
#pragma once

#include "kv_index.h"

namespace rax {

// The pages of a row of `len` tokens: `full` filled ones and, if `part` > 0, one more with so many tokens.
struct RowPages {
  int full, part, invalid;
  RAX_HD int all() const { return full + (part > 0); }
};
// a length outside [0, max_pages << page_shift] is invalid: such a row holds nothing
RAX_HD RowPages row_pages(int len, int page_shift, int max_pages) {
  RowPages p{0, 0, 0};
  if (len < 0 || (long long)len > ((long long)max_pages << page_shift)) {
    p.invalid = 1;
    return p;
  }
  p.full = len >> page_shift;
  p.part = len & ((1 << page_shift) - 1);
  return p;
}

// a parent outside [-1, rows) is invalid and stands for none
RAX_HD int parent_or_none(int parent, int rows) { return parent >= 0 && parent < rows ? parent : -1; }

// What a row's children change in the number of holders of its page at column c: each child holds the
// full pages; of the partly filled one the first child keeps it and the others have their own.
RAX_HD int holders_change(RowPages p, int c, int children) {
  if (c < p.full) return children - 1;
  return c == p.full && p.part > 0 && children == 0 ? -1 : 0;
}

// Columns of a strip (a workgroup takes a strip of all rows), and the strip of a workgroup of `strips` ones: strips that
// share cache lines on one die.
constexpr int kForkColumns = 4;
RAX_HD int strip_of_block(int block, int strips) {
  const int per = (strips + kDies - 1) / kDies, place = block / kDies;
  const int s = place < per ? block % kDies * per + place : strips;
  return s < strips ? s : strips;
}

}  // namespace rax
