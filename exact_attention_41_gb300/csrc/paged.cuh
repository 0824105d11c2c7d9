// Geometry shared by the kernels of attn_fwd_paged.
#pragma once

#include "kernels.h"

namespace attn {

// One sequence of a paged call: its query rows [q0, q0 + lq) and key count.
struct PagedSeq {
  int q0, lq, lk;
  int err;  // error bits to raise; a bad length leaves no rows or no keys
};

__device__ __forceinline__ PagedSeq paged_seq(const PagedArgs &a, int i) {
  PagedSeq s;
  s.err = 0;
  s.q0 = a.cu_q[i];
  const int64_t n = (int64_t)a.cu_q[i + 1] - s.q0;
  if (s.q0 < 0 || n < 0 || s.q0 + n > a.total_q) {
    s.err = kErrBadSeqlen;
    s.lq = s.lk = 0;
    return s;
  }
  s.lq = (int)n;
  const int cached = a.cache_seqlens[i];
  const int64_t lk = (int64_t)cached + (a.appended ? s.lq : 0);
  s.lk = (int)lk;
  // rows of a sequence with a bad key count get the result of no keys
  if (cached < 0) {
    s.err = kErrBadSeqlen;
    s.lk = 0;
  } else if (lk > (int64_t)a.max_pages * a.page_size) {
    s.err = kErrCacheOverflow;
    s.lk = 0;
  }
  return s;
}

// Physical page of logical page pg of sequence i, or -1 when it lies outside
// the pool.  pg must be below max_pages.
__device__ __forceinline__ int paged_page(const PagedArgs &a, int i, int pg) {
  const int page = a.block_table ? a.block_table[(int64_t)i * a.max_pages + pg] : i;
  return page >= 0 && page < a.num_pages ? page : -1;
}

}  // namespace attn
