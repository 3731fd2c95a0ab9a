// call_check.hpp - the argument checks that the C entry points of the training and
// block operators share (fno_train.cpp, fno_block_ops.cpp). Host code only.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/fno.h"

namespace fno {

inline size_t esize(int dtype) { return dtype == FNO_F32 ? 4 : 2; }
inline bool valid_dtype(fno_dtype_t d) { return d == FNO_F32 || d == FNO_F16 || d == FNO_BF16; }
inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline fno_status_t status_of(hipError_t e) {
  if (e == hipSuccess) return FNO_OK;
  return e == hipErrorOutOfMemory ? FNO_ERR_OUT_OF_MEMORY : FNO_ERR_DEVICE;
}

// The arguments of one call: inputs may share memory with each other, an
// output with nothing. Every pointer is held to its alignment.
class Spans {
 public:
  void in(const void *p, size_t n, size_t align) { add(p, n, align, false); }
  void out(const void *p, size_t n, size_t align) { add(p, n, align, true); }
  bool ok() const {
    if (bad_) return false;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((s_[i].out || s_[j].out) && s_[i].a < s_[j].a + s_[j].n && s_[j].a < s_[i].a + s_[i].n) return false;
    return true;
  }

 private:
  struct Span {
    uintptr_t a;
    size_t n;
    bool out;
  };
  void add(const void *p, size_t n, size_t align, bool out) {
    if (!p) return;
    if (!aligned(p, align)) bad_ = true;
    s_[n_++] = Span{(uintptr_t)p, n, out};
  }
  Span s_[24];
  int n_ = 0;
  bool bad_ = false;
};

// values one operator handles: byte offsets stay far inside 64 bits
constexpr long kMaxValues = 1L << 40;
constexpr long kMaxRow = 1L << 31;

inline bool values_in_range(long a, long b, long c) {
  return a <= kMaxValues && b <= kMaxValues / a && c <= kMaxValues / (a * b);
}

}  // namespace fno
