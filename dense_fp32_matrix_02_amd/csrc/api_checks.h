// Argument checks shared by the host sides of the FP8 and routing calls: pure
// host code, before any HIP call.
#pragma once

#include <climits>
#include <cstdint>

#include "sgemm_mi355_route.h"

namespace sgemm_impl {

typedef unsigned __int128 Bytes;

constexpr int kMostRows = INT_MAX - 1024;  // row and column numbers stay ints with a tile of headroom

inline int element_size(int type) { return type == SGEMM_MI355_F32 ? 4 : 2; }
inline bool known_type(int type) {
  return type == SGEMM_MI355_F32 || type == SGEMM_MI355_BF16 || type == SGEMM_MI355_F16;
}
inline int at_least_1(int x) { return x > 1 ? x : 1; }
inline int blocks_of(int n) { return n / 128 + (n % 128 != 0); }

// A call's matrices: each one's address, extent and alignment. check() gives
// the first error: a null pointer, a misaligned one, an extent past the
// address space, or an output that overlaps another matrix.
class Matrices {
 public:
  // rows x cols elements of `size` bytes, row stride ld elements.
  void dense(const void* p, int64_t rows, int64_t cols, int64_t ld, int size, bool output) {
    if (rows <= 0 || cols <= 0) return;
    add(p, ((Bytes)(rows - 1) * (Bytes)ld + (Bytes)cols) * (Bytes)size, size, output);
  }
  // `count` matrices of rows x cols elements, element (i, r, c) at i*stride + r*s_r + c*s_c.
  void strided(const void* p, int64_t count, int64_t stride, int64_t rows, int64_t s_r, int64_t cols, int64_t s_c,
               int size, bool output) {
    if (count <= 0 || rows <= 0 || cols <= 0) return;
    add(p, ((Bytes)(count - 1) * (Bytes)stride + (Bytes)(rows - 1) * (Bytes)s_r + (Bytes)(cols - 1) * (Bytes)s_c + 1) *
               (Bytes)size,
        size, output);
  }
  int check() const {
    for (int i = 0; i < n_; ++i)
      if (m_[i].p == nullptr) return SGEMM_MI355_ERR_NULL;
    for (int i = 0; i < n_; ++i)
      if (((uintptr_t)m_[i].p & (m_[i].align - 1)) != 0) return SGEMM_MI355_ERR_ALIGN;
    for (int i = 0; i < n_; ++i)
      if (m_[i].bytes > (Bytes)1 << 62) return SGEMM_MI355_ERR_EXTENT;
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < n_; ++j)
        if (i != j && m_[i].output) {
          const Bytes a = (uintptr_t)m_[i].p, b = (uintptr_t)m_[j].p;
          if (a < b + m_[j].bytes && b < a + m_[i].bytes) return SGEMM_MI355_ERR_ALIAS;
        }
    return SGEMM_MI355_OK;
  }

 private:
  struct Matrix {
    const void* p;
    Bytes bytes;
    unsigned align;
    bool output;
  };
  void add(const void* p, Bytes bytes, int align, bool output) { m_[n_++] = Matrix{p, bytes, (unsigned)align, output}; }
  Matrix m_[10];
  int n_ = 0;
};

// Whether rows x cols elements at strides s_r, s_c all have places of their own.
inline bool apart(int64_t rows, int64_t s_r, int64_t cols, int64_t s_c) {
  if (rows > 1 && s_r < 1) return false;
  if (cols > 1 && s_c < 1) return false;
  if (rows <= 1 || cols <= 1) return true;
  return (Bytes)s_r > (Bytes)(cols - 1) * (Bytes)s_c || (Bytes)s_c > (Bytes)(rows - 1) * (Bytes)s_r;
}

// A launch counts its threads in 32 bits.
inline bool launchable(int64_t blocks, int threads) { return blocks * threads <= (int64_t)UINT32_MAX; }

inline int done(hipError_t err) { return err == hipSuccess ? SGEMM_MI355_OK : SGEMM_MI355_ERR_LAUNCH; }

}  // namespace sgemm_impl
