// Host-side pieces that the library's translation units share: scratch memory,
// pointer checks, the launch counter.  Definitions in bcjr_api.cu.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace bcjr {
namespace host {

// Adds n to bcjr_launch_count.
void counted_launch(int n = 1);

// Stream-ordered scratch from the library-private pool of the current device.
int scratch_alloc(void** mem, size_t bytes, cudaStream_t st);

// BCJR_OK for a device or managed pointer aligned to 4 bytes (or null, where allowed).
int check_dev_ptr(const void* p, bool nullable);

// Takes (reads and clears) the error flag of the matrix kernels of bcjr_dense.cu on the current device.
int take_dense_error(int* flag);

// Carves one stream-ordered allocation into 256-byte aligned pieces.
struct Arena {
  size_t off = 0;
  char* base = nullptr;
  template <class T>
  T* take(size_t count) {
    size_t bytes = (count * sizeof(T) + 255) & ~size_t(255);
    T* p = reinterpret_cast<T*>(base ? base + off : nullptr);
    off += bytes;
    return p;
  }
};

}  // namespace host
}  // namespace bcjr
