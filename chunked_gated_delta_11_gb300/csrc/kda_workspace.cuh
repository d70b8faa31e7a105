// kda_workspace.cuh -- device memory that a call needs while its kernels run.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace kda {

// A workspace of the caller's, or one allocated on the stream for this call.
class Workspace {
 public:
  Workspace(void* given, size_t bytes, size_t need, cudaStream_t stream) : stream_(stream) {
    if (need == 0) return;
    if (given) {
      ok_ = (reinterpret_cast<uintptr_t>(given) & 15u) == 0 && bytes >= need;
      ptr_ = given;
    } else if (cudaMallocAsync(&ptr_, need, stream) == cudaSuccess) {
      own_ = true;
    } else {
      cudaGetLastError();
      ok_ = false;
    }
  }
  ~Workspace() {
    if (own_) cudaFreeAsync(ptr_, stream_);
  }
  Workspace(const Workspace&) = delete;
  Workspace& operator=(const Workspace&) = delete;
  bool ok() const { return ok_; }
  void* get() const { return ptr_; }

 private:
  cudaStream_t stream_;
  void* ptr_ = nullptr;
  bool own_ = false, ok_ = true;
};

}  // namespace kda
