// device_scope.h -- the device of a handle, for the length of a call.
#pragma once

#include <cuda_runtime.h>

namespace sgd {

// A call's launches, copies and default stream are those of its handle's
// device, whichever the caller has current; the caller's is current again
// afterwards.  (Nothing is set where it is the same one.)
class DeviceScope {
 public:
  explicit DeviceScope(int device) {
    ok_ = cudaGetDevice(&before_) == cudaSuccess;
    if (ok_ && before_ != device) ok_ = moved_ = cudaSetDevice(device) == cudaSuccess;
  }
  ~DeviceScope() {
    if (moved_) cudaSetDevice(before_);
  }
  DeviceScope(const DeviceScope &) = delete;
  DeviceScope &operator=(const DeviceScope &) = delete;
  bool ok() const { return ok_; }

 private:
  int before_ = 0;
  bool ok_ = false, moved_ = false;
};

}  // namespace sgd
