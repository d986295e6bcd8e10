// call_order.h - the calls of one handle run in the order they are made,
// whatever streams they are made on.
#pragma once

#include <cuda_runtime.h>

#include "rnn.h"

namespace rnn {

// One event, recorded behind each call: a call on another stream waits for it
// on the device, and the host waits for it before it changes what calls read.
// Calls captured into a graph run when the graph does: they are not ordered
// here, and the host then waits for the device.
class CallOrder {
 public:
  rnn_status_t create() {
    return cudaEventCreateWithFlags(&done_, cudaEventDisableTiming) == cudaSuccess ? RNN_OK : RNN_CUDA_ERROR;
  }
  void destroy() {
    if (done_) cudaEventDestroy(done_);
    done_ = nullptr;
  }
  // Before a call's first launch on s.
  rnn_status_t enter(cudaStream_t s) {
    cudaStreamCaptureStatus st;
    if (cudaStreamIsCapturing(s, &st) != cudaSuccess) return RNN_CUDA_ERROR;
    capturing_ = st != cudaStreamCaptureStatusNone;
    if (capturing_) {
      captured_ = true;
      return RNN_OK;
    }
    // ids, unlike stream handles, are never used again
    if (cudaStreamGetId(s, &id_) != cudaSuccess) return RNN_CUDA_ERROR;
    if (pending_ && id_ != last_ && cudaStreamWaitEvent(s, done_, 0) != cudaSuccess) return RNN_CUDA_ERROR;
    return RNN_OK;
  }
  // Behind its last launch, whether or not all of them succeeded.
  rnn_status_t leave(cudaStream_t s) {
    if (capturing_) return RNN_OK;
    if (cudaEventRecord(done_, s) != cudaSuccess) return RNN_CUDA_ERROR;
    last_ = id_;
    pending_ = true;
    return RNN_OK;
  }
  // Until no call is under way.
  rnn_status_t wait() {
    if (captured_) return cudaDeviceSynchronize() == cudaSuccess ? RNN_OK : RNN_CUDA_ERROR;
    if (pending_ && cudaEventSynchronize(done_) != cudaSuccess) return RNN_CUDA_ERROR;
    pending_ = false;
    return RNN_OK;
  }

 private:
  cudaEvent_t done_ = nullptr;
  unsigned long long id_ = 0, last_ = 0;
  bool pending_ = false, capturing_ = false, captured_ = false;
};

}  // namespace rnn
