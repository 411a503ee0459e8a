// Host-side helpers that the files holding C entry points share: argument
// checks, error texts and the library-owned workspace (defined in fs_api.cu).
#pragma once

#include <cstdint>
#include <mutex>
#include <cuda_runtime.h>

#include "flashsample.h"

namespace fs {

// Per-(device, stream) scratch of the training operators, of fixed size.
// `ticket` and `count` are zero between calls: the last block of the launch
// that used them leaves them so.  A call's launches are enqueued under one
// CallLock and run in their order, so the calls of one stream may share it.
constexpr int kTrainMaxBlocks = 2048;
struct alignas(256) TrainScratch {
  unsigned int ticket;
  unsigned int pad;
  unsigned long long count;             // tokens (or sequences) that take part
  float coef, first_coef;               // clip_grad_norm: the scaling launch multiplies by both
  float pad2[2];
  double sums[kTrainMaxBlocks][4];      // one row per block
  alignas(256) unsigned char small[FS_SMALL_WORKSPACE];   // workspace of calls that bring none
};

// Held by a call from its first use of the stream's workspace until its last
// launch is enqueued.  What one launch leaves there for the next (a count, a
// factor, parts to merge) would otherwise be overwritten by a call that
// another host thread enqueues on the same stream in between.
class CallLock {
 public:
  explicit CallLock(cudaStream_t stream);

 private:
  std::unique_lock<std::mutex> lock_;
};

void api_begin();                       // clears fs_last_error()
fs_status api_fail(fs_status s, const char* fmt, ...);
fs_status api_launched(cudaError_t e, const char* what);
// A non-null device pointer of the current device with this alignment.
fs_status api_check_array(const void* p, size_t align, const char* name);
// B >= 0, 0 < d <= 65536 a multiple of 8, V >= 0, both below 2^31.
fs_status api_check_shapes(int64_t B, int64_t d, int64_t V);
// The injected launch failure (FS_FAULT_LAUNCH), where one is set.
fs_status api_check_launch();
// Whether a call's launches after its first are to fail (FS_FAULT_LATER_LAUNCH).
bool api_later_launch_fails();
fs_status api_error_word(int** out, cudaStream_t stream);
fs_status api_train_scratch(cudaStream_t stream, TrainScratch** out);

#define FS_API_TRY(expr)              \
  do {                                \
    fs_status _s = (expr);            \
    if (_s != FS_OK) return _s;       \
  } while (0)

}  // namespace fs
