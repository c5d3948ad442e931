// Host-side helpers shared by the files that implement the C ABI (sdpa_api.cu defines them).
#pragma once

#include "common.cuh"
#include "../../include/sdpa.h"

namespace sdpa {

// Device address of the error word on the current device.
int error_word(unsigned** out);

bool aligned16(const void* ptr);
bool aligned4(const void* ptr);
bool overlaps(const void* a, size_t na, const void* b, size_t nb);
size_t elem_size(int dtype);

// Validates the layout of one [B, H, L, D] tensor and returns its byte extent in *bytes.
bool check_layout(const sdpa_layout_t& l, int B, int H, int L, int D, size_t es, Layout* out, size_t* bytes);

uint64_t wait_limit_ns();  // time limit of a bounded wait inside a kernel
int sm_count();            // SMs of the current device, 0 if unknown
int status_of(cudaError_t e);

struct EventPair {
  cudaEvent_t start = nullptr, stop = nullptr;
};
bool begin_launch(EventPair* ev, cudaStream_t s);
void end_launch(int kernel, const EventPair& ev, bool timed, cudaError_t e, cudaStream_t s);

// Launches one kernel through `fn`, counting it and, when timing is on, bracketing it with
// events on its stream.
template <typename Fn>
cudaError_t launch_one(int kernel, cudaStream_t s, Fn fn) {
  EventPair ev;
  const bool timed = begin_launch(&ev, s);
  const cudaError_t e = fn();
  end_launch(kernel, ev, timed, e, s);
  return e;
}

}  // namespace sdpa
