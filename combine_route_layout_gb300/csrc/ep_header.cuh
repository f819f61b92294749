// The first bytes of a router's or a product's workspace: error bits, and what
// its kernels expect to be zero when they start (tickets). A handle's first call
// puts a kernel ahead of its own that clears them and leaves the handle's mark
// there. Where it finds the mark it does nothing, so that error bits wait for their
// report whatever runs after them: a call that is being captured puts the kernel
// into its graph, once a capture, since a graph may run later, or never, or often.
// The mark also says that a report reads no left-over memory.
#pragma once

#include <atomic>

#include "ep_kernels.cuh"

namespace ep {

constexpr size_t kHeaderBytes = 1024;
constexpr size_t kTicketOffset = 256;

struct Header {
  uint32_t* words = nullptr;   // [0] error bits, [1] mark
  uint32_t mark = 0;
  bool ready = false;          // a call that was not captured has cleared it
  unsigned long long capture = 0;   // the capture whose graph clears it
};

static __global__ void clear_header_kernel(uint32_t* words, uint32_t mark) {
  const bool cleared = words[1] == mark;
  __syncthreads();
  if (!cleared) words[threadIdx.x] = threadIdx.x == 1 ? mark : 0u;
}

inline void open_header(Header* h, void* workspace) {
  static std::atomic<uint32_t> next{1};
  h->words = static_cast<uint32_t*>(workspace);
  h->mark = 0x45500000u + next.fetch_add(1);
  h->ready = false;
}

inline cudaError_t header_ready(Header* h, cudaStream_t st) {
  if (h->ready) return cudaSuccess;
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  unsigned long long id = 0;
  cudaError_t e = cudaStreamGetCaptureInfo(st, &cap, &id);
  if (e != cudaSuccess) return e;
  const bool capturing = cap != cudaStreamCaptureStatusNone;
  if (capturing && id == h->capture) return cudaSuccess;
  clear_header_kernel<<<1, kHeaderBytes / 4, 0, st>>>(h->words, h->mark);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (capturing) {
    h->capture = id;
  } else {
    h->ready = true;
  }
  return cudaSuccess;
}

// Wait for `st`, then read and clear the error bits.
inline cudaError_t header_report(Header* h, cudaStream_t st, uint32_t* bits) {
  uint32_t got[2] = {0, 0};
  *bits = 0;
  cudaError_t e = cudaMemcpyAsync(got, h->words, sizeof(got), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess || got[1] != h->mark || got[0] == 0) return e;
  *bits = got[0];
  e = cudaMemsetAsync(h->words, 0, sizeof(uint32_t), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return e;
}

// Zero everything behind the mark, on `st`, and wait: what a kernel that gave up left
// behind. A graph captured on a handle that had run clears nothing itself.
inline cudaError_t header_renew(Header* h, cudaStream_t st) {
  cudaError_t e = cudaMemsetAsync(h->words + 2, 0, kHeaderBytes - 2 * sizeof(uint32_t), st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  return e;
}

}  // namespace ep
