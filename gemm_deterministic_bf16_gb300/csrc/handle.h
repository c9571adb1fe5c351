// handle.h -- the library handle and the host helpers shared by the C ABI's
// source files: error mapping, workspace layout, overlap checks, timing.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <vector>

#include "common.cuh"
#include "tc.h"

constexpr int kTicketWords = detffn::kTcsTickets + 2 * detffn::kTcsRanges;

struct detffn_handle_s {
  int device = 0;
  int sm_count = 0;
  uint16_t* d_silu = nullptr;   // [65536] BF16 SiLU by gate bit pattern
  float* d_dsilu = nullptr;     // [65536] FP32 SiLU' by gate bit pattern
  int* d_status = nullptr;      // device status word (bounded waits)
  int* d_tickets = nullptr;     // tree tickets of the few-token kernels (kTcsTickets words) and the fused
                                // forward's range counters (2 x kTcsRanges words), zero between calls
  detffn::Waits wt;                     // the current call's wait settings (status word, poll limit, test stall)
  int flags = 0;                // the current call's option flags
  // A second stream and two events (made at creation) for the overlapped
  // dHidden reduction (DETFFN_FLAG_OVERLAP_DHIDDEN).
  cudaStream_t side = nullptr;
  cudaEvent_t ev_fork = nullptr, ev_join = nullptr;
  std::vector<uint16_t> h_silu;
  std::vector<float> h_dsilu;
  // Measurement: event pairs around launches while profiling is on.
  struct Rec {
    const char* name;
    cudaEvent_t a, b;
    double bytes, flops;
    int launches;
  };
  bool prof = false;
  std::vector<Rec> recs;
};

namespace detffn {

// Records the CUDA error behind a DETFFN_ERR_CUDA (detffn_last_cuda_error).
void note_cuda_error(cudaError_t e);

inline detffn_status cu(cudaError_t e) {
  if (e == cudaSuccess) return DETFFN_OK;
  note_cuda_error(e);
  return DETFFN_ERR_CUDA;
}

#define TRY(expr)                              \
  do {                                         \
    detffn_status _s = (expr);                 \
    if (_s != DETFFN_OK) return _s;            \
  } while (0)
#define TRYCU(expr) TRY(cu(expr))

// Runs `launch`; while profiling, brackets it with an event pair on `st`.
template <class F>
detffn_status timed(detffn_handle h, cudaStream_t st, const char* name, double bytes,
                    double flops, F&& launch, int launches = 1) {
  if (!h || !h->prof) return launch();
  detffn_handle_s::Rec r{name, nullptr, nullptr, bytes, flops, launches};
  if (cudaEventCreate(&r.a) != cudaSuccess || cudaEventCreate(&r.b) != cudaSuccess) return DETFFN_ERR_CUDA;
  cudaEventRecord(r.a, st);
  const detffn_status s = launch();
  cudaEventRecord(r.b, st);
  h->recs.push_back(r);
  return s;
}

struct Arena {
  char* base;
  size_t off = 0;
  explicit Arena(void* b) : base(static_cast<char*>(b)) {}
  template <class T>
  T* take(long long count) {
    off = (off + 255) & ~(size_t)255;
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off += (size_t)count * sizeof(T);
    return p;
  }
};

inline bool overlap(const void* a, long long na, const void* b, long long nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace detffn
