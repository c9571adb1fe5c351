// block.h -- launchers of the operators around the FFN: norms joined with the
// residual stream, 8-bit activation checkpoints.
#pragma once

#include "common.cuh"

namespace detffn {

// Rows of one tensor: element (m, c) at p + m * ld + c.
struct Rows {
  const void* p = nullptr;
  long long ld = 0;
};

constexpr long long kJoinMaxH = 32768;
// Column sums of the backward pass are taken over this many row sets at
// most, whatever the GPU, so that their order depends on the call alone (its
// sizes, types, operands and 16-byte alignment).
constexpr int kJoinSets = 152;

struct JoinArgs {
  long long M = 0;
  int H = 0;
  int dtype = 0, pdtype = 0;
  float scale = 1.0f, eps = 0.0f;
  const void* w_post = nullptr;
  const void* w_pre = nullptr;
  const void* gate = nullptr;
  long long gate_rs = 0;
  int gate_cs = 0;
  Rows x, z, out, y;          // forward
  Rows r, dr, dy, dx, dz;     // backward (and z)
  void* dgate = nullptr;      // laid out as the gate, contiguous
  void* dw_post = nullptr;
  void* dw_pre = nullptr;
  float* part = nullptr;      // backward: column partials [kind][set][H], then [set] for a scalar gate
};

cudaError_t join_forward_f32(const JoinArgs& a, cudaStream_t st);
cudaError_t join_forward_f16(const JoinArgs& a, cudaStream_t st);
cudaError_t join_forward_bf16(const JoinArgs& a, cudaStream_t st);
cudaError_t join_backward_f32(const JoinArgs& a, cudaStream_t st);
cudaError_t join_backward_f16(const JoinArgs& a, cudaStream_t st);
cudaError_t join_backward_bf16(const JoinArgs& a, cudaStream_t st);

constexpr int kCkptBlock = 64;  // elements of a row that share a scale

struct CkptArgs {
  long long M = 0, I = 0;
  int dtype = 0;
  const void* gate = nullptr;   // pack: in; unpack: out
  const void* up = nullptr;
  int8_t* gq = nullptr;
  int8_t* uq = nullptr;
  float* gs = nullptr;
  float* us = nullptr;
  const void* dh = nullptr;     // backward
  void *dU = nullptr, *dG = nullptr, *h = nullptr;
};

cudaError_t launch_ckpt8_pack(const CkptArgs& a, int sm_count, cudaStream_t st);
cudaError_t launch_ckpt8_unpack(const CkptArgs& a, int sm_count, cudaStream_t st);
cudaError_t launch_ckpt8_silu_bwd(const CkptArgs& a, int sm_count, cudaStream_t st);

}  // namespace detffn
