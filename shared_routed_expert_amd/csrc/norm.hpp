// Arguments of the norm in front of the MoE layer (see include/srmoe.h).
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace srmoe {

struct NormArgs {
  const uint16_t* x;
  size_t x_stride;
  const uint16_t* residual;   // null: none
  uint16_t* residual_out;     // null: not written
  const float* weight;
  float eps;
  int T, H;
  bool block;                 // scales of 128 columns, else of a row
  uint16_t* y;                // null: not written
  uint8_t* xq;                // null: not written
  float* sx;
};

hipError_t launch_add_rms_norm(const NormArgs&, hipStream_t);

}  // namespace srmoe
