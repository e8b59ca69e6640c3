// fp8.hpp -- arguments and launchers of the 8-bit product and its quantisation.  Not part of the ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_stage.hpp"
#include "verify.hpp"

namespace lora {

constexpr uint32_t kFp8MaxK = 65536;  // columns of a product
struct QuantArgs {
  const void *x;  // [n][x_stride]
  uint8_t *codes; // [n][c_stride]
  float *scale;   // [ceil(n / block_rows)][s_stride]
  long long x_stride, c_stride, s_stride;
  int n, k;
  FastDiv per_row;  // workgroup units of a row (block_rows 1: threads; 128: workgroups)
};
hipError_t launch_quantize_fp8(const QuantArgs &a, int dtype, int block_rows, hipStream_t st);

struct Fp8Args {
  const uint8_t *W, *x;          // [n_out][w_stride], [n][x_stride]
  const float *w_scale, *x_scale;  // [ceil(n_out / 128)][ws_stride], [n][xs_stride]
  void *y;                       // [n][y_stride]
  long long w_stride, x_stride, ws_stride, xs_stride, y_stride;
  int n_out, k, n;
};
hipError_t launch_matmul_fp8(const Fp8Args &a, int dtype, hipStream_t st);

}  // namespace lora
