// fp8_host.cpp -- the C ABI of the 8-bit product and its quantisation.
//
// Host side only, like lora_host.cpp: argument checks before any launch.
// Nothing here allocates, frees, synchronises or reads device memory.
#include <hip/hip_runtime.h>

#include <climits>

#include "../../include/lora_mi355x.h"
#include "fp8.hpp"
#include "host.hpp"

using namespace lora;

namespace {

constexpr uint32_t kMaxOut = 1u << 26;
constexpr uint32_t kMaxStride = 1u << 22;  // of a product's rows: a tile's offsets stay within 32 bits

uint32_t blocks_of(uint32_t k) { return (k + kFp8Block - 1) / kFp8Block; }

// Rows of k codes and their scales.
int check_codes(const char *what, const char *name, const void *codes, uint32_t stride, uint32_t k, const float *scale,
                uint32_t scale_stride, uint32_t n) {
  if (stride < k) return fail(LORA_ERR_STRIDE, "%s: %s row stride %u < its row of %u codes", what, name, stride, k);
  if (stride % 16) return fail(LORA_ERR_UNSUPPORTED, "%s: %s row stride %u must be a multiple of 16", what, name, stride);
  if (scale_stride < blocks_of(k))
    return fail(LORA_ERR_STRIDE, "%s: %s scale stride %u < its row of %u scales", what, name, scale_stride, blocks_of(k));
  if (n && (!codes || !scale))
    return fail(LORA_ERR_NULL_PTR, "%s: %s codes %p and scales %p must be non-NULL", what, name, codes, (const void *)scale);
  if (n && !aligned16(codes)) return fail(LORA_ERR_UNSUPPORTED, "%s: %s %p must be 16-byte aligned", what, name, codes);
  if (n && (uintptr_t)scale % 4)
    return fail(LORA_ERR_UNSUPPORTED, "%s: %s scales %p must be aligned to their 4 bytes", what, name, (const void *)scale);
  return LORA_OK;
}

}  // namespace

extern "C" {

int lora_quantize_fp8(int32_t dtype, uint32_t n_rows, uint32_t k, const void *x, uint32_t x_row_stride, uint32_t block_rows,
                      void *codes, uint32_t codes_row_stride, float *scale, uint32_t scale_row_stride, void *stream) {
  clear_err();
  const char *what = "lora_quantize_fp8";
  if (int e = check_type(what, dtype)) return e;
  if (block_rows != 1 && block_rows != (uint32_t)kFp8Block)
    return fail(LORA_ERR_UNSUPPORTED, "%s: block_rows %u is neither 1 nor %d", what, block_rows, kFp8Block);
  if (k == 0 || k % 16 || k > (uint32_t)INT_MAX / 2)
    return fail(k == 0 || k > (uint32_t)INT_MAX / 2 ? LORA_ERR_SHAPE : LORA_ERR_UNSUPPORTED,
                "%s: [n_rows %u x k %u]: k must be a multiple of 16 in 16..%d", what, n_rows, k, INT_MAX / 2);
  if ((uint64_t)n_rows * blocks_of(k) * 8 > (uint64_t)INT_MAX - 256)
    return fail(LORA_ERR_SHAPE, "%s: [n_rows %u x k %u] has more than 2^28 - 33 row blocks", what, n_rows, k);
  if (int e = check_rows(what, dtype, "x", x, x_row_stride, k, n_rows)) return e;
  if (int e = check_codes(what, "codes", codes, codes_row_stride, k, scale, scale_row_stride, n_rows)) return e;
  if (n_rows == 0) return LORA_OK;
  if (int e = check_device(what)) return e;
  QuantArgs a{};
  a.x = x;
  a.codes = (uint8_t *)codes;
  a.scale = scale;
  a.x_stride = x_row_stride;
  a.c_stride = codes_row_stride;
  a.s_stride = scale_row_stride;
  a.n = (int)n_rows;
  a.k = (int)k;
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] { return launch_quantize_fp8(a, dtype, (int)block_rows, st); });
}

// No form needs one.
size_t lora_matmul_fp8_workspace_bytes(int32_t, uint32_t, uint32_t, uint32_t) { return 0; }

int lora_matmul_fp8(int32_t dtype, uint32_t n_out, uint32_t k_in, const void *W, uint32_t w_row_stride, const float *w_scale,
                    uint32_t w_scale_stride, const void *x, uint32_t x_row_stride, const float *x_scale, uint32_t x_scale_stride,
                    uint32_t n, void *y, uint32_t y_row_stride, void *, size_t, void *stream) {
  clear_err();
  const char *what = "lora_matmul_fp8";
  if (int e = check_type(what, dtype)) return e;
  if (n_out == 0 || n_out > kMaxOut || k_in == 0 || k_in > kFp8MaxK)
    return fail(LORA_ERR_SHAPE, "%s: [n %u] x [n_out %u x k_in %u]: n_out must be in 1..%u and k_in in 1..%u", what, n, n_out, k_in,
                kMaxOut, kFp8MaxK);
  if (n_out % 8 || k_in % 16)
    return fail(LORA_ERR_UNSUPPORTED, "%s: [n %u] x [n_out %u x k_in %u]: n_out must be a multiple of 8 and k_in of 16", what, n,
                n_out, k_in);
  if (n > kMaxRows)
    return fail(LORA_ERR_SHAPE, "%s: [n %u] x [n_out %u x k_in %u]: n exceeds the limit %u", what, n, n_out, k_in, kMaxRows);
  if (int e = check_codes(what, "W", W, w_row_stride, k_in, w_scale, w_scale_stride, n)) return e;
  if (int e = check_codes(what, "x", x, x_row_stride, k_in, x_scale, x_scale_stride, n)) return e;
  if (int e = check_rows(what, dtype, "y", y, y_row_stride, n_out, n)) return e;
  if (w_row_stride > kMaxStride || x_row_stride > kMaxStride || x_scale_stride > kMaxStride)
    return fail(LORA_ERR_STRIDE, "%s: row strides of W %u, x %u and x's scales %u must be at most %u", what, w_row_stride, x_row_stride,
                x_scale_stride, kMaxStride);
  if (n == 0) return LORA_OK;
  if (int e = check_device(what)) return e;
  Fp8Args a{};
  a.W = (const uint8_t *)W;
  a.x = (const uint8_t *)x;
  a.w_scale = w_scale;
  a.x_scale = x_scale;
  a.y = y;
  a.w_stride = w_row_stride;
  a.x_stride = x_row_stride;
  a.ws_stride = w_scale_stride;
  a.xs_stride = x_scale_stride;
  a.y_stride = y_row_stride;
  a.n_out = (int)n_out;
  a.k = (int)k_in;
  a.n = (int)n;
  hipStream_t st = (hipStream_t)stream;
  return timed(what, st, [&] { return launch_matmul_fp8(a, dtype, st); });
}

}  // extern "C"
