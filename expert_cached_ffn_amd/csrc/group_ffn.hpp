// The FP8 experts of ft_moe_grouped_ffn (arguments as there, checked by it).
#pragma once

#include "ft_internal.hpp"

namespace ft {

struct Fp8Ffn {
  const ft_expert_layout *L;
  const void *slot_pool;
  int n_slots;
  const int32_t *slot_of_expert;
  const void *shared_blob;
  const void *x;
  int T, k, E;
  const int32_t *expert_offsets, *sorted_rows;
  float *y_rows, *y_shared;
  bool gate_up, down;  // stages to run
  void *workspace;
};

size_t fp8_ffn_workspace_bytes(int32_t T, int32_t k, int32_t H, int32_t I);
ft_status fp8_ffn(const Fp8Ffn &f, hipStream_t stream);

// Rows to codes and scales, checked by the caller (fp8.hip).
ft_status fp8_quantize_launch(const void *x, int x_dtype, int64_t ldx, int64_t n, int K, int block_rows, uint8_t *codes,
                              int64_t ldc, float *scales, hipStream_t stream);

}  // namespace ft
