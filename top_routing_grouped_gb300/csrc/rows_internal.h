// rows_internal.h -- what the host side of the sorted rows (api_rows.cu) and their kernels share.
#pragma once
#include "../../include/moe_rows.h"
#include "moe_internal.h"

namespace moe {
namespace rows {

constexpr int kMaxK = 64;
constexpr int kMaxSortExperts = 1024;
// Most blocks of slots that a sort's first launch counts: two an SM (524288 slots of 256 experts with their rows of 200
// bf16: 53.7 us, with one an SM 56.9; a sort of 131072 slots 7.1-11.8 us by the experts, 6.6-10.6).
constexpr int kCountBlocks = 304;
__host__ __device__ inline int count_pitch(int E) { return (E + 3) / 4 * 4; }  // words of a block's counts

struct Args {
  const void* idx;  // null: the positions are given in slot_pos
  bool idx64;
  int64_t T;
  int k, E;
  int32_t *counts, *slot_pos, *row_slot;
  const char* x;  // rows of row_bytes (0: none are moved)
  int64_t row_bytes, ld_bytes, R;
  char* x_rows;
  const uint32_t* x_words;  // ... with `words` 32-bit words beside each (null: none)
  uint32_t* row_words;
  int64_t words;
  const float* gates;  // null: none
  float* row_gates;
};

// Whether a sort of N slots counts them in a launch of its own, into [kCountBlocks, count_pitch(E)] words.
bool counts_first(int64_t N);
cudaError_t launch_rows(const Args& a, int32_t* counted, cudaStream_t st);

cudaError_t launch_combine(const void* y, bool y_bf16, int64_t R, const int32_t* slot_pos, const float* gates, int64_t T,
                           int k, int64_t d, const void* residual, void* out, bool out_bf16, cudaStream_t st);
cudaError_t launch_combine_backward(const void* dout, bool dout_bf16, const int32_t* slot_pos, const float* gates, int64_t T,
                                    int k, int64_t d, int64_t R, const void* y, void* dy, bool y_bf16, float* dgates,
                                    cudaStream_t st);

}  // namespace rows
}  // namespace moe
