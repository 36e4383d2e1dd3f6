// Host-side checks and conversions shared by the C entry points (internal to libmamba2).
#pragma once

#include <stddef.h>

#include "kernels.h"

namespace mamba2 {

// Records the error's text for mamba2_last_cuda_error and gives MAMBA2_ERR_CUDA.
mamba2_status cuda_fail(cudaError_t e);

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline bool aligned16(const void* p) { return aligned_to(p, 16); }

inline size_t act_size(mamba2_dtype a) { return a == MAMBA2_F32 ? 4 : 2; }
inline bool act_ok(mamba2_dtype a) { return a == MAMBA2_F32 || a == MAMBA2_BF16; }

// Slot range, then shared slots, then coverage of [0, rows).
mamba2_status validate_batch(const mamba2_recurrent_batch* rb, int32_t num_slots, int32_t rows, bool need_cu);

// Fills cu and slot/fresh; tiles are set by the caller.
void fill_table(SeqTable& t, const mamba2_recurrent_batch* rb);

// SMs of the current device.
int device_sm_count();

}  // namespace mamba2
