// Host helpers shared by the library's translation units: the per-thread record behind
// wush_last_error_detail() and the launch forms.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "wush.h"

#ifndef WUSH_USE_PDL
#define WUSH_USE_PDL 1
#endif

namespace wush {

// Records the failing call behind a WUSH_ERR_CUDA of this host thread; returns WUSH_ERR_CUDA.
int record_cuda_failure(int code, const char* what, const char* file, int line, bool driver);

// Tensor map of a row-major u8 matrix, 128-byte swizzle, boxes of box_cols x box_rows.
int encode_u8_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t cols, int box_cols, int box_rows);

// Address of the current device's error word, and the bound of in-kernel waits.
int device_error_word(unsigned int** word);
unsigned long long wait_limit_ns();

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace wush
