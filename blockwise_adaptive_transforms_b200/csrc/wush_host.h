// Host helpers shared by the library's translation units: the per-thread record behind
// wush_last_error_detail() and the launch forms.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "wush.h"

#ifndef WUSH_USE_PDL
#define WUSH_USE_PDL 1
#endif

namespace wush {

// Records the failing call behind a WUSH_ERR_CUDA of this host thread; returns WUSH_ERR_CUDA.
int record_cuda_failure(int code, const char* what, const char* file, int line, bool driver);

inline bool is_aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

}  // namespace wush
