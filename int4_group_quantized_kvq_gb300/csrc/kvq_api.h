// kvq_api.h -- what the files of the extern "C" boundary share: the per-thread error string
// and the checks of arguments.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "kvq.h"

namespace kvq {

// Set the calling thread's error string and return `code`; clear it and return KVQ_OK.
int fail(int code, const char* fmt, ...);
int ok();
int cuda_fail(cudaError_t e, const char* what);

// Geometry shared by every call on a K/V cache.  Returns KVQ_OK or an error (with the message set).
int check_cfg(const kvq_cache_config* c);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool is_pow2_in(int x, int lo, int hi) { return x >= lo && x <= hi && (x & (x - 1)) == 0; }

}  // namespace kvq
