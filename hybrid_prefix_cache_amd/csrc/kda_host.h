// kda_host.h -- host-side helpers shared by the C entry points: the thread's
// error text, argument predicates, metadata shipping and per-kernel timing.
// Defined in kda_api.cpp, validating() in kda_kv_api.cpp, check_paths in kda_tree_api.cpp.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <vector>

#include "../../include/kda.h"

namespace kda {

// Sets the thread's error text and returns st; ok() clears it.
kda_status fail(kda_status st, const char* fmt, ...);
kda_status ok();
kda_status hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline bool valid_dtype(int d) { return d == KDA_F32 || d == KDA_BF16; }

// KDA_VALIDATE=1: device tables are read back and checked before a call.
bool validating();

kda_status check_conv_pool(const kda_conv_pool* p);

// KDA_VALIDATE=1: the accepted paths of n requests, read back to *p and *c and checked.
kda_status check_paths(const char* what, const int32_t* path, const int32_t* count, int32_t n, int32_t tokens,
                       std::vector<int32_t>* p, std::vector<int32_t>* c, hipStream_t st);

// Copies a host table into the workspace through kernel arguments.
kda_status ship_metadata(uint8_t* ws, const std::vector<uint8_t>& blob, hipStream_t st);

// Brackets one launch with events when timing is enabled.
class Launch {
 public:
  Launch(const char* name, hipStream_t st);
  ~Launch();

 private:
  const char* name_;
  hipStream_t st_;
  hipEvent_t ev0_ = nullptr, ev1_ = nullptr;
};

}  // namespace kda
