// kda_host.h -- host-side helpers shared by the C entry points: the thread's
// error text, argument predicates, metadata shipping and per-kernel timing.
// Defined in kda_api.cpp.
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
