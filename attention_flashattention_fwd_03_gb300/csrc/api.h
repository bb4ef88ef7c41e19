// api.h -- what the files that hold C entry points share: per-device set-up, tensor-map
// encoding, argument checks and the wait limits (all defined in api.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <cstdint>

#include "gbattn.h"
#include "internal.h"

#define GBATTN_API extern "C" __attribute__((visibility("default")))

namespace gbattn {

struct DeviceState {
  bool initialized = false;
  int status = ATTN_OK;
  int num_sms = 0;
  unsigned* flags = nullptr;
};

// One-time checks and kernel attributes of the current device; returns a status.
int device_state(DeviceState** out);

// The driver's cuTensorMapEncodeTiled.
int encoder(PFN_cuTensorMapEncodeTiled_v12000* fn);

// Tiled map over a bf16 tensor of `rank` dims (innermost first), 128-byte swizzle.
int encode_bf16(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* base,
                int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                const uint32_t* box);

inline bool aligned(const void* p, uintptr_t a) {
  return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

constexpr uint64_t kMaxDim = 1ull << 31;  // keeps every TMA coordinate inside int32

// See attn_test_set_failure.
extern std::atomic<unsigned long long> g_wait_limit_ns;  // limit of every wait in the kernels
extern std::atomic<int> g_withhold_copy;

FwdParams fwd_params(void* o, float* lse, int B, int Hq, int Hkv, int Tq, int Tk, int D,
                     int causal, float scale, unsigned* flags);

}  // namespace gbattn
