// Device helpers of the kernels between the FFN steps (paged cache, attention, norm), beside
// device_common.h, whose code the decode kernels' counter summary is tied to.
#pragma once

#include "device_common.h"

namespace sfn {

// The larger of v and the v of lane l ^ BIT (BIT 16 or 32), the same in both lanes.
template <int BIT>
__device__ __forceinline__ float swap_pair_max(float v) {
  float a = v, b = v;
  lane_swap<BIT>(a, b);
  return fmaxf(a, b);
}

// The largest v of the 64 lanes, in every lane.
__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_mov<SFN_DPP_XOR1>(v));
  v = fmaxf(v, dpp_mov<SFN_DPP_XOR2>(v));
  v = fmaxf(v, dpp_mov<SFN_DPP_HALF_MIRROR>(v));
  v = fmaxf(v, dpp_mov<SFN_DPP_ROW_MIRROR>(v));
  v = swap_pair_max<16>(v);
  return swap_pair_max<32>(v);
}

// Between a wave's writes to LDS and its lanes' reads of each other's: LDS does a wave's
// accesses in order, so this only keeps the compiler from moving them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 2^x by the hardware's exponential (one instruction; results below the smallest normal
// number flush to zero, which for softmax weights relative to the row's largest is nothing).
__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }

typedef __attribute__((ext_vector_type(2))) float f32x2_t;

// Two fp32 values rounded to bf16 (nearest, ties to even; NaN stays NaN), a in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2_t{a, b}), bf16x2_t));
}

}  // namespace sfn
