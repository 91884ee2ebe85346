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

// 16 bytes of a row as fp32 values, and back.
template <int WT>
struct Row16;
template <>
struct Row16<WT_BF16> {
  static constexpr int kVals = 8;
  __device__ __forceinline__ static void widen(const uint4& v, float* f) {
    const uint32_t p[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(p[i] << 16);
      f[2 * i + 1] = __uint_as_float(p[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ static uint4 narrow(const float* f) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
};
template <>
struct Row16<WT_F32> {
  static constexpr int kVals = 4;
  __device__ __forceinline__ static void widen(const uint4& v, float* f) {
    f[0] = __uint_as_float(v.x);
    f[1] = __uint_as_float(v.y);
    f[2] = __uint_as_float(v.z);
    f[3] = __uint_as_float(v.w);
  }
  __device__ __forceinline__ static uint4 narrow(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

}  // namespace sfn
