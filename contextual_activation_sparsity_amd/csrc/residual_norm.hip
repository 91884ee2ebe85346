// The update of the residual stream between two blocks, with the norms on either side of
// it: h_out = h + scale gate N(y; w_post), x_out = N(h_out; w_pre), N(v; w) =
// v / sqrt(mean(v^2) + eps) w. One workgroup per token holds the row in registers, so
// every input is read once and every output written once, with the two sums of squares
// (fp32) between. x_out is computed from the fp32 row, before h_out is rounded: each
// output is rounded once. HBM bound for many tokens: 8192 of 8192 values with both norms and a
// gate 124 us, 5.4 TB/s where a large copy reaches 5.1 (non-temporal accesses 122 to 127, gate
// and weights read before the first sum 128). One token of 4096: 2.8 us back to back in a
// graph, the launch, one round of loads and the workgroup-wide sums.

#include "kernels.h"
#include "serving_common.h"
#include "sparse_ffn.h"

namespace sfn {

namespace {

constexpr int kNormVals = 8;  // values a thread handles together

template <int WT>
__device__ __forceinline__ void load8(const SFN_GLOBAL char* p, int64_t i, float* f) {
  if constexpr (WT == WT_BF16) {
    const uint4 v = ld16(p + i * 16);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
    const uint4 a = ld16(p + i * 32), b = ld16(p + i * 32 + 16);
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
  }
}

template <int WT>
__device__ __forceinline__ void store8(SFN_GLOBAL char* p, int64_t i, const float* f) {
  if constexpr (WT == WT_BF16) {
    *reinterpret_cast<SFN_GLOBAL u32x4_t*>(p + i * 16) =
        u32x4_t{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  } else {
    *reinterpret_cast<SFN_GLOBAL f32x4_t*>(p + i * 32) = f32x4_t{f[0], f[1], f[2], f[3]};
    *reinterpret_cast<SFN_GLOBAL f32x4_t*>(p + i * 32 + 16) = f32x4_t{f[4], f[5], f[6], f[7]};
  }
}

template <int NT>
__device__ __forceinline__ float block_sum(float v, float* s_part) {
  v = wave_sum(v);
  if constexpr (NT == 64) return v;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  __syncthreads();  // the previous sum has been read
  if (lane == 0) s_part[wave] = v;
  __syncthreads();
  float t = 0.f;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) t += s_part[w];
  return t;
}

template <int HT, int YT, int WT, int NT, int NV>
__global__ __launch_bounds__(NT) void residual_norm_kernel(NormArgs a) {
  __shared__ float s_part[NT / 64];
  const int t = blockIdx.x, tid = threadIdx.x;
  const int nch = a.d / kNormVals;
  const int64_t row = (int64_t)t * nch;
  const float inv_d = 1.0f / (float)a.d;
  float h[NV][kNormVals];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = tid + v * NT;
    if (i < nch) load8<HT>(gp(a.h), row + i, h[v]);
    else
#pragma unroll
      for (int j = 0; j < kNormVals; ++j) h[v][j] = 0.f;
  }
  if (a.y) {
    float y[NV][kNormVals];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = tid + v * NT;
      if (i < nch) load8<YT>(gp(a.y), row + i, y[v]);
      else
#pragma unroll
        for (int j = 0; j < kNormVals; ++j) y[v][j] = 0.f;
    }
    float s = 1.f;
    if (a.w_post) {
      float q = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int j = 0; j < kNormVals; ++j) q = fmaf(y[v][j], y[v][j], q);
      q = block_sum<NT>(q, s_part);
      s = 1.0f / sqrtf(fmaf(q, inv_d, a.eps));
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = tid + v * NT;
      if (i >= nch) continue;
      if (a.w_post) {
        float w[kNormVals];
        load8<WT>(gp(a.w_post), i, w);
#pragma unroll
        for (int j = 0; j < kNormVals; ++j) y[v][j] = y[v][j] * s * w[j];
      }
      if (a.gate) {
        float g[kNormVals];
        load8<WT>(gp(a.gate) + (int64_t)t * a.gate_stride, i, g);
#pragma unroll
        for (int j = 0; j < kNormVals; ++j) y[v][j] *= g[j];
      }
#pragma unroll
      for (int j = 0; j < kNormVals; ++j) h[v][j] = fmaf(a.scale, y[v][j], h[v][j]);
      if (a.h_out) store8<HT>(gp(a.h_out), row + i, h[v]);
    }
  }
  if (!a.x_out) return;
  float q = 0.f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int j = 0; j < kNormVals; ++j) q = fmaf(h[v][j], h[v][j], q);
  q = block_sum<NT>(q, s_part);
  const float s = 1.0f / sqrtf(fmaf(q, inv_d, a.eps));
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int i = tid + v * NT;
    if (i >= nch) continue;
    float w[kNormVals];
    load8<WT>(gp(a.w_pre), i, w);
#pragma unroll
    for (int j = 0; j < kNormVals; ++j) w[j] = h[v][j] * s * w[j];
    store8<WT>(gp(a.x_out), row + i, w);
  }
}

// One 8-value chunk to a thread where the row allows it: 4000 tokens of 4096 values 32.6 us
// with 512 threads, 35.5 with 256 of two chunks, one token 2.8 and 3.5 us; 20000 tokens of 512
// values 21 us with one wave, 34 with 256 threads. Rows past 512 chunks: 8192 values of up to
// kFewRows tokens with 1024 threads (one token 3.4 us, with 512 threads 3.7), of more with 512
// (1000 tokens 14.1 us, with 1024 threads 16.5).
constexpr int kFewRows = 256;

template <int HT, int YT, int WT, int NT, int NV>
void launch_as(const NormArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL((residual_norm_kernel<HT, YT, WT, NT, NV>), dim3(a.T), dim3(NT), 0, stream, a);
}

template <int HT, int YT, int WT>
void launch_sized(const NormArgs& a, hipStream_t stream) {
  const int nch = a.d / kNormVals;
  if (nch <= 64) launch_as<HT, YT, WT, 64, 1>(a, stream);
  else if (nch <= 128) launch_as<HT, YT, WT, 128, 1>(a, stream);
  else if (nch <= 256) launch_as<HT, YT, WT, 256, 1>(a, stream);
  else if (nch <= 512) launch_as<HT, YT, WT, 512, 1>(a, stream);
  else if (nch <= 1024 && a.T > kFewRows) launch_as<HT, YT, WT, 512, 2>(a, stream);
  else if (nch <= 1024) launch_as<HT, YT, WT, 1024, 1>(a, stream);
  else launch_as<HT, YT, WT, 1024, 2>(a, stream);
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, int hdtype, int ydtype, int wdtype, hipStream_t stream) {
  const int k = (hdtype == SFN_BF16 ? 4 : 0) | (ydtype == SFN_BF16 ? 2 : 0) | (wdtype == SFN_BF16 ? 1 : 0);
  switch (k) {
    case 0: launch_sized<WT_F32, WT_F32, WT_F32>(a, stream); break;
    case 1: launch_sized<WT_F32, WT_F32, WT_BF16>(a, stream); break;
    case 2: launch_sized<WT_F32, WT_BF16, WT_F32>(a, stream); break;
    case 3: launch_sized<WT_F32, WT_BF16, WT_BF16>(a, stream); break;
    case 4: launch_sized<WT_BF16, WT_F32, WT_F32>(a, stream); break;
    case 5: launch_sized<WT_BF16, WT_F32, WT_BF16>(a, stream); break;
    case 6: launch_sized<WT_BF16, WT_BF16, WT_F32>(a, stream); break;
    default: launch_sized<WT_BF16, WT_BF16, WT_BF16>(a, stream); break;
  }
  return hipGetLastError();
}

}  // namespace sfn
