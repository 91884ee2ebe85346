// The paged key/value cache in 8 bits: its writes (with the rotation of queries and keys) and
// reads of whole rows.

#include <algorithm>

#include "cache8.h"
#include "kernels.h"
#include "serving_common.h"
#include "sparse_ffn.h"

namespace sfn {

namespace {

// ---- append --------------------------------------------------------------------------
//
// One workgroup per token (of a few tokens, two). Queries are turned as kv_append_kernel turns them:
// a thread keeps the cosines and sines of 16 bytes of values and walks the heads with them. A row of
// K or V (one head's dh values) belongs to dh / 8 neighbouring lanes: the row's largest magnitude is
// a maximum over those lanes, its power of two a shift of that maximum's bits, and each value is
// rounded once, by the hardware's conversion to e4m3. A lane has four values and the four that they
// are turned with, so that nothing is loaded twice and their cosines and sines are read once for all
// of the lane's rows (against eight neighbouring values, with the partners and the cosines read for
// each row: 2000 tokens of 32 / 32 heads 35.2 -> 20.7 us, 6000 of 16 / 16 55.6 -> 36.5).
// Keys are turned in 64 bits: both products of a bf16 or fp32 value and an fp32 cosine are
// exact there, so a code is the one nearest to the rotated value but for one rounding to 53
// bits, whatever the order of operations; in 32 bits one value in a million would fall on the
// other side of a border between two codes. On the way to 32 bits the value is rounded to odd
// (cut, its last bit set if anything was lost), which a second rounding does not notice.
// Bound by memory: 8000 tokens, 64 / 8 heads of 128, 316 MB in 67 us, 4.7 TB/s where a large copy
// reaches 5.1; with the products in 32 bits it would be 62. Past-the-caches reads, the cache's
// rows before the queries and 512 threads gave 3 to 8% more time there. Where keys and values
// are most of it, each wave waits for its rows: 6000 tokens of 16 / 16 heads, 123 MB, 3.4 TB/s.
// Four tokens 3.0 us in a graph, 3.6 where each launch is timed alone: latency.
// Four values of a row.
template <int WT>
__device__ __forceinline__ void load4(const SFN_GLOBAL char* p, float* f) {
  if constexpr (WT == WT_BF16) {
    const uint64_t v = *reinterpret_cast<const SFN_GLOBAL uint64_t*>(p);
    f[0] = __uint_as_float((uint32_t)v << 16);
    f[1] = __uint_as_float((uint32_t)v & 0xffff0000u);
    f[2] = __uint_as_float((uint32_t)(v >> 32) << 16);
    f[3] = __uint_as_float((uint32_t)(v >> 32) & 0xffff0000u);
  } else {
    Row16<WT>::widen(ld16(p), f);
  }
}

// d in 32 bits, rounded to odd.
__device__ __forceinline__ float to_odd(double d) {
  uint32_t f = __float_as_uint((float)d);
  const double back = (double)__uint_as_float(f);
  if (back != d) f = (f - (fabs(back) > fabs(d) ? 1u : 0u)) | 1u;  // a NaN stays one
  return __uint_as_float(f);
}

// The largest v of each N consecutive lanes (N 8 or 16), in all of them.
template <int N>
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, dpp_mov<SFN_DPP_XOR1>(v));
  v = fmaxf(v, dpp_mov<SFN_DPP_XOR2>(v));
  v = fmaxf(v, dpp_mov<SFN_DPP_HALF_MIRROR>(v));
  if constexpr (N == 16) v = fmaxf(v, dpp_mov<SFN_DPP_ROW_MIRROR>(v));
  return v;
}

__device__ __forceinline__ bool finite(float x) { return (__float_as_uint(x) & 0x7f800000u) != 0x7f800000u; }

template <int WT, int DH>
__global__ __launch_bounds__(256) void kv8_append_kernel(Kv8AppendArgs a) {
  constexpr int E = Row16<WT>::kVals, kB = 16 / E, L = DH / 8;  // values of 16 bytes, bytes of one, lanes of a row
  const int t = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
  const int slot = gp(a.slot)[t];
  const int lg = a.page_shift;
  const bool put = slot >= 0 && (slot >> lg) < a.n_pages;  // a token without a slot writes no key or value
  const int half = a.rot / 2;
  const SFN_GLOBAL float* rope = nullptr;
  if (half) rope = gp(a.rope) + (int64_t)min(max(gp(a.pos)[t], 0), a.n_pos - 1) * a.rot;

  // queries
  if (blockIdx.y == 0) {
    const SFN_GLOBAL char* q = gp(a.q) + (int64_t)t * a.q_stride;
    SFN_GLOBAL char* qo = gp(a.q_out) + (int64_t)t * a.h_q * DH * kB;
    auto load = [&](int at, float (&f)[E]) { Row16<WT>::widen(ld16(q + at), f); };
    auto store = [&](int at, const float (&f)[E]) {
      const uint4 x = Row16<WT>::narrow(f);
      *reinterpret_cast<SFN_GLOBAL u32x4_t*>(qo + at) = u32x4_t{x.x, x.y, x.z, x.w};
    };
    const int units = half / E;
    if (units && a.h_q) {
      const int u = tid % units, step = nt / units;
      float c[E], s[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        c[i] = rope[u * E + i];
        s[i] = rope[half + u * E + i];
      }
      for (int h = tid / units; h < a.h_q && tid < units * step; h += step) {
        const int at = h * DH * kB + u * 16;
        float x[E], y[E], xr[E], yr[E];
        load(at, x);
        load(at + half * kB, y);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          xr[i] = x[i] * c[i] - y[i] * s[i];
          yr[i] = y[i] * c[i] + x[i] * s[i];
        }
        store(at, xr);
        store(at + half * kB, yr);
      }
    }
    const int rest = (DH - a.rot) / E;  // units of a head that are not turned
    for (int i = tid; i < a.h_q * rest; i += nt) {
      const int at = (i / rest * DH + a.rot) * kB + (i % rest) * 16;
      float x[E];
      load(at, x);
      store(at, x);
    }
  }
  if (!put || (gridDim.y == 2 && blockIdx.y == 0)) return;

  // keys, then values; whole waves take part in the maxima
  const int64_t cell = (((int64_t)(slot >> lg) * a.h_kv) << lg) + (slot & ((1 << lg) - 1));  // head 0's row in the cache
  const int rows = 2 * a.h_kv, lane = tid % L;
  const bool turned = 8 * lane < a.rot;
  float c[4], s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = turned ? rope[4 * lane + i] : 0.f;
    s[i] = turned ? rope[half + 4 * lane + i] : 0.f;
  }
  for (int r0 = 0; r0 < rows; r0 += nt / L) {
    const int r = r0 + tid / L;
    const bool mine = r < rows, key = r < a.h_kv;
    const int h = key ? r : r - a.h_kv;
    // the lane's values: four from `lo` on, and their partners from `hi` on
    const int lo = key && !turned ? 8 * lane : 4 * lane, hi = key ? lo + (turned ? half : 4) : lo + DH / 2;
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (mine) {
      const SFN_GLOBAL char* row = (key ? gp(a.k) + (int64_t)t * a.k_stride : gp(a.v) + (int64_t)t * a.v_stride) + h * DH * kB;
      load4<WT>(row + lo * kB, x);
      load4<WT>(row + hi * kB, x + 4);
      if (key && turned) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const double u = x[i], w = x[4 + i], cd = c[i], sd = s[i];
          x[i] = to_odd(u * cd - w * sd);
          x[4 + i] = to_odd(w * cd + u * sd);
        }
      }
    }
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, finite(x[i]) ? fabsf(x[i]) : 0.f);
    const int b = exp_of_row(group_max<L>(top));
    const float scale = __uint_as_float((uint32_t)(254 - b) << 23);  // 2^(127 - b)
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)  // e4m3 has no infinity: it becomes NaN, as NaN does
      y[i] = finite(x[i]) ? fminf(fmaxf(x[i] * scale, -448.f), 448.f) : __uint_as_float(0x7fc00000u);
    if (mine) {
      const int64_t to = cell + ((int64_t)h << lg);
      SFN_GLOBAL char* const codes = (key ? gp(a.k_cache) : gp(a.v_cache)) + to * DH;
      *reinterpret_cast<SFN_GLOBAL uint32_t*>(codes + lo) = pack_e4m3(y[0], y[1], y[2], y[3]);
      *reinterpret_cast<SFN_GLOBAL uint32_t*>(codes + hi) = pack_e4m3(y[4], y[5], y[6], y[7]);
      if (lane == 0) (key ? gp(a.k_exp) : gp(a.v_exp))[to] = (uint8_t)b;
    }
  }
}

// ---- read ----------------------------------------------------------------------------
//
// Rows of K and V by slots, as the values they stand for: exact in bf16 and fp32 (four bits of
// significand and a power of two). Bound by memory: 60000 tokens, 8 heads of 128, 370 MB in 70 us,
// 5.3 TB/s, in bf16; 20000 in fp32, 205 MB in 40.5 us. A lane turns 16 codes into bf16 (with 8: 79
// us), 8 into fp32 (with 16 its stores lie too far apart: 122 us), and a workgroup takes as many
// tokens as give all of its lanes a piece (60000 tokens of 2 heads of 64, one token to a workgroup
// 16 us, with eight 10.9). Codes are read once and past the caches; results that the caches would
// not hold go past them too (70 instead of 77 us), others do not (2000 tokens 3.7 instead of 4.2).
template <int WT>
constexpr int kReadCodes = WT == WT_BF16 ? 16 : 8;

template <int WT, int DH, bool PAST>
__global__ __launch_bounds__(256) void kv8_read_kernel(Kv8ReadArgs a) {
  constexpr int kB = WT == WT_BF16 ? 2 : 4, E = kReadCodes<WT>, L = DH / E;
  const int lg = a.page_shift, per = 2 * a.h_kv * L;  // lanes of a token
  for (int i = threadIdx.x; i < a.tokens * per; i += blockDim.x) {
    const int t = blockIdx.x * a.tokens + i / per, r = i % per / L, at = (i % L) * E;
    if (t >= a.T) return;
    const int slot = gp(a.slot)[t];
    const bool held = slot >= 0 && (slot >> lg) < a.n_pages, key = r < a.h_kv;
    const int h = key ? r : r - a.h_kv;
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = 0.f;
    if (held) {
      const int64_t from = ((((int64_t)(slot >> lg) * a.h_kv) + h) << lg) + (slot & ((1 << lg) - 1));
      const SFN_GLOBAL char* p = (key ? gp(a.k_cache) : gp(a.v_cache)) + from * DH + at;
      const float scale = scale_of((key ? gp(a.k_exp) : gp(a.v_exp))[from]);
      typedef __attribute__((ext_vector_type(E / 4))) uint32_t Codes;
      const Codes w = __builtin_nontemporal_load(reinterpret_cast<const SFN_GLOBAL Codes*>(p));
#pragma unroll
      for (int e = 0; e < E; e += 4) values_of(w[e / 4], scale, x + e);
    }
    SFN_GLOBAL char* to = (key ? gp(a.k_out) + (int64_t)t * a.k_stride : gp(a.v_out) + (int64_t)t * a.v_stride) + (h * DH + at) * kB;
#pragma unroll
    for (int e = 0; e < E; e += 16 / kB) {
      u32x4_t v;
      if constexpr (WT == WT_BF16)
        v = u32x4_t{pack_bf16(x[e], x[e + 1]), pack_bf16(x[e + 2], x[e + 3]), pack_bf16(x[e + 4], x[e + 5]), pack_bf16(x[e + 6], x[e + 7])};
      else
        v = __builtin_bit_cast(u32x4_t, (f32x4_t{x[e], x[e + 1], x[e + 2], x[e + 3]}));
      SFN_GLOBAL u32x4_t* const o = reinterpret_cast<SFN_GLOBAL u32x4_t*>(to + e * kB);
      if constexpr (PAST) __builtin_nontemporal_store(v, o);
      else *o = v;
    }
  }
}

// Up to so many tokens, a token's queries and its rows of the cache are a workgroup each, which run
// side by side (4 tokens, 32 / 8 heads, when each took half a microsecond more than now, 3.53 us where
// one after the other took 4.00); more fill the chip as they are (8000 tokens, 64 / 8 heads, 67 us against 73, 2000 of 32 / 32 20.9 against 20.6).
constexpr int kApart = 1024;
constexpr int64_t kHeld = 64 << 20;  // bytes that are written past the caches if there are more

int threads_for(int items) { return items <= 64 ? 64 : items <= 128 ? 128 : 256; }

template <int WT>
void launch_append(const Kv8AppendArgs& a, int dh, int threads, hipStream_t stream) {
  if (dh == 64) hipLaunchKernelGGL((kv8_append_kernel<WT, 64>), dim3(a.T, a.T <= kApart ? 2 : 1), dim3(threads), 0, stream, a);
  else hipLaunchKernelGGL((kv8_append_kernel<WT, 128>), dim3(a.T, a.T <= kApart ? 2 : 1), dim3(threads), 0, stream, a);
}
template <int WT, int DH>
void launch_read(Kv8ReadArgs a, hipStream_t stream) {
  const int per = 2 * a.h_kv * DH / kReadCodes<WT>;
  a.tokens = std::clamp(256 / per, 1, 16);
  const dim3 grid((a.T + a.tokens - 1) / a.tokens), threads(threads_for(a.tokens * per));
  if ((int64_t)a.T * a.h_kv * DH * (WT == WT_BF16 ? 4 : 8) > kHeld) hipLaunchKernelGGL((kv8_read_kernel<WT, DH, true>), grid, threads, 0, stream, a);
  else hipLaunchKernelGGL((kv8_read_kernel<WT, DH, false>), grid, threads, 0, stream, a);
}

}  // namespace

hipError_t launch_kv8_append(const Kv8AppendArgs& a, int dh, int dtype, hipStream_t stream) {
  const int e = dtype == SFN_BF16 ? 8 : 4, threads = threads_for(std::max(a.h_q * std::max(a.rot / 2, dh - a.rot) / e, 2 * a.h_kv * dh / 8));
  if (dtype == SFN_BF16) launch_append<WT_BF16>(a, dh, threads, stream);
  else launch_append<WT_F32>(a, dh, threads, stream);
  return hipGetLastError();
}

hipError_t launch_kv8_read(const Kv8ReadArgs& a, int dh, int dtype, hipStream_t stream) {
  if (dtype == SFN_BF16) {
    if (dh == 64) launch_read<WT_BF16, 64>(a, stream);
    else launch_read<WT_BF16, 128>(a, stream);
  } else {
    if (dh == 64) launch_read<WT_F32, 64>(a, stream);
    else launch_read<WT_F32, 128>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace sfn
