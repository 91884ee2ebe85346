// The paged key/value cache's bookkeeping and writes: the plan of a step (which pages each
// request holds, where each new token goes) and the append of the step's keys and values.

#include <algorithm>

#include "kernels.h"
#include "serving_common.h"
#include "sparse_ffn.h"

namespace sfn {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanWaves = kPlanThreads / 64;

// ---- plan ----------------------------------------------------------------------------
//
// With p tokens to a page, request r holds h = ceil(held / p) pages and needs
// m = ceil((ctx + new) / p). Requests with m < h give back entries [m, h) of their table
// row, pushed on the stack of free pages in request order; then those with m > h take
// m - h pages each from its top, in request order. Three prefix sums over the requests
// (new tokens, pages taken, pages given back) place everything, so each output element is
// computed on its own: token i finds its request by binary search, and a taken page is
// either a given-back one (the last ones pushed) or an old stack entry.
//
// One launch: every workgroup repeats the prefix sums over all requests (12 bytes each, at
// most 4096 of them, from the L2) and then does its share of the outputs; with a second
// launch or a grid-wide wait the outputs would start later than the repeated sums end. No
// workgroup reads what another writes: released entries are read from rows that take
// nothing, taken entries are written into rows that release nothing; when more is given
// back than taken only stack entries at and above n_free are written, and then no stack
// entry is read, otherwise none is written. The same inputs may therefore be planned again
// with the same result. Bound by latency: launch, one round of loads, the sums, a search, and
// the reads it leads to. Four requests 3.3 us, 1024 requests with 25000 tokens 5.8 us.
__device__ __forceinline__ int upper(const int* cu, int n, int v) {
  // the r with cu[r] <= v < cu[r + 1], for 0 <= v < cu[n]
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

__global__ __launch_bounds__(kPlanThreads) void kv_plan_kernel(KvPlanArgs a) {
  extern __shared__ int s_cu[];  // three arrays of R + 1: new tokens, pages taken, pages given back
  __shared__ int s_wave[3][kPlanWaves];
  __shared__ int s_bad;
  const int R = a.R, lg = a.page_shift, pm = (1 << lg) - 1;
  int* const s_new = s_cu;
  int* const s_take = s_cu + (R + 1);
  int* const s_rel = s_cu + 2 * (R + 1);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) s_bad = 0;
  const int given = gp(a.n_free)[0];
  const bool counted = given >= 0 && given <= a.n_pages;
  const int n_free = counted ? given : 0;
  __syncthreads();
  const int per = (R + kPlanThreads - 1) / kPlanThreads;
  const int r0 = tid * per, r1 = min(R, r0 + per);
  int sum[3] = {0, 0, 0};
  int bad = 0;
  for (int r = r0; r < r1; ++r) {
    const int held = gp(a.held)[r], ctx = gp(a.ctx)[r], nw = gp(a.fresh)[r];
    const int64_t cap = (int64_t)a.max_pages << lg;
    int n = 0, t = 0, b = 0;
    if (held < 0 || ctx < 0 || nw < 0 || ctx > held || held > cap || (int64_t)ctx + nw > cap || nw > a.max_tokens) {
      bad = 1;
    } else {
      const int h = (held + pm) >> lg, m = (ctx + nw + pm) >> lg;
      n = nw;
      t = max(m - h, 0);
      b = max(h - m, 0);
    }
    s_new[r + 1] = n;  // this request's own counts; turned into running sums below
    s_take[r + 1] = t;
    s_rel[r + 1] = b;
    sum[0] += n;
    sum[1] += t;
    sum[2] += b;
  }
  if (bad) s_bad = 1;
  int incl[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    incl[k] = wave_incl_scan(sum[k]);
    if (lane == 63) s_wave[k][wave] = incl[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    int base = incl[k] - sum[k];
    for (int w = 0; w < wave; ++w) base += s_wave[k][w];
    int* dst = k == 0 ? s_new : k == 1 ? s_take : s_rel;
    for (int r = r0; r < r1; ++r) {
      base += dst[r + 1];
      dst[r + 1] = base;
    }
    if (tid == 0) dst[0] = 0;
  }
  __syncthreads();
  const int T = s_new[R], takes = s_take[R], rels = s_rel[R];
  // the stack's room is compared first: rels alone may be near 2^31
  const int status = (s_bad || !counted || T > a.max_tokens || rels > a.n_pages - n_free) ? -1 : max(takes - (n_free + rels), 0);
  const bool ok = status == 0;
  // the first workgroups place the tokens, the others everything that goes by request or page:
  // each is a chain of dependent reads, and the chains run side by side
  const bool tokens = (int)blockIdx.x < a.token_groups;
  const int gid = (tokens ? blockIdx.x : blockIdx.x - a.token_groups) * kPlanThreads + tid;
  const int gsz = (tokens ? a.token_groups : gridDim.x - a.token_groups) * kPlanThreads;

  auto released = [&](int i) {  // number i of the pages given back
    const int r = upper(s_rel, R, i);
    const int m = (gp(a.ctx)[r] + gp(a.fresh)[r] + pm) >> lg;
    return gp(a.table)[(int64_t)r * a.max_pages + m + i - s_rel[r]];
  };
  auto taken = [&](int j) {  // number j of the pages taken
    const int top = n_free + rels - 1 - j;
    return top >= n_free ? released(top - n_free) : gp(a.free_pages)[top];
  };
  if (tokens) {
    for (int t = gid; t < a.max_tokens; t += gsz) {
      int pos = 0, slot = -1;
      if (ok && t < T) {
        const int r = upper(s_new, R, t);
        pos = gp(a.ctx)[r] + t - s_new[r];
        const int e = pos >> lg, h = (gp(a.held)[r] + pm) >> lg;
        const int page = e < h ? gp(a.table)[(int64_t)r * a.max_pages + e] : taken(s_take[r] + e - h);
        slot = (page << lg) + (pos & pm);
      }
      gp(a.pos)[t] = pos;
      gp(a.slot)[t] = slot;
    }
    return;
  }
  for (int r = gid; r < R; r += gsz) {
    gp(a.kv_len)[r] = ok ? gp(a.ctx)[r] + gp(a.fresh)[r] : 0;
    gp(a.cu)[r + 1] = ok ? s_new[r + 1] : 0;
  }
  if (ok) {
    for (int j = gid; j < takes; j += gsz) {
      const int r = upper(s_take, R, j);
      const int h = (gp(a.held)[r] + pm) >> lg;
      gp(a.table)[(int64_t)r * a.max_pages + h + j - s_take[r]] = taken(j);
    }
    for (int i = gid; i < rels - takes; i += gsz) gp(a.free_pages)[n_free + i] = released(i);
  }
  if (gid == 0) {
    gp(a.cu)[0] = 0;
    gp(a.n_free_out)[0] = ok ? n_free + rels - takes : given;
    gp(a.status)[0] = status;
  }
}

// ---- append --------------------------------------------------------------------------
//
// One workgroup per token. A rotation unit is one 16-byte chunk of the first half of a
// head's rotated values and the chunk half a rotation later; a thread keeps one unit's
// cosines and sines in registers and walks the heads with them, q's heads first, then k's.
// What is not rotated (the values, and the rest of each head) is copied. bf16 values are
// widened, turned in fp32 and rounded once. Every byte is read once and written once (counted:
// 169 and 164 MB of 8000 tokens, 64 / 8 heads of 128): HBM bound, 62 us, 5.3 TB/s where a large
// copy reaches 5.1; four tokens 2.8 us, latency. Non-temporal stores take 58 us instead of 63
// alone, but the attention that follows reads what is written here.
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

template <int WT>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a) {
  constexpr int E = Row16<WT>::kVals;
  constexpr int kB = WT == WT_BF16 ? 2 : 4;
  const int t = blockIdx.x, tid = threadIdx.x, nt = blockDim.x;
  const int slot = gp(a.slot)[t];
  const int lg = a.page_shift;
  const bool put = slot >= 0 && (slot >> lg) < a.n_pages;  // a token without a slot writes no key or value
  const int heads = a.h_q + (put ? a.h_kv : 0);
  const int head_bytes = a.dh * kB;
  const int64_t cell = put ? (((int64_t)(slot >> lg) * a.h_kv) << lg) + (slot & ((1 << lg) - 1)) : 0;  // head 0's row in the cache
  const SFN_GLOBAL char* q = gp(a.q) + (int64_t)t * a.q_stride;
  const SFN_GLOBAL char* k = gp(a.k) + (int64_t)t * a.k_stride;
  const SFN_GLOBAL char* v = gp(a.v) + (int64_t)t * a.v_stride;
  SFN_GLOBAL char* qo = gp(a.q_out) + (int64_t)t * a.h_q * head_bytes;
  auto src_of = [&](int h) { return h < a.h_q ? q + h * head_bytes : k + (h - a.h_q) * head_bytes; };
  auto dst_of = [&](int h) {
    return h < a.h_q ? qo + h * head_bytes : gp(a.k_cache) + (cell + ((int64_t)(h - a.h_q) << lg)) * head_bytes;
  };
  auto ld = [](const SFN_GLOBAL char* p) { return ld16(p); };
  auto st = [](SFN_GLOBAL char* p, const uint4& x) {
    *reinterpret_cast<SFN_GLOBAL u32x4_t*>(p) = u32x4_t{x.x, x.y, x.z, x.w};
  };
  const int half = a.rot / 2, units = half / E;
  if (units) {
    const int u = tid % units, step = nt / units;
    const int p = min(max(gp(a.pos)[t], 0), a.n_pos - 1);
    const SFN_GLOBAL float* cs = gp(a.rope) + (int64_t)p * a.rot + u * E;
    float c[E], s[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
      c[i] = cs[i];
      s[i] = cs[half + i];
    }
    for (int h = tid / units; h < heads && tid < units * step; h += step) {
      const SFN_GLOBAL char* src = src_of(h) + u * 16;
      float x[E], y[E], xr[E], yr[E];
      Row16<WT>::widen(ld(src), x);
      Row16<WT>::widen(ld(src + half * kB), y);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        xr[i] = x[i] * c[i] - y[i] * s[i];
        yr[i] = y[i] * c[i] + x[i] * s[i];
      }
      SFN_GLOBAL char* dst = dst_of(h) + u * 16;
      st(dst, Row16<WT>::narrow(xr));
      st(dst + half * kB, Row16<WT>::narrow(yr));
    }
  }
  const int rest = (a.dh - a.rot) / E;  // chunks of a head that are not rotated
  if (rest) {
    for (int i = tid; i < heads * rest; i += nt) {
      const int h = i / rest, at = a.rot * kB + (i % rest) * 16;
      st(dst_of(h) + at, ld(src_of(h) + at));
    }
  }
  if (put) {
    const int nch = a.dh / E;
    for (int i = tid; i < a.h_kv * nch; i += nt) {
      const int h = i / nch, at = (i % nch) * 16;
      st(gp(a.v_cache) + (cell + ((int64_t)h << lg)) * head_bytes + at, ld(v + h * head_bytes + at));
    }
  }
}

}  // namespace

hipError_t launch_kv_plan(const KvPlanArgs& a, hipStream_t stream) {
  // a workgroup for every 512 tokens (more than 200 would only repeat the sums), and two for
  // every 512 requests, which take or give back a page each now and then
  KvPlanArgs b = a;
  b.token_groups = (a.max_tokens + kPlanThreads - 1) / kPlanThreads;
  if (b.token_groups > 200) b.token_groups = 200;
  const int g = b.token_groups + 2 * ((a.R + kPlanThreads - 1) / kPlanThreads);
  hipLaunchKernelGGL(kv_plan_kernel, dim3(g), dim3(kPlanThreads), 3 * (a.R + 1) * sizeof(int), stream, b);
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs& a, int dtype, hipStream_t stream) {
  // as many threads as a token has units and chunks, from one wave to four: 8000 tokens of 4 / 2
  // heads of 64 take 6.4 us with one wave and 10.0 with four; of 12 / 4 heads 8.8 with two waves
  // and 10.5 with four
  const int e = dtype == SFN_BF16 ? 8 : 4;
  const int items = std::max((a.h_q + a.h_kv) * std::max(a.rot / 2, a.dh - a.rot) / e, a.h_kv * a.dh / e);
  const int threads = items <= 64 ? 64 : items <= 128 ? 128 : 256;
  if (dtype == SFN_BF16)
    hipLaunchKernelGGL(kv_append_kernel<WT_BF16>, dim3(a.T), dim3(threads), 0, stream, a);
  else
    hipLaunchKernelGGL(kv_append_kernel<WT_F32>, dim3(a.T), dim3(threads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace sfn
