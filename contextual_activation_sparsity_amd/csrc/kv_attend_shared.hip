// Attention of requests that share a prefix, whose keys and values are read once for all of them.

#include "attend_device.h"

namespace sfn {

namespace {

// ---- the parts -----------------------------------------------------------------------
//
// With m, l and o the running maximum, sum of weights and weighted sum of the values over some
// of a row's keys, those over two sets of keys join to
//   m = max(m1, m2),  l = l1 2^(m1 - m) + l2 2^(m2 - m),  o = o1 2^(m1 - m) + o2 2^(m2 - m),
// so the keys of the prefix are attended to once by the rows of all requests' tokens together
// (all of them see all of it), each request's other keys by its own rows, and the parts are joined.
// One launch does both: the first workgroups take row tiles and splits of the prefix, which the
// products or the latency of its few stages bound, the others the requests' own keys, which
// memory binds; side by side they take about as long as the longer of them. As two launches (a
// prefix's and the requests', then the join) 6 fp32 chunks over 300 shared keys took 14.1 us where
// this takes 9.3, 8 tokens after 2000 shared keys 19.7 (13.2), 48 after 8000 48.2 (46.0), 32 chunks
// after 60000 665 (641).
// WAY is how a workgroup takes the rows of one key head: 1 and 2 are split attention with 16 and 32
// rows, 3 is tile attention. All tokens have at least as many rows as one request's, so the prefix's
// way is never the smaller one. The registers of a launch are those of its larger way: with 16 rows
// in both parts three workgroups share a compute unit, otherwise two.
// 48 single tokens after 8000 shared keys, each with up to 1000 of its own, 32 / 8 heads of 128,
// bf16, 123 MB: 43.2 us, 37 in this launch and 6 to 7 in the join, 2.8 TB/s. The requests' part
// alone takes 22 us with three workgroups to a compute unit and 31 with two; two tiles of keys held
// at once there (255 registers), or the first page guessed from the shared length, gave 1 to 2%.
// The prefix in tiles serves requests whose own keys go through split attention, as all of them
// would in calls without a prefix, whose maximum is exact. It is here too then: the 48 tokens are off
// by 0.0018 of the result instead of 0.0021, for 43.1 instead of 42.6 us (64 after 30000 66.0 and
// 65.1, 32 chunks of up to 8 after 20000 84.2 and 80.7).
template <int WT, int CT, int DH, int WAY, int KIND, bool EXACT, int SIZE_A, int SIZE_B>
__device__ __forceinline__ void attend_way(const AttendArgs& a, uint32_t bx, int split, int r, char (&s_a)[SIZE_A], char (&s_b)[SIZE_B],
                                           float (&s_m)[4][32], float (&s_l)[4][32]) {
  if constexpr (WAY == 3)
    tile_attention<CT, DH, 1, KIND, EXACT>(a, bx, split, r, s_a, s_b, reinterpret_cast<uint32_t(&)[4]>(s_m));
  else
    split_attention<WT, CT, DH, WAY, 4, KIND>(a, bx, split, r, reinterpret_cast<float(&)[4][16 * WAY]>(s_m),
                                              reinterpret_cast<float(&)[4][16 * WAY]>(s_l), PermutedRows<DH>{s_a, s_b});
}

template <int WT, int CT, int DH, int PREFIX_WAY, int OWN_WAY>
__global__ __launch_bounds__(256, PREFIX_WAY == 1 ? 3 : 2) void attend_shared_kernel(SharedArgs x) {
  static_assert(OWN_WAY <= PREFIX_WAY, "more rows in the prefix's part");
  constexpr int SIZE = 2 * kTileKeys * DH * 2;  // a stage of K and of V, or four waves' 16 rows in fp32
  static_assert(SIZE == 4 * 16 * DH * 4, "the ways' arrays are of one size");
  __shared__ __attribute__((aligned(16))) char s_a[SIZE];
  __shared__ __attribute__((aligned(16))) char s_b[PREFIX_WAY == 1 ? 16 : SIZE];
  __shared__ float s_m[4][32], s_l[4][32];
  const int i = blockIdx.x - x.prefix_groups;
  const AttendArgs& a = x.own;
  if (i < 0) {
    const int per = x.prefix.row_tiles * x.prefix.h_kv, split = blockIdx.x / per;
    attend_way<WT, CT, DH, PREFIX_WAY, ATTEND_PREFIX, OWN_WAY != 3>(x.prefix, blockIdx.x - split * per, split, 0, s_a, s_b, s_m, s_l);
  } else {
    const int per = a.row_tiles * a.h_kv, t = i / per, S = a.S | 1, r = t / S;
    attend_way<WT, CT, DH, OWN_WAY, ATTEND_OWN, false>(a, i - t * per, t - r * S, r, s_a, s_b, s_m, s_l);
  }
}

// Joins one output row of a call over a shared prefix: the parts of the keys behind it (a, by request
// or by token) and of the prefix (p, by token), which count where the request's tokens come after it.
template <int WT, int DH, bool WAVE>
__global__ __launch_bounds__(256) void attend_join_shared_kernel(SharedArgs x) {
  const AttendArgs &a = x.own, &p = x.prefix;
  constexpr int NT = WAVE ? 64 : 256;        // threads of a row
  constexpr int LD = DH / 4, NS = NT / LD;   // lanes of a row's values, parts side by side
  constexpr int U = 8;                       // loads in flight
  constexpr int NP = 2 * kMaxSplits, NK = NP / NT;
  __shared__ float s_w[WAVE ? 4 : 1][NP];
  __shared__ float s_red[8];
  __shared__ f32x4_t s_o[256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tid = WAVE ? lane : threadIdx.x;
  const int i = blockIdx.x, r = blockIdx.z, head = WAVE ? blockIdx.y * 4 + wave : blockIdx.y;
  if (WAVE && head >= a.h_q) return;
  float* const w_of = s_w[WAVE ? wave : 0];
  const Request<ATTEND_OWN> req(a, r);
  if (i >= req.n) return;
  const int shared = Request<ATTEND_OWN>::shared_len(a);
  const int mine = splits_used(a, req, i, head);
  const int all = mine + (req.past >= shared ? (shared + p.chunk - 1) / p.chunk : 0);
  const int64_t at_a = (req.place(a, r, i) * a.h_q + head) * a.S;
  const int64_t at_p = ((int64_t)req.in_prefix(a, p.max_new, r, i) * a.h_q + head) * p.S;
  const SFN_GLOBAL f32x2_t* ml_a = reinterpret_cast<const SFN_GLOBAL f32x2_t*>(gp(a.part_ml)) + at_a;
  const SFN_GLOBAL f32x2_t* ml_p = reinterpret_cast<const SFN_GLOBAL f32x2_t*>(gp(p.part_ml)) + at_p;
  const int d4 = tid % LD, s0 = tid / LD;
  const SFN_GLOBAL f32x4_t* o_a = reinterpret_cast<const SFN_GLOBAL f32x4_t*>(gp(a.part_o) + at_a * DH) + d4;
  const SFN_GLOBAL f32x4_t* o_p = reinterpret_cast<const SFN_GLOBAL f32x4_t*>(gp(p.part_o) + at_p * DH) + d4;
  auto part = [&](int s) { return s < mine ? o_a[(int64_t)s * LD] : o_p[(int64_t)(s - mine) * LD]; };
  f32x4_t v[U];  // the first of them on their way while the weights are found
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = part(min(s0 + u * NS, all - 1));

  float m[NK], l[NK], M = kNegInf;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const int s = tid + k * NT;
    f32x2_t x = {kNegInf, 0.f};
    if (s < all) x = s < mine ? ml_a[s] : ml_p[s - mine];
    m[k] = x[0];
    l[k] = x[1];
    M = fmaxf(M, m[k]);
  }
  M = wave_max(M);
  if constexpr (!WAVE) {
    if (lane == 0) s_red[wave] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  }
  float L = 0.f;
#pragma unroll
  for (int k = 0; k < NK; ++k) {
    const float w = m[k] == kNegInf ? 0.f : exp2_f(m[k] - M);
    w_of[tid + k * NT] = w;
    L += w * l[k];
  }
  L = wave_sum(L);
  if constexpr (!WAVE) {
    if (lane == 0) s_red[4 + wave] = L;
    __syncthreads();
    L = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
  } else {
    wave_sync();
  }
  f32x4_t o = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < all; s += U * NS) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * NS < all) o += v[u] * w_of[s + u * NS];  // also for weight 0: NaN scores show
    if (s + U * NS < all) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = part(min(s + (U + u) * NS, all - 1));
    }
  }
  f32x4_t* const o_of = s_o + (WAVE ? 64 * wave : 0);
  o_of[tid] = o;
  if constexpr (WAVE) wave_sync();
  else __syncthreads();
  if (tid < LD) {
#pragma unroll
    for (int s = 1; s < NS; ++s) o += o_of[s * LD + d4];
    store_row<WT, DH>(a, req.t0 + i, head, 4 * d4, o, L);
  }
}

template <int WT, int CT, int DH, int PREFIX_WAY, int OWN_WAY>
void launch_ways(const SharedArgs& a, hipStream_t stream) {
  const int groups = a.prefix_groups + a.own.R * (a.own.S | 1) * a.own.row_tiles * a.own.h_kv;
  hipLaunchKernelGGL((attend_shared_kernel<WT, CT, DH, PREFIX_WAY, OWN_WAY>), dim3(groups), dim3(256), 0, stream, a);
}

template <int WT, int CT, int DH>
void launch_shared(SharedArgs a, hipStream_t stream) {
  a.prefix_groups = a.prefix.row_tiles * a.prefix.h_kv * a.prefix.S;
  auto way = [](const AttendArgs& p) { return p.tile_rows == 16 ? 1 : p.tile_rows == 32 ? 2 : 3; };
  const int prefix = way(a.prefix), own = way(a.own);
  if (prefix == 1) launch_ways<WT, CT, DH, 1, 1>(a, stream);
  else if (prefix == 2 && own == 1) launch_ways<WT, CT, DH, 2, 1>(a, stream);
  else if (prefix == 2) launch_ways<WT, CT, DH, 2, 2>(a, stream);
  else if constexpr (WT == WT_BF16) {
    if (own == 1) launch_ways<WT, CT, DH, 3, 1>(a, stream);
    else if (own == 2) launch_ways<WT, CT, DH, 3, 2>(a, stream);
    else launch_ways<WT, CT, DH, 3, 3>(a, stream);
  }
  const AttendArgs& o = a.own;
  if ((int64_t)o.R * o.max_new * o.h_q >= kJoinByWave)
    hipLaunchKernelGGL((attend_join_shared_kernel<WT, DH, true>), dim3(o.max_new, (o.h_q + 3) / 4, o.R), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((attend_join_shared_kernel<WT, DH, false>), dim3(o.max_new, o.h_q, o.R), dim3(256), 0, stream, a);
}

}  // namespace

// The prefix's keys are the same for all its row tiles, so that their splits can be chosen to fill
// the chip evenly: of numbers of workgroups up to kQuarterRounds quarters of a round (two to a compute
// unit) the one with the lowest cost, which is the stages of the longest chain of rounds, each as
// long as writing and joining kPartsOfStage rows of parts. 32 chunks of up to 16 tokens after
// 60000 shared keys, 64 / 8 heads, in 8 bits: 641 us, unsplit (152 workgroups) 1186.
// kPartsOfStage 3000, with 6500 in brackets, bf16, 32 / 8 heads: 48 single tokens after 8000 shared
// keys 42.9 us (45.9), 64 after 30000 66.1 (68.9), 4 chunks of 16 after 8000, 64 / 8 heads, 35.4
// (41.4), 4 prompts of 150 after 4000 47.4 (55.1). With 1500 48 after 8000 in 8 bits take 41.3 us, with
// 3000 37.7; other shapes were not weighed in 8 bits.
constexpr int kSlots = 512, kQuarterRounds = 16, kPartsOfStage = 3000;
AttendPlan prefix_plan(int T, int h_q, int h_kv, int dtype, int max_shared) {
  AttendPlan p = attend_plan(1, h_q, h_kv, dtype, T, max_shared, 0);
  if (p.tile_rows != kTileRows) return p;
  const int64_t base = (int64_t)h_kv * p.row_tiles, span = std::max(1, max_shared), rows = (int64_t)T * h_q;
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  int64_t best = INT64_MAX;
  for (int k = 0; k <= kQuarterRounds; ++k) {
    const int64_t s = k ? std::min<int64_t>(k * (kSlots / 4) / base, kMaxSplits) : 1;
    if (s < 1) continue;
    const int64_t chunk = up(up(span, s), kTileKeys) * kTileKeys, S = up(span, chunk);
    const int64_t cost = up(base * S, kSlots) * (chunk / kTileKeys) * kPartsOfStage + rows * S;
    if (cost < best) {
      best = cost;
      p.chunk = (int)chunk;
      p.S = (int)S;
    }
  }
  return p;
}

// Rows of parts: at least one for each row; of tiles with split keys at most so many tiles' as
// workgroups are tried.
int64_t prefix_most_parts(int T, int h_q, int h_kv, int dtype, int max_shared) {
  const int64_t rows = (int64_t)T * h_q, other = attend_most_parts(1, h_q, h_kv, dtype, T, max_shared);
  const int64_t splits = std::clamp<int64_t>((max_shared + kTileKeys - 1) / kTileKeys, 1, kMaxSplits);
  return std::max({rows, other, std::min(rows * splits, (int64_t)kTileRows * kQuarterRounds * (kSlots / 4))});
}

hipError_t launch_kv_attend_shared(const SharedArgs& a, int dh, int dtype, hipStream_t stream) {
  by_type(dh, dtype, a.own.k_exp != nullptr, [&](auto wt, auto ct, auto d) { launch_shared<wt(), ct(), d()>(a, stream); });
  return hipGetLastError();
}

}  // namespace sfn
