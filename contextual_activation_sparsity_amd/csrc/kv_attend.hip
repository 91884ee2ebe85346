// Attention of each request's new tokens over its pages of the key/value cache.

#include "attend_device.h"

namespace sfn {

namespace {

template <int WT, int CT, int DH, int RT, int NW>
__global__ __launch_bounds__(64 * NW, NW == 8 || RT == 2 ? 2 : 3) void attend_split_kernel(AttendArgs a) {
  __shared__ float s_m[NW][16 * RT], s_l[NW][16 * RT];
  __shared__ __attribute__((aligned(16))) float s_o[NW][16 * RT][DH + 4];
  split_attention<WT, CT, DH, RT, NW, ATTEND_PLAIN>(a, blockIdx.x, blockIdx.y, blockIdx.z, s_m, s_l, PaddedRows<DH, 16 * RT, NW>{s_o});
}

template <int CT, int DH, int KG>
__global__ __launch_bounds__(256 * KG, 2) void attend_tile_kernel(AttendArgs a) {
  __shared__ __attribute__((aligned(16))) char s_a[KG * 2 * kTileKeys * DH * 2];
  __shared__ __attribute__((aligned(16))) char s_b[KG * 2 * kTileKeys * DH * 2];
  __shared__ uint32_t s_odd[4 * KG];
  tile_attention<CT, DH, KG, ATTEND_PLAIN, false>(a, blockIdx.x, blockIdx.y, blockIdx.z, s_a, s_b, s_odd);
}

// Joins the splits of one output row (a token's query head): one workgroup for a row, or one
// wave where there are rows enough to fill the chip that way and at most 64 splits. The parts
// lie by request and token, so that their first loads need not wait for the lengths; what
// was never written is not used.
template <int WT, int DH, bool WAVE>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  constexpr int NT = WAVE ? 64 : 256;        // threads of a row
  constexpr int LD = DH / 4, NS = NT / LD;   // lanes of a row's values, splits side by side
  constexpr int U = 8;                       // loads in flight
  __shared__ float s_w[256];
  __shared__ float s_red[8];
  __shared__ f32x4_t s_o[256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, tid = WAVE ? lane : threadIdx.x;
  const int i = blockIdx.x, r = blockIdx.z, head = WAVE ? blockIdx.y * 4 + wave : blockIdx.y;
  if (WAVE && head >= a.h_q) return;
  float* const w_of = s_w + (WAVE ? 64 * wave : 0);
  const int64_t part = (((int64_t)r * a.max_new + i) * a.h_q + head) * a.S;
  const int d4 = tid % LD, s0 = tid / LD;
  const SFN_GLOBAL f32x4_t* src = reinterpret_cast<const SFN_GLOBAL f32x4_t*>(gp(a.part_o) + part * DH) + d4;
  const f32x2_t ml = reinterpret_cast<const SFN_GLOBAL f32x2_t*>(gp(a.part_ml))[part + min(tid, a.S - 1)];
  f32x4_t v[U];
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = src[(int64_t)min(s0 + u * NS, a.S - 1) * LD];

  const Request<ATTEND_PLAIN> req(a, r);
  if (i >= req.n) return;
  const int t0 = req.t0, used = splits_used(a, req, i, head);

  const float m = tid < used ? ml[0] : kNegInf, l = tid < used ? ml[1] : 0.f;
  float M = wave_max(m);
  if constexpr (!WAVE) {
    if (lane == 0) s_red[wave] = M;
    __syncthreads();
    M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  }
  const float w = m == kNegInf ? 0.f : exp2_f(m - M);
  w_of[tid] = w;
  float L = wave_sum(w * l);
  if constexpr (!WAVE) {
    if (lane == 0) s_red[4 + wave] = L;
    __syncthreads();
    L = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
  } else {
    wave_sync();
  }
  f32x4_t o = {0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < used; s += U * NS) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u * NS < used) o += v[u] * w_of[s + u * NS];  // also for weight 0: NaN scores show
    if (s + U * NS < used) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = src[(int64_t)min(s + (U + u) * NS, a.S - 1) * LD];
    }
  }
  f32x4_t* const o_of = s_o + (WAVE ? 64 * wave : 0);
  o_of[tid] = o;
  if constexpr (WAVE) wave_sync();
  else __syncthreads();
  if (tid < LD) {
#pragma unroll
    for (int s = 1; s < NS; ++s) o += o_of[s * LD + d4];
    store_row<WT, DH>(a, t0 + i, head, 4 * d4, o, L);
  }
}

// Tile kernel: up to this many workgroups get two groups of waves (one to a compute unit),
// and few row tiles are split into at most as many. 16-token chunks of R requests, 64 / 8 heads,
// ragged up to 4000 keys, with 256 workgroups at most, with 384 and with 512 (then one group of
// waves and two workgroups to a compute unit): R = 4 24.6, 27.4 and 26.4 us; 8 36.8, 41.8, 39.8;
// 12 54.8, 57.1, 52.0; 16 58.4, 69.1, 62.3; 17 77.9, 87.0, 71.2; 24 81.5, 95.5, 95.3. The division
// is of whole row tiles, so that 17 requests are 136 workgroups where 16 are 256.
constexpr int kTileFill = 256;
// Unsplit items, 8 waves or 4: 256 items of up to 300 keys (32 / 8 heads) 8.5 us with 8; 512
// items 15.5 with 8, 13.8 with 4 (three workgroups to a compute unit then), 4096 items 92 and 63.
constexpr int kWideMost = 256;

template <int WT, int CT, int DH>
void launch_sized(const AttendArgs& a, hipStream_t stream) {
  // heads first: the row tiles of a key head lie a multiple of h_kv apart, so that with 8 (or
  // 16, ...) key heads they share an XCD's L2
  // An odd number of splits (the one too many ends at once): workgroups go to the shader
  // engines in turn, and with 4 splits of ragged lengths one engine would get all the first,
  // full splits and another all the last ones. 128 requests of up to 8000 keys, 32 / 8 heads,
  // 4 splits: 477 us without it, 332 with it; 4 splits of 64 requests of up to 3000 100 and 78 us.
  const dim3 grid(a.row_tiles * a.h_kv, a.S | 1, a.R), block(256);
  if (a.tile_rows == kTileRows) {
    if constexpr (WT == WT_BF16) {
      if ((int64_t)a.R * a.S * a.row_tiles * a.h_kv > kTileFill)
        hipLaunchKernelGGL((attend_tile_kernel<CT, DH, 1>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((attend_tile_kernel<CT, DH, 2>), grid, dim3(512), 0, stream, a);
    }
  } else {
    // one workgroup for all of an item's keys and a compute unit for each: more waves
    const bool wide = a.S == 1 && (int64_t)a.R * a.row_tiles * a.h_kv <= kWideMost;
    const dim3 threads(wide ? 512 : 256);
    if (a.tile_rows == 16 && wide) hipLaunchKernelGGL((attend_split_kernel<WT, CT, DH, 1, 8>), grid, threads, 0, stream, a);
    else if (a.tile_rows == 16) hipLaunchKernelGGL((attend_split_kernel<WT, CT, DH, 1, 4>), grid, threads, 0, stream, a);
    else if (wide) hipLaunchKernelGGL((attend_split_kernel<WT, CT, DH, 2, 8>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((attend_split_kernel<WT, CT, DH, 2, 4>), grid, threads, 0, stream, a);
  }
  if (a.S > 1) {
    if (a.S <= 64 && (int64_t)a.R * a.max_new * a.h_q >= kJoinByWave)
      hipLaunchKernelGGL((attend_join_kernel<WT, DH, true>), dim3(a.max_new, (a.h_q + 3) / 4, a.R), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((attend_join_kernel<WT, DH, false>), dim3(a.max_new, a.h_q, a.R), dim3(256), 0, stream, a);
  }
}

}  // namespace

// How the keys are split, by measurement (GPU time in a graph, bf16, heads of 128):
//   - At least kFill workgroups, two to a compute unit: one token over 131000 keys, 64 / 8
//     heads, takes 86 us with 512, 88 with 768 and 90 with 1024 (with fewer waves to share
//     the memory with, each streams better, and there are fewer parts to join).
//   - Several requests: finer, since their lengths differ and the last workgroup is waited
//     for; down to kLeast keys, but at most kMost workgroups. Each with the other side, 32 / 8
//     heads, ragged: 8 requests of up to 2000 keys 13.5 us, with splits of 512 16.5; 32 of up to
//     800 17.3 (20.3); 48 of up to 8000 149, with 2048 workgroups 157, with 4096 149; 256 of up
//     to 500 (2048 items) 56 unsplit, 63 with 4096 workgroups.
//   - Up to kWhole keys: no split and no second launch. 32 / 32 heads, each call from Python:
//     201 keys 5.7 us against 7.7 in two launches, 301 keys 7.2 against 7.7, but 501 keys 10.5
//     against 8.3 (one compute unit's load rate bounds an unsplit item).
//   - Tile kernel: a round of its two wave groups (128 keys) takes as long as writing and joining
//     kPartsOfRound parts, the second launch as long as kPartsOfJoin; few row tiles are split
//     if that gains. Split and unsplit: 12 tokens of 3 requests, 8 / 1 heads, 160 keys 12.1 and
//     11.0 us, 412 keys 12.2 and 14.6; 16 of 8 requests, 32 / 8 heads, 416 keys 16.7 and 15.4,
//     1016 keys 20.5 and 23.2; a prompt of 400 tokens, 32 / 8 heads, 22.2 and 14.8.
constexpr int kPartsOfRound = 6500, kPartsOfJoin = 10000;
constexpr int kFill = 512, kLeast = 128, kMost = 3200, kWhole = 384;
AttendPlan attend_plan(int R, int h_q, int h_kv, int dtype, int max_new, int max_len, int window) {
  AttendPlan p{};
  const int64_t rows = (int64_t)max_new * (h_q / h_kv);
  const bool bf = dtype == SFN_BF16;
  p.tile_rows = rows <= 16 ? 16 : rows <= 32 || !bf ? 32 : kTileRows;
  p.tile_keys = p.tile_rows == kTileRows ? kTileKeys : bf ? 32 : 16;
  p.row_tiles = (int)((rows + p.tile_rows - 1) / p.tile_rows);
  const int64_t base = (int64_t)R * h_kv * p.row_tiles;
  const bool tile = p.tile_rows == kTileRows;
  const int64_t step = tile ? kTileKeys : 4 * p.tile_keys;  // splits are multiples of it
  auto splits = [&](int64_t span) {
    int64_t s = tile ? std::max<int64_t>(1, kTileFill / base) : (kFill + base - 1) / base;
    if (!tile && R > 1) s = std::max<int64_t>(s, std::min<int64_t>((span + kLeast - 1) / kLeast, kMost / base));
    return !tile && span <= kWhole ? 1 : std::min<int64_t>(s, kMaxSplits);
  };
  // keys one row tile can span
  int64_t span = std::max(1, max_len);
  if (window > 0) span = std::min<int64_t>(span, (int64_t)window + p.tile_rows + p.tile_keys);
  const int64_t s = splits(span);
  int64_t chunk = ((span + s - 1) / s + step - 1) / step * step;
  if (tile && chunk < span) {
    auto rounds = [](int64_t keys) { return (keys + 2 * kTileKeys - 1) / (2 * kTileKeys); };
    const int64_t parts = (int64_t)R * max_new * h_q * ((span + chunk - 1) / chunk);
    if ((rounds(span) - rounds(chunk)) * kPartsOfRound <= kPartsOfJoin + parts) chunk = (span + step - 1) / step * step;
  }
  p.chunk = (int)chunk;
  p.S = (int)((span + chunk - 1) / chunk);
  p.parts = p.S > 1 ? (int64_t)R * max_new * h_q * p.S : 0;
  return p;
}

// A split call launches at most this many workgroups (by the rules above: fewer than 2 kFill, or
// kMost of several requests; kTileFill of the tile kernel), each with a tile's rows of parts; nor
// can a row have more splits than its keys have steps. More new tokens may mean fewer parts (up
// to none), so this is taken over all calls within the bounds.
int64_t attend_most_parts(int R, int h_q, int h_kv, int dtype, int max_new, int max_len) {
  const bool bf = dtype == SFN_BF16;
  const int g = h_q / h_kv;
  auto parts = [&](int64_t tokens, int64_t keys, int64_t step, int64_t rows_launched) {
    const int64_t s = std::min<int64_t>((keys + step - 1) / step, kMaxSplits);
    return s > 1 ? std::min((int64_t)R * tokens * h_q * s, rows_launched) : 0;
  };
  const int64_t split = max_len <= kWhole ? 0
                                          : parts(bf ? std::min(max_new, 32 / g) : max_new, max_len, 4 * (bf ? 32 : 16),
                                                  32 * (R > 1 ? std::max(2 * kFill, kMost) : 2 * kFill));
  const int64_t tile = bf && (int64_t)max_new * g > 32 ? parts(max_new, max_len, kTileKeys, (int64_t)kTileRows * kTileFill) : 0;
  return std::max(split, tile);
}

hipError_t launch_kv_attend(const AttendArgs& a, int dh, int dtype, hipStream_t stream) {
  by_type(dh, dtype, a.k_exp != nullptr, [&](auto wt, auto ct, auto d) { launch_sized<wt(), ct(), d()>(a, stream); });
  return hipGetLastError();
}

}  // namespace sfn
