// Attention of each request's new tokens over its pages of the key/value cache.

#include <algorithm>

#include "device_common.h"
#include "kernels.h"
#include "sparse_ffn.h"

namespace sfn {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;

constexpr float kNegInf = -__builtin_huge_valf();

// ---- split attention -----------------------------------------------------------------
//
// A workgroup takes 16 RT rows of one key head's queries (row rho of a request is its
// token rho / g, head rho % g of the g query heads that share the key head, so grouped
// heads fill the matrix tile) and one split of the keys; its four waves take every fourth
// tile of the split, each with a softmax of its own (running maximum and sum, fp32), and
// join at the end. K, Q, P and V go from memory to the matrix cores through registers
// alone. The scores are computed as S^T = K Q^T, whose tile leaves one query row per lane
// (lane & 15) and its keys in the lane's registers, so maxima and sums need two lane swaps
// and P^T is already laid out as the right operand of O^T = V^T P^T:
//   bf16: 32 keys a tile, two 16 x 16 score tiles; the P operand wants 8 keys a lane, and
//   as the order of the contracted keys is free, lane quarter q takes keys 4q..4q+3 of
//   either score tile, which are the ones it holds. V rows are read as they lie (VW values
//   a lane); the left operand of output block e takes element e of each lane's values
//   (a byte permute packs two keys), so O's rows come out as dh = VW (4q + i) + e.
//   fp32: 16 keys a tile; the 16x16x4 product takes one key per lane quarter, so step i
//   takes keys 4q + i: again the ones the lane holds, with no packing.
// Masked scores are -inf; a row that sees no key keeps l = 0 and gives zeros. Values of
// keys past the end of the sequence are zeroed, whatever the cache holds there.
template <int WT, int DH>
struct AttnTile {
  static constexpr bool kBf = WT == WT_BF16;
  static constexpr int KB = kBf ? 2 : 4;           // bytes of a value
  static constexpr int KT = kBf ? 32 : 16;         // keys of a tile
  static constexpr int NG = KT / 16;               // 16-key groups (each within a page)
  static constexpr int NQ = DH * KB / 64;          // 16-byte chunks a lane holds of a row (K, Q)
  static constexpr int VW = kBf && DH == 128 ? 8 : 4;  // values a lane reads of a V row
  static constexpr int NB = DH / (16 * VW);        // times that
  static constexpr int NO = DH / 16;               // output blocks
};

// Whether a word holds a value that is not finite (fp32, or either bf16 half).
template <int WT>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  const bool hi = (w & 0x7f800000u) == 0x7f800000u;
  return WT == WT_BF16 ? hi || (w & 0x7f80u) == 0x7f80u : hi;
}

// The word with those values replaced by 0.
template <int WT>
__device__ __forceinline__ uint32_t finite_part(uint32_t w) {
  if (WT == WT_F32) return not_finite<WT>(w) ? 0u : w;
  if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
  if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
  return w;
}

// acc += V^T P^T of one tile: v the lane's words of V (group, key 4q + j, piece, word), p
// its weights (group, key 4q + i).
template <int WT, int DH>
__device__ __forceinline__ void add_weighted(
    const uint32_t (&v)[AttnTile<WT, DH>::NG][4][AttnTile<WT, DH>::NB][AttnTile<WT, DH>::VW * AttnTile<WT, DH>::KB / 4],
    const f32x4_t (&p)[AttnTile<WT, DH>::NG], f32x4_t (&acc)[AttnTile<WT, DH>::NO]) {
  using C = AttnTile<WT, DH>;
  if constexpr (C::kBf) {
    // the weights are rounded to bf16, as V is: the matrix cores take both operands in one
    // type, and the rounding (at most 2^-8 of each weight, of either sign) adds no more to
    // the result than rounding it to bf16 at the end does. Their sum is not rounded.
    const bf16x8_t pf = __builtin_bit_cast(
        bf16x8_t, make_uint4(pack_bf16(p[0][0], p[0][1]), pack_bf16(p[0][2], p[0][3]), pack_bf16(p[1][0], p[1][1]),
                             pack_bf16(p[1][2], p[1][3])));
#pragma unroll
    for (int e = 0; e < C::VW; ++e) {
      const uint32_t sel = (e & 1) ? 0x07060302u : 0x05040100u;
      uint32_t w[4];
#pragma unroll
      for (int h = 0; h < 4; ++h)
        w[h] = __builtin_amdgcn_perm(v[h >> 1][2 * (h & 1) + 1][0][e >> 1], v[h >> 1][2 * (h & 1)][0][e >> 1], sel);
      acc[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(w[0], w[1], w[2], w[3])),
                                                       pf, acc[e], 0, 0, 0);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
        for (int e = 0; e < C::VW; ++e)
          acc[nb * C::VW + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[0][i][nb][e]), p[0][i],
                                                                     acc[nb * C::VW + e], 0, 0, 0);
  }
}

// The same for the values of key kk that are not finite, and only into the rows that see it.
template <int WT, int DH>
__device__ __forceinline__ void add_one_key(
    const uint32_t (&v)[AttnTile<WT, DH>::NG][4][AttnTile<WT, DH>::NB][AttnTile<WT, DH>::VW * AttnTile<WT, DH>::KB / 4],
    const f32x4_t (&p)[AttnTile<WT, DH>::NG], int kk, int q, bool sees, f32x4_t (&acc)[AttnTile<WT, DH>::NO]) {
  using C = AttnTile<WT, DH>;
  float w = 0.f;  // the weight, in the lanes that hold the key
#pragma unroll
  for (int u = 0; u < C::NG; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) w = 16 * u + 4 * q + i == kk ? p[u][i] : w;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
    for (int e = 0; e < C::VW; ++e) {
      // the key's value, likewise; it goes through the products as operand element 0
      uint32_t x = 0;
#pragma unroll
      for (int u = 0; u < C::NG; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x = 16 * u + 4 * q + j == kk ? (C::kBf ? v[u][j][nb][e >> 1] >> (16 * (e & 1)) & 0xffffu : v[u][j][nb][e]) : x;
      x = not_finite<WT>(x) ? x : 0u;
      f32x4_t& o = acc[nb * C::VW + e];
      f32x4_t t;
      if constexpr (C::kBf)
        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(x, 0, 0, 0)),
                                                    __builtin_bit_cast(bf16x8_t, make_uint4(pack_bf16(w, 0.f), 0, 0, 0)),
                                                    o, 0, 0, 0);
      else
        t = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x), w, o, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = sees ? t[i] : o[i];
    }
}

template <int WT, int DH, int RT>
__global__ __launch_bounds__(256, RT == 1 ? 3 : RT == 2 ? 2 : 1) void attend_split_kernel(AttendArgs a) {
  using C = AttnTile<WT, DH>;
  constexpr int KT = C::KT, NG = C::NG, NQ = C::NQ, VW = C::VW, NB = C::NB, NO = C::NO, KB = C::KB;
  __shared__ float s_m[4][16 * RT], s_l[4][16 * RT];
  __shared__ __attribute__((aligned(16))) float s_o[16 * RT][DH + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, q = lane >> 4;
  int b = blockIdx.x;
  const int hk = b % a.h_kv;
  b /= a.h_kv;
  const int rtile = b % a.row_tiles;
  b /= a.row_tiles;
  const int split = b % a.S, r = b / a.S;

  const int t0 = min(max(gp(a.cu)[r], 0), a.T), t1 = min(max(gp(a.cu)[r + 1], t0), a.T);
  const int n = t1 - t0, g = a.g, rows = n * g;
  const int rho0 = rtile * 16 * RT;
  if (rho0 >= rows) return;
  const int len = min(max(gp(a.kv_len)[r], 0), a.max_len);
  const int past = len - n;  // position of the first new token
  const int rho1 = min(rho0 + 16 * RT, rows) - 1;
  // keys that some row of the tile sees
  const int hi = max(0, min(past + rho1 / g + 1, len));
  const int lo = a.window > 0 ? max(0, past + rho0 / g + 1 - a.window) : 0;
  const int lo_al = lo & ~(KT - 1);
  const int k0 = lo_al + split * a.chunk, k1 = min(k0 + a.chunk, hi);
  if (split > 0 && k0 >= hi) return;
  // keys that every row sees
  const int hi_all = min(past + rho0 / g + 1, len);
  const int lo_all = a.window > 0 ? max(0, past + rho1 / g + 1 - a.window) : 0;

  const int row_bytes = DH * KB;
  const int lg = a.page_shift, pm = (1 << lg) - 1;
  const SFN_GLOBAL int32_t* table = gp(a.table) + (int64_t)r * a.max_pages;

  // Q: right operand, lane's row c, chunk s: values 64 s / KB + 16 q / KB ...
  uint4 qf[RT][NQ];
  int row_hi[RT], row_lo[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int rho = rho0 + 16 * x + c;
    const bool ok = rho < rows;
    const int rr = ok ? rho : rho0;
    const int tok = rr / g, head = hk * g + rr % g;
    const SFN_GLOBAL char* src = gp(a.q) + (int64_t)(t0 + tok) * a.q_stride + head * row_bytes + 16 * q;
#pragma unroll
    for (int s = 0; s < NQ; ++s) qf[x][s] = ld16(src + 64 * s);
    row_hi[x] = ok ? min(past + tok + 1, len) : 0;
    row_lo[x] = a.window > 0 ? past + tok + 1 - a.window : 0;
  }

  f32x4_t acc[RT][NO];
  float m[RT], l[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    m[x] = kNegInf;
    l[x] = 0.f;
#pragma unroll
    for (int o = 0; o < NO; ++o) acc[x][o] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }

  for (int kt = k0 + wave * KT; kt < k1; kt += 4 * KT) {
    uint4 kf[NG][NQ];
    uint32_t vf[NG][4][NB][VW * KB / 4];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      const int key = min(kt + 16 * u, (k1 - 1) & ~15);
      const int page = min(max(table[key >> lg], 0), a.n_pages - 1);
      const int64_t row = (((int64_t)page * a.h_kv + hk) << lg) + (key & pm);
      const SFN_GLOBAL char* kp = gp(a.k) + (row + c) * row_bytes + 16 * q;
#pragma unroll
      for (int s = 0; s < NQ; ++s) kf[u][s] = ld16(kp + 64 * s);
      const SFN_GLOBAL char* vp = gp(a.v) + (row + 4 * q) * row_bytes + c * VW * KB;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const SFN_GLOBAL char* p = vp + j * row_bytes + nb * 16 * VW * KB;
          if constexpr (VW * KB == 16) {
            const uint4 w = ld16(p);
            vf[u][j][nb][0] = w.x;
            vf[u][j][nb][1] = w.y;
            vf[u][j][nb][2] = w.z;
            vf[u][j][nb][3] = w.w;
          } else {
            const uint64_t w = *reinterpret_cast<const SFN_GLOBAL uint64_t*>(p);
            vf[u][j][nb][0] = (uint32_t)w;
            vf[u][j][nb][1] = (uint32_t)(w >> 32);
          }
        }
    }
    const bool full = kt >= lo_all && kt + KT <= hi_all;  // every row sees every key of the tile
    if (kt + KT > len) {
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int w = 0; w < VW * KB / 4; ++w)
              vf[u][j][nb][w] = kt + 16 * u + 4 * q + j < len ? vf[u][j][nb][w] : 0u;
    }
    // A masked key has weight 0, but 0 times a value that is not finite is NaN: a tile with a
    // masked key and such a value takes the long way below, so that no token's result
    // depends on tokens it does not see.
    bool odd = false;
    if (!full) {
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int w = 0; w < VW * KB / 4; ++w) odd |= not_finite<WT>(vf[u][j][nb][w]);
      odd = __any(odd);
    }
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      f32x4_t s[NG];
#pragma unroll
      for (int u = 0; u < NG; ++u) {
        s[u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          if constexpr (C::kBf) {
            s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, kf[u][i]),
                                                           __builtin_bit_cast(bf16x8_t, qf[x][i]), s[u], 0, 0, 0);
          } else {
            const f32x4_t kk = __builtin_bit_cast(f32x4_t, kf[u][i]), qq = __builtin_bit_cast(f32x4_t, qf[x][i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(kk[e], qq[e], s[u], 0, 0, 0);
          }
        }
      }
      // scores in units of log2: p = 2^(s - m)
      float top = kNegInf;
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v = s[u][i] * a.scale_log2;
          if (!full) {
            const int key = kt + 16 * u + 4 * q + i;
            v = key < row_hi[x] && key >= row_lo[x] ? v : kNegInf;
          }
          s[u][i] = v;
          top = fmaxf(top, v);
        }
      top = swap_pair_max<16>(top);
      top = swap_pair_max<32>(top);
      const float mn = fmaxf(m[x], top);
      const float ms = mn == kNegInf ? 0.f : mn;
      if (__any(mn > m[x])) {
        const float al = exp2_f(m[x] - ms);
        l[x] *= al;
#pragma unroll
        for (int o = 0; o < NO; ++o)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[x][o][i] *= al;
        m[x] = mn;
      }
      float add = 0.f;
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[u][i] = exp2_f(s[u][i] - ms);
          add += s[u][i];
        }
      l[x] += add;
      if (odd) {
        // the finite values for all, then the others key by key into the rows that see them
        uint32_t fin[NG][4][NB][VW * KB / 4];
#pragma unroll
        for (int u = 0; u < NG; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int w = 0; w < VW * KB / 4; ++w) fin[u][j][nb][w] = finite_part<WT>(vf[u][j][nb][w]);
        add_weighted<WT, DH>(fin, s, acc[x]);
#pragma unroll 1
        for (int kk = 0; kk < KT; ++kk)
          add_one_key<WT, DH>(vf, s, kk, q, kt + kk < row_hi[x] && kt + kk >= row_lo[x], acc[x]);
      } else {
        add_weighted<WT, DH>(vf, s, acc[x]);
      }
    }
  }

  // join the four waves: a common maximum, then each adds its share in wave order
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    l[x] = swap_pair_sum<16>(l[x]);
    l[x] = swap_pair_sum<32>(l[x]);
    if (q == 0) {
      s_m[wave][16 * x + c] = m[x];
      s_l[wave][16 * x + c] = l[x];
    }
  }
  __syncthreads();
  float w_self[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const int i = 16 * x + c;
    const float M = fmaxf(fmaxf(s_m[0][i], s_m[1][i]), fmaxf(s_m[2][i], s_m[3][i]));
    w_self[x] = m[x] == kNegInf ? 0.f : exp2_f(m[x] - M);
  }
  for (int w = 0; w < 4; ++w) {
    if (wave == w) {
#pragma unroll
      for (int x = 0; x < RT; ++x)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              float* o = &s_o[16 * x + c][16 * VW * nb + VW * (4 * q + i) + e];
              const float v = acc[x][nb * VW + e][i] * w_self[x];
              *o = w == 0 ? v : *o + v;
            }
    }
    __syncthreads();
  }
  for (int i = tid; i < 16 * RT * (DH / 4); i += 256) {
    const int x = i / (DH / 4), d4 = (i % (DH / 4)) * 4;
    const int rho = rho0 + x;
    if (rho >= rows) continue;
    const int tok = rho / g, head = hk * g + rho % g;
    const float M = fmaxf(fmaxf(s_m[0][x], s_m[1][x]), fmaxf(s_m[2][x], s_m[3][x]));
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) L += s_m[w][x] == kNegInf ? 0.f : exp2_f(s_m[w][x] - M) * s_l[w][x];
    f32x4_t o = *reinterpret_cast<const f32x4_t*>(&s_o[x][d4]);
    const int64_t orow = (int64_t)(t0 + tok) * a.h_q + head;
    if (a.S == 1) {
      const float inv = L == 0.f ? 0.f : 1.0f / L;
      o *= inv;
      if constexpr (C::kBf) {
        *reinterpret_cast<SFN_GLOBAL uint64_t*>(gp(a.out) + (orow * DH + d4) * 2) =
            (uint64_t)pack_bf16(o[0], o[1]) | (uint64_t)pack_bf16(o[2], o[3]) << 32;
      } else {
        *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.out) + (orow * DH + d4) * 4) = o;
      }
    } else {
      const int64_t at = orow * a.S + split;
      *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.part_o) + at * DH + d4) = o;
      if (d4 == 0) {
        gp(a.part_ml)[2 * at] = M;
        gp(a.part_ml)[2 * at + 1] = L;
      }
    }
  }
}

// Joins the splits of one output row (a token's query head): one workgroup per row.
template <int WT, int DH>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a, int tile_rows) {
  constexpr int KT = AttnTile<WT, DH>::KT;
  constexpr int LD = DH / 4, NS = 256 / LD;  // lanes of a row, splits side by side
  __shared__ float s_w[256];
  __shared__ float s_red[8];
  __shared__ f32x4_t s_o[NS][LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int b = blockIdx.x;
  const int head = b % a.h_q;
  b /= a.h_q;
  const int i = b % a.max_new, r = b / a.max_new;
  const int t0 = min(max(gp(a.cu)[r], 0), a.T), t1 = min(max(gp(a.cu)[r + 1], t0), a.T);
  const int n = t1 - t0, g = a.g;
  if (i >= n) return;
  const int len = min(max(gp(a.kv_len)[r], 0), a.max_len), past = len - n;
  const int rho0 = (i * g + head % g) / tile_rows * tile_rows;
  const int rho1 = min(rho0 + tile_rows, n * g) - 1;
  const int hi = max(0, min(past + rho1 / g + 1, len));
  const int lo = a.window > 0 ? max(0, past + rho0 / g + 1 - a.window) : 0;
  const int span = hi - (lo & ~(KT - 1));
  const int used = span > 0 ? (span + a.chunk - 1) / a.chunk : 1;  // <= S <= 256
  const int64_t orow = (int64_t)(t0 + i) * a.h_q + head;
  float m = kNegInf, l = 0.f;
  if (tid < used) {
    m = gp(a.part_ml)[2 * (orow * a.S + tid)];
    l = gp(a.part_ml)[2 * (orow * a.S + tid) + 1];
  }
  float M = m;
#pragma unroll
  for (int x = 1; x < 64; x <<= 1) M = fmaxf(M, shfl_xor_f(M, x));
  if (lane == 0) s_red[wave] = M;
  __syncthreads();
  M = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
  const float w = m == kNegInf ? 0.f : exp2_f(m - M);
  s_w[tid] = w;
  const float L4 = wave_sum(w * l);
  if (lane == 0) s_red[4 + wave] = L4;
  __syncthreads();
  const float L = (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
  const int d4 = tid % LD, s0 = tid / LD;
  f32x4_t o = {0.f, 0.f, 0.f, 0.f};
  const SFN_GLOBAL f32x4_t* src = reinterpret_cast<const SFN_GLOBAL f32x4_t*>(gp(a.part_o) + orow * a.S * DH) + d4;
  for (int s = s0; s < used; s += NS) {
    const f32x4_t v = src[(int64_t)s * LD];
    o += v * s_w[s];  // also for weight 0: NaN scores show
  }
  s_o[s0][d4] = o;
  __syncthreads();
  if (tid < LD) {
    for (int s = 1; s < NS; ++s) o += s_o[s][d4];
    o *= L == 0.f ? 0.f : 1.0f / L;
    if constexpr (WT == WT_BF16) {
      *reinterpret_cast<SFN_GLOBAL uint64_t*>(gp(a.out) + (orow * DH + 4 * d4) * 2) =
          (uint64_t)pack_bf16(o[0], o[1]) | (uint64_t)pack_bf16(o[2], o[3]) << 32;
    } else {
      *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.out) + (orow * DH + 4 * d4) * 4) = o;
    }
  }
}

template <int WT, int DH>
void launch_split(const AttendArgs& a, int RT, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.R * a.S * a.row_tiles * a.h_kv)), block(256);
  if (RT == 1) hipLaunchKernelGGL((attend_split_kernel<WT, DH, 1>), grid, block, 0, stream, a);
  else if (RT == 2) hipLaunchKernelGGL((attend_split_kernel<WT, DH, 2>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((attend_split_kernel<WT, DH, 4>), grid, block, 0, stream, a);
  if (a.S > 1) {
    const dim3 rows((unsigned)((int64_t)a.R * a.max_new * a.h_q));
    hipLaunchKernelGGL((attend_join_kernel<WT, DH>), rows, block, 0, stream, a, 16 * RT);
  }
}

}  // namespace

AttendPlan attend_plan(int R, int h_q, int h_kv, int dtype, int max_new, int max_len, int window) {
  AttendPlan p;
  const int kt = dtype == SFN_BF16 ? 32 : 16;
  const int64_t rows = (int64_t)max_new * (h_q / h_kv);
  p.RT = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const int64_t tiles = (rows + 16 * p.RT - 1) / (16 * p.RT);
  p.row_tiles = (int)tiles;
  // keys one row tile can span
  int64_t span = max_len;
  if (window > 0 && (int64_t)window + max_new + kt < span) span = (int64_t)window + max_new + kt;
  if (span < 1) span = 1;
  const int64_t base = (int64_t)R * h_kv * tiles;
  const int64_t step = 4 * kt;  // a tile for each wave
  int64_t s = (1024 + base - 1) / base;
  if (s > 256) s = 256;
  p.S_most = (int)std::min<int64_t>(s, std::max<int64_t>(1, ((int64_t)max_len + step - 1) / step));
  int64_t chunk = ((span + s - 1) / s + step - 1) / step * step;
  p.chunk = (int)chunk;
  p.S = (int)((span + chunk - 1) / chunk);
  return p;
}

hipError_t launch_kv_attend(const AttendArgs& a, int RT, int dh, int dtype, hipStream_t stream) {
  if (dtype == SFN_BF16) {
    if (dh == 64) launch_split<WT_BF16, 64>(a, RT, stream);
    else launch_split<WT_BF16, 128>(a, RT, stream);
  } else {
    if (dh == 64) launch_split<WT_F32, 64>(a, RT, stream);
    else launch_split<WT_F32, 128>(a, RT, stream);
  }
  return hipGetLastError();
}

}  // namespace sfn
