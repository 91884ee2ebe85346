// Attention of each request's new tokens over its pages of the key/value cache.

#include <algorithm>
#include <type_traits>

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

// The same for the values of key kk that are not finite, and only into the rows that see
// it. vp: the lane's first value of that key's row.
template <int WT, int DH>
__device__ __forceinline__ void add_one_key(const SFN_GLOBAL char* vp, const f32x4_t (&p)[AttnTile<WT, DH>::NG], int kk, int q,
                                            bool sees, f32x4_t (&acc)[AttnTile<WT, DH>::NO]) {
  using C = AttnTile<WT, DH>;
  float w = 0.f;  // the weight, in the lanes that hold the key
#pragma unroll
  for (int u = 0; u < C::NG; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) w = 16 * u + i == kk - 4 * q ? p[u][i] : w;
  const bool mine = (kk >> 2 & 3) == q;
#pragma unroll
  for (int nb = 0; nb < C::NB; ++nb) {
#pragma unroll
    for (int e = 0; e < C::VW; ++e) {
      // the key's value goes through the products as operand element 0
      uint32_t x = C::kBf ? reinterpret_cast<const SFN_GLOBAL uint16_t*>(vp)[nb * 16 * C::VW + e]
                          : reinterpret_cast<const SFN_GLOBAL uint32_t*>(vp)[nb * 16 * C::VW + e];
      x = mine && not_finite<WT>(x) ? x : 0u;
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

  // the cache row of the first key of key's group of 16
  auto row_of = [&](int key) -> int64_t {
    const int page = min(max(table[key >> lg], 0), a.n_pages - 1);
    return (((int64_t)page * a.h_kv + hk) << lg) + (key & pm & ~15);
  };

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
      const int64_t row = row_of(min(kt + 16 * u, (k1 - 1) & ~15));
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
              vf[u][j][nb][w] = 16 * u + j < len - kt - 4 * q ? vf[u][j][nb][w] : 0u;
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
      if (odd) {
        // the finite values for all rows first; the others key by key into the rows that see
        // them, read again
#pragma unroll
        for (int u = 0; u < NG; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int w = 0; w < VW * KB / 4; ++w) vf[u][j][nb][w] = finite_part<WT>(vf[u][j][nb][w]);
      }
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
            const int key = 16 * u + i, at = kt + 4 * q;
            v = key < row_hi[x] - at && key >= row_lo[x] - at ? v : kNegInf;
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
      add_weighted<WT, DH>(vf, s, acc[x]);
      if (odd) {
#pragma unroll 1
        for (int kk = 0; kk < KT && kt + kk < len; ++kk)
          add_one_key<WT, DH>(gp(a.v) + (row_of(kt + kk) + (kk & 15)) * row_bytes + c * VW * KB, s, kk, q,
                              kt + kk < row_hi[x] && kt + kk >= row_lo[x], acc[x]);
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

// ---- tile attention ------------------------------------------------------------------
//
// bf16, more query rows than the split kernel's registers hold: a workgroup takes 128 rows
// of one key head's queries, 32 to a wave, and walks the keys (or one split of them) 64 at
// a time. K and V come to LDS by asynchronous 16-byte loads, one stage ahead of the
// products, and serve all four waves. As above the scores are S^T = K Q^T, in 32 x 32 tiles:
// a lane has one query row (lane & 31) and half of its keys, the lane 32 away the others.
// Their order is once more what the next product needs: in step t of 16 keys, lane half h
// holds keys 16 t + 4h..+3 and 16 t + 8 + 4h..+3, and V^T's operand is read in that order
// by transposing LDS reads (16 lanes turn 4 keys x 16 values). The 16-byte chunks of the
// rows in LDS are permuted (by exclusive or with bits of the row) so that the lanes of one
// read fall on different banks; the loads write LDS in lane order, so it is their source
// addresses that are permuted.
// The running maximum is raised only when a score passes it by more than kSlack (in log2):
// softmax does not depend on the number subtracted, 2^8 is far from any overflow in fp32,
// and most tiles then leave the accumulators alone.
typedef __attribute__((ext_vector_type(16))) float f32x16_t;
typedef __attribute__((ext_vector_type(4))) short i16x4_t;
#define SFN_LDS __attribute__((address_space(3)))

constexpr int kTileRows = 128, kTileKeys = 64;
constexpr float kSlack = 8.f;
constexpr int kWaitLoads = 0x0f70;  // s_waitcnt vmcnt(0) (the other counters at their maximum)

__device__ __forceinline__ uint2 read_transposed(const SFN_LDS char* p) {
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SFN_LDS i16x4_t*)p));
}
__device__ __forceinline__ bf16x8_t read_frag(const SFN_LDS char* p) {
  return *reinterpret_cast<const SFN_LDS bf16x8_t*>(p);
}

// 16 bytes a lane from base + offset to LDS at lds + 16 lane, without waiting. Written as
// assembly because the compiler, which cannot tell which LDS the builtin writes, would let
// every LDS read after it wait for the data. No register is written, so nothing of the
// compiler's is in flight; whoever reads the LDS waits for vmcnt(0) and a barrier first.
__device__ __forceinline__ void load_to_lds(const SFN_GLOBAL char* base, uint32_t offset, SFN_LDS char* lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"((uint32_t)(uintptr_t)lds), "v"(offset), "s"(base)
               : "memory", "m0");
}

// One wave's state over its 32 rows, and where its lanes read and load.
template <int DH>
struct TileWave {
  static constexpr int ROW = DH * 2;           // bytes of a row
  static constexpr int NC = DH / 8;            // 16-byte chunks of a row
  static constexpr int RI = 64 / NC;           // rows of one wave-wide load
  static constexpr int NS = DH / 16, ND = DH / 32, KT = kTileKeys;
  // chunk ch of row `row` lies at these places
  __device__ __forceinline__ static int k_place(int row, int ch) { return ch ^ (DH == 128 ? row & 15 : row >> 1 & 7); }
  __device__ __forceinline__ static int v_place(int row, int ch) { return ch ^ (DH == 128 ? (row & 3) << 2 : (row >> 1 & 1) << 2); }

  bf16x8_t q[NS];
  f32x16_t acc[ND];
  float m, l;
  int row_lo, row_hi;  // the keys that the lane's row sees
  int c, h;

  // Loads this wave's 16 rows of a stage: kp and vp are those rows in the cache, kl and vl
  // the wave's part of the stage.
  __device__ __forceinline__ static void load(const SFN_GLOBAL char* kp, const SFN_GLOBAL char* vp, SFN_LDS char* kl, SFN_LDS char* vl,
                                              int lane) {
#pragma unroll
    for (int i = 0; i < 16 / RI; ++i) {
      const int row = i * RI + lane / NC, ch = lane % NC;  // the wave's rows start at a multiple of 16
      const uint32_t ko = row * ROW + k_place(row, ch) * 16, vo = row * ROW + v_place(row, ch) * 16;
      load_to_lds(kp, ko, kl + i * 1024);
      load_to_lds(vp, vo, vl + i * 1024);
    }
  }

  // acc += V^T P^T over the stage. With CLEAN, values that are not finite count as 0 and the
  // return says whether there were any.
  template <bool CLEAN>
  __device__ __forceinline__ bool add_values(const SFN_LDS char* v, const uint32_t (&pw)[2][8]) {
    const int vrow = 4 * h + (c & 15) / 4, vcol = 16 * (c >> 4) + 4 * (c & 3);
    bool odd = false;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      const int col = 32 * d + vcol;
      // 16 rows further the places repeat
      const SFN_LDS char* at = v + vrow * ROW + v_place(vrow, col >> 3) * 16 + (col & 7) * 2;
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const bf16x8_t p = __builtin_bit_cast(bf16x8_t, make_uint4(pw[t >> 1][4 * (t & 1)], pw[t >> 1][4 * (t & 1) + 1],
                                                                   pw[t >> 1][4 * (t & 1) + 2], pw[t >> 1][4 * (t & 1) + 3]));
        uint2 x = read_transposed(at + 16 * t * ROW), y = read_transposed(at + (16 * t + 8) * ROW);
        if constexpr (CLEAN) {
          odd |= not_finite<WT_BF16>(x.x) | not_finite<WT_BF16>(x.y) | not_finite<WT_BF16>(y.x) | not_finite<WT_BF16>(y.y);
          x = make_uint2(finite_part<WT_BF16>(x.x), finite_part<WT_BF16>(x.y));
          y = make_uint2(finite_part<WT_BF16>(y.x), finite_part<WT_BF16>(y.y));
        }
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(x.x, x.y, y.x, y.y)), p, acc[d], 0, 0, 0);
      }
    }
    return odd;
  }

  // The values that are not finite, key by key, into the rows that see the key.
  __device__ __forceinline__ void add_not_finite(const SFN_LDS char* v, const uint32_t (&pw)[2][8], int kt) {
#pragma unroll 1
    for (int kk = 0; kk < KT; ++kk) {
      uint32_t w = 0;  // the key's weight, in the lanes that hold it
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w = 32 * kb + 8 * (i >> 2) + (i & 3) == kk - 4 * h ? pw[kb][i >> 1] >> (16 * (i & 1)) & 0xffffu : w;
      int first = 4 * h;  // of the lane's values; opaque, so that no address is kept through the main loop
      asm("" : "+v"(first));
      const float p = __uint_as_float(__shfl((int)w, c + 32 * (kk >> 2 & 1), 64) << 16);
      const bool sees = kt + kk < row_hi && kt + kk >= row_lo;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const int col = 32 * d + 2 * i + first;  // the lane's values acc[d][i .. i + 3]
          const uint64_t x4 = *reinterpret_cast<const SFN_LDS uint64_t*>(v + kk * ROW + v_place(kk, col >> 3) * 16 + (col & 7) * 2);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = (uint32_t)(x4 >> (16 * e)) << 16;
            if (sees && not_finite<WT_F32>(x)) acc[d][i + e] = fmaf(p, __uint_as_float(x), acc[d][i + e]);
          }
        }
    }
  }

  // The stage's 64 keys from kt on. full: every row sees every key.
  __device__ __forceinline__ void step(const SFN_LDS char* k, const SFN_LDS char* v, int kt, bool full,
                                       float scale_log2) {
    f32x16_t s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const SFN_LDS char* at = k + c * ROW + k_place(c, 2 * i + h) * 16;  // the places repeat 32 rows further
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_frag(at + 32 * kb * ROW), q[i], s[kb], 0, 0, 0);
    }
    if (!full) {
      const int hi = row_hi - kt - 4 * h, lo = row_lo - kt - 4 * h;
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int key = 32 * kb + 8 * (i >> 2) + (i & 3);  // from the lane's first one on
          s[kb][i] = key < hi && key >= lo ? s[kb][i] : kNegInf;
        }
    }
    float top = kNegInf;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[kb][i]);
    top = swap_pair_max<32>(top) * scale_log2;  // the scale is positive
    if (__any(top > m + kSlack)) {
      const float mn = fmaxf(m, top);
      const float al = mn == kNegInf ? 0.f : exp2_f(m - mn);
      m = mn;
      l *= al;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] *= al;
    }
    const float ms = m == kNegInf ? 0.f : m;
    uint32_t pw[2][8];
    float add = 0.f;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = exp2_f(fmaf(s[kb][i], scale_log2, -ms)), p1 = exp2_f(fmaf(s[kb][i + 1], scale_log2, -ms));
        add += p0 + p1;
        pw[kb][i >> 1] = pack_bf16(p0, p1);
      }
    l += add;
    if (full) {
      add_values<false>(v, pw);
    } else if (__any(add_values<true>(v, pw))) {
      add_not_finite(v, pw, kt);
    }
  }
};

template <int DH>
__global__ __launch_bounds__(256, 2) void attend_tile_kernel(AttendArgs a) {
  using W = TileWave<DH>;
  constexpr int ND = W::ND, NC = W::NC, ROW = W::ROW, KT = kTileKeys;
  __shared__ __attribute__((aligned(16))) char s_k[2][KT * ROW], s_v[2][KT * ROW];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  W w;
  const int c = w.c = lane & 31, h = w.h = lane >> 5;
  int b = blockIdx.x;
  const int hk = b % a.h_kv;
  b /= a.h_kv;
  const int rtile = a.row_tiles - 1 - b % a.row_tiles;  // the longest first
  b /= a.row_tiles;
  const int split = b % a.S, r = b / a.S;

  const int t0 = min(max(gp(a.cu)[r], 0), a.T), t1 = min(max(gp(a.cu)[r + 1], t0), a.T);
  const int n = t1 - t0, g = a.g, rows = n * g;
  const int rho0 = rtile * kTileRows;
  if (rho0 >= rows) return;
  const int len = min(max(gp(a.kv_len)[r], 0), a.max_len);
  const int past = len - n;
  const int rho1 = min(rho0 + kTileRows, rows) - 1;
  const int hi = max(0, min(past + rho1 / g + 1, len));
  const int lo = a.window > 0 ? max(0, past + rho0 / g + 1 - a.window) : 0;
  const int k0 = (lo & ~(KT - 1)) + split * a.chunk, k1 = min(k0 + a.chunk, hi);
  if (split > 0 && k0 >= hi) return;

  // this wave's rows
  const int w0 = rho0 + 32 * wave, w1 = min(w0 + 32, rows) - 1;  // none if w0 > w1
  const int some_hi = w0 <= w1 ? min(past + w1 / g + 1, len) : 0;  // keys that some row of it sees
  const int some_lo = a.window > 0 ? past + w0 / g + 1 - a.window : 0;
  const int all_hi = min(past + w0 / g + 1, len);  // and that every row sees
  const int all_lo = a.window > 0 ? past + w1 / g + 1 - a.window : 0;
  const bool ok = w0 + c < rows;
  const int rho = ok ? w0 + c : rho0, tok = rho / g, head = hk * g + rho % g;
  w.row_hi = ok ? min(past + tok + 1, len) : 0;
  w.row_lo = a.window > 0 ? past + tok + 1 - a.window : 0;
  w.m = kNegInf;
  w.l = 0.f;
  {
    const SFN_GLOBAL char* src = gp(a.q) + (int64_t)(t0 + tok) * a.q_stride + head * ROW + 16 * h;
#pragma unroll
    for (int s = 0; s < W::NS; ++s) w.q[s] = __builtin_bit_cast(bf16x8_t, ld16(src + 32 * s));
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) w.acc[d][i] = 0.f;
  }

  const int lg = a.page_shift, pm = (1 << lg) - 1;
  const SFN_GLOBAL int32_t* table = gp(a.table) + (int64_t)r * a.max_pages;
  // byte offset in the cache of this wave's 16 rows of the stage at kt (one group, one page)
  auto rows_at = [&](int kt) -> int64_t {
    const int key = min(kt + 16 * wave, (k1 - 1) & ~15);
    const int page = min(max(table[key >> lg], 0), a.n_pages - 1);
    return ((((int64_t)page * a.h_kv + hk) << lg) + (key & pm)) * ROW;
  };
  SFN_LDS char* const kl = (SFN_LDS char*)&s_k[0][0];
  SFN_LDS char* const vl = (SFN_LDS char*)&s_v[0][0];
  const int mine = 16 * wave * ROW;

  int64_t at = k0 < k1 ? rows_at(k0) : 0;
  if (k0 < k1) W::load(gp(a.k) + at, gp(a.v) + at, kl + mine, vl + mine, lane);
  int buf = 0;
  for (int kt = k0; kt < k1; kt += KT, buf ^= KT * ROW) {
    const bool more = kt + KT < k1;
    if (more) at = rows_at(kt + KT);
    // this wave's part of the stage has arrived; after the barrier everyone's has, and the
    // other buffer is free
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    __syncthreads();
    if (kt + KT > len) {  // the last stage: what the page holds past the sequence becomes 0
      for (int i = tid; i < (kt + KT - len) * NC; i += 256)
        *reinterpret_cast<uint4*>(&s_v[buf ? 1 : 0][(KT - 1 - i / NC) * ROW + (i % NC) * 16]) = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    const int nx = buf ^ KT * ROW;
    if (more) W::load(gp(a.k) + at, gp(a.v) + at, kl + nx + mine, vl + nx + mine, lane);
    if (kt < some_hi && kt + KT > some_lo)
      w.step(kl + buf, vl + buf, kt, kt >= all_lo && kt + KT <= all_hi, a.scale_log2);
  }

  const float l = swap_pair_sum<32>(w.l);
  if (!ok) return;
  const int64_t orow = (int64_t)(t0 + tok) * a.h_q + head;
  if (a.S == 1) {
    const float inv = l == 0.f ? 0.f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<SFN_GLOBAL uint64_t*>(gp(a.out) + (orow * DH + 32 * d + 2 * i + 4 * h) * 2) =
            (uint64_t)pack_bf16(w.acc[d][i] * inv, w.acc[d][i + 1] * inv) |
            (uint64_t)pack_bf16(w.acc[d][i + 2] * inv, w.acc[d][i + 3] * inv) << 32;
  } else {
    const int64_t at = orow * a.S + split;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.part_o) + at * DH + 32 * d + 2 * i + 4 * h) =
            f32x4_t{w.acc[d][i], w.acc[d][i + 1], w.acc[d][i + 2], w.acc[d][i + 3]};
    if (h == 0) {
      gp(a.part_ml)[2 * at] = w.m;
      gp(a.part_ml)[2 * at + 1] = l;
    }
  }
}

// Joins the splits of one output row (a token's query head): one workgroup per row.
template <int WT, int DH>
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs a) {
  const int KT = a.tile_keys, tile_rows = a.tile_rows;
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
void launch_sized(const AttendArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((int64_t)a.R * a.S * a.row_tiles * a.h_kv)), block(256);
  if (a.tile_rows == kTileRows) {
    if constexpr (WT == WT_BF16) hipLaunchKernelGGL((attend_tile_kernel<DH>), grid, block, 0, stream, a);
  } else if (a.tile_rows == 16) {
    hipLaunchKernelGGL((attend_split_kernel<WT, DH, 1>), grid, block, 0, stream, a);
  } else {
    hipLaunchKernelGGL((attend_split_kernel<WT, DH, 2>), grid, block, 0, stream, a);
  }
  if (a.S > 1) {
    const dim3 rows((unsigned)((int64_t)a.R * a.max_new * a.h_q));
    hipLaunchKernelGGL((attend_join_kernel<WT, DH>), rows, block, 0, stream, a);
  }
}

}  // namespace

// workgroups that fill the chip once: as many as are resident
#ifndef X_SLOTS1
#define X_SLOTS1 768
#define X_SLOTS2 512
#define X_SLOTST 512
#define X_MAXS 256
#endif
AttendPlan attend_plan(int R, int h_q, int h_kv, int dtype, int max_new, int max_len, int window) {
  AttendPlan p;
  const int64_t rows = (int64_t)max_new * (h_q / h_kv);
  const bool bf = dtype == SFN_BF16;
  p.tile_rows = rows <= 16 ? 16 : rows <= 32 || !bf ? 32 : kTileRows;
  p.tile_keys = p.tile_rows == kTileRows ? kTileKeys : bf ? 32 : 16;
  const int64_t tiles = (rows + p.tile_rows - 1) / p.tile_rows;
  p.row_tiles = (int)tiles;
  // keys one row tile can span
  int64_t span = max_len;
  if (window > 0 && (int64_t)window + max_new + p.tile_keys < span) span = (int64_t)window + max_new + p.tile_keys;
  if (span < 1) span = 1;
  const int64_t base = (int64_t)R * h_kv * tiles;
  const int64_t step = p.tile_rows == kTileRows ? p.tile_keys : 4 * p.tile_keys;  // a tile for each wave
  const int64_t slots = p.tile_rows == 16 ? X_SLOTS1 : p.tile_rows == 32 ? X_SLOTS2 : X_SLOTST;
  int64_t s = (slots + base - 1) / base;
  if (s > X_MAXS) s = X_MAXS;
  p.S_most = (int)std::min<int64_t>(s, std::max<int64_t>(1, ((int64_t)max_len + step - 1) / step));
  const int64_t chunk = ((span + s - 1) / s + step - 1) / step * step;
  p.chunk = (int)chunk;
  p.S = (int)((span + chunk - 1) / chunk);
  return p;
}

hipError_t launch_kv_attend(const AttendArgs& a, int dh, int dtype, hipStream_t stream) {
  if (dtype == SFN_BF16) {
    if (dh == 64) launch_sized<WT_BF16, 64>(a, stream);
    else launch_sized<WT_BF16, 128>(a, stream);
  } else {
    if (dh == 64) launch_sized<WT_F32, 64>(a, stream);
    else launch_sized<WT_F32, 128>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace sfn
