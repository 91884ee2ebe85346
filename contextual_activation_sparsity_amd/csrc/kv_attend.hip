// Attention of each request's new tokens over its pages of the key/value cache.

#include <algorithm>

#include "kernels.h"
#include "serving_common.h"
#include "sparse_ffn.h"

namespace sfn {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;

constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kMaxSplits = 256;  // the join kernel's threads

// ---- split attention -----------------------------------------------------------------
//
// For few query rows to a key head (up to 32), and for fp32. A workgroup takes 16 RT rows of
// one key head's queries (row rho of a request is its token rho / g, head rho % g of the g
// query heads that share the key head, so grouped heads fill the matrix tile) and one split
// of the keys; its NW waves take every NW-th tile of the split, each with a softmax of its
// own (running maximum and sum, fp32), and join at the end. K, Q, P and V go from memory to
// the matrix cores through registers alone: at these sizes the products are far from their
// bound, and streaming through LDS (as the tile kernel does) took 102 us where this takes
// 83. Nor do registers for two tiles at once help (105 against 93 us with 8 waves): twelve
// waves of 16 KB each already keep more than enough bytes under way.
// The scores are computed as S^T = K Q^T, whose tile leaves one query row per lane (lane & 15)
// and its keys in the lane's registers, so maxima and sums need two lane swaps and P^T is
// already laid out as the right operand of O^T = V^T P^T:
//   bf16: 32 keys a tile, two 16 x 16 score tiles; the P operand wants 8 keys a lane, and
//   as the order of the contracted keys is free, lane quarter q takes keys 4q..4q+3 of
//   either score tile, which are the ones it holds. V rows are read as they lie (VW values
//   a lane); the left operand of output block e takes element e of each lane's values
//   (a byte permute packs two keys), so O's rows come out as dh = VW (4q + i) + e.
//   fp32: 16 keys a tile; the 16x16x4 product takes one key per lane quarter, so step i
//   takes keys 4q + i: again the ones the lane holds, with no packing.
// Masked scores are -inf; a row that sees no key keeps l = 0 and gives zeros. Values of
// keys past the end of the sequence are zeroed, whatever the cache holds there.
// Rows of one tile: bound by the read of K and V, each once (counted: 537 and 853 MB). One token
// over 131000 keys, 64 / 8 heads of 128: 82.7 us, 6.5 TB/s (a plain read kernel reaches 5.8 to
// 6.8); 48 requests of up to 8000 keys, 32 / 8 heads: 141.6 us, 6.0 TB/s; non-temporal loads,
// since nothing is read twice, gave 7% of that. fp32 twice the bytes: 168 and 272 us. A short call
// is a chain of dependent reads (lengths and pages, keys, the join), each about a microsecond:
// 201 keys, 32 heads, 4 us.
// fp32 with more rows reads K and V again for every tile of 32, and is bound by the products,
// which wait for each tile's loads: two requests of 1000 tokens after 4000 others, 32 / 8 heads
// of 128, 1387 us, 106 TFLOP/s where an fp32 product of 8192 x 8192 reaches 154.
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

// Values d4 .. d4 + 3 of one output row, from their unscaled sums and the sum of weights.
template <int WT, int DH>
__device__ __forceinline__ void store_row(const AttendArgs& a, int token, int head, int d4, f32x4_t o, float L) {
  o *= L == 0.f ? 0.f : 1.0f / L;
  const int64_t at = ((int64_t)token * a.h_q + head) * DH + d4;
  if constexpr (WT == WT_BF16)
    *reinterpret_cast<SFN_GLOBAL uint64_t*>(gp(a.out) + at * 2) =
        (uint64_t)pack_bf16(o[0], o[1]) | (uint64_t)pack_bf16(o[2], o[3]) << 32;
  else
    *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.out) + at * 4) = o;
}

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

// sum + both bf16 halves of w, in fp32.
__device__ __forceinline__ float add_pair(uint32_t w, float sum) {
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), __builtin_bit_cast(bf16x2_t, 0x3f803f80u), sum, false);
}

// acc += V^T P^T of one tile: v the lane's words of V (group, key 4q + j, piece, word), p
// its weights (group, key 4q + i); l += the lane's weights.
template <int WT, int DH>
__device__ __forceinline__ void add_weighted(
    const uint32_t (&v)[AttnTile<WT, DH>::NG][4][AttnTile<WT, DH>::NB][AttnTile<WT, DH>::VW * AttnTile<WT, DH>::KB / 4],
    const f32x4_t (&p)[AttnTile<WT, DH>::NG], f32x4_t (&acc)[AttnTile<WT, DH>::NO], float& l) {
  using C = AttnTile<WT, DH>;
  if constexpr (C::kBf) {
    // the weights are rounded to bf16, as V is: the matrix cores take both operands in one
    // type, and the rounding (at most 2^-8 of each weight, of either sign) adds no more to
    // the result than rounding it to bf16 at the end does. Their sum, in fp32, is of the
    // rounded weights, so that the result is a true mean of the rows of V: what one large
    // weight loses by its rounding cancels.
    const uint4 pw = make_uint4(pack_bf16(p[0][0], p[0][1]), pack_bf16(p[0][2], p[0][3]), pack_bf16(p[1][0], p[1][1]),
                                pack_bf16(p[1][2], p[1][3]));
    l = add_pair(pw.x, add_pair(pw.y, l)) + add_pair(pw.z, add_pair(pw.w, 0.f));
    const bf16x8_t pf = __builtin_bit_cast(bf16x8_t, pw);
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
    l += (p[0][0] + p[0][1]) + (p[0][2] + p[0][3]);
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
  asm("" : "+v"(vp));  // no address of this is kept through the main loop
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

// One tile of keys in a lane's registers.
template <int WT, int DH>
struct KeyTile {
  using C = AttnTile<WT, DH>;
  uint4 k[C::NG][C::NQ];
  uint32_t v[C::NG][4][C::NB][C::VW * C::KB / 4];

  // row: the cache row of each group's first key
  __device__ __forceinline__ void load(const AttendArgs& a, const int64_t (&row)[C::NG], int c, int q) {
    constexpr int ROW = DH * C::KB;
#pragma unroll
    for (int u = 0; u < C::NG; ++u) {
      const SFN_GLOBAL char* kp = gp(a.k) + (row[u] + c) * ROW + 16 * q;
#pragma unroll
      for (int s = 0; s < C::NQ; ++s) k[u][s] = ldg16(kp + 64 * s);
    }
#pragma unroll
    for (int u = 0; u < C::NG; ++u) {
      const SFN_GLOBAL char* vp = gp(a.v) + (row[u] + 4 * q) * ROW + c * C::VW * C::KB;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb) {
          const SFN_GLOBAL char* p = vp + j * ROW + nb * 16 * C::VW * C::KB;
          if constexpr (C::VW * C::KB == 16) {
            const uint4 w = ldg16(p);
            v[u][j][nb][0] = w.x;
            v[u][j][nb][1] = w.y;
            v[u][j][nb][2] = w.z;
            v[u][j][nb][3] = w.w;
          } else {
            const uint64_t w = __builtin_nontemporal_load(reinterpret_cast<const SFN_GLOBAL uint64_t*>(p));
            v[u][j][nb][0] = (uint32_t)w;
            v[u][j][nb][1] = (uint32_t)(w >> 32);
          }
        }
    }
  }

  // Zeroes the values of keys from `keys` on (keys of the tile that the sequence has); returns
  // whether some other value is not finite, and makes those 0 too.
  __device__ __forceinline__ bool clean(int keys, int q) {
    uint32_t top = 0;  // the largest magnitude bits seen: of the bf16 halves, or of the fp32 words
#pragma unroll
    for (int u = 0; u < C::NG; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
          for (int w = 0; w < C::VW * C::KB / 4; ++w) {
            uint32_t& x = v[u][j][nb][w];
            x = 16 * u + j < keys - 4 * q ? x : 0u;
            if constexpr (C::kBf) {
              typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;
              top = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, top),
                                                                           __builtin_bit_cast(u16x2_t, x & 0x7fff7fffu)));
            } else {
              top = max(top, x & 0x7fffffffu);
            }
          }
    const bool odd = C::kBf ? (top & 0xffffu) >= 0x7f80u || top >= 0x7f800000u : top >= 0x7f800000u;
    if (!__any(odd)) return false;
#pragma unroll
    for (int u = 0; u < C::NG; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nb = 0; nb < C::NB; ++nb)
#pragma unroll
          for (int w = 0; w < C::VW * C::KB / 4; ++w) v[u][j][nb][w] = finite_part<WT>(v[u][j][nb][w]);
    return true;
  }
};

// The rows of a tile that starts at row rho0: which token and which of the g heads.
struct RowMap {
  int tok0, rem0, mul, g;
  __device__ __forceinline__ RowMap(const AttendArgs& a, int rho0) : mul(a.g_mul), g(a.g) {
    tok0 = rho0 ? rho0 / g : 0;
    rem0 = rho0 - tok0 * g;
  }
  // of row rho0 + i, i < 128: g_mul is 2^21 / g rounded up, and i + rem0 < 128 + 1024
  __device__ __forceinline__ int token(int i) const { return tok0 + (int)((uint32_t)(i + rem0) * (uint32_t)mul >> 21); }
  __device__ __forceinline__ int head(int i, int tok) const { return i + rem0 - (tok - tok0) * g; }
};

template <int WT, int DH, int RT, int NW>
__global__ __launch_bounds__(64 * NW, NW == 8 || RT == 2 ? 2 : 3) void attend_split_kernel(AttendArgs a) {
  using C = AttnTile<WT, DH>;
  constexpr int KT = C::KT, NG = C::NG, NQ = C::NQ, VW = C::VW, NB = C::NB, NO = C::NO, KB = C::KB;
  constexpr int TR = 16 * RT, ROW = DH * KB;
  __shared__ float s_m[NW][TR], s_l[NW][TR];
  __shared__ __attribute__((aligned(16))) float s_o[NW][TR][DH + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int rtile = a.row_tiles == 1 ? 0 : blockIdx.x / a.h_kv, hk = blockIdx.x - rtile * a.h_kv;
  const int split = blockIdx.y, r = blockIdx.z;

  // the cache row of the first key of a group of 16, from the request's page table; a key past
  // the sequence may name any page, of this cache
  const int lg = a.page_shift, pm = (1 << lg) - 1;
  const SFN_GLOBAL int32_t* table = gp(a.table) + (int64_t)r * a.max_pages;
  auto page_of = [&](int key) { return __builtin_amdgcn_readfirstlane(table[min(key >> lg, a.max_pages - 1)]); };
  auto row_in = [&](int page, int key) -> int64_t {
    return (((int64_t)min(max(page, 0), a.n_pages - 1) * a.h_kv + hk) << lg) + (key & pm & ~15);
  };
  // without a window the first keys do not depend on the lengths: their pages are read with them
  int page[NG];
#pragma unroll
  for (int u = 0; u < NG; ++u) page[u] = page_of(split * a.chunk + wave * KT + 16 * u);

  const int t0 = min(max(gp(a.cu)[r], 0), a.T), t1 = min(max(gp(a.cu)[r + 1], t0), a.T);
  const int n = t1 - t0, g = a.g, rows = min(n, a.max_new) * g;
  const int len = min(max(gp(a.kv_len)[r], 0), a.max_len);
  const int rho0 = rtile * TR;
  if (rho0 >= rows) return;
  const int past = len - n;  // position of the first new token
  const RowMap map(a, rho0);
  const int last = min(TR, rows - rho0) - 1, tok1 = map.token(last);
  // keys that some row of the tile sees, and that every row sees
  const int hi = max(0, min(past + tok1 + 1, len));
  const int lo = a.window > 0 ? max(0, past + map.tok0 + 1 - a.window) : 0;
  const int hi_all = min(past + map.tok0 + 1, len);
  const int lo_all = a.window > 0 ? max(0, past + tok1 + 1 - a.window) : 0;
  const int k0 = (lo & ~(KT - 1)) + split * a.chunk, k1 = min(k0 + a.chunk, hi);
  if (split > 0 && k0 >= hi) return;

  const int kw = k0 + wave * KT;
  KeyTile<WT, DH> tile;
  auto find = [&](int kt) {
#pragma unroll
    for (int u = 0; u < NG; ++u) page[u] = page_of(kt + 16 * u);
  };
  // the tile at kt, from the pages found for it, and then the pages of the one after it
  auto fetch = [&](int kt) {
    int64_t row[NG];
#pragma unroll
    for (int u = 0; u < NG; ++u) row[u] = row_in(page[u], kt + 16 * u);
    tile.load(a, row, c, q);
    if (kt + NW * KT < k1) find(kt + NW * KT);
  };
  if (kw < k1) {
    if (lo > 0) find(kw);
    fetch(kw);
  }

  // Q: right operand, lane's row c, chunk s: values 64 s / KB + 16 q / KB ...
  uint4 qf[RT][NQ];
  int row_hi[RT], row_lo[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    const bool ok = 16 * x + c <= last;
    const int i = ok ? 16 * x + c : 0, tok = map.token(i), head = hk * g + map.head(i, tok);
    const SFN_GLOBAL char* src = gp(a.q) + (int64_t)(t0 + tok) * a.q_stride + head * ROW + 16 * q;
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

  for (int kt = kw; kt < k1;) {
    // A masked key has weight 0, but 0 times a value that is not finite is NaN: a tile with a
    // masked key and such a value takes the long way below, so that no token's result
    // depends on tokens it does not see.
    const bool full = kt >= lo_all && kt + KT <= hi_all;  // every row sees every key of the tile
    const bool odd = full ? false : tile.clean(len - kt, q);
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      f32x4_t s[NG];
#pragma unroll
      for (int u = 0; u < NG; ++u) {
        const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
        if constexpr (C::kBf) {
          s[u] = zero;
#pragma unroll
          for (int i = 0; i < NQ; ++i)
            s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, tile.k[u][i]),
                                                           __builtin_bit_cast(bf16x8_t, qf[x][i]), s[u], 0, 0, 0);
        } else {
          // four sums side by side: half the rounding error of one chain of dh additions (sharp
          // scores, 600 keys: 4.4e-7 of the result against 1.1e-6), for 10.0 instead of 9.8 us
          // of the windowed fp32 chunk
          f32x4_t part[4] = {zero, zero, zero, zero};
#pragma unroll
          for (int i = 0; i < NQ; ++i) {
            const f32x4_t kk = __builtin_bit_cast(f32x4_t, tile.k[u][i]), qq = __builtin_bit_cast(f32x4_t, qf[x][i]);
#pragma unroll
            for (int e = 0; e < 4; ++e) part[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(kk[e], qq[e], part[e], 0, 0, 0);
          }
          s[u] = (part[0] + part[1]) + (part[2] + part[3]);
        }
      }
      // p = 2^(scale s - m), scale and m in units of log2, with one rounding
      float top = kNegInf;
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!full) {
            const int key = 16 * u + i, at = kt + 4 * q;
            s[u][i] = key < row_hi[x] - at && key >= row_lo[x] - at ? s[u][i] : kNegInf;
          }
          top = fmaxf(top, s[u][i]);
        }
      top = swap_pair_max<16>(top);
      top = swap_pair_max<32>(top) * a.scale_log2;  // the scale is positive
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
#pragma unroll
      for (int u = 0; u < NG; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][i] = exp2_f(fmaf(s[u][i], a.scale_log2, -ms));
      add_weighted<WT, DH>(tile.v, s, acc[x], l[x]);
      if (odd) {
        // the values that are not finite: key by key, read again, into the rows that see them
#pragma unroll 1
        for (int kk = 0; kk < KT && kt + kk < len; ++kk)
          add_one_key<WT, DH>(gp(a.v) + (row_in(page_of(kt + kk), kt + kk) + (kk & 15)) * ROW + c * VW * KB, s, kk, q,
                              kt + kk < row_hi[x] && kt + kk >= row_lo[x], acc[x]);
      }
    }
    kt += NW * KT;
    if (kt < k1) fetch(kt);
  }

  // join the waves: a common maximum, then the sums in wave order
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    l[x] = swap_pair_sum<16>(l[x]);
    l[x] = swap_pair_sum<32>(l[x]);
    if (q == 0) s_m[wave][16 * x + c] = m[x];
  }
  __syncthreads();
  float M[RT];
#pragma unroll
  for (int x = 0; x < RT; ++x) {
    M[x] = s_m[0][16 * x + c];
#pragma unroll
    for (int w = 1; w < NW; ++w) M[x] = fmaxf(M[x], s_m[w][16 * x + c]);
    const float w_self = m[x] == kNegInf ? 0.f : exp2_f(m[x] - M[x]);
    if (q == 0) s_l[wave][16 * x + c] = l[x] * w_self;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < VW; e += 4)
          *reinterpret_cast<f32x4_t*>(&s_o[wave][16 * x + c][16 * VW * nb + VW * (4 * q + i) + e]) =
              f32x4_t{acc[x][nb * VW + e][i], acc[x][nb * VW + e + 1][i], acc[x][nb * VW + e + 2][i], acc[x][nb * VW + e + 3][i]} * w_self;
  }
  __syncthreads();
  for (int i = tid; i < (last + 1) * (DH / 4); i += 64 * NW) {
    const int x = i / (DH / 4), d4 = (i % (DH / 4)) * 4;
    const int tok = map.token(x), head = hk * g + map.head(x, tok);
    float L = 0.f;
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      L += s_l[w][x];
      o += *reinterpret_cast<const f32x4_t*>(&s_o[w][x][d4]);
    }
    if (a.S == 1) {
      store_row<WT, DH>(a, t0 + tok, head, d4, o, L);
    } else {
      const int64_t at = (((int64_t)r * a.max_new + tok) * a.h_q + head) * a.S + split;
      *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.part_o) + at * DH + d4) = o;
      if (d4 == 0) {
        float top = s_m[0][x];
#pragma unroll
        for (int w = 1; w < NW; ++w) top = fmaxf(top, s_m[w][x]);
        *reinterpret_cast<SFN_GLOBAL f32x2_t*>(gp(a.part_ml) + 2 * at) = f32x2_t{top, L};
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
// and most tiles then leave the accumulators alone. It costs accuracy where one key has most of
// the weight: with the exact maximum that key's weight is 1, which bf16 holds exactly, with a
// lagging one it is rounded like the others. Sharp scores (deviation 2), error against 64 bits
// relative to the result: 0.0021 for the 16-token chunk and 0.0022 for prompts; with kSlack 0
// 0.0018 and 0.0019, like the split kernel, and 1 to 4% longer for chunks, 6 to 9% for prompts.
// Two requests of 2048 tokens after 8192 others, 32 / 8 heads of 128: 619 GFLOP in 580 to 625
// us by the box, 990 to 1065 TFLOP/s, where a sustained bf16 product of 8192 x 8192 reaches
// 1385. What bounds it is power, and how full the matrix cores are: they are busy half of the
// clocks (the library's product keeps them busy 69%), with no bank conflict in LDS, and the
// clock falls to 1.6 to 1.9 GHz, as it does for that product, where a kernel bound by memory runs
// at 2.5. Fewer clocks a key have brought lower clocks: leaving out the whole softmax saves 3%.
// Heads of 64 have as much softmax for half the products: 370 us, 837 TFLOP/s. The four requests'
// 16-token chunk (82 MB of K and V) reads at 5.8 TB/s between a start of 2 us and the joins.
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

// 16 bytes a lane from `from` + offset to LDS at lds + 16 lane, without waiting. A read of LDS
// afterwards waits for the data unless the compiler can tell that it reads another array: the
// stages lie in two arrays for that, and the loop takes turns with them (one array: 688 instead
// of 603 us on the 2048-token prompts, 32.4 instead of 28.9 us on the 16-token chunk). The
// buffer form, because the waits for LDS are then counted and not for everything (620 and 30.2 us).
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t offset, SFN_LDS char* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(from, (SFN_LDS void*)lds, 16, offset, 0, 0, 0);
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
    const __amdgpu_buffer_rsrc_t kr = __builtin_amdgcn_make_buffer_rsrc((void*)kp, 0, 16 * ROW, 0x00027000);
    const __amdgpu_buffer_rsrc_t vr = __builtin_amdgcn_make_buffer_rsrc((void*)vp, 0, 16 * ROW, 0x00027000);
#pragma unroll
    for (int i = 0; i < 16 / RI; ++i) {
      const int row = i * RI + lane / NC, ch = lane % NC;  // the wave's rows start at a multiple of 16
      const uint32_t ko = row * ROW + k_place(row, ch) * 16, vo = row * ROW + v_place(row, ch) * 16;
      load_to_lds(kr, ko, kl + i * 1024);
      load_to_lds(vr, vo, vl + i * 1024);
    }
  }

  // acc += V^T P^T over the stage
  __device__ __forceinline__ void add_values(const SFN_LDS char* stage, int voff, const uint32_t (&pw)[2][8]) {
    const int vrow = 4 * h + (c & 15) / 4, vcol = 16 * (c >> 4) + 4 * (c & 3);
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const bf16x8_t p = __builtin_bit_cast(bf16x8_t, make_uint4(pw[t >> 1][4 * (t & 1)], pw[t >> 1][4 * (t & 1) + 1],
                                                                 pw[t >> 1][4 * (t & 1) + 2], pw[t >> 1][4 * (t & 1) + 3]));
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const int col = 32 * d + vcol;
        // 16 rows further the places repeat
        int place = voff + vrow * ROW + v_place(vrow, col >> 3) * 16 + (col & 7) * 2;
        asm("" : "+v"(place));  // one step from the array, so that the compiler sees which array it is
        const SFN_LDS char* at = stage + place;
        const uint2 x = read_transposed(at + 16 * t * ROW), y = read_transposed(at + (16 * t + 8) * ROW);
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, make_uint4(x.x, x.y, y.x, y.y)), p, acc[d], 0, 0, 0);
      }
    }
  }

  // The values that are not finite, read again from the cache, key by key, into the rows that
  // see the key. row(key): where its row of V begins.
  template <class Row>
  __device__ __forceinline__ void add_not_finite(Row row, const uint32_t (&pw)[2][8], int kt, int keys) {
#pragma unroll 1
    for (int kk = 0; kk < keys; ++kk) {
      uint32_t w = 0;  // the key's weight, in the lanes that hold it
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          w = 32 * kb + 8 * (i >> 2) + (i & 3) == kk - 4 * h ? pw[kb][i >> 1] >> (16 * (i & 1)) & 0xffffu : w;
      int first = 8 * h;  // of the lane's values, in bytes; opaque, so that no address is kept through the main loop
      asm("" : "+v"(first));
      const float p = __uint_as_float(__shfl((int)w, c + 32 * (kk >> 2 & 1), 64) << 16);
      const bool sees = kt + kk < row_hi && kt + kk >= row_lo;
      const SFN_GLOBAL char* v = row(kt + kk);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const uint64_t x4 = *reinterpret_cast<const SFN_GLOBAL uint64_t*>(v + 64 * d + 4 * i + first);  // of acc[d][i .. i + 3]
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t x = (uint32_t)(x4 >> (16 * e)) << 16;
            acc[d][i + e] = sees && not_finite<WT_F32>(x) ? fmaf(p, __uint_as_float(x), acc[d][i + e]) : acc[d][i + e];
          }
        }
    }
  }

  // The stage's 64 keys from kt on. full: every row sees every key. odd: values that are not
  // finite were taken out of the stage (see add_not_finite).
  template <class Row>
  __device__ __forceinline__ void step(const SFN_LDS char* stage, int koff, int voff, int kt, bool full, bool odd, float scale_log2,
                                       Row row, int keys) {
    // the matrix products first: the compute unit's other workgroup then falls out of step and
    // does its softmax meanwhile (614 -> 589 us on the 2048-token prompts)
    __builtin_amdgcn_s_setprio(1);
    f32x16_t s[2];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; ++i) s[kb][i] = 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const SFN_LDS char* at = stage + (koff + c * ROW + k_place(c, 2 * i + h) * 16);  // the places repeat 32 rows further
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) s[kb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(read_frag(at + 32 * kb * ROW), q[i], s[kb], 0, 0, 0);
    }
    __builtin_amdgcn_s_setprio(0);
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
    float add[2] = {l, 0.f};
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float p0 = exp2_f(fmaf(s[kb][i], scale_log2, -ms)), p1 = exp2_f(fmaf(s[kb][i + 1], scale_log2, -ms));
        pw[kb][i >> 1] = pack_bf16(p0, p1);
        add[kb] = add_pair(pw[kb][i >> 1], add[kb]);
      }
    l = add[0] + add[1];
    __builtin_amdgcn_s_setprio(1);
    add_values(stage, voff, pw);
    __builtin_amdgcn_s_setprio(0);
    if (__builtin_expect(odd, 0)) add_not_finite(row, pw, kt, keys);
  }
};

// KG groups of four waves: with two of them (a split of the keys for few row tiles) each takes
// every second stage, with buffers of its own, and the groups join in LDS at the end, so that
// there are half as many parts to write and join as with two workgroups.
template <int DH, int KG>
__global__ __launch_bounds__(256 * KG, 2) void attend_tile_kernel(AttendArgs a) {
  using W = TileWave<DH>;
  constexpr int ND = W::ND, NC = W::NC, ROW = W::ROW, KT = kTileKeys;
  constexpr int STAGE = KT * ROW;  // bytes of a stage of K, and of V
  // two arrays, so that the compiler knows that the reads of one need not wait for the loads
  // into the other; of each, a group's K stage and its V stage
  __shared__ __attribute__((aligned(16))) char s_a[KG * 2 * STAGE];
  __shared__ __attribute__((aligned(16))) char s_b[KG * 2 * STAGE];
  const int tid = threadIdx.x & 255, lane = threadIdx.x & 63;
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // in its group
  W w;
  const int c = w.c = lane & 31, h = w.h = lane >> 5;
  const int hk = a.row_tiles == 1 ? blockIdx.x : blockIdx.x % a.h_kv;
  const int rtile = a.row_tiles == 1 ? 0 : a.row_tiles - 1 - blockIdx.x / a.h_kv;  // the longest first
  const int split = blockIdx.y, r = blockIdx.z;

  // byte offset in the cache of this wave's 16 rows of the stage at kt (one group of keys, in
  // one page; past the sequence any page of the cache)
  const int lg = a.page_shift, pm = (1 << lg) - 1;
  const SFN_GLOBAL int32_t* table = gp(a.table) + (int64_t)r * a.max_pages;
  auto page_of = [&](int kt) { return __builtin_amdgcn_readfirstlane(table[min((kt + 16 * wave) >> lg, a.max_pages - 1)]); };
  auto rows_in = [&](int page, int kt) -> int64_t {
    return ((((int64_t)min(max(page, 0), a.n_pages - 1) * a.h_kv + hk) << lg) + ((kt + 16 * wave) & pm)) * ROW;
  };
  // without a window the first stage does not depend on the lengths: its page is read with them
  int page = page_of(split * a.chunk + kg * KT);

  const int t0 = min(max(gp(a.cu)[r], 0), a.T), t1 = min(max(gp(a.cu)[r + 1], t0), a.T);
  const int n = t1 - t0, g = a.g, rows = min(n, a.max_new) * g;
  const int len = min(max(gp(a.kv_len)[r], 0), a.max_len);
  const int rho0 = rtile * kTileRows;
  if (rho0 >= rows) return;
  const int past = len - n;
  const RowMap map(a, rho0);
  const int last = min(kTileRows, rows - rho0) - 1;  // the tile's last row
  // keys that some row of the tile sees, and that every row sees
  const int tok1 = map.token(last);
  const int hi = max(0, min(past + tok1 + 1, len));
  const int lo = a.window > 0 ? max(0, past + map.tok0 + 1 - a.window) : 0;
  const int tile_hi = min(past + map.tok0 + 1, len);
  const int tile_lo = a.window > 0 ? past + tok1 + 1 - a.window : 0;
  const int k0 = (lo & ~(KT - 1)) + split * a.chunk, k1 = min(k0 + a.chunk, hi);
  if (split > 0 && k0 >= hi) return;

  const int group = kg * 2 * STAGE, mine = group + 16 * wave * ROW;
  const int kg0 = k0 + kg * KT;
  if (kg0 < k1) {
    if (lo > 0) page = page_of(kg0);
    const int64_t at = rows_in(page, kg0);
    W::load(gp(a.k) + at, gp(a.v) + at, (SFN_LDS char*)s_a + mine, (SFN_LDS char*)s_a + STAGE + mine, lane);
  }

  // this wave's rows
  const int i0 = 32 * wave, i1 = min(i0 + 31, last);  // none if i0 > last
  const int wt0 = map.token(i0), wt1 = map.token(max(i1, 0));
  const int some_hi = i0 <= last ? min(past + wt1 + 1, len) : 0;  // keys that some row of it sees
  const int some_lo = a.window > 0 ? past + wt0 + 1 - a.window : 0;
  const int all_hi = min(past + wt0 + 1, len);  // and that every row sees
  const int all_lo = a.window > 0 ? past + wt1 + 1 - a.window : 0;
  const bool ok = i0 + c <= last;
  const int i = ok ? i0 + c : 0, tok = map.token(i), head = hk * g + map.head(i, tok);
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
      for (int e = 0; e < 16; ++e) w.acc[d][e] = 0.f;
  }
  auto v_row = [&](int key) {
    const int p = min(max(table[key >> lg], 0), a.n_pages - 1);
    return gp(a.v) + ((((int64_t)p * a.h_kv + hk) << lg) + (key & pm)) * ROW;
  };

  // a round, a stage for each group: the keys from kr on, in cur; the next ones go into nxt
  auto round = [&](char* cur, char* nxt, int kr) __attribute__((always_inline)) {
    const int kt = kr + kg * KT, kn = kt + KG * KT;
    if (kn < k1) page = page_of(kn);
    // this wave's part of the stage has arrived; after the barrier everyone's has, and the
    // other array is free
    __builtin_amdgcn_s_waitcnt(kWaitLoads);
    __syncthreads();
    // A stage with masked keys: what the page holds past the sequence becomes 0, and so do
    // values that are not finite (0 times one of them is NaN); those count in a way of their own
    bool odd = false;
    if (kr + KG * KT > tile_hi || kr < tile_lo) {
      for (int e = kt < k1 ? tid : KT * NC; e < KT * NC; e += 256) {
        uint4* const at = reinterpret_cast<uint4*>(cur + group + STAGE + e * 16);
        const uint4 x = *at;
        if (kt + e / NC >= len) {
          *at = make_uint4(0, 0, 0, 0);
        } else if (not_finite<WT_BF16>(x.x) | not_finite<WT_BF16>(x.y) | not_finite<WT_BF16>(x.z) | not_finite<WT_BF16>(x.w)) {
          *at = make_uint4(finite_part<WT_BF16>(x.x), finite_part<WT_BF16>(x.y), finite_part<WT_BF16>(x.z), finite_part<WT_BF16>(x.w));
          odd = true;
        }
      }
      odd = __syncthreads_or(odd);
    }
    if (kn < k1) {
      const int64_t at = rows_in(page, kn);
      W::load(gp(a.k) + at, gp(a.v) + at, (SFN_LDS char*)nxt + mine, (SFN_LDS char*)nxt + STAGE + mine, lane);
    }
    if (kt < min(some_hi, k1) && kt + KT > some_lo)
      w.step((SFN_LDS char*)cur, group, group + STAGE, kt, kt >= all_lo && kt + KT <= all_hi, odd, a.scale_log2, v_row,
             min(KT, len - kt));
  };
  for (int kr = k0; kr < k1; kr += KG * KT) {
    round(s_a, s_b, kr);
    kr += KG * KT;
    if (kr >= k1) break;
    round(s_b, s_a, kr);
  }

  float l = swap_pair_sum<32>(w.l);
  __syncthreads();  // the stages have been read: their LDS is free
  if constexpr (KG == 2) {
    // the second group's sums through LDS, 16 bytes a lane and step, each pair of waves in a
    // part of its own (where the wave below then puts its rows)
    f32x4_t* const at = reinterpret_cast<f32x4_t*>(s_a + wave * 32 * DH * 4) + lane;
    float* const ml = reinterpret_cast<float*>(s_b) + 2 * tid;
    if (kg == 1) {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          at[(d * 4 + e) * 64] = f32x4_t{w.acc[d][4 * e], w.acc[d][4 * e + 1], w.acc[d][4 * e + 2], w.acc[d][4 * e + 3]};
      ml[0] = w.m;
      ml[1] = l;
    }
    __syncthreads();
    if (kg == 1) return;
    const float mo = ml[0], lo2 = ml[1];
    const float M = fmaxf(w.m, mo);
    const float f = w.m == kNegInf ? 0.f : exp2_f(w.m - M), fo = mo == kNegInf ? 0.f : exp2_f(mo - M);
    w.m = M;
    l = l * f + lo2 * fo;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const f32x4_t o = at[(d * 4 + e) * 64];
#pragma unroll
        for (int j = 0; j < 4; ++j) w.acc[d][4 * e + j] = w.acc[d][4 * e + j] * f + o[j] * fo;
      }
    wave_sync();  // the rows below go where other lanes read these sums
  }
  // Rows out through LDS, so that whole rows are written at once (a lane's values are 4 of
  // every 8 of its row). 16-byte places are permuted like the stages'.
  constexpr int OC = DH / 4;  // 16-byte places of an fp32 row
  char* const out = KG == 1 ? (wave < 2 ? s_a : s_b) + (wave & 1) * 32 * DH * 4 : s_a + wave * 32 * DH * 4;
  const bool whole = a.S == 1;
  const float inv = whole ? (l == 0.f ? 0.f : 1.0f / l) : 1.f;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<f32x4_t*>(out + c * DH * 4 + (((8 * d + 2 * e + h) ^ (c & 15)) * 16)) =
          f32x4_t{w.acc[d][4 * e], w.acc[d][4 * e + 1], w.acc[d][4 * e + 2], w.acc[d][4 * e + 3]} * inv;
  // the lane's row in the output or in the parts, -1 if it has none
  const int64_t orow = whole ? (int64_t)(t0 + tok) * a.h_q + head : (((int64_t)r * a.max_new + tok) * a.h_q + head) * a.S + split;
  const int own = ok ? (int)orow : -1;
  if (!whole && h == 0 && ok) *reinterpret_cast<SFN_GLOBAL f32x2_t*>(gp(a.part_ml) + 2 * orow) = f32x2_t{w.m, l};
  wave_sync();
  constexpr int RO = 64 / OC;  // rows of one step
  const int ch = lane % OC;
#pragma unroll
  for (int x = 0; x < 32; x += RO) {
    const int rr = x + lane / OC;
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(out + rr * DH * 4 + ((ch ^ (rr & 15)) * 16));
    const int64_t to = __shfl(own, rr, 64);
    if (to < 0) continue;
    if (whole)
      *reinterpret_cast<SFN_GLOBAL uint64_t*>(gp(a.out) + (to * DH + 4 * ch) * 2) =
          (uint64_t)pack_bf16(v[0], v[1]) | (uint64_t)pack_bf16(v[2], v[3]) << 32;
    else
      *reinterpret_cast<SFN_GLOBAL f32x4_t*>(gp(a.part_o) + to * DH + 4 * ch) = v;
  }
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

  const int t0 = min(max(gp(a.cu)[r], 0), a.T), t1 = min(max(gp(a.cu)[r + 1], t0), a.T);
  const int n = t1 - t0;
  if (i >= n) return;
  const int len = min(max(gp(a.kv_len)[r], 0), a.max_len), past = len - n;
  // the row tile that the row was in, and the keys that it saw
  const int g = a.g, rho0 = (i * g + head % g) / a.tile_rows * a.tile_rows;
  const int rho1 = min(rho0 + a.tile_rows, min(n, a.max_new) * g) - 1;
  const int hi = max(0, min(past + rho1 / g + 1, len));
  const int lo = a.window > 0 ? max(0, past + rho0 / g + 1 - a.window) : 0;
  const int span = hi - (lo & ~(a.tile_keys - 1));
  const int used = span > 0 ? (span + a.chunk - 1) / a.chunk : 1;  // <= S

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
// From so many rows on a wave joins one instead of a workgroup: 28.7 against 31.8 us there,
// 10.1 against 11.2 us for the 888 rows of an fp32 chunk, but 91.5 against 89.8 us for 64 rows
// of 64 splits.
constexpr int kJoinByWave = 512;
// Unsplit items, 8 waves or 4: 256 items of up to 300 keys (32 / 8 heads) 8.5 us with 8; 512
// items 15.5 with 8, 13.8 with 4 (three workgroups to a compute unit then), 4096 items 92 and 63.
constexpr int kWideMost = 256;

template <int WT, int DH>
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
        hipLaunchKernelGGL((attend_tile_kernel<DH, 1>), grid, block, 0, stream, a);
      else hipLaunchKernelGGL((attend_tile_kernel<DH, 2>), grid, dim3(512), 0, stream, a);
    }
  } else {
    // one workgroup for all of an item's keys and a compute unit for each: more waves
    const bool wide = a.S == 1 && (int64_t)a.R * a.row_tiles * a.h_kv <= kWideMost;
    const dim3 threads(wide ? 512 : 256);
    if (a.tile_rows == 16 && wide) hipLaunchKernelGGL((attend_split_kernel<WT, DH, 1, 8>), grid, threads, 0, stream, a);
    else if (a.tile_rows == 16) hipLaunchKernelGGL((attend_split_kernel<WT, DH, 1, 4>), grid, threads, 0, stream, a);
    else if (wide) hipLaunchKernelGGL((attend_split_kernel<WT, DH, 2, 8>), grid, threads, 0, stream, a);
    else hipLaunchKernelGGL((attend_split_kernel<WT, DH, 2, 4>), grid, threads, 0, stream, a);
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
