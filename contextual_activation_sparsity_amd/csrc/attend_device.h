// Attention of new tokens over pages of the key/value cache: what the kernels of a call's requests
// (kv_attend.hip) and of a call over a shared prefix (kv_attend_shared.hip) are made of.
#pragma once

#include <algorithm>
#include <type_traits>

#include "cache8.h"
#include "kernels.h"
#include "serving_common.h"
#include "sparse_ffn.h"

namespace sfn {

namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;

constexpr float kNegInf = -__builtin_huge_valf();
constexpr int kMaxSplits = 256;  // the join kernel's threads

// What the cache holds: values of the tokens' type, or e4m3 codes and a power of two to a row.
enum { CT_SAME = 0, CT_E4M3 = 1 };

// What a launch, or a workgroup's share of one, attends to: each request's keys; the prefix that
// all requests of a call share; or each request's keys behind that prefix.
enum { ATTEND_PLAIN = 0, ATTEND_PREFIX = 1, ATTEND_OWN = 2 };

// One request: its tokens are [t0, t0 + n), the first of them stands at position `past`, and its
// keys [from, len) are read. The prefix is attended to by all tokens as one request, all of which
// see every key of it (past = len); the part behind it starts there for a request whose tokens
// all come after it, and otherwise reads everything from the request's own pages.
// The prefix's part is made for min(T, R max_new) tokens, `most`. The call's tokens are
// [cu[0], cu[R]); only where some request has more than max_new can they be more than that, and
// then the first max_new of each request follow each other there.
template <int KIND>
struct Request {
  int t0, n, len, past, from;
  __device__ __forceinline__ Request(const AttendArgs& a, int r) {
    // every word is read at once: a read that waits for another is a microsecond of a short call
    const int c0 = gp(a.cu)[r], c1 = gp(a.cu)[KIND == ATTEND_PREFIX ? a.R : r + 1];
    if constexpr (KIND != ATTEND_PREFIX) len = gp(a.kv_len)[r];
    const int shared = KIND == ATTEND_PLAIN ? 0 : shared_len(a);
    t0 = min(max(c0, 0), a.T);
    n = min(max(c1, t0), a.T) - t0;
    from = 0;
    if constexpr (KIND == ATTEND_PREFIX) {
      past = len = shared;
      return;
    }
    len = min(max(len, 0), a.max_len);
    if constexpr (KIND == ATTEND_OWN) {
      len = min(len, shared + a.max_own);
      if (len - n >= shared) from = shared;
      else len = min(len, a.max_own);
    }
    past = len - n;
  }
  __device__ __forceinline__ static int shared_len(const AttendArgs& a) { return min(max(gp(a.shared)[0], 0), a.max_shared); }
  // Where token `tok` of request r has its parts, in tokens: by request, or by token where those
  // are fewer (calls over a shared prefix, which have parts of every row, split or not).
  __device__ __forceinline__ int64_t place(const AttendArgs& a, int r, int tok) const {
    if (KIND == ATTEND_OWN && a.by_token) return t0 + tok;
    return (int64_t)r * a.max_new + tok;
  }
  __device__ __forceinline__ static int start(const AttendArgs& a, int r) { return min(max(gp(a.cu)[r], 0), a.T); }
  // Token `tok` is the step's token first() + tok: for the prefix, whose `most` and whose requests'
  // bound are max_new and each_new, not the same for all where there are more.
  __device__ __forceinline__ int first(const AttendArgs& a, int tok) const {
    if (KIND != ATTEND_PREFIX || n <= a.max_new) return t0;
    int at = 0, it = -tok;  // where there is none, nothing asks for what it gets
#pragma unroll 1
    for (int r = 0; r < a.R; ++r) {  // all of them, so that the loop is the wave's and not the lane's
      const int from = start(a, r), m = min(max(start(a, r + 1) - from, 0), a.each_new);
      it = tok >= at && tok < at + m ? from - at : it;
      at += m;
    }
    return it;
  }
  // And back, for token i < max_new of request r; one that the prefix's part is not made for
  // (offsets that descend) is given another.
  __device__ __forceinline__ int in_prefix(const AttendArgs& a, int most, int r, int i) const {
    const int c0 = start(a, 0);
    int at = t0 + i - c0;
    if (most < a.T && start(a, a.R) - c0 > most) {
      at = i;
#pragma unroll 1
      for (int s = 0; s < r; ++s) at += min(max(start(a, s + 1) - start(a, s), 0), a.max_new);
    }
    return min(max(at, 0), most - 1);
  }
};

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
// An 8-bit cache has half the bytes, so that the time in which a wave turns codes into bf16 counts:
// its loads are under way meanwhile, keys and values apart. The 48 requests read 411 MB in 80 us, 5.1
// TB/s (with both loaded after the products, as above: 106 us for the call, with the keys' loads
// ahead 83), one token over 131000 keys 270 MB in 46 us, 5.9 TB/s (54.7 and 49.3 for the call). Tiles
// of 64 keys do not fit in the registers; two tiles of 32 held at once gave 84.2 for 82.9 us.
template <int WT, int CT, int DH>
struct AttnTile {
  static constexpr bool kBf = WT == WT_BF16, k8 = CT == CT_E4M3;
  static constexpr int KB = kBf ? 2 : 4;           // bytes of a value
  static constexpr int CB = k8 ? 1 : KB;           // and in the cache
  static constexpr int KT = kBf ? 32 : 16;         // keys of a tile
  static constexpr int NG = KT / 16;               // 16-key groups (each within a page)
  static constexpr int NQ = DH * KB / 64;          // 16-byte chunks a lane holds of a row (K, Q)
  static constexpr int VW = (kBf || k8) && DH == 128 ? 8 : 4;  // values a lane reads of a V row
  static constexpr int NB = DH / (16 * VW);        // times that
  static constexpr int NO = DH / 16;               // output blocks
  // Where in its row chunk s of lane quarter q starts (values). The order of the contracted
  // values is free, so a lane takes 16 codes at once and the chunks that they make follow.
  __device__ __forceinline__ static int chunk_at(int s, int q) {
    constexpr int E = 16 / KB, NC = k8 ? 16 / E : 1;
    return k8 ? 64 * (s / NC) + 16 * q + E * (s % NC) : 4 * E * s + E * q;
  }
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
    const uint32_t (&v)[AttnTile<WT, CT_SAME, DH>::NG][4][AttnTile<WT, CT_SAME, DH>::NB]
                       [AttnTile<WT, CT_SAME, DH>::VW * AttnTile<WT, CT_SAME, DH>::KB / 4],
    const f32x4_t (&p)[AttnTile<WT, CT_SAME, DH>::NG], f32x4_t (&acc)[AttnTile<WT, CT_SAME, DH>::NO], float& l) {
  using C = AttnTile<WT, CT_SAME, DH>;
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
template <int WT, int CT, int DH>
__device__ __forceinline__ void add_one_key(const SFN_GLOBAL char* vp, const f32x4_t (&p)[AttnTile<WT, CT, DH>::NG], int kk, int q,
                                            bool sees, f32x4_t (&acc)[AttnTile<WT, CT, DH>::NO]) {
  using C = AttnTile<WT, CT, DH>;
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
      uint32_t x;
      if constexpr (C::k8) x = not_a_number(vp[nb * 16 * C::VW + e]) ? (C::kBf ? 0x7fc0u : 0x7fc00000u) : 0u;
      else if constexpr (C::kBf) x = reinterpret_cast<const SFN_GLOBAL uint16_t*>(vp)[nb * 16 * C::VW + e];
      else x = reinterpret_cast<const SFN_GLOBAL uint32_t*>(vp)[nb * 16 * C::VW + e];
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
template <int WT, int CT, int DH>
struct KeyTile {
  using C = AttnTile<WT, CT, DH>;
  uint4 k[C::NG][C::NQ];
  uint32_t v[C::NG][4][C::NB][C::VW * C::KB / 4];

  // row: the cache row of each group's first key
  __device__ __forceinline__ void load_keys(const AttendArgs& a, const int64_t (&row)[C::NG], int c, int q) {
    constexpr int ROW = DH * C::KB;
#pragma unroll
    for (int u = 0; u < C::NG; ++u) {
      const SFN_GLOBAL char* kp = gp(a.k) + (row[u] + c) * ROW + 16 * q;
#pragma unroll
      for (int s = 0; s < C::NQ; ++s) k[u][s] = ldg16(kp + 64 * s);
    }
  }
  __device__ __forceinline__ void load_values(const AttendArgs& a, const int64_t (&row)[C::NG], int c, int q) {
    constexpr int ROW = DH * C::KB;
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

  // Chunk i of the key's row in group u.
  __device__ __forceinline__ uint4 key_chunk(int u, int i) const { return k[u][i]; }
  __device__ __forceinline__ void add_values(const f32x4_t (&p)[C::NG], f32x4_t (&acc)[C::NO], float& l) const {
    add_weighted<WT, DH>(v, p, acc, l);
  }

  // Zeroes the values of keys from `keys` on (keys of the tile that the sequence has) and, where
  // OWN, before `from` (places of the prefix's tokens, which may never have been written; with NaN
  // there 48 tokens after 8016 shared keys took 86 us through weigh()'s long way instead of 44);
  // returns whether some other value is not finite, and makes those 0 too.
  template <bool OWN>
  __device__ __forceinline__ bool clean(int from, int keys, int q) {
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
            x = 16 * u + j < keys - 4 * q && (!OWN || 16 * u + j >= from - 4 * q) ? x : 0u;
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

// The same of an 8-bit cache: the codes and their rows' bytes, turned into values of the tokens'
// type as they go into the products, keys and values times their row's power of two (exact in
// bf16: four bits of significand).
template <int WT, int DH>
struct KeyTile<WT, CT_E4M3, DH> {
  using C = AttnTile<WT, CT_E4M3, DH>;
  static constexpr int NR = DH / 64, NV = C::VW / 4;  // 16-byte loads of a K row, words of a V row
  uint4 k[C::NG][NR];
  uint32_t v[C::NG][4][NV];
  uint32_t kb[C::NG], vb[C::NG];  // the bytes of key c, and of keys 4q .. 4q + 3

  __device__ __forceinline__ void load_keys(const AttendArgs& a, const int64_t (&row)[C::NG], int c, int q) {
#pragma unroll
    for (int u = 0; u < C::NG; ++u) {
      // one address for the wave and an offset for the lane
      const SFN_GLOBAL char* kp = gp(a.k) + row[u] * DH;
      const uint32_t at = c * DH + 16 * q;
#pragma unroll
      for (int s = 0; s < NR; ++s) k[u][s] = ldg16(kp + (at + 64 * s));
      kb[u] = (gp(a.k_exp) + row[u])[(uint32_t)c];
    }
  }
  __device__ __forceinline__ void load_values(const AttendArgs& a, const int64_t (&row)[C::NG], int c, int q) {
#pragma unroll
    for (int u = 0; u < C::NG; ++u) {
      const SFN_GLOBAL char* vp = gp(a.v) + row[u] * DH;
      const uint32_t at = 4 * q * DH + c * C::VW;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (NV == 2) {
          const uint64_t w = __builtin_nontemporal_load(reinterpret_cast<const SFN_GLOBAL uint64_t*>(vp + (at + j * DH)));
          v[u][j][0] = (uint32_t)w;
          v[u][j][1] = (uint32_t)(w >> 32);
        } else {
          v[u][j][0] = __builtin_nontemporal_load(reinterpret_cast<const SFN_GLOBAL uint32_t*>(vp + (at + j * DH)));
        }
      }
      vb[u] = *reinterpret_cast<const SFN_GLOBAL uint32_t*>(gp(a.v_exp) + row[u] + (uint32_t)(4 * q));
    }
  }

  __device__ __forceinline__ uint4 key_chunk(int u, int i) const {
    const float scale = scale_of(kb[u]);
    if constexpr (C::kBf) {
      const uint4 w = k[u][i >> 1];
      const uint32_t a = i & 1 ? w.z : w.x, b = i & 1 ? w.w : w.y;
      return make_uint4(pair_of<false>(a, scale), pair_of<true>(a, scale), pair_of<false>(b, scale), pair_of<true>(b, scale));
    } else {
      const uint4 w = k[u][i >> 2];
      float f[4];
      values_of((i & 3) == 0 ? w.x : (i & 3) == 1 ? w.y : (i & 3) == 2 ? w.z : w.w, scale, f);
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
  }

  __device__ __forceinline__ void add_values(const f32x4_t (&p)[C::NG], f32x4_t (&acc)[C::NO], float& l) const {
    if constexpr (C::kBf) {
#pragma unroll
      for (int u = 0; u < C::NG; u += 2) {
        // rounded to bf16, and their sum, as in add_weighted
        uint4 pw = make_uint4(pack_bf16(p[u][0], p[u][1]), pack_bf16(p[u][2], p[u][3]), pack_bf16(p[u + 1][0], p[u + 1][1]),
                                    pack_bf16(p[u + 1][2], p[u + 1][3]));
        l = add_pair(pw.x, add_pair(pw.y, l)) + add_pair(pw.z, add_pair(pw.w, 0.f));
        float scale[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t b = vb[u + h];
          asm("" : "+v"(b), "+v"(pw.w));  // not before the weights are there: turned values take four times the registers
#pragma unroll
          for (int j = 0; j < 4; ++j) scale[h][j] = scale_of(b >> (8 * j) & 0xffu);
        }
#pragma unroll
        for (int e = 0; e < C::VW; e += 2) {
          uint32_t x[2][4];  // values e and e + 1 of the lane's eight keys
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              x[h][j] = e & 2 ? pair_of<true>(v[u + h][j][e >> 2], scale[h][j]) : pair_of<false>(v[u + h][j][e >> 2], scale[h][j]);
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const uint32_t sel = o ? 0x07060302u : 0x05040100u;
            const uint4 w = make_uint4(__builtin_amdgcn_perm(x[0][1], x[0][0], sel), __builtin_amdgcn_perm(x[0][3], x[0][2], sel),
                                       __builtin_amdgcn_perm(x[1][1], x[1][0], sel), __builtin_amdgcn_perm(x[1][3], x[1][2], sel));
            acc[e + o] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w), __builtin_bit_cast(bf16x8_t, pw),
                                                                 acc[e + o], 0, 0, 0);
          }
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < C::NG; ++u) {
        l += (p[u][0] + p[u][1]) + (p[u][2] + p[u][3]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < C::VW; e += 4) {
            float f[4];
            values_of(v[u][j][e >> 2], scale_of(vb[u] >> (8 * j) & 0xffu), f);
#pragma unroll
            for (int o = 0; o < 4; ++o) acc[e + o] = __builtin_amdgcn_mfma_f32_16x16x4f32(f[o], p[u][j], acc[e + o], 0, 0, 0);
          }
      }
    }
  }

  template <bool OWN>
  __device__ __forceinline__ bool clean(int from, int keys, int q) {
    uint32_t odd = 0;
#pragma unroll
    for (int u = 0; u < C::NG; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int w = 0; w < NV; ++w) {
          uint32_t& x = v[u][j][w];
          x = 16 * u + j < keys - 4 * q && (!OWN || 16 * u + j >= from - 4 * q) ? x : 0u;
          odd |= nan_codes(x);
        }
    if (!__any(odd != 0)) return false;
#pragma unroll
    for (int u = 0; u < C::NG; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int w = 0; w < NV; ++w) {
          uint32_t& x = v[u][j][w];
          asm("" : "+v"(x));  // opaque, so that nothing of the first pass is kept for this rare one
          x = without_nan(x);
        }
    return true;
  }
};

// Where the waves' sums of the rows lie in LDS: [wave][row][value], padded so that the rows of
// one write fall on different banks.
template <int DH, int TR, int NW>
struct PaddedRows {
  float (&o)[NW][TR][DH + 4];
  __device__ __forceinline__ f32x4_t* at(int wave, int row, int d) const { return reinterpret_cast<f32x4_t*>(&o[wave][row][d]); }
};
// The same in two arrays of [wave][16 rows][value], for rows 0 .. 15 and 16 .. 31, where there is no
// room for padding: the 16-byte places of a row are permuted by the row instead.
template <int DH>
struct PermutedRows {
  char *a, *b;
  __device__ __forceinline__ f32x4_t* at(int wave, int row, int d) const {
    return reinterpret_cast<f32x4_t*>((row < 16 ? a : b) + (wave * 16 + (row & 15)) * DH * 4 + ((d >> 2) ^ (row & 15)) * 16);
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

template <int WT, int CT, int DH, int RT, int NW, int KIND, class Lds>
__device__ __forceinline__ void split_attention(const AttendArgs& a, uint32_t bx, int split, int r, float (&s_m)[NW][16 * RT],
                                                float (&s_l)[NW][16 * RT], Lds s_o) {
  using C = AttnTile<WT, CT, DH>;
  constexpr int KT = C::KT, NG = C::NG, NQ = C::NQ, VW = C::VW, NB = C::NB, NO = C::NO, KB = C::KB;
  constexpr int TR = 16 * RT, ROW = DH * KB;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int rtile = a.row_tiles == 1 ? 0 : bx / a.h_kv, hk = bx - rtile * a.h_kv;

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

  const Request<KIND> req(a, r);
  const int t0 = req.t0, len = req.len, past = req.past;
  const int g = a.g, rows = min(req.n, a.max_new) * g;
  const int rho0 = rtile * TR;
  if (rho0 >= rows) return;
  const RowMap map(a, rho0);
  const int last = min(TR, rows - rho0) - 1, tok1 = map.token(last);
  // keys that some row of the tile sees, and that every row sees
  const int hi = max(0, min(past + tok1 + 1, len));
  const int lo = a.window > 0 ? max(0, past + map.tok0 + 1 - a.window) : req.from;
  const int hi_all = min(past + map.tok0 + 1, len);
  const int lo_all = a.window > 0 ? max(0, past + tok1 + 1 - a.window) : req.from;
  const int k0 = (lo & ~(KT - 1)) + split * a.chunk, k1 = min(k0 + a.chunk, hi);
  if (split > 0 && k0 >= hi) return;

  const int kw = k0 + wave * KT;
  KeyTile<WT, CT, DH> tile;
  auto find = [&](int kt) {
#pragma unroll
    for (int u = 0; u < NG; ++u) page[u] = page_of(kt + 16 * u);
  };
  // the tile at kt, from the pages found for it, and then the pages of the one after it
  int64_t row[NG];
  auto place = [&](int kt) {
#pragma unroll
    for (int u = 0; u < NG; ++u) row[u] = row_in(page[u], kt + 16 * u);
  };
  auto fetch = [&](int kt) {
    place(kt);
    tile.load_keys(a, row, c, q);
    tile.load_values(a, row, c, q);
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
    const SFN_GLOBAL char* src = gp(a.q) + (int64_t)(req.first(a, tok) + tok) * a.q_stride + head * ROW;
#pragma unroll
    for (int s = 0; s < NQ; ++s) qf[x][s] = ld16(src + C::chunk_at(s, q) * KB);
    row_hi[x] = ok ? min(past + tok + 1, len) : 0;
    row_lo[x] = a.window > 0 ? past + tok + 1 - a.window : req.from;
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

  auto scores = [&](int x, f32x4_t (&s)[NG]) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      const f32x4_t zero = {0.f, 0.f, 0.f, 0.f};
      if constexpr (C::kBf) {
        s[u] = zero;
#pragma unroll
        for (int i = 0; i < NQ; ++i)
          s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, tile.key_chunk(u, i)),
                                                         __builtin_bit_cast(bf16x8_t, qf[x][i]), s[u], 0, 0, 0);
      } else {
        // four sums side by side: half the rounding error of one chain of dh additions (sharp
        // scores, 600 keys: 4.4e-7 of the result against 1.1e-6), for 10.0 instead of 9.8 us
        // of the windowed fp32 chunk
        f32x4_t part[4] = {zero, zero, zero, zero};
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          const f32x4_t kk = __builtin_bit_cast(f32x4_t, tile.key_chunk(u, i)), qq = __builtin_bit_cast(f32x4_t, qf[x][i]);
#pragma unroll
          for (int e = 0; e < 4; ++e) part[e] = __builtin_amdgcn_mfma_f32_16x16x4f32(kk[e], qq[e], part[e], 0, 0, 0);
        }
        s[u] = (part[0] + part[1]) + (part[2] + part[3]);
      }
    }
  };
  auto weigh = [&](int x, f32x4_t (&s)[NG], int kt, bool full, bool odd) __attribute__((always_inline)) {
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
    tile.add_values(s, acc[x], l[x]);
    if (odd) {
      // the values that are not finite: key by key, read again, into the rows that see them
#pragma unroll 1
      for (int kk = 0; kk < KT && kt + kk < len; ++kk)
        add_one_key<WT, CT, DH>(gp(a.v) + ((row_in(page_of(kt + kk), kt + kk) + (kk & 15)) * DH + c * VW) * C::CB, s, kk, q,
                                kt + kk < row_hi[x] && kt + kk >= row_lo[x], acc[x]);
    }
  };
  for (int kt = kw; kt < k1;) {
    const bool full = kt >= lo_all && kt + KT <= hi_all;  // every row sees every key of the tile
    const int next = kt + NW * KT;
    // A masked key has weight 0, but 0 times a value that is not finite is NaN: a tile with a
    // masked key and such a value takes the long way in weigh(), so that no token's result
    // depends on tokens it does not see.
    if constexpr (C::k8) {
      // turning codes into values takes more time than the products, so the loads are under way
      // meanwhile: the next tile's keys from here on, its values after this one's
      f32x4_t s[RT][NG];
#pragma unroll
      for (int x = 0; x < RT; ++x) scores(x, s[x]);
      if (next < k1) {
        place(next);
        tile.load_keys(a, row, c, q);
      }
      const bool odd = full ? false : tile.template clean<KIND == ATTEND_OWN>(req.from - kt, len - kt, q);
#pragma unroll
      for (int x = 0; x < RT; ++x) weigh(x, s[x], kt, full, odd);
      if (next < k1) {
        tile.load_values(a, row, c, q);
        if (next + NW * KT < k1) find(next + NW * KT);
      }
    } else {
      const bool odd = full ? false : tile.template clean<KIND == ATTEND_OWN>(req.from - kt, len - kt, q);
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        f32x4_t s[NG];
        scores(x, s);
        weigh(x, s, kt, full, odd);
      }
      if (next < k1) fetch(next);
    }
    kt = next;
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
          *s_o.at(wave, 16 * x + c, 16 * VW * nb + VW * (4 * q + i) + e) =
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
      o += *s_o.at(w, x, d4);
    }
    if (KIND == ATTEND_PLAIN && a.S == 1) {
      store_row<WT, DH>(a, t0 + tok, head, d4, o, L);
    } else {
      const int64_t at = (req.place(a, r, tok) * a.h_q + head) * a.S + split;
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
// us by the machine, 990 to 1065 TFLOP/s, where a sustained bf16 product of 8192 x 8192 reaches
// 1385. What bounds it is power, and how full the matrix cores are: they are busy half of the
// clocks (the library's product keeps them busy 69%), with no bank conflict in LDS, and the
// clock falls to 1.6 to 1.9 GHz, as it does for that product, where a kernel bound by memory runs
// at 2.5. Fewer clocks a key have brought lower clocks: leaving out the whole softmax saves 3%.
// An 8-bit cache costs the conversion of each stage, once for 128 rows, and its writes to LDS: 655 to
// 690 us by the machine, 900 to 945 TFLOP/s (up to 730 us where each launch is timed alone), the matrix
// cores busy 40% of clocks of 1.9 to 2.0 GHz. One in six of
// LDS's busy clocks is a conflict of those writes; a layout without any gave 0.5%. The 8-bit matrix
// product with Q in two e4m3 parts would need no conversion, but its sums are off by up to 2.8e-4 of
// the products' norm, which is not 32 bits.
// Heads of 64 have as much softmax for half the products: 370 us, 837 TFLOP/s (8 bits: 410). The four requests'
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
template <int CT, int DH>
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
          uint64_t x4;  // of acc[d][i .. i + 3]
          if constexpr (CT == CT_E4M3) x4 = *reinterpret_cast<const SFN_GLOBAL uint32_t*>(v + (64 * d + 4 * i + first) / 2);
          else x4 = *reinterpret_cast<const SFN_GLOBAL uint64_t*>(v + 64 * d + 4 * i + first);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t x;
            if constexpr (CT == CT_E4M3) x = not_a_number((uint32_t)(x4 >> (8 * e))) ? 0x7fc00000u : 0u;
            else x = (uint32_t)(x4 >> (16 * e)) << 16;
            acc[d][i + e] = sees && not_finite<WT_F32>(x) ? fmaf(p, __uint_as_float(x), acc[d][i + e]) : acc[d][i + e];
          }
        }
    }
  }

  // The stage's 64 keys from kt on. full: every row sees every key. odd: values that are not
  // finite were taken out of the stage (see add_not_finite).
  template <class Row>
  __device__ __forceinline__ void step(const SFN_LDS char* stage, int koff, int voff, int kt, bool full, bool odd, float scale_log2,
                                       Row row, int keys, float slack) {
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
    if (__any(top > m + slack)) {
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
    // The products' code begins at 32 bytes: what other code a launch holds moves it otherwise, and
    // the 2048-token prompts with it (on one machine 622 or 632 us by its place, 615 here; 16-token chunks
    // the same). Heads of 64 gain nothing.
    if constexpr (DH == 128) asm volatile(".p2align 5");
    add_values(stage, voff, pw);
    __builtin_amdgcn_s_setprio(0);
    if (__builtin_expect(odd, 0)) add_not_finite(row, pw, kt, keys);
  }
};

// Of an 8-bit cache: a wave's 16 rows of a stage of K or of V on their way through registers. They
// are read while the products of the stage before are under way, turned into bf16 and written to
// LDS after them, so that the products read the same stages as above.
template <int DH>
struct CodeRows {
  static constexpr int LR = DH / 16, RI = 64 / LR, N = 16 / RI;  // lanes of a row, rows of one load, loads
  uint4 w[N];
  uint32_t b[N];
  __device__ __forceinline__ void load(const SFN_GLOBAL char* rows, const SFN_GLOBAL uint8_t* exps, int lane) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t row = i * RI + lane / LR;  // one address for the wave and an offset for the lane
      w[i] = ld16(rows + (row * DH + (lane % LR) * 16));
      b[i] = exps[row];
    }
  }
  // place(row, ch): where chunk ch (8 values) of a row lies; to: the wave's part of the stage
  template <class Place>
  __device__ __forceinline__ void put(SFN_LDS char* to, int lane, Place place) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int row = i * RI + lane / LR, ch = (lane % LR) * 2;
      const float s = scale_of(b[i]);
      const uint4 x = w[i];
      *reinterpret_cast<SFN_LDS u32x4_t*>(to + row * DH * 2 + place(row, ch) * 16) =
          u32x4_t{pair_of<false>(x.x, s), pair_of<true>(x.x, s), pair_of<false>(x.y, s), pair_of<true>(x.y, s)};
      *reinterpret_cast<SFN_LDS u32x4_t*>(to + row * DH * 2 + place(row, ch + 1) * 16) =
          u32x4_t{pair_of<false>(x.z, s), pair_of<true>(x.z, s), pair_of<false>(x.w, s), pair_of<true>(x.w, s)};
    }
  }
};

// KG groups of four waves: with two of them (a split of the keys for few row tiles) each takes
// every second stage, with buffers of its own, and the groups join in LDS at the end, so that
// there are half as many parts to write and join as with two workgroups.
// s_a and s_b are two arrays, so that the compiler knows that the reads of one need not wait for
// the loads into the other; of each, a group's K stage and its V stage.
// EXACT: the maximum does not lag (kSlack 0).
template <int CT, int DH, int KG, int KIND, bool EXACT>
__device__ __forceinline__ void tile_attention(const AttendArgs& a, uint32_t bx, int split, int r, char (&s_a)[KG * 2 * kTileKeys * DH * 2],
                                               char (&s_b)[KG * 2 * kTileKeys * DH * 2], uint32_t (&s_odd)[4 * KG]) {
  using W = TileWave<CT, DH>;
  constexpr bool k8 = CT == CT_E4M3;
  constexpr int CROW = k8 ? DH : DH * 2;  // bytes of a row in the cache
  constexpr int ND = W::ND, NC = W::NC, ROW = W::ROW, KT = kTileKeys;
  constexpr int STAGE = KT * ROW;  // bytes of a stage of K, and of V
  const int tid = threadIdx.x & 255, lane = threadIdx.x & 63;
  const int kg = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 8);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);  // in its group
  W w;
  const int c = w.c = lane & 31, h = w.h = lane >> 5;
  const int hk = a.row_tiles == 1 ? bx : bx % a.h_kv;
  const int rtile = a.row_tiles == 1 ? 0 : a.row_tiles - 1 - bx / a.h_kv;  // the longest first

  // the first in the cache of this wave's 16 rows of the stage at kt (one group of keys, in
  // one page; past the sequence any page of the cache)
  const int lg = a.page_shift, pm = (1 << lg) - 1;
  const SFN_GLOBAL int32_t* table = gp(a.table) + (int64_t)r * a.max_pages;
  auto page_of = [&](int kt) { return __builtin_amdgcn_readfirstlane(table[min((kt + 16 * wave) >> lg, a.max_pages - 1)]); };
  auto rows_in = [&](int page, int kt) -> int64_t {
    return (((int64_t)min(max(page, 0), a.n_pages - 1) * a.h_kv + hk) << lg) + ((kt + 16 * wave) & pm);
  };
  // without a window the first stage does not depend on the lengths: its page is read with them
  int page = page_of(split * a.chunk + kg * KT);

  const Request<KIND> req(a, r);
  const int t0 = req.t0, len = req.len, past = req.past;
  const int g = a.g, rows = min(req.n, a.max_new) * g;
  const int rho0 = rtile * kTileRows;
  if (rho0 >= rows) return;
  const RowMap map(a, rho0);
  const int last = min(kTileRows, rows - rho0) - 1;  // the tile's last row
  // keys that some row of the tile sees, and that every row sees
  const int tok1 = map.token(last);
  const int hi = max(0, min(past + tok1 + 1, len));
  const int lo = a.window > 0 ? max(0, past + map.tok0 + 1 - a.window) : req.from;
  const int tile_hi = min(past + map.tok0 + 1, len);
  const int tile_lo = a.window > 0 ? past + tok1 + 1 - a.window : req.from;
  const int k0 = (lo & ~(KT - 1)) + split * a.chunk, k1 = min(k0 + a.chunk, hi);
  if (split > 0 && k0 >= hi) return;

  const int group = kg * 2 * STAGE, mine = group + 16 * wave * ROW;
  const int kg0 = k0 + kg * KT;
  CodeRows<DH> kc{}, vc{};
  auto load = [&](char* stage, int64_t row) __attribute__((always_inline)) {
    if constexpr (k8) {
      kc.load(gp(a.k) + row * CROW, gp(a.k_exp) + row, lane);
      vc.load(gp(a.v) + row * CROW, gp(a.v_exp) + row, lane);
    } else {
      W::load(gp(a.k) + row * ROW, gp(a.v) + row * ROW, (SFN_LDS char*)stage + mine, (SFN_LDS char*)stage + STAGE + mine, lane);
    }
  };
  auto put = [&](char* stage) __attribute__((always_inline)) {
    if constexpr (k8) {
      kc.put((SFN_LDS char*)stage + mine, lane, W::k_place);
      vc.put((SFN_LDS char*)stage + STAGE + mine, lane, W::v_place);
    }
  };
  if (kg0 < k1) {
    if (lo > 0) page = page_of(kg0);
    load(s_a, rows_in(page, kg0));
  }

  // this wave's rows
  const int i0 = 32 * wave, i1 = min(i0 + 31, last);  // none if i0 > last
  const int wt0 = map.token(i0), wt1 = map.token(max(i1, 0));
  const int some_hi = i0 <= last ? min(past + wt1 + 1, len) : 0;  // keys that some row of it sees
  const int some_lo = a.window > 0 ? past + wt0 + 1 - a.window : req.from;
  const int all_hi = min(past + wt0 + 1, len);  // and that every row sees
  const int all_lo = a.window > 0 ? past + wt1 + 1 - a.window : req.from;
  const bool ok = i0 + c <= last;
  const int i = ok ? i0 + c : 0, tok = map.token(i), head = hk * g + map.head(i, tok);
  w.row_hi = ok ? min(past + tok + 1, len) : 0;
  w.row_lo = a.window > 0 ? past + tok + 1 - a.window : req.from;
  w.m = kNegInf;
  w.l = 0.f;
  {
    const SFN_GLOBAL char* src = gp(a.q) + (int64_t)(req.first(a, tok) + tok) * a.q_stride + head * ROW + 16 * h;
#pragma unroll
    for (int s = 0; s < W::NS; ++s) w.q[s] = __builtin_bit_cast(bf16x8_t, ld16(src + 32 * s));
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int e = 0; e < 16; ++e) w.acc[d][e] = 0.f;
  }
  auto v_row = [&](int key) {
    const int p = min(max(table[key >> lg], 0), a.n_pages - 1);
    return gp(a.v) + ((((int64_t)p * a.h_kv + hk) << lg) + (key & pm)) * CROW;
  };
  if (kg0 < k1) put(s_a);

  // a round, a stage for each group: the keys from kr on, in cur; the next ones go into nxt
  auto round = [&](char* cur, char* nxt, int kr) __attribute__((always_inline)) {
    const int kt = kr + kg * KT, kn = kt + KG * KT;
    if (kn < k1) page = page_of(kn);
    // this wave's part of the stage has arrived; after the barrier everyone's has, and the
    // other array is free
    if constexpr (!k8) __builtin_amdgcn_s_waitcnt(kWaitLoads);
    __syncthreads();
    // A stage with masked keys: what the page holds past the sequence, or in places of the
    // prefix's, becomes 0, and so do values that are not finite (0 times one of them is NaN);
    // those count in a way of their own
    bool odd = false;
    if (kr + KG * KT > tile_hi || kr < tile_lo) {
      for (int e = kt < k1 ? tid : KT * NC; e < KT * NC; e += 256) {
        uint4* const at = reinterpret_cast<uint4*>(cur + group + STAGE + e * 16);
        const uint4 x = *at;
        if (kt + e / NC >= len || (KIND == ATTEND_OWN && kt + e / NC < req.from)) {
          *at = make_uint4(0, 0, 0, 0);
        } else if (not_finite<WT_BF16>(x.x) | not_finite<WT_BF16>(x.y) | not_finite<WT_BF16>(x.z) | not_finite<WT_BF16>(x.w)) {
          *at = make_uint4(finite_part<WT_BF16>(x.x), finite_part<WT_BF16>(x.y), finite_part<WT_BF16>(x.z), finite_part<WT_BF16>(x.w));
          odd = true;
        }
      }
      // whether any wave's part of it had one
      const bool any = __any(odd);
      if (lane == 0) s_odd[KG == 1 ? wave : kg * 4 + wave] = any;
      __syncthreads();
      uint32_t all = 0;
#pragma unroll
      for (int w = 0; w < 4 * KG; ++w) all |= s_odd[w];
      odd = __builtin_amdgcn_readfirstlane(all) != 0;
    }
    if (kn < k1) load(nxt, rows_in(page, kn));
    if (kt < min(some_hi, k1) && kt + KT > some_lo)
      w.step((SFN_LDS char*)cur, group, group + STAGE, kt, kt >= all_lo && kt + KT <= all_hi, odd, a.scale_log2, v_row,
             min(KT, len - kt), EXACT ? 0.f : kSlack);
    if (k8 && kn < k1) put(nxt);
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
  const bool whole = KIND == ATTEND_PLAIN && a.S == 1;
  const float inv = whole ? (l == 0.f ? 0.f : 1.0f / l) : 1.f;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<f32x4_t*>(out + c * DH * 4 + (((8 * d + 2 * e + h) ^ (c & 15)) * 16)) =
          f32x4_t{w.acc[d][4 * e], w.acc[d][4 * e + 1], w.acc[d][4 * e + 2], w.acc[d][4 * e + 3]} * inv;
  // the lane's row in the output or in the parts, -1 if it has none
  const int64_t orow = whole ? (int64_t)(t0 + tok) * a.h_q + head : (req.place(a, r, tok) * a.h_q + head) * a.S + split;
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

// The splits that wrote parts of the row of token i and head `head` of a request: those of the
// keys that some row of its row tile saw. At most S.
template <int KIND>
__device__ __forceinline__ int splits_used(const AttendArgs& a, const Request<KIND>& req, int i, int head) {
  const int g = a.g, rho0 = (i * g + head % g) / a.tile_rows * a.tile_rows;
  const int rho1 = min(rho0 + a.tile_rows, min(req.n, a.max_new) * g) - 1;
  const int hi = max(0, min(req.past + rho1 / g + 1, req.len));
  const int lo = a.window > 0 ? max(0, req.past + rho0 / g + 1 - a.window) : req.from;
  const int span = hi - (lo & ~(a.tile_keys - 1));
  return span > 0 ? (span + a.chunk - 1) / a.chunk : 1;
}

// From so many rows on a wave joins one instead of a workgroup: 28.7 against 31.8 us there,
// 10.1 against 11.2 us for the 888 rows of an fp32 chunk, but 91.5 against 89.8 us for 64 rows
// of 64 splits.
constexpr int kJoinByWave = 512;

// Calls f<WT, CT, DH>() for a cache's types and head size.
template <class F>
void by_type(int dh, int dtype, bool e4m3, F f) {
  auto sized = [&](auto wt, auto ct) {
    if (dh == 64) f(wt, ct, std::integral_constant<int, 64>());
    else f(wt, ct, std::integral_constant<int, 128>());
  };
  auto typed = [&](auto wt) {
    if (e4m3) sized(wt, std::integral_constant<int, CT_E4M3>());
    else sized(wt, std::integral_constant<int, CT_SAME>());
  };
  if (dtype == SFN_BF16) typed(std::integral_constant<int, WT_BF16>());
  else typed(std::integral_constant<int, WT_F32>());
}

}  // namespace
}  // namespace sfn
