// C ABI of the sparse gated-FFN library: argument validation, workspace sizing and
// dispatch to the HIP kernels. Every argument is checked before any HIP call, so the
// error paths run (and are tested) on machines without a GPU.

#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <exception>

#include "kernels.h"
#include "sparse_ffn.h"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
// 4-byte alignment of an optional int32 or fp32 pointer (NULL passes)
bool aligned4_or_null(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

int wbytes(int wdtype) { return wdtype == SFN_BF16 ? 2 : 4; }

// Shape, enum and alignment checks shared by every call on an FFN layer.
int check_ffn(const sfn_ffn* ffn, bool need_up_down) {
  if (!ffn) return SFN_EINVAL;
  if (ffn->wdtype != SFN_F32 && ffn->wdtype != SFN_BF16) return SFN_EDTYPE;
  if (ffn->act != SFN_ACT_SILU && ffn->act != SFN_ACT_RELU) return SFN_EINVAL;
  if (ffn->d < 1 || ffn->d > SFN_MAX_D || ffn->f < 1 || ffn->f > SFN_MAX_F) return SFN_ESHAPE;
  if ((ffn->d * wbytes(ffn->wdtype)) % 16 != 0) return SFN_EALIGN;
  if (!ffn->w_gate) return SFN_EINVAL;
  if (need_up_down && (!ffn->w_up || !ffn->w_down_t)) return SFN_EINVAL;
  if (!aligned16(ffn->w_gate)) return SFN_EALIGN;
  if (ffn->w_up && !aligned16(ffn->w_up)) return SFN_EALIGN;
  if (ffn->w_down_t && !aligned16(ffn->w_down_t)) return SFN_EALIGN;
  if (ffn->b_gate && (reinterpret_cast<uintptr_t>(ffn->b_gate) & 3u)) return SFN_EALIGN;
  return SFN_OK;
}

int check_svd(const sfn_svd* s) {
  if (!s) return SFN_EINVAL;
  if (s->reserved != 0) return SFN_EINVAL;
  if (s->d < 1 || s->d > SFN_MAX_D || s->f < 1 || s->f > SFN_MAX_F) return SFN_ESHAPE;
  if (s->r < 1 || s->r > SFN_MAX_RANK || s->r > s->d) return SFN_ESHAPE;
  if (s->d % 8 != 0 || s->r % 8 != 0) return SFN_EALIGN;
  if (!s->q || !s->l || !s->tau) return SFN_EINVAL;
  if (!aligned16(s->q) || !aligned16(s->l)) return SFN_EALIGN;
  if ((reinterpret_cast<uintptr_t>(s->tau) & 3u) || (s->b && (reinterpret_cast<uintptr_t>(s->b) & 3u)))
    return SFN_EALIGN;
  return SFN_OK;
}

int check_ws(void* ws, size_t ws_bytes, size_t need) {
  if (!ws || ws_bytes < need) return SFN_EWORKSPACE;
  if (!aligned256(ws)) return SFN_EALIGN;
  return SFN_OK;
}

int hip_status(hipError_t e) { return e == hipSuccess ? SFN_OK : SFN_EHIP; }

// Validation and launch of one decode step on a workspace (sparse_ffn_decode and its
// allocation-free variant).
int decode_validate(const sfn_ffn* ffn, const void* x, int32_t B, const float* t, const int32_t* cand,
                    const int32_t* n_cand, const uint8_t* mask_in, float* y, const int32_t* active_idx,
                    const int32_t* n_active) {
  const int st = check_ffn(ffn, y != nullptr);
  if (st != SFN_OK) return st;
  if (!x) return SFN_EINVAL;
  if (!aligned16(x)) return SFN_EALIGN;
  if (B < 1 || B > SFN_MAX_BATCH) return SFN_ESHAPE;
  if ((cand == nullptr) != (n_cand == nullptr)) return SFN_EINVAL;
  if (cand && (B != 1 || mask_in)) return SFN_EINVAL;
  if (y && !aligned16(y)) return SFN_EALIGN;
  if (!aligned4_or_null(t) || !aligned4_or_null(cand) || !aligned4_or_null(n_cand) ||
      !aligned4_or_null(active_idx) || !aligned4_or_null(n_active))
    return SFN_EALIGN;
  return SFN_OK;
}

size_t decode_need(const sfn_ffn* ffn, int32_t B) {
  return sfn::decode_workspace_bytes(ffn->d, ffn->f, wbytes(ffn->wdtype), B > 1 ? SFN_MAX_BATCH : 1);
}

int decode_launch(const sfn_ffn* ffn, const void* x, int32_t B, const float* t, const int32_t* cand,
                  const int32_t* n_cand, const uint8_t* mask_in, float* y, int32_t* active_idx, int32_t* n_active,
                  void* ws, void* stream) {
  const int wb = wbytes(ffn->wdtype);
  sfn::DecodeArgs a{};
  a.wg = static_cast<const char*>(ffn->w_gate);
  a.wu = static_cast<const char*>(ffn->w_up);
  a.wd = static_cast<const char*>(ffn->w_down_t);
  a.bias = ffn->b_gate;
  a.x = static_cast<const char*>(x);
  a.t = t;
  a.cand = cand;
  a.n_cand = n_cand;
  a.mask_in = mask_in;
  a.y = y;
  a.active_idx = active_idx;
  a.n_active = n_active;
  a.d = ffn->d;
  a.f = ffn->f;
  a.nch = ffn->d * wb / 16;
  a.row_bytes = ffn->d * wb;
  a.nb = B;
  a.act = ffn->act;
  a.G = sfn::decode_grid(ffn->f);
  a.n_red = sfn::decode_reducers(a.G, B, ffn->d);
  sfn::decode_carve(a, ws, wb);
  return hip_status(sfn::launch_decode(a, ffn->wdtype, static_cast<hipStream_t>(stream)));
}

// Scratch of sparse_ffn_decode_noalloc: a file-scope device array, one copy on each GPU
// the library runs on, zero when the code object is loaded. Kernels never see its name:
// host code takes its device address from hipGetSymbolAddress, once per device with that
// device current, and passes that address like a workspace.
constexpr size_t kNoAllocScratchBytes = SFN_NOALLOC_SCRATCH_BYTES;
__device__ __attribute__((aligned(256))) unsigned char scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 64;
std::atomic<void*> g_scratch_ptr[kMaxDevices];

// The current device's address of `scratch` (resolved on the first call on each device;
// host threads that race store the same value).
int scratch_ptr(void** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return SFN_EHIP;
  void* p = g_scratch_ptr[dev].load(std::memory_order_acquire);
  if (!p) {
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || !p) return SFN_EHIP;
    g_scratch_ptr[dev].store(p, std::memory_order_release);
  }
  *out = p;
  return SFN_OK;
}

}  // namespace

extern "C" {

size_t sparse_ffn_workspace_size(const sfn_ffn* ffn, int32_t max_tokens) {
  try {
    if (check_ffn(ffn, false) != SFN_OK || max_tokens < 1 || max_tokens > 65536) return 0;
    const int wb = wbytes(ffn->wdtype);
    const int nb = max_tokens > 1 ? SFN_MAX_BATCH : 1;
    size_t need = sfn::decode_workspace_bytes(ffn->d, ffn->f, wb, nb);
    const size_t chunk = sfn::chunk_workspace_bytes(ffn->d, ffn->f, ffn->wdtype, max_tokens < SFN_MAX_CHUNK ? max_tokens : SFN_MAX_CHUNK);
    if (chunk > need) need = chunk;
    const size_t cal = sfn::calibrate_workspace_bytes(ffn->d, ffn->f, ffn->wdtype, max_tokens);
    if (cal > need) need = cal;
    return need;
  } catch (...) {
    return 0;
  }
}

size_t svd_predict_workspace_size(const sfn_svd* svd) {
  try {
    if (check_svd(svd) != SFN_OK) return 0;
    return sfn::svd_workspace_bytes(svd->d, svd->f, svd->r);
  } catch (...) {
    return 0;
  }
}

const char* sparse_ffn_strerror(int status) {
  switch (status) {
    case SFN_OK: return "success";
    case SFN_EINVAL: return "invalid argument (null pointer, bad enum or out-of-range scalar)";
    case SFN_ESHAPE: return "unsupported shape (d, f, r, batch or chunk size out of range)";
    case SFN_EDTYPE: return "unsupported dtype";
    case SFN_EWORKSPACE: return "workspace missing or smaller than the size query returns";
    case SFN_EALIGN: return "pointer or row not 16-byte aligned (workspace: 256-byte)";
    case SFN_EUNSUPPORTED: return "request not implemented by this library";
    case SFN_EHIP: return "HIP runtime error on launch";
    case SFN_ETOOLARGE:
      return "request needs more scratch than sparse_ffn_decode_noalloc's fixed array (SFN_NOALLOC_SCRATCH_BYTES)";
    default: return "unknown status";
  }
}

int sparse_ffn_decode(const sfn_ffn* ffn, const void* x, int32_t B, const float* t, const int32_t* cand,
                      const int32_t* n_cand, const uint8_t* mask_in, float* y, int32_t* active_idx,
                      int32_t* n_active, void* ws, size_t ws_bytes, void* stream) {
  try {
    int st = decode_validate(ffn, x, B, t, cand, n_cand, mask_in, y, active_idx, n_active);
    if (st != SFN_OK) return st;
    st = check_ws(ws, ws_bytes, decode_need(ffn, B));
    if (st != SFN_OK) return st;
    return decode_launch(ffn, x, B, t, cand, n_cand, mask_in, y, active_idx, n_active, ws, stream);
  } catch (...) {
    return SFN_EHIP;
  }
}

int sparse_ffn_decode_noalloc(const sfn_ffn* ffn, const void* x, int32_t B, const float* t, const int32_t* cand,
                              const int32_t* n_cand, const uint8_t* mask_in, float* y, int32_t* active_idx,
                              int32_t* n_active, void* stream) {
  try {
    int st = decode_validate(ffn, x, B, t, cand, n_cand, mask_in, y, active_idx, n_active);
    if (st != SFN_OK) return st;
    if (decode_need(ffn, B) > kNoAllocScratchBytes) return SFN_ETOOLARGE;
    void* ws = nullptr;
    st = scratch_ptr(&ws);
    if (st != SFN_OK) return st;
    return decode_launch(ffn, x, B, t, cand, n_cand, mask_in, y, active_idx, n_active, ws, stream);
  } catch (...) {
    return SFN_EHIP;
  }
}

int sparse_ffn_decode_parallel(const sfn_ffn* ffn, const void* x, const int32_t* cand, const int32_t* n_cand,
                               float* y, void* ws, size_t ws_bytes, void* stream) {
  try {
    int st = check_ffn(ffn, true);
    if (st != SFN_OK) return st;
    if (!x || !cand || !n_cand || !y) return SFN_EINVAL;
    if (!aligned16(x) || !aligned16(y)) return SFN_EALIGN;
    if (!aligned4_or_null(cand) || !aligned4_or_null(n_cand)) return SFN_EALIGN;
    const int wb = wbytes(ffn->wdtype);
    st = check_ws(ws, ws_bytes, sfn::decode_workspace_bytes(ffn->d, ffn->f, wb, 1));
    if (st != SFN_OK) return st;

    sfn::DecodeArgs a{};
    a.wg = static_cast<const char*>(ffn->w_gate);
    a.wu = static_cast<const char*>(ffn->w_up);
    a.wd = static_cast<const char*>(ffn->w_down_t);
    a.bias = ffn->b_gate;
    a.x = static_cast<const char*>(x);
    a.cand = cand;
    a.n_cand = n_cand;
    a.y = y;
    a.d = ffn->d;
    a.f = ffn->f;
    a.nch = ffn->d * wb / 16;
    a.row_bytes = ffn->d * wb;
    a.nb = 1;
    a.act = ffn->act;
    a.G = sfn::decode_grid(ffn->f);
    a.n_red = sfn::decode_reducers(a.G, 1, ffn->d);
    sfn::decode_carve(a, ws, wb);
    return hip_status(sfn::launch_decode_parallel(a, ffn->wdtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

int sparse_ffn_calibrate(const sfn_ffn* ffn, const void* x_cal, int32_t n, float k, float* t_out,
                         float* scores_out, void* ws, size_t ws_bytes, void* stream) {
  try {
    int st = check_ffn(ffn, false);
    if (st != SFN_OK) return st;
    if (!x_cal || !t_out) return SFN_EINVAL;
    if (!aligned16(x_cal)) return SFN_EALIGN;
    if (n < 1 || n > 65536) return SFN_ESHAPE;
    if (!(k >= 0.0f && k <= 1.0f)) return SFN_EINVAL;
    if ((int64_t)n * ffn->f > (int64_t)1 << 31) return SFN_ESHAPE;
    if (scores_out && (reinterpret_cast<uintptr_t>(scores_out) & 15u)) return SFN_EALIGN;
    st = check_ws(ws, ws_bytes, sfn::calibrate_workspace_bytes(ffn->d, ffn->f, ffn->wdtype, n));
    if (st != SFN_OK) return st;
    return hip_status(sfn::launch_calibrate(*ffn, x_cal, n, k, t_out, scores_out, ws, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

int svd_predict(const sfn_svd* svd, const void* x, int32_t* cand_idx, int32_t* n_cand, float* p_out, void* ws,
                size_t ws_bytes, void* stream) {
  try {
    int st = check_svd(svd);
    if (st != SFN_OK) return st;
    if (!x || !cand_idx || !n_cand) return SFN_EINVAL;
    if (!aligned16(x)) return SFN_EALIGN;
    if (p_out && (reinterpret_cast<uintptr_t>(p_out) & 3u)) return SFN_EALIGN;
    st = check_ws(ws, ws_bytes, sfn::svd_workspace_bytes(svd->d, svd->f, svd->r));
    if (st != SFN_OK) return st;
    return hip_status(sfn::launch_svd_predict(*svd, x, cand_idx, n_cand, p_out, ws, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

namespace {

size_t round256(size_t b) { return (b + 255) & ~(size_t)255; }

// Fused SVD pipeline workspace: the decode scratch for one token, then z [r] fp32.
size_t svd_pipeline_z_offset(const sfn_ffn* ffn) { return round256(sfn::decode_workspace_bytes(ffn->d, ffn->f, 2, 1)); }
size_t svd_pipeline_bytes(const sfn_ffn* ffn, const sfn_svd* svd) {
  return svd_pipeline_z_offset(ffn) + round256((size_t)svd->r * sizeof(float));
}

int check_svd_pipeline(const sfn_ffn* ffn, const sfn_svd* svd) {
  int st = check_ffn(ffn, true);
  if (st != SFN_OK) return st;
  st = check_svd(svd);
  if (st != SFN_OK) return st;
  if (ffn->wdtype != SFN_BF16) return SFN_EDTYPE;  // the predictor takes the bf16 token
  if (svd->d != ffn->d || svd->f != ffn->f) return SFN_ESHAPE;
  return SFN_OK;
}

}  // namespace

size_t sparse_ffn_svd_workspace_size(const sfn_ffn* ffn, const sfn_svd* svd) {
  try {
    if (check_svd_pipeline(ffn, svd) != SFN_OK) return 0;
    return svd_pipeline_bytes(ffn, svd);
  } catch (...) {
    return 0;
  }
}

int sparse_ffn_decode_svd(const sfn_ffn* ffn, const sfn_svd* svd, const void* x, int32_t pipeline, float* y,
                          int32_t* idx, int32_t* n_idx, void* ws, size_t ws_bytes, void* stream) {
  try {
    int st = check_svd_pipeline(ffn, svd);
    if (st != SFN_OK) return st;
    if (!x) return SFN_EINVAL;
    if (pipeline != SFN_PIPE_SEQUENTIAL && pipeline != SFN_PIPE_PARALLEL) return SFN_EINVAL;
    if (pipeline == SFN_PIPE_PARALLEL && !y) return SFN_EINVAL;
    if (!y && !idx && !n_idx) return SFN_EINVAL;  // nothing to compute
    if (!aligned16(x)) return SFN_EALIGN;
    if (y && !aligned16(y)) return SFN_EALIGN;
    if ((idx && (reinterpret_cast<uintptr_t>(idx) & 3u)) || (n_idx && (reinterpret_cast<uintptr_t>(n_idx) & 3u)))
      return SFN_EALIGN;
    st = check_ws(ws, ws_bytes, svd_pipeline_bytes(ffn, svd));
    if (st != SFN_OK) return st;

    float* z = reinterpret_cast<float*>(static_cast<char*>(ws) + svd_pipeline_z_offset(ffn));
    sfn::DecodeArgs a{};
    a.wg = static_cast<const char*>(ffn->w_gate);
    a.wu = static_cast<const char*>(ffn->w_up);
    a.wd = static_cast<const char*>(ffn->w_down_t);
    a.bias = ffn->b_gate;
    a.x = static_cast<const char*>(x);
    a.y = y;
    a.active_idx = idx;
    a.n_active = n_idx;
    a.pl = static_cast<const char*>(svd->l);
    a.pz = z;
    a.ptau = svd->tau;
    a.pb = svd->b;
    a.pr = svd->r;
    a.d = ffn->d;
    a.f = ffn->f;
    a.nch = ffn->d * 2 / 16;
    a.row_bytes = ffn->d * 2;
    a.nb = 1;
    a.act = ffn->act;
    a.G = sfn::decode_grid(ffn->f);
    a.n_red = sfn::decode_reducers(a.G, 1, ffn->d);
    sfn::decode_carve(a, ws, 2);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    hipError_t e = sfn::launch_svd_z(*svd, x, z, s);
    if (e != hipSuccess) return SFN_EHIP;
    e = pipeline == SFN_PIPE_PARALLEL ? sfn::launch_decode_parallel(a, SFN_BF16, s) : sfn::launch_decode(a, SFN_BF16, s);
    return hip_status(e);
  } catch (...) {
    return SFN_EHIP;
  }
}

int ffn_dense_chunk(const sfn_ffn* ffn, const void* x, int32_t n, float* y, void* ws, size_t ws_bytes,
                    void* stream) {
  try {
    int st = check_ffn(ffn, true);
    if (st != SFN_OK) return st;
    if (!x || !y) return SFN_EINVAL;
    if (!aligned16(x) || !aligned16(y)) return SFN_EALIGN;
    if (n < 1 || n > SFN_MAX_CHUNK) return SFN_ESHAPE;
    st = check_ws(ws, ws_bytes, sfn::chunk_workspace_bytes(ffn->d, ffn->f, ffn->wdtype, n));
    if (st != SFN_OK) return st;
    return hip_status(sfn::launch_dense_chunk(*ffn, x, n, y, ws, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

namespace {

int check_kv(const sfn_kv* kv, bool need_data) {
  if (!kv) return SFN_EINVAL;
  if (kv->dtype != SFN_F32 && kv->dtype != SFN_BF16) return SFN_EDTYPE;
  if (kv->reserved != 0) return SFN_EINVAL;
  if (kv->page < 16 || kv->page > 256 || (kv->page & (kv->page - 1))) return SFN_ESHAPE;
  if (kv->n_pages < 1 || (int64_t)kv->n_pages * kv->page > INT32_MAX) return SFN_ESHAPE;
  if (kv->h_kv < 1 || kv->h_kv > SFN_MAX_HEADS) return SFN_ESHAPE;
  if (kv->dh != 64 && kv->dh != 128) return SFN_ESHAPE;
  if (need_data && (!kv->k || !kv->v)) return SFN_EINVAL;
  if (!aligned16(kv->k) || !aligned16(kv->v)) return SFN_EALIGN;
  return SFN_OK;
}

int check_kv8(const sfn_kv8* kv, bool need_data) {
  if (!kv) return SFN_EINVAL;
  const int st = check_kv(&kv->kv, need_data);
  if (st != SFN_OK) return st;
  if (need_data && (!kv->k_exp || !kv->v_exp)) return SFN_EINVAL;
  return aligned16(kv->k_exp) && aligned16(kv->v_exp) ? SFN_OK : SFN_EALIGN;
}

int page_shift(int page) { return __builtin_ctz((unsigned)page); }

// A token stride in elements: room for `heads` heads, 16-byte steps.
int check_rows(const void* p, int64_t stride, int heads, const sfn_kv* kv) {
  if (!aligned16(p)) return SFN_EALIGN;
  if (stride < (int64_t)heads * kv->dh || stride > (int64_t)1 << 32) return SFN_ESHAPE;
  return stride * wbytes(kv->dtype) % 16 == 0 ? SFN_OK : SFN_EALIGN;
}

// The shape arguments of an attention call, and its division of the work.
int check_attend(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new, int32_t max_len) {
  if (R < 1 || R > SFN_MAX_REQUESTS || T < 0 || T > SFN_MAX_STEP_TOKENS) return SFN_ESHAPE;
  if (h_q < 1 || h_q > SFN_MAX_HEADS || h_q % kv->h_kv) return SFN_ESHAPE;
  if (max_new < 1 || max_new > SFN_MAX_STEP_TOKENS || max_len < 0 || max_len > 1 << 30) return SFN_ESHAPE;
  return SFN_OK;
}

size_t attend_bytes(const sfn_kv* kv, int64_t parts) {
  return sfn::kWsHeader + round256((size_t)parts * kv->dh * sizeof(float)) + round256((size_t)parts * 2 * sizeof(float));
}

}  // namespace

int kv_cache_plan(const sfn_kv* kv, int32_t R, int32_t max_pages, int32_t max_tokens, const int32_t* held_len,
                  const int32_t* ctx_len, const int32_t* new_len, int32_t* table, int32_t* free_pages,
                  const int32_t* n_free, int32_t* n_free_out, int32_t* cu, int32_t* kv_len, int32_t* pos,
                  int32_t* slot, int32_t* status, void* stream) {
  try {
    const int st = check_kv(kv, false);
    if (st != SFN_OK) return st;
    if (R < 1 || R > SFN_MAX_REQUESTS || max_tokens < 1 || max_tokens > SFN_MAX_STEP_TOKENS) return SFN_ESHAPE;
    if (max_pages < 1 || (int64_t)R * max_pages > INT32_MAX || (int64_t)max_pages * kv->page > INT32_MAX) return SFN_ESHAPE;
    const void* all[] = {held_len, ctx_len, new_len, table, free_pages, n_free, n_free_out, cu, kv_len, pos, slot, status};
    for (const void* p : all) {
      if (!p) return SFN_EINVAL;
      if (!aligned4_or_null(p)) return SFN_EALIGN;
    }
    // outputs that are read as inputs while they are written
    const void* in[] = {held_len, ctx_len, new_len, n_free};
    const void* out[] = {table, free_pages, n_free_out, cu, kv_len, pos, slot, status};
    for (const void* i : in)
      for (const void* o : out)
        if (i == o) return SFN_EINVAL;
    sfn::KvPlanArgs a{held_len, ctx_len, new_len, table, free_pages, n_free, n_free_out, cu, kv_len, pos, slot, status,
                      R, max_pages, max_tokens, kv->n_pages, page_shift(kv->page)};
    return hip_status(sfn::launch_kv_plan(a, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

namespace {

// The arguments that both kinds of cache take alike.
int check_append(const sfn_kv* kv, int32_t h_q, const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                 int64_t v_stride, const int32_t* pos, const int32_t* slot, const float* rope, int32_t n_pos, int32_t rot,
                 const void* q_out) {
  int st;
  if ((h_q > 0) != (q != nullptr) || (h_q > 0) != (q_out != nullptr)) return SFN_EINVAL;
  if (!k || !v || !slot) return SFN_EINVAL;
  if (rope ? !pos : rot != 0) return SFN_EINVAL;
  if (rope && (rot < 16 || rot > kv->dh || rot % 16 || n_pos < 1)) return SFN_ESHAPE;
  if (h_q && (st = check_rows(q, q_stride, h_q, kv)) != SFN_OK) return st;
  if ((st = check_rows(k, k_stride, kv->h_kv, kv)) != SFN_OK) return st;
  if ((st = check_rows(v, v_stride, kv->h_kv, kv)) != SFN_OK) return st;
  if (!aligned16(q_out) || !aligned16(rope) || !aligned4_or_null(pos) || !aligned4_or_null(slot)) return SFN_EALIGN;
  return SFN_OK;
}

}  // namespace

int kv_cache_append(const sfn_kv* kv, int32_t T, int32_t h_q, const void* q, int64_t q_stride, const void* k,
                    int64_t k_stride, const void* v, int64_t v_stride, const int32_t* pos, const int32_t* slot,
                    const float* rope, int32_t n_pos, int32_t rot, void* q_out, void* stream) {
  try {
    int st = check_kv(kv, true);
    if (st != SFN_OK) return st;
    if (T < 0 || T > SFN_MAX_STEP_TOKENS || h_q < 0 || h_q > SFN_MAX_HEADS) return SFN_ESHAPE;
    if (T == 0) return SFN_OK;  // empty arrays may have null addresses
    if ((st = check_append(kv, h_q, q, q_stride, k, k_stride, v, v_stride, pos, slot, rope, n_pos, rot, q_out)) != SFN_OK) return st;
    const int64_t e = wbytes(kv->dtype);
    sfn::KvAppendArgs a{};
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.q_stride = q_stride * e;
    a.k_stride = k_stride * e;
    a.v_stride = v_stride * e;
    a.q_out = static_cast<char*>(q_out);
    a.k_cache = static_cast<char*>(kv->k);
    a.v_cache = static_cast<char*>(kv->v);
    a.pos = pos;
    a.slot = slot;
    a.rope = rope;
    a.T = T;
    a.h_q = h_q;
    a.h_kv = kv->h_kv;
    a.dh = kv->dh;
    a.rot = rope ? rot : 0;
    a.n_pos = n_pos;
    a.n_pages = kv->n_pages;
    a.page_shift = page_shift(kv->page);
    return hip_status(sfn::launch_kv_append(a, kv->dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

int kv8_cache_append(const sfn_kv8* kv, int32_t T, int32_t h_q, const void* q, int64_t q_stride, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, const int32_t* pos, const int32_t* slot,
                     const float* rope, int32_t n_pos, int32_t rot, void* q_out, void* stream) {
  try {
    int st = check_kv8(kv, true);
    if (st != SFN_OK) return st;
    if (T < 0 || T > SFN_MAX_STEP_TOKENS || h_q < 0 || h_q > SFN_MAX_HEADS) return SFN_ESHAPE;
    if (T == 0) return SFN_OK;
    const sfn_kv* c = &kv->kv;
    if ((st = check_append(c, h_q, q, q_stride, k, k_stride, v, v_stride, pos, slot, rope, n_pos, rot, q_out)) != SFN_OK) return st;
    const int64_t e = wbytes(c->dtype);
    sfn::Kv8AppendArgs a{};
    a.q = static_cast<const char*>(q);
    a.k = static_cast<const char*>(k);
    a.v = static_cast<const char*>(v);
    a.q_stride = q_stride * e;
    a.k_stride = k_stride * e;
    a.v_stride = v_stride * e;
    a.q_out = static_cast<char*>(q_out);
    a.k_cache = static_cast<char*>(c->k);
    a.v_cache = static_cast<char*>(c->v);
    a.k_exp = kv->k_exp;
    a.v_exp = kv->v_exp;
    a.pos = pos;
    a.slot = slot;
    a.rope = rope;
    a.T = T;
    a.h_q = h_q;
    a.h_kv = c->h_kv;
    a.rot = rope ? rot : 0;
    a.n_pos = n_pos;
    a.n_pages = c->n_pages;
    a.page_shift = page_shift(c->page);
    return hip_status(sfn::launch_kv8_append(a, c->dh, c->dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

int kv8_cache_read(const sfn_kv8* kv, int32_t T, const int32_t* slot, void* k_out, int64_t k_stride, void* v_out,
                   int64_t v_stride, void* stream) {
  try {
    int st = check_kv8(kv, true);
    if (st != SFN_OK) return st;
    if (T < 0 || T > SFN_MAX_STEP_TOKENS) return SFN_ESHAPE;
    if (T == 0) return SFN_OK;
    const sfn_kv* c = &kv->kv;
    if (!slot || !k_out || !v_out) return SFN_EINVAL;
    if ((st = check_rows(k_out, k_stride, c->h_kv, c)) != SFN_OK) return st;
    if ((st = check_rows(v_out, v_stride, c->h_kv, c)) != SFN_OK) return st;
    if (!aligned4_or_null(slot)) return SFN_EALIGN;
    const int64_t e = wbytes(c->dtype);
    sfn::Kv8ReadArgs a{};
    a.k_cache = static_cast<const char*>(c->k);
    a.v_cache = static_cast<const char*>(c->v);
    a.k_exp = kv->k_exp;
    a.v_exp = kv->v_exp;
    a.slot = slot;
    a.k_out = static_cast<char*>(k_out);
    a.v_out = static_cast<char*>(v_out);
    a.k_stride = k_stride * e;
    a.v_stride = v_stride * e;
    a.T = T;
    a.h_kv = c->h_kv;
    a.n_pages = c->n_pages;
    a.page_shift = page_shift(c->page);
    return hip_status(sfn::launch_kv8_read(a, c->dh, c->dtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

namespace {

size_t attend_size(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new, int32_t max_len) {
  if (check_attend(kv, R, T, h_q, max_new, max_len) != SFN_OK) return 0;
  return attend_bytes(kv, sfn::attend_most_parts(R, h_q, kv->h_kv, kv->dtype, max_new, max_len));
}

// What every attention launch has in common.
sfn::AttendArgs attend_args(const sfn_kv* kv, const uint8_t* k_exp, const uint8_t* v_exp, int32_t T, int32_t h_q, const void* q,
                            int64_t q_stride, const int32_t* cu, const int32_t* kv_len, float scale, void* out) {
  sfn::AttendArgs a{};
  a.k = static_cast<const char*>(kv->k);
  a.v = static_cast<const char*>(kv->v);
  a.k_exp = k_exp;
  a.v_exp = v_exp;
  a.q = static_cast<const char*>(q);
  a.q_stride = q_stride * wbytes(kv->dtype);
  a.cu = cu;
  a.kv_len = kv_len;
  a.out = static_cast<char*>(out);
  a.T = T;
  a.h_q = h_q;
  a.h_kv = kv->h_kv;
  a.g = h_q / kv->h_kv;
  a.g_mul = ((1 << 21) + a.g - 1) / a.g;
  a.page_shift = page_shift(kv->page);
  a.n_pages = kv->n_pages;
  a.scale_log2 = scale * 1.44269504088896340736f;
  return a;
}

// Its division of the work, and where its parts lie: at w, as part_bytes(kv, p.parts) count them.
void set_plan(sfn::AttendArgs& a, const sfn::AttendPlan& p, const sfn_kv* kv, char* w, int64_t parts) {
  a.part_o = reinterpret_cast<float*>(w);
  a.part_ml = reinterpret_cast<float*>(w + round256((size_t)parts * kv->dh * sizeof(float)));
  a.tile_rows = p.tile_rows;
  a.tile_keys = p.tile_keys;
  a.row_tiles = p.row_tiles;
  a.S = p.S;
  a.chunk = p.chunk;
}

int attend(const sfn_kv* kv, const uint8_t* k_exp, const uint8_t* v_exp, int32_t R, int32_t T, int32_t h_q, const void* q, int64_t q_stride,
           const int32_t* table, int32_t max_pages, const int32_t* cu, const int32_t* kv_len, int32_t max_new, int32_t max_len, float scale,
           int32_t window, void* out, void* ws, size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_attend(kv, R, T, h_q, max_new, max_len)) != SFN_OK) return st;
  if (max_pages < 1) return SFN_ESHAPE;
  if ((int64_t)max_pages * kv->page < max_len) max_len = max_pages * kv->page;
  if (T == 0) return SFN_OK;
  if (!q || !table || !cu || !kv_len || !out) return SFN_EINVAL;
  if (!(scale > 0.0f) || !std::isfinite(scale) || window < 0) return SFN_EINVAL;
  if ((st = check_rows(q, q_stride, h_q, kv)) != SFN_OK) return st;
  if (!aligned16(out) || !aligned4_or_null(table) || !aligned4_or_null(cu) || !aligned4_or_null(kv_len)) return SFN_EALIGN;
  if (window >= max_len) window = 0;  // every key is within it
  const sfn::AttendPlan p = sfn::attend_plan(R, h_q, kv->h_kv, kv->dtype, max_new, max_len, window);
  if ((int64_t)R * p.S * p.row_tiles * kv->h_kv > INT32_MAX) return SFN_ESHAPE;
  if ((st = check_ws(ws, ws_bytes, attend_bytes(kv, p.parts))) != SFN_OK) return st;
  sfn::AttendArgs a = attend_args(kv, k_exp, v_exp, T, h_q, q, q_stride, cu, kv_len, scale, out);
  set_plan(a, p, kv, static_cast<char*>(ws) + sfn::kWsHeader, p.parts);
  a.table = table;
  a.max_pages = max_pages;
  a.R = R;
  a.max_new = max_new;
  a.max_len = max_len;
  a.window = window;
  return hip_status(sfn::launch_kv_attend(a, kv->dh, kv->dtype, static_cast<hipStream_t>(stream)));
}

// Keys that a launch over the rest of the sequences may span: it begins with a whole tile.
int32_t own_span(int32_t max_own) { return max_own + 64; }

int check_shared(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new, int32_t max_shared, int32_t max_own) {
  if (max_shared < 0 || max_own < 0 || (int64_t)max_shared + max_own > 1 << 30) return SFN_ESHAPE;
  return check_attend(kv, R, T, h_q, max_new, max_shared + max_own);
}

// Tokens of a call over a shared prefix that can have parts: every one that is computed has, of
// both sets of keys. The step may have others (other calls', or room that a captured step leaves).
int32_t shared_tokens(int32_t R, int32_t T, int32_t max_new) { return (int32_t)std::min<int64_t>(T, (int64_t)R * max_new); }

size_t shared_bytes(const sfn_kv* kv, int64_t own, int64_t prefix) {
  return attend_bytes(kv, own) + attend_bytes(kv, prefix) - sfn::kWsHeader;
}

size_t shared_size(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new, int32_t max_shared, int32_t max_own) {
  if (check_shared(kv, R, T, h_q, max_new, max_shared, max_own) != SFN_OK) return 0;
  const int32_t t = shared_tokens(R, T > 0 ? T : 1, max_new);
  const int64_t own = sfn::attend_most_parts(R, h_q, kv->h_kv, kv->dtype, max_new, own_span(max_own));
  const int64_t prefix = sfn::prefix_most_parts(t, h_q, kv->h_kv, kv->dtype, max_shared);
  return shared_bytes(kv, std::max(own, (int64_t)t * h_q), std::max(prefix, (int64_t)t * h_q));
}

int attend_shared(const sfn_kv* kv, const uint8_t* k_exp, const uint8_t* v_exp, int32_t R, int32_t T, int32_t h_q, const void* q,
                  int64_t q_stride, const int32_t* prefix, int32_t prefix_pages, const int32_t* shared_len, const int32_t* table,
                  int32_t max_pages, const int32_t* cu, const int32_t* kv_len, int32_t max_new, int32_t max_shared, int32_t max_own,
                  float scale, void* out, void* ws, size_t ws_bytes, void* stream) {
  int st;
  if ((st = check_shared(kv, R, T, h_q, max_new, max_shared, max_own)) != SFN_OK) return st;
  if (max_pages < 1 || prefix_pages < 1) return SFN_ESHAPE;
  if ((int64_t)prefix_pages * kv->page < max_shared) max_shared = prefix_pages * kv->page;
  if (T == 0) return SFN_OK;
  if (!q || !prefix || !shared_len || !table || !cu || !kv_len || !out) return SFN_EINVAL;
  if (!(scale > 0.0f) || !std::isfinite(scale)) return SFN_EINVAL;
  if ((st = check_rows(q, q_stride, h_q, kv)) != SFN_OK) return st;
  if (!aligned16(out)) return SFN_EALIGN;
  for (const int32_t* p : {prefix, shared_len, table, cu, kv_len})
    if (!aligned4_or_null(p)) return SFN_EALIGN;
  max_new = std::min(max_new, T);
  const sfn::AttendPlan po = sfn::attend_plan(R, h_q, kv->h_kv, kv->dtype, max_new, own_span(max_own), 0);
  const int32_t tokens = shared_tokens(R, T, max_new);
  const sfn::AttendPlan pp = sfn::prefix_plan(tokens, h_q, kv->h_kv, kv->dtype, max_shared);
  // one launch of 256 threads to a workgroup, whose threads are counted in 32 bits
  if ((int64_t)R * (po.S | 1) * po.row_tiles * kv->h_kv + (int64_t)pp.S * pp.row_tiles * kv->h_kv > UINT32_MAX / 256) return SFN_ESHAPE;
  const int64_t rows = (int64_t)tokens * h_q, own_parts = rows * po.S, prefix_parts = rows * pp.S;
  if ((st = check_ws(ws, ws_bytes, shared_bytes(kv, own_parts, prefix_parts))) != SFN_OK) return st;
  char* const w = static_cast<char*>(ws) + sfn::kWsHeader;
  sfn::SharedArgs a{};
  a.own = attend_args(kv, k_exp, v_exp, T, h_q, q, q_stride, cu, kv_len, scale, out);
  a.own.R = R;
  a.own.shared = shared_len;
  a.own.max_shared = max_shared;
  a.own.max_own = max_own;
  a.own.by_token = T < (int64_t)R * max_new;
  a.prefix = a.own;
  set_plan(a.own, po, kv, w, own_parts);
  a.own.table = table;
  a.own.max_pages = max_pages;
  a.own.max_new = max_new;
  a.own.max_len = (int32_t)std::min<int64_t>((int64_t)max_pages * kv->page, max_shared + max_own);
  set_plan(a.prefix, pp, kv, w + (attend_bytes(kv, own_parts) - sfn::kWsHeader), prefix_parts);
  a.prefix.table = prefix;
  a.prefix.max_pages = prefix_pages;
  a.prefix.max_new = tokens;
  a.prefix.each_new = max_new;
  a.prefix.max_len = max_shared;
  return hip_status(sfn::launch_kv_attend_shared(a, kv->dh, kv->dtype, static_cast<hipStream_t>(stream)));
}

}  // namespace

size_t kv_cache_attend_workspace_size(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new,
                                      int32_t max_len) {
  try {
    return check_kv(kv, false) == SFN_OK ? attend_size(kv, R, T, h_q, max_new, max_len) : 0;
  } catch (...) {
    return 0;
  }
}

int kv_cache_attend(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, const void* q, int64_t q_stride,
                    const int32_t* table, int32_t max_pages, const int32_t* cu, const int32_t* kv_len,
                    int32_t max_new, int32_t max_len, float scale, int32_t window, void* out, void* ws,
                    size_t ws_bytes, void* stream) {
  try {
    const int st = check_kv(kv, true);
    if (st != SFN_OK) return st;
    return attend(kv, nullptr, nullptr, R, T, h_q, q, q_stride, table, max_pages, cu, kv_len, max_new, max_len, scale, window, out, ws,
                  ws_bytes, stream);
  } catch (...) {
    return SFN_EHIP;
  }
}

size_t kv8_cache_attend_workspace_size(const sfn_kv8* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new,
                                       int32_t max_len) {
  try {
    return check_kv8(kv, false) == SFN_OK ? attend_size(&kv->kv, R, T, h_q, max_new, max_len) : 0;
  } catch (...) {
    return 0;
  }
}

int kv8_cache_attend(const sfn_kv8* kv, int32_t R, int32_t T, int32_t h_q, const void* q, int64_t q_stride,
                     const int32_t* table, int32_t max_pages, const int32_t* cu, const int32_t* kv_len,
                     int32_t max_new, int32_t max_len, float scale, int32_t window, void* out, void* ws,
                     size_t ws_bytes, void* stream) {
  try {
    const int st = check_kv8(kv, true);
    if (st != SFN_OK) return st;
    return attend(&kv->kv, kv->k_exp, kv->v_exp, R, T, h_q, q, q_stride, table, max_pages, cu, kv_len, max_new, max_len, scale, window, out,
                  ws, ws_bytes, stream);
  } catch (...) {
    return SFN_EHIP;
  }
}

size_t kv_cache_attend_shared_workspace_size(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new,
                                             int32_t max_shared, int32_t max_own) {
  try {
    return check_kv(kv, false) == SFN_OK ? shared_size(kv, R, T, h_q, max_new, max_shared, max_own) : 0;
  } catch (...) {
    return 0;
  }
}

int kv_cache_attend_shared(const sfn_kv* kv, int32_t R, int32_t T, int32_t h_q, const void* q, int64_t q_stride,
                           const int32_t* prefix, int32_t prefix_pages, const int32_t* shared_len,
                           const int32_t* table, int32_t max_pages, const int32_t* cu, const int32_t* kv_len,
                           int32_t max_new, int32_t max_shared, int32_t max_own, float scale, void* out, void* ws,
                           size_t ws_bytes, void* stream) {
  try {
    const int st = check_kv(kv, true);
    if (st != SFN_OK) return st;
    return attend_shared(kv, nullptr, nullptr, R, T, h_q, q, q_stride, prefix, prefix_pages, shared_len, table, max_pages, cu, kv_len,
                         max_new, max_shared, max_own, scale, out, ws, ws_bytes, stream);
  } catch (...) {
    return SFN_EHIP;
  }
}

size_t kv8_cache_attend_shared_workspace_size(const sfn_kv8* kv, int32_t R, int32_t T, int32_t h_q, int32_t max_new,
                                              int32_t max_shared, int32_t max_own) {
  try {
    return check_kv8(kv, false) == SFN_OK ? shared_size(&kv->kv, R, T, h_q, max_new, max_shared, max_own) : 0;
  } catch (...) {
    return 0;
  }
}

int kv8_cache_attend_shared(const sfn_kv8* kv, int32_t R, int32_t T, int32_t h_q, const void* q, int64_t q_stride,
                            const int32_t* prefix, int32_t prefix_pages, const int32_t* shared_len,
                            const int32_t* table, int32_t max_pages, const int32_t* cu, const int32_t* kv_len,
                            int32_t max_new, int32_t max_shared, int32_t max_own, float scale, void* out, void* ws,
                            size_t ws_bytes, void* stream) {
  try {
    const int st = check_kv8(kv, true);
    if (st != SFN_OK) return st;
    return attend_shared(&kv->kv, kv->k_exp, kv->v_exp, R, T, h_q, q, q_stride, prefix, prefix_pages, shared_len, table, max_pages, cu,
                         kv_len, max_new, max_shared, max_own, scale, out, ws, ws_bytes, stream);
  } catch (...) {
    return SFN_EHIP;
  }
}

int residual_norm(const sfn_norm* norm, int32_t T, const void* h, int32_t hdtype, const void* y, int32_t ydtype,
                  const void* gate, int64_t gate_stride, void* h_out, void* x_out, void* stream) {
  try {
    if (!norm) return SFN_EINVAL;
    for (int dt : {norm->wdtype, hdtype, ydtype})
      if (dt != SFN_F32 && dt != SFN_BF16) return SFN_EDTYPE;
    if (norm->d < 8 || norm->d > SFN_MAX_D || T < 0 || T > SFN_MAX_STEP_TOKENS) return SFN_ESHAPE;
    if (norm->d % 8) return SFN_EALIGN;
    if (T == 0) return SFN_OK;
    if (!(norm->eps >= 0.0f) || !std::isfinite(norm->eps) || !std::isfinite(norm->scale)) return SFN_EINVAL;
    if (!h || (!h_out && !x_out)) return SFN_EINVAL;
    if (x_out && !norm->w_pre) return SFN_EINVAL;
    if (!y && (h_out || gate)) return SFN_EINVAL;
    if (gate && gate_stride != 0 && gate_stride < norm->d) return SFN_ESHAPE;
    if (gate && gate_stride % 8) return SFN_EALIGN;
    const void* all[] = {h, y, gate, h_out, x_out, norm->w_post, norm->w_pre};
    for (const void* p : all)
      if (!aligned16(p)) return SFN_EALIGN;
    sfn::NormArgs a{};
    a.h = static_cast<const char*>(h);
    a.y = static_cast<const char*>(y);
    a.w_post = static_cast<const char*>(norm->w_post);
    a.w_pre = static_cast<const char*>(norm->w_pre);
    a.gate = static_cast<const char*>(gate);
    a.gate_stride = gate_stride * wbytes(norm->wdtype);
    a.h_out = static_cast<char*>(h_out);
    a.x_out = static_cast<char*>(x_out);
    a.scale = norm->scale;
    a.eps = norm->eps;
    a.T = T;
    a.d = norm->d;
    return hip_status(sfn::launch_residual_norm(a, hdtype, ydtype, norm->wdtype, static_cast<hipStream_t>(stream)));
  } catch (...) {
    return SFN_EHIP;
  }
}

}  // extern "C"
