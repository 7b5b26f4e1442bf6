// na_ops_api.cu -- the extern "C" entry points of the packed attention, the
// norms around a block, and the layer made of them: argument checks and
// workspace layout.
#include <cmath>
#include <cstdint>

#include "na2d_internal.h"

#define NA_EXPORT extern "C" __attribute__((visibility("default")))

namespace na2d {
namespace {

// A pointer the call uses, aligned to `to` bytes; NULL is bad only if needed.
bool bad(const void* ptr, bool needed, uintptr_t to = 16) {
  return ptr ? (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0 : needed;
}
na_status from_cuda(cudaError_t e) { return e == cudaSuccess ? NA_OK : NA_ERR_CUDA; }
bool known(na_dtype dt) { return dt == NA_F32 || dt == NA_F16 || dt == NA_BF16; }
size_t elem_size(na_dtype dt) { return dt == NA_F32 ? 4 : 2; }

constexpr int kMaxTokens = 1 << 30;

// Sizes of a packed batch; the pointers are the caller's.
na_status check_packed(int nseq, int total_q, int total_k, int heads_q, int heads_k, int d, int causal, int window,
                       float scale, na_dtype dt, PackedArgs* p) {
  if (!known(dt) || nseq < 0 || total_q < 0 || total_k < 0) return NA_ERR_INVALID_ARG;
  if (heads_q < 1 || heads_k < 1 || heads_q % heads_k) return NA_ERR_INVALID_ARG;
  if (d != 16 && d != 32 && d != 64 && d != 128) return NA_ERR_INVALID_ARG;
  if ((causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return NA_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || scale <= 0.f) return NA_ERR_INVALID_ARG;
  // block numbers are 32 bits, a grid has 65535 key heads at most, and the
  // kernels step over rows and keys in ints
  if (heads_k > 65535 || total_q > kMaxTokens || total_k > kMaxTokens || ((long double)total_q + total_k) * heads_q * d >= (long double)(1ll << 40))
    return NA_ERR_UNSUPPORTED;
  *p = PackedArgs{};
  p->nseq = nseq;
  p->total_q = total_q;
  p->total_k = total_k;
  p->hq = heads_q;
  p->hk = heads_k;
  p->group = heads_q / heads_k;
  p->d = d;
  p->causal = causal;
  p->window = window;
  p->scale = scale;
  return NA_OK;
}

constexpr int kMaxChannels = 8192;  // a row lies in one block's registers

na_status check_norm(long long rows, int C, long long gates, int rms, int post, float eps, float scale, na_dtype dt,
                     NormArgs* p) {
  if (!known(dt) || rows < 0 || C < 1 || gates < 0) return NA_ERR_INVALID_ARG;
  if ((rms != 0 && rms != 1) || (post != 0 && post != 1)) return NA_ERR_INVALID_ARG;
  if (!std::isfinite(eps) || eps < 0.f || !std::isfinite(scale)) return NA_ERR_INVALID_ARG;
  if (gates > 0 && rows % gates) return NA_ERR_INVALID_ARG;
  if (C > kMaxChannels || (long double)rows * C >= (long double)(1ll << 40)) return NA_ERR_UNSUPPORTED;
  *p = NormArgs{};
  p->rows = rows;
  p->C = C;
  p->gate_rows = rows > 0 ? (gates > 0 ? rows / gates : rows) : 1;
  p->rms = rms;
  p->post = post;
  p->eps = eps;
  p->scale = scale;
  return NA_OK;
}

}  // namespace
}  // namespace na2d

using namespace na2d;

// ------------------------------------------------------- packed attention
NA_EXPORT size_t na_packed_workspace_bytes(int nseq, int total_q, int total_k, int heads_q, int heads_k, int d,
                                           na_dtype dt) {
  PackedArgs p;
  if (check_packed(nseq, total_q, total_k, heads_q, heads_k, d, 0, 0, 1.f, dt, &p) != NA_OK) return 0;
  if (nseq == 0 || total_q == 0) return 0;
  return packed_workspace_bytes(p, dt);
}

NA_EXPORT na_status na_packed_forward(const void* q, const void* k, const void* v, const int* cu_q, const int* cu_k,
                                      const int* len_k, void* out, float* lse, void* workspace,
                                      size_t workspace_bytes, int nseq, int total_q, int total_k, int heads_q,
                                      int heads_k, int d, int causal, int window, float scale, na_dtype dt,
                                      void* stream) {
  PackedArgs p;
  const na_status st = check_packed(nseq, total_q, total_k, heads_q, heads_k, d, causal, window, scale, dt, &p);
  if (st != NA_OK) return st;
  if (nseq == 0 || total_q == 0) return NA_OK;
  const bool keys = total_k > 0;
  if (bad(q, true) || bad(out, true) || bad(k, keys) || bad(v, keys)) return NA_ERR_INVALID_ARG;
  if (bad(cu_q, true, 4) || bad(cu_k, true, 4) || bad(len_k, false, 4) || bad(lse, false, 4)) return NA_ERR_INVALID_ARG;
  const size_t need = packed_workspace_bytes(p, dt);
  if (bad(workspace, need > 0, 256) || (need && workspace_bytes < need)) return NA_ERR_INVALID_ARG;
  if (status_word(&p.status) != cudaSuccess) return NA_ERR_CUDA;
  p.q = q;
  p.k = k;
  p.v = v;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.len_k = len_k;
  p.out = out;
  p.lse = lse;
  return from_cuda(launch_packed_forward(p, workspace, dt, (cudaStream_t)stream));
}

NA_EXPORT size_t na_packed_backward_workspace_bytes(int nseq, int total_q, int total_k, int heads_q, int heads_k,
                                                    int d, na_dtype dt) {
  PackedArgs p;
  if (check_packed(nseq, total_q, total_k, heads_q, heads_k, d, 0, 0, 1.f, dt, &p) != NA_OK) return 0;
  if (nseq == 0 || total_q == 0) return 0;
  return packed_backward_workspace_bytes(p, dt);
}

NA_EXPORT na_status na_packed_backward(const void* q, const void* k, const void* v, const void* out, const float* lse,
                                       const void* dout, const int* cu_q, const int* cu_k, void* dq, void* dk,
                                       void* dv, void* workspace, size_t workspace_bytes, int nseq, int total_q,
                                       int total_k, int heads_q, int heads_k, int d, int causal, int window,
                                       float scale, na_dtype dt, void* stream) {
  PackedArgs p;
  const na_status st = check_packed(nseq, total_q, total_k, heads_q, heads_k, d, causal, window, scale, dt, &p);
  if (st != NA_OK) return st;
  if (nseq == 0 || (total_q == 0 && total_k == 0)) return NA_OK;
  const bool rows = total_q > 0, keys = total_k > 0;
  if (bad(q, rows) || bad(out, rows) || bad(dout, rows) || bad(dq, rows) || bad(lse, rows, 4)) return NA_ERR_INVALID_ARG;
  if (bad(k, keys) || bad(v, keys) || bad(dk, keys) || bad(dv, keys)) return NA_ERR_INVALID_ARG;
  if (bad(cu_q, true, 4) || bad(cu_k, true, 4)) return NA_ERR_INVALID_ARG;
  const size_t need = rows ? packed_backward_workspace_bytes(p, dt) : 0;
  if (bad(workspace, need > 0, 256) || workspace_bytes < need) return NA_ERR_INVALID_ARG;
  if (status_word(&p.status) != cudaSuccess) return NA_ERR_CUDA;
  p.q = q;
  p.k = k;
  p.v = v;
  p.o = out;
  p.lse_in = lse;
  p.dout = dout;
  p.cu_q = cu_q;
  p.cu_k = cu_k;
  p.dq = dq;
  p.dk = dk;
  p.dv = dv;
  return from_cuda(launch_packed_backward(p, workspace, dt, (cudaStream_t)stream));
}

// ------------------------------------------------------------------- norms
NA_EXPORT na_status na_norm_forward(const void* x, const void* o, const void* post_w, const void* post_b,
                                    const void* gate, const void* w, const void* b, void* y, void* h, long long rows,
                                    int C, long long gates, int rms, int post, float eps, float scale, na_dtype dt,
                                    void* stream) {
  NormArgs p;
  const na_status st = check_norm(rows, C, gates, rms, post, eps, scale, dt, &p);
  if (st != NA_OK) return st;
  if (rows == 0) return NA_OK;  // whatever the pointers: those of empty buffers may be NULL
  if ((gate != nullptr) != (gates > 0)) return NA_ERR_INVALID_ARG;
  if ((!o && (post || gate)) || (!post && (post_w || post_b)) || (!h && (w || b))) return NA_ERR_INVALID_ARG;
  if ((o != nullptr) != (y != nullptr) || (!y && !h)) return NA_ERR_INVALID_ARG;  // without o, y is x
  if (bad(x, true)) return NA_ERR_INVALID_ARG;
  for (const void* ptr : {o, post_w, post_b, gate, w, b, (const void*)y, (const void*)h})
    if (bad(ptr, false)) return NA_ERR_INVALID_ARG;
  p.x = x;
  p.o = o;
  p.pw = post_w;
  p.pb = post_b;
  p.gate = gate;
  p.w = w;
  p.b = b;
  p.y = y;
  p.h = h;
  if (status_word(&p.status) != cudaSuccess) return NA_ERR_CUDA;
  return from_cuda(launch_norm_forward(p, dt, (cudaStream_t)stream));
}

NA_EXPORT size_t na_norm_backward_workspace_bytes(long long rows, int C, long long gates, na_dtype dt) {
  NormArgs p;
  if (check_norm(rows, C, gates, 0, 0, 0.f, 1.f, dt, &p) != NA_OK || rows == 0) return 0;
  return norm_workspace_bytes(rows, C, p.gate_rows, dt);
}

NA_EXPORT na_status na_norm_backward(const void* y, const void* o, const void* post_w, const void* post_b,
                                     const void* gate, const void* w, const void* dy, const void* dh, void* dx,
                                     void* d_o, float* dw, float* db, float* dpost_w, float* dpost_b, float* dgate,
                                     void* workspace, size_t workspace_bytes, long long rows, int C, long long gates,
                                     int rms, int post, float eps, float scale, na_dtype dt, void* stream) {
  NormArgs p;
  const na_status st = check_norm(rows, C, gates, rms, post, eps, scale, dt, &p);
  if (st != NA_OK) return st;
  if (rows == 0) return NA_ERR_UNSUPPORTED;  // the sums over no rows would stay unwritten
  if ((gate != nullptr) != (gates > 0) || (!gate && dgate)) return NA_ERR_INVALID_ARG;
  if ((!o && (post || gate)) || (!post && (post_w || post_b || dpost_w || dpost_b))) return NA_ERR_INVALID_ARG;
  if (!dh && (w || dw || db)) return NA_ERR_INVALID_ARG;
  if ((!dy && !dh) || (o != nullptr) != (d_o != nullptr)) return NA_ERR_INVALID_ARG;
  if (bad(y, dh != nullptr) || bad(dx, true) || bad(workspace, true, 256)) return NA_ERR_INVALID_ARG;
  for (const void* ptr : {o, post_w, post_b, gate, w, dy, dh, (const void*)d_o, (const void*)dw, (const void*)db,
                          (const void*)dpost_w, (const void*)dpost_b, (const void*)dgate})
    if (bad(ptr, false)) return NA_ERR_INVALID_ARG;
  if (workspace_bytes < norm_workspace_bytes(rows, C, p.gate_rows, dt)) return NA_ERR_INVALID_ARG;
  p.x = y;
  p.o = o;
  p.pw = post_w;
  p.pb = post_b;
  p.gate = gate;
  p.w = w;
  p.dy = dy;
  p.dh = dh;
  p.dx = dx;
  p.dout = d_o;
  p.dw = dw;
  p.db = db;
  p.dpw = dpost_w;
  p.dpb = dpost_b;
  p.dgate = dgate;
  p.partial = (float*)workspace;
  if (status_word(&p.status) != cudaSuccess) return NA_ERR_CUDA;
  return from_cuda(launch_norm_backward(p, dt, (cudaStream_t)stream));
}

// ------------------------------------------------------------------- layer
// The two maps between the layer's steps lie in front of the block's own
// workspace.
NA_EXPORT size_t na2d_layer_workspace_bytes(int B, int H, int W, int heads, int dh, int ksize, na_dtype dt) {
  const size_t block = na2d_block_workspace_bytes(B, H, W, heads, dh, ksize, dt);
  if (block == 0) return 0;
  const size_t map = (size_t)B * H * W * heads * dh * elem_size(dt);
  return 2 * ((map + 255) / 256 * 256) + block;
}

NA_EXPORT na_status na2d_layer_forward(const void* x, const void* w, const void* b, const void* wqkv,
                                       const void* bqkv, const void* wo, const void* bo, const void* rpb,
                                       const void* post_w, const void* post_b, const void* gate, void* y,
                                       void* workspace, size_t workspace_bytes, int B, int H, int W, int heads, int dh,
                                       int ksize, int gates, int rms, int post, float eps, float scale, na_dtype dt,
                                       void* stream) {
  // everything is checked before anything runs: the block's arguments by its
  // kernel choice and workspace size, which enqueue nothing
  const int kind = na2d_forward_kernel(B, heads, H, W, dh, ksize, dt);
  if (kind < 0) return (na_status)-kind;
  if (B == 0 || heads == 0) return NA_OK;
  const size_t need = na2d_layer_workspace_bytes(B, H, W, heads, dh, ksize, dt);
  if (need == 0) return NA_ERR_INVALID_ARG;
  const long long rows = (long long)B * H * W;
  const int C = heads * dh;
  NormArgs unused;
  const na_status ok = check_norm(rows, C, gates, rms, post, eps, scale, dt, &unused);
  if (ok != NA_OK) return ok;
  if ((gate != nullptr) != (gates > 0) || (!post && (post_w || post_b))) return NA_ERR_INVALID_ARG;
  for (const void* ptr : {x, wqkv, wo, (const void*)y})
    if (bad(ptr, true)) return NA_ERR_INVALID_ARG;
  for (const void* ptr : {w, b, bqkv, bo, rpb, post_w, post_b, gate})
    if (bad(ptr, false)) return NA_ERR_INVALID_ARG;
  if (bad(workspace, true, 256) || workspace_bytes < need) return NA_ERR_INVALID_ARG;
  const size_t map = ((size_t)rows * C * elem_size(dt) + 255) / 256 * 256;
  char* ws = static_cast<char*>(workspace);
  na_status st = na_norm_forward(x, nullptr, nullptr, nullptr, nullptr, w, b, nullptr, ws, rows, C, 0, rms, 0, eps,
                                 1.f, dt, stream);
  if (st == NA_OK)
    st = na2d_block_forward(ws, wqkv, bqkv, wo, bo, rpb, ws + map, ws + 2 * map, workspace_bytes - 2 * map, B, H, W,
                            heads, dh, ksize, dt, stream);
  if (st == NA_OK)
    st = na_norm_forward(x, ws + map, post_w, post_b, gate, nullptr, nullptr, y, nullptr, rows, C, gates, rms, post,
                         eps, scale, dt, stream);
  return st;
}
