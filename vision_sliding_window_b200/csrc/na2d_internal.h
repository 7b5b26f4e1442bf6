// na2d_internal.h -- launchers shared between the C-ABI front end
// (na2d_api.cu) and the kernel translation units.  Not part of the ABI.
#pragma once

#include <cuda_runtime.h>

#include "na2d.h"

namespace na2d {

struct Shape {
  int B, heads, H, W, d, ks;
  long long queries() const { return (long long)B * heads * H * W; }
};

// SIMT kernels (na2d_simt.cu): every dtype, every supported shape.
cudaError_t launch_forward_simt(const void* q, const void* k, const void* v, const void* rpb,
                                void* out, const Shape& s, na_dtype dt, cudaStream_t st);
cudaError_t launch_qk_rpb_simt(const void* q, const void* k, const void* rpb, float* attn,
                               const Shape& s, na_dtype dt, cudaStream_t st);
cudaError_t launch_softmax_simt(float* attn, long long rows, int ks, float scale, cudaStream_t st);
cudaError_t launch_av_simt(const float* attn, const void* v, void* out, const Shape& s,
                           na_dtype dt, cudaStream_t st);

// Backward (na2d_bwd.cu): every dtype and head size; the workspace holds
// two float64 per query.
size_t backward_workspace_bytes(const Shape& s);
cudaError_t launch_backward_simt(const void* q, const void* k, const void* v, const void* rpb, const void* dout,
                                 void* dq, void* dk, void* dv, float* drpb, void* workspace, const Shape& s,
                                 na_dtype dt, cudaStream_t st);

// na2d_forward_host with every copy and the kernel in order on the
// caller's stream (na2d_api.cu); used by na2d_forward_host_noalloc.
na_status forward_host_serial(const void* q_host, const void* k_host, const void* v_host, const void* rpb_host,
                              void* out_host, void* workspace, size_t workspace_bytes, int B, int heads, int H,
                              int W, int d, int ksize, na_dtype dt, void* stream);

// SASA (na2d_sasa.cu): the zero-padded copies of q, k, v and the padded
// output live in the caller's workspace (four 256-byte aligned parts).
size_t sasa_workspace_bytes(const Shape& s, size_t es);
cudaError_t launch_sasa_pad(const void* q, const void* k, const void* v, void* workspace, const Shape& s, size_t es,
                            cudaStream_t st, void** qp, void** kp, void** vp, void** outp);
cudaError_t launch_sasa_crop(const void* outp, void* out, const Shape& s, size_t es, cudaStream_t st);

// NA block (na2d_block.cu): projections in cuBLAS around na2d_forward.
size_t block_workspace_bytes(int B, int H, int W, int heads, int dh, size_t es);
na_status run_block(const void* x, const void* wqkv, const void* bqkv, const void* wo, const void* bo, const void* rpb,
                    void* y, void* workspace, int B, int H, int W, int heads, int dh, int ks, na_dtype dt,
                    cudaStream_t st);

// NA over 1-3 axes with dilation (na2d_nd.cu).
cudaError_t launch_forward_nd(const void* q, const void* k, const void* v, const void* rpb, void* out, int B,
                              int heads, const int (&L)[3], int d, const int (&ks)[3], const int (&dil)[3],
                              na_dtype dt, cudaStream_t st);

// Device address of the current device's status word (na2d_api.cu).
cudaError_t status_word(unsigned** out);

// Norms around a block (na_norm.cu).
struct NormArgs {
  const void *x, *o, *pw, *pb, *gate, *w, *b;  // x is y in the backward pass
  void *y, *h;
  const void *dy, *dh;
  void *dx, *dout;  // dout: the gradient of o
  float *dw, *db, *dpw, *dpb, *dgate, *partial;
  long long rows, gate_rows;  // gate_rows rows share a row of the gate
  int C, rms, post;
  float eps, scale;
  unsigned* status;
  int lanes, pieces;  // set by the launchers
  long long chunks, chunk_rows;
};
size_t norm_workspace_bytes(long long rows, int C, long long gate_rows, na_dtype dt);
cudaError_t launch_norm_forward(const NormArgs& p, na_dtype dt, cudaStream_t st);
cudaError_t launch_norm_backward(NormArgs p, na_dtype dt, cudaStream_t st);

// Attention over packed sequences (na_packed_*.cu).
struct PackedArgs {
  const void *q, *k, *v;
  void* out;
  float* lse;
  const int *cu_q, *cu_k, *len_k;
  const void *o, *dout;  // backward: the forward's output and its gradient
  const float* lse_in;
  void *dq, *dk, *dv;
  int nseq, total_q, total_k, hq, hk, group, d, causal, window;
  float scale;
  // Sequences' keys are cut into at most max_pieces pieces that are joined
  // afterwards (1: not cut), of piece_keys keys each, or (0) the same number of
  // pieces for every sequence; and the pieces' results
  int path, piece_keys, max_pieces;
  float *part_o, *part_lse;  // [max_pieces][total_q][hq][d] and [max_pieces][total_q][hq];
                             // backward: [max_pieces][2][total_k][hk][d], dv and dk
  float2* terms;  // backward: (lse log2 e, out . dout) of every row, [total_q][hq]
  // fp16 backward on the tensor cores: the powers of two that lift a row's
  // weights' gradients into the type's range, [total_q][hq] and, for dk, of a
  // sequence and key head, [nseq][hk]
  float *row_lifts, *lifts;
  unsigned* status;
};
// Row tiles of 128 that a block of the tensor-core forward owns.
constexpr int packed_row_tiles(int d) { return d > 64 ? 2 : 1; }
enum { kPathSimt, kPathRows, kPathTc };
// Sets path, piece_keys and max_pieces (na_packed_simt.cu).
void packed_plan(PackedArgs* p, na_dtype dt);
cudaError_t launch_packed_forward_rows(const PackedArgs& p, na_dtype dt, cudaStream_t st);  // na_packed_rows.cu
cudaError_t launch_packed_forward_tc(const PackedArgs& p, na_dtype dt, cudaStream_t st);    // na_packed_tc.cu
void packed_backward_plan(PackedArgs* p, na_dtype dt);  // sets path and max_pieces
cudaError_t launch_packed_backward_tc(const PackedArgs& p, na_dtype dt, cudaStream_t st);   // na_packed_tc_bwd.cu
cudaError_t launch_packed_dkdv_join(const PackedArgs& p, na_dtype dt, cudaStream_t st);     // there too: adds pieces
size_t packed_workspace_bytes(const PackedArgs& p, na_dtype dt);
size_t packed_backward_workspace_bytes(const PackedArgs& p, na_dtype dt);
cudaError_t launch_packed_forward(PackedArgs p, void* workspace, na_dtype dt, cudaStream_t st);
cudaError_t launch_packed_backward(PackedArgs p, void* workspace, na_dtype dt, cudaStream_t st);

// Tensor-core fused forward (na2d_tc.cu), fp16/bf16.
bool forward_tc_supported(const Shape& s, na_dtype dt);
cudaError_t launch_forward_tc(const void* q, const void* k, const void* v, const void* rpb,
                              void* out, const Shape& s, na_dtype dt, unsigned* status,
                              cudaStream_t st);

}  // namespace na2d
