// Internal launch interface between the host API (api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "decode_common.cuh"

namespace pd {

// SIMT decode (any dtype / D in {64,128,256} / page size / group)
bool simt_supports(int q_dtype, int kv_dtype, int D);
// Launch, or (ctas != nullptr) only report resident blocks per SM.
cudaError_t launch_decode_simt(const DecodeParams& p, int q_dtype, int kv_dtype, dim3 grid,
                               cudaStream_t st, int* ctas = nullptr);

// Tensor-core decode (register-direct page loads + mma.sync); see decode_mma.cuh.
struct MmaConfig {
  int threads;       // block size
  int smem_bytes;    // dynamic shared memory
  int ctas_per_sm;   // occupancy (0 until queried)
};
// Launch (cfg == nullptr) or just query the launch configuration (cfg != nullptr).
cudaError_t launch_mma_bf16(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                           MmaConfig* cfg);
cudaError_t launch_mma_f16(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                           MmaConfig* cfg);
cudaError_t launch_mma_fp8(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                           MmaConfig* cfg);
// The same for pages of 8 rows (single token): two pages per 16-row tile.
cudaError_t launch_mma_pair_bf16(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                                 MmaConfig* cfg);
cudaError_t launch_mma_pair_f16(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                                MmaConfig* cfg);
cudaError_t launch_mma_pair_fp8(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                                MmaConfig* cfg);
// The same for the multi-query form (p.q_len > 1).
cudaError_t launch_mma_mq_bf16(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                               MmaConfig* cfg);
cudaError_t launch_mma_mq_f16(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                              MmaConfig* cfg);
cudaError_t launch_mma_mq_fp8(const DecodeParams& p, int q_dtype, dim3 grid, cudaStream_t st,
                              MmaConfig* cfg);

// Sets the thread's last-error message (api.cu).
void record_error(const char* msg);

// merge_state_inplace and append_paged_kv
cudaError_t launch_merge_state(void* V, float* S, const void* V_other, const float* S_other, int N,
                               int H, int D, int v_dtype, cudaStream_t st);
// R-way merge of fp32 partial states into out (out_dtype) and S_out; partner r's rows
// at V_parts + r * rstride (rstride = N*H*D: [R,N,H,D] with S [R,N,H]; or N*H*(D+1):
// one packed [out | lse] block per partner, S_parts = V_parts + N*H*D).
cudaError_t launch_merge_states(void* out, float* S_out, const float* V_parts, const float* S_parts,
                                int R, int N, int H, int D, int out_dtype, long long rstride,
                                cudaStream_t st);
// RoPE applied to the appended K rows (mode 0: none, 1 rotate-half, 2 interleaved).
struct AppendRope {
  const int32_t* positions;                // [T] position of each new token
  int mode;
  unsigned long long F[kMaxHalfDim];       // fixed-point turns per frequency
};
// 8-bit cache with a scale per block of rows (DecodeParams::scales): the tensor-core decode
// (decode_bs.cuh; tm: the pages as boxes of 16 rows) and the SIMT one.
cudaError_t launch_bs_e4m3(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                           cudaStream_t st, MmaConfig* cfg);
cudaError_t launch_bs_int(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                          cudaStream_t st, MmaConfig* cfg);
// The same for any page size and rows per scale: tiles gathered row by row.
cudaError_t launch_bs_rows_e4m3(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                                cudaStream_t st, MmaConfig* cfg);
cudaError_t launch_bs_rows_int(const DecodeParams& p, const CUtensorMap& tm, int q_dtype, dim3 grid,
                               cudaStream_t st, MmaConfig* cfg);
cudaError_t launch_decode_simt_bs(const DecodeParams& p, int q_dtype, int kv_dtype, dim3 grid,
                                  cudaStream_t st, int* ctas = nullptr);
// Append to such a cache: grid x = slots of touched blocks, grid y = blocks of kAppendWarps (K | V,
// head) pairs.
constexpr int kAppendWarps = 4;
inline long long append_bs_grid_y(int H_kv) { return (2ll * H_kv + kAppendWarps - 1) / kAppendWarps; }
struct AppendBsParams {
  uint8_t* pages;
  float* scales;
  const void* k_new;
  const void* v_new;
  const int32_t* append_indptr;  // [B+1] new tokens of each sequence
  const int32_t* indptr;         // page table after the append
  const int32_t* values;
  const int32_t* length_info;    // [B] last page lengths after the append
  unsigned* err;
  long long k_stride, v_stride;  // elements from token to token
  long long max_pages, nnz;
  int T, B, H_kv, P, S;
};
cudaError_t launch_append_bs(const AppendBsParams& a, int D, int in_dtype, int kv_dtype, cudaStream_t st);

// qk_norm_rope
struct QkParams {
  const void* q;
  const void* k;
  const void* q_weight;  // nullptr: no norm
  const void* k_weight;
  const int32_t* positions;
  const double* freq;    // [rd / 2] radians per position
  void* q_out;
  void* k_out;
  long long q_stride, k_stride, q_out_stride, k_out_stride;  // elements from token to token
  long long q_head, k_head, q_out_head, k_out_head;          // elements from head to head
  int T, Hq, Hk, D, rd, mode, w_dtype;
  int parts;  // warps that share a token's heads (set by the launch)
  float eps, inv_D, w_offset, attention_factor;
};
cudaError_t launch_qk_norm_rope(const QkParams& a, int dtype, int num_sms, cudaStream_t st);

cudaError_t launch_append(void* pages, const void* k_new, const void* v_new,
                          const int64_t* slot_mapping, int T, int H_kv, int D, int P,
                          long long max_pages, int in_dtype, int kv_dtype, float k_scale,
                          float v_scale, unsigned* err, const AppendRope& rope, cudaStream_t st);

}  // namespace pd
