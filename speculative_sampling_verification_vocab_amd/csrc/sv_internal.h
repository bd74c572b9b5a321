// Internal launch interface between the C ABI layer and the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sv_host.h"
#include "sv_host_quant.h"
#include "sv_host_sample.h"
#include "sv_host_tree.h"

namespace sv {

// SAMPLE: statistics, then either decisions and sampling (s.decide) or
// sampling with the decisions in its prologue, then pick: four or three
// launches.  events[k] (if present, k < n_events) is recorded before launch k
// and events[launches] after the last one.
hipError_t launch_sample_pipeline(const VerifyShape& s, const VerifyIO& io, const VerifyWorkspace& ws,
                                  hipStream_t st, void* const* events, int n_events);
// SAMPLE_EARLY_EXIT: K + 2 launches (position i's statistics, each block
// first deciding position i - 1 of its sequence; then sampling, which decides
// position K - 1, and pick); events as above.
hipError_t launch_early_exit_pipeline(const VerifyShape& s, const VerifyIO& io, const VerifyWorkspace& ws,
                                      hipStream_t st, void* const* events, int n_events);
// GREEDY: greedy -> greedy_finalize.
hipError_t launch_greedy(const VerifyShape& s, const VerifyIO& io, const VerifyWorkspace& ws, hipStream_t st);
hipError_t launch_greedy_finalize(const VerifyShape& s, const VerifyIO& io, const VerifyWorkspace& ws,
                                  hipStream_t st);

// nsel_pos (host, nsel_period entries) set: context x uses the first
// nsel_pos[x % nsel_period] of its S cluster ids and writes compact rows of
// stride L; otherwise every context uses n_sel ids and rows of n_sel * cs.
hipError_t launch_head(const void* h, const void* W, const int32_t* cluster_ids, int B, int K, int d, int V,
                       int cluster_size, int n_sel, void* compact, void* dense, int dense_dtype,
                       hipStream_t st, const int32_t* nsel_pos = nullptr, int nsel_period = 0, int S = 0,
                       int L = 0, int compact_dtype = 0);

// Head over one shortlist shared by every row: C[M, n_sel*cs] = h[M, d] * W_S^T.
// partial (null: no K split) holds head_static_workspace_bytes(M, d, N).
hipError_t launch_head_static(const void* h, const void* W, const int32_t* cluster_ids, int M, int d, int V,
                              int cluster_size, int n_sel, void* out, int out_dtype, float* partial,
                              hipStream_t st);

// Read-only stream of bytes (a multiple of 32 KiB) for the roofline reference.
hipError_t launch_read_stream(const void* src, size_t bytes, void* sink, hipStream_t st);

// KV-cache commit: copy, then lengths and status (two launches).
hipError_t launch_kv_commit(void* cache, const void* staging, const int32_t* accepted_len, int32_t* cache_len,
                            int32_t* status, int P, int B, int K, int Lmax, int64_t row_bytes, int elem_bytes,
                            bool vec_ok, hipStream_t st);

// Rows into the 8-bit block format (one launch).
hipError_t launch_quantize_rows(const void* x, int R, int d, int dtype, void* codes, void* scales, hipStream_t st);

// Head on a quantised weight: h's rows quantised into the workspace (with
// plan.own_h by the product's blocks, with no launch), the product, and with
// plan.split > 1 the sum of the slices.
hipError_t launch_head_quantized(const void* h, const void* W_codes, const void* W_scales, const int32_t* cluster_ids,
                                 int M, int d, int V, int cluster_size, int n_sel, void* out, int out_dtype,
                                 const HeadQPlan& plan, const HeadQWorkspace& w, void* workspace, hipStream_t st);

// Quantised KV cache: commit (one launch, or two when new_len is cache_len)
// and read (one launch).
hipError_t launch_kv_commit_quantized(void* codes, void* scales, const void* staging, const int32_t* accepted_len,
                                      const int32_t* cache_len, int32_t* new_len, int32_t* status, int P, int B, int K,
                                      int Lmax, int E, int dtype, const KvQPlan& plan, hipStream_t st);
hipError_t launch_kv_read_quantized(const void* codes, const void* scales, const int32_t* cache_len, void* out,
                                    int32_t* status, int P, int B, int Lmax, int Lout, int E, int dtype,
                                    const KvQPlan& plan, hipStream_t st);

// Token log-probabilities: one launch for rows of up to kLpRowTiles tiles
// (s.NP == 0), else parts of rows, then their join and the alternatives.
hipError_t launch_logprobs(const LogprobsShape& s, const LogprobsWorkspace& w, const void* logits,
                           const int32_t* tokens, int dtype, float temperature, float* logprobs, float* entropy,
                           int32_t* top_ids, float* top_logprobs, void* workspace, hipStream_t st);

// Attention of a tree over the cache: one launch, and a second one where blocks
// share the keys of a row (plan.split > 1 or plan.ranges > 0), which joins them.
hipError_t launch_tree_attention(const AttnPointers& io, bool quantized, int B, int N, int Hq, int Hkv, int D, int L,
                                 float scale, int window, int sinks, int dtype, const AttnPlan& plan, void* workspace,
                                 hipStream_t st);

// Walk along a tree and commit of its path: one launch, or two when new_len is cache_len.
hipError_t launch_tree_commit(void* cache, const void* staging, const TreeCommitIO& io, int P, int B, int N, int L,
                              const TreeCopyPlan& plan, hipStream_t st);
hipError_t launch_tree_commit_quantized(void* codes, void* scales, const void* staging, const TreeCommitIO& io, int P,
                                        int B, int N, int L, int E, int dtype, const KvQPlan& plan, hipStream_t st);

// Tokens drawn with request settings (one launch).
hipError_t launch_sample_tokens(const void* logits, const float* uniforms, int R, int V, int dtype,
                                const SampleSettings& set, int32_t* tokens, hipStream_t st);

}  // namespace sv
