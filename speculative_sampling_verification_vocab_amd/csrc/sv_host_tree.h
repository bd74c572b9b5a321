// Host half of the operators of a step with a tree of drafts: geometry and
// argument checks.  Plain C++ with no HIP types, like sv_host.h.
#pragma once

#include "sv_host_quant.h"

namespace sv {

constexpr int kMaxNodes = SPEC_MAX_NODES;
constexpr int32_t kMaxLength = 1 << 30;  // cache positions: sums with depths and windows stay in int32

// ---- attention ------------------------------------------------------------------

// Launch plan of spec_tree_attention and its quantised form.  The rows of one
// KV head are its G = Hq / Hkv query heads of every node, node by node; a block
// takes `rows` of them against one split of the keys.
struct AttnPlan {
  int32_t R;       // rows per (sequence, KV head)
  int32_t dp;      // head size rounded up to 64, 128 or 256
  bool shared;     // the block's waves have rows of their own and share the keys; else keys of their own
  int32_t mt;      // tiles of 16 rows per wave
  int32_t rows;    // rows per block
  int32_t groups;  // blocks that share the rows of a KV head
  int32_t split;   // blocks that share the keys
  size_t slots;    // B * Hkv * groups * split: partial results, and blocks but for the round-up
  unsigned grid;
  size_t stats, acc, total;  // workspace byte offsets (split > 1)
};

constexpr int kAttnStage = 64;         // keys that the waves of a block share at a time
constexpr int kAttnBlocksWanted = 512; // 2 per CU
constexpr int kAttnSplitKeys = 512;    // at least so many cache positions per split

inline spec_status_t check_attention(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t L_max,
                                     spec_dtype_t dtype, bool aligned, AttnPlan* p, bool* empty) {
  if (!valid_dtype(dtype) || B < 0 || N < 0 || Hq < 1 || Hkv < 1 || D < 1 || L_max < 0) return SPEC_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || N > kMaxNodes || D % 8 != 0 || D > 256 || L_max > kMaxLength) return SPEC_ERR_UNSUPPORTED;
  if ((long long)Hkv * D > (1 << 22) || Hq > (1 << 22)) return SPEC_ERR_UNSUPPORTED;  // 32 rows' offsets stay in uint32
  *empty = B == 0 || N == 0;
  if (*empty) return SPEC_OK;
  size_t n = 0;
  if (!mul_fits((size_t)B * (size_t)(L_max > N ? L_max : N), (size_t)Hq * (size_t)D * elem_size(dtype), kMaxBytes, &n))
    return SPEC_ERR_UNSUPPORTED;
  p->R = N * (Hq / Hkv);
  p->dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  p->shared = aligned && dtype == SPEC_BF16 && p->dp <= 128 && p->R > 64;
  p->mt = p->shared ? (p->R <= 128 ? 2 : 4) : p->R <= 16 || p->dp == 256 ? 1 : 2;
  p->rows = 16 * p->mt * (p->shared ? kWavesPerBlock : 1);
  p->groups = (p->R + p->rows - 1) / p->rows;
  const unsigned long long pairs = (unsigned long long)B * Hkv * p->groups;
  if (pairs > max_blocks(kBlock) / 64) return SPEC_ERR_UNSUPPORTED;
  long long s = (p->shared && p->mt == 4 ? kAttnBlocksWanted / 2 : kAttnBlocksWanted) / pairs;
  const long long most_splits = ((long long)L_max + N + kAttnSplitKeys - 1) / kAttnSplitKeys;
  if (s > most_splits) s = most_splits;
  p->split = s < 1 ? 1 : (int32_t)s;
  p->slots = (size_t)pairs * p->split;
  const size_t eight = ((size_t)B * Hkv * p->split + 7) / 8 * 8 * p->groups;
  if (eight > max_blocks(kBlock)) return SPEC_ERR_UNSUPPORTED;
  p->grid = (unsigned)eight;
  p->stats = p->acc = p->total = 0;
  if (p->split > 1) {
    const size_t rows = p->slots * (size_t)p->rows;
    if (rows > kMaxBytes / ((size_t)D * 4 + 8)) return SPEC_ERR_UNSUPPORTED;
    p->acc = align256(rows * 8);
    p->total = p->acc + align256(rows * (size_t)D * 4);
  }
  return SPEC_OK;
}

// Workspace bytes of a call on any buffers.
inline spec_status_t attention_workspace(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t L_max,
                                         spec_dtype_t dtype, size_t* bytes) {
  AttnPlan p{};
  bool empty = false;
  size_t most = 0;
  for (int aligned = 0; aligned < 2; ++aligned) {
    const spec_status_t sc = check_attention(B, N, Hq, Hkv, D, L_max, dtype, aligned != 0, &p, &empty);
    if (sc != SPEC_OK) return sc;
    if (!empty && p.total > most) most = p.total;
  }
  *bytes = most;
  return SPEC_OK;
}

struct AttnPointers {
  const void *q, *k_cache, *k_scales, *v_cache, *v_scales, *k_new, *v_new;
  const int32_t *parents, *cache_len;
  const void* out;
};

// spec_tree_attention (quantized: its 8-bit form).
inline spec_status_t validate_attention(const AttnPointers& a, bool quantized, int32_t B, int32_t N, int32_t Hq,
                                        int32_t Hkv, int32_t D, int32_t L_max, float scale, int32_t window,
                                        int32_t sinks, spec_dtype_t dtype, const void* workspace,
                                        size_t workspace_bytes, AttnPlan* p, bool* empty) {
  size_t need = 0;
  const spec_status_t sw = attention_workspace(B, N, Hq, Hkv, D, L_max, dtype, &need);
  if (sw != SPEC_OK) return sw;
  // Values go to shared memory in whole 16-byte pieces.
  const bool aligned = quantized || ((uintptr_t)a.k_cache % 16 == 0 && (uintptr_t)a.v_cache % 16 == 0);
  const spec_status_t sc = check_attention(B, N, Hq, Hkv, D, L_max, dtype, aligned, p, empty);
  if (sc != SPEC_OK) return sc;
  if (!(scale > 0.0f && isfinite(scale)) || window < 0 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  if (*empty) return SPEC_OK;
  if (!a.q || !a.k_new || !a.v_new || !a.parents || !a.cache_len || !a.out) return SPEC_ERR_INVALID_ARG;
  if (L_max > 0 && (!a.k_cache || !a.v_cache || (quantized && (!a.k_scales || !a.v_scales)))) return SPEC_ERR_INVALID_ARG;
  const uintptr_t es = (uintptr_t)elem_size(dtype);
  if ((uintptr_t)a.q % es || (uintptr_t)a.k_new % es || (uintptr_t)a.v_new % es || (uintptr_t)a.out % es ||
      (uintptr_t)a.parents % 4 || (uintptr_t)a.cache_len % 4)
    return SPEC_ERR_INVALID_ARG;
  if (!quantized && ((uintptr_t)a.k_cache % es || (uintptr_t)a.v_cache % es)) return SPEC_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < need)) return SPEC_ERR_WORKSPACE;
  return SPEC_OK;
}

// ---- commit of a tree's path ----------------------------------------------------

// What both commits check; the buffers of the cache are the callers'.
struct TreeCommitIO {
  const int32_t *tokens, *parents, *sampled, *cache_len;
  int32_t *new_len, *accepted_len, *out_tokens, *path, *status;
};

inline spec_status_t check_tree_commit(const TreeCommitIO& io, int32_t P, int32_t B, int32_t N, int32_t L_max,
                                       int32_t E, spec_dtype_t dtype, bool* empty) {
  if (!valid_dtype(dtype)) return SPEC_ERR_INVALID_ARG;
  if (P < 0 || B < 0 || N < 1 || L_max < 0 || E < 0) return SPEC_ERR_INVALID_ARG;
  if (N > kMaxNodes) return SPEC_ERR_UNSUPPORTED;
  *empty = B == 0;
  if (*empty) return SPEC_OK;
  const int32_t* in[] = {io.tokens, io.parents, io.sampled, io.cache_len};
  const size_t in_bytes[] = {(size_t)B * N * 4, (size_t)B * N * 4, (size_t)B * N * 4, (size_t)B * 4};
  const int32_t* out[] = {io.new_len, io.accepted_len, io.out_tokens, io.path, io.status};
  const size_t out_bytes[] = {(size_t)B * 4, (size_t)B * 4, (size_t)B * N * 4, (size_t)B * N * 4, (size_t)B * 4};
  for (const int32_t* p : in)
    if (!p || (uintptr_t)p % 4) return SPEC_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i) {
    const bool optional = i >= 3;  // path and status
    if ((!out[i] && !optional) || (uintptr_t)out[i] % 4) return SPEC_ERR_INVALID_ARG;
    if (!out[i]) continue;
    // Blocks read the inputs while others write the outputs: new_len is
    // cache_len itself (the lengths then follow in a launch of their own) or
    // apart from every input, and so is every other output.
    for (int j = 0; j < 4; ++j) {
      if (i == 0 && j == 3 && out[i] == in[j]) continue;
      if (overlap(out[i], out_bytes[i], in[j], in_bytes[j])) return SPEC_ERR_INVALID_ARG;
    }
    for (int j = 0; j < i; ++j)
      if (out[j] && overlap(out[i], out_bytes[i], out[j], out_bytes[j])) return SPEC_ERR_INVALID_ARG;
  }
  return SPEC_OK;
}

// Units (16-byte vectors or elements) of a path's entries, in chunks of one
// block; chunks is 0 where there is nothing to move.
struct TreeCopyPlan {
  int32_t unit_bytes, units;  // units per entry
  uint32_t chunks;            // blocks per (plane, sequence)
};

// Units that a thread moves: of a path through N nodes, about as many entries
// as a binary tree of that size is deep are expected; longer paths loop.
inline uint32_t tree_chunks(int32_t N, int32_t rows, size_t units, int per_thread) {
  int32_t expect = 1;
  while (expect < 31 && (1 << expect) <= N) ++expect;
  if (expect > rows) expect = rows;
  const size_t c = ((size_t)expect * units + (size_t)per_thread * kBlock - 1) / ((size_t)per_thread * kBlock);
  return (uint32_t)(c < 1 ? 1 : c > 64 ? 64 : c);
}

inline spec_status_t validate_tree_commit(const void* cache, const void* staging, const TreeCommitIO& io, int32_t P,
                                          int32_t B, int32_t N, int32_t L_max, int32_t E, spec_dtype_t dtype,
                                          TreeCopyPlan* plan, bool* empty) {
  const spec_status_t sc = check_tree_commit(io, P, B, N, L_max, E, dtype, empty);
  if (sc != SPEC_OK || *empty) return sc;
  const size_t es = elem_size(dtype), planes = (size_t)P * (size_t)B;
  size_t rows = 0, bytes = 0;
  if (!mul_fits(planes, (size_t)(L_max > N ? L_max : N), kMaxBytes, &rows) ||
      !mul_fits(rows, (size_t)E * es, kMaxBytes, &bytes))
    return SPEC_ERR_INVALID_ARG;
  plan->chunks = 0;
  plan->unit_bytes = (int32_t)es;
  plan->units = 0;
  if (P == 0 || L_max == 0 || E == 0) return SPEC_OK;
  if (!cache || !staging || (uintptr_t)cache % es || (uintptr_t)staging % es) return SPEC_ERR_INVALID_ARG;
  const size_t row = (size_t)E * es;
  if (row % 16 == 0 && (uintptr_t)cache % 16 == 0 && (uintptr_t)staging % 16 == 0) plan->unit_bytes = 16;
  plan->units = (int32_t)(row / plan->unit_bytes);
  if ((size_t)plan->units * N > 0x7fffffffu / 2) return SPEC_ERR_UNSUPPORTED;  // unit numbers stay in int32
  plan->chunks = tree_chunks(N, N < L_max ? N : L_max, (size_t)plan->units, 4);
  if (planes * plan->chunks > max_blocks(kBlock)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

inline spec_status_t validate_tree_commit_quantized(const void* codes, const void* scales, const void* staging,
                                                    const TreeCommitIO& io, int32_t P, int32_t B, int32_t N,
                                                    int32_t L_max, int32_t E, spec_dtype_t dtype, KvQPlan* plan,
                                                    bool* empty) {
  const spec_status_t sc = check_tree_commit(io, P, B, N, L_max, E, dtype, empty);
  if (sc != SPEC_OK || *empty) return sc;
  const size_t es = elem_size(dtype), planes = (size_t)P * (size_t)B;
  size_t rows = 0, bytes = 0;
  if (!mul_fits(planes, (size_t)(L_max > N ? L_max : N), kMaxBytes, &rows) ||
      !mul_fits(rows, (size_t)E * es, kMaxBytes, &bytes))
    return SPEC_ERR_INVALID_ARG;
  *plan = KvQPlan{};
  plan->copies = P > 0 && L_max > 0 && E > 0;
  plan->nb = quant_blocks(E);
  if (!plan->copies) return SPEC_OK;
  if (!codes || !scales || !staging || (uintptr_t)staging % es) return SPEC_ERR_INVALID_ARG;
  plan->vec = E % 8 == 0 && (uintptr_t)staging % 16 == 0 && (uintptr_t)codes % 8 == 0;
  if ((size_t)N * (size_t)plan->nb * 16 > 0x7fffffffu / 2) return SPEC_ERR_UNSUPPORTED;  // unit numbers stay in int32
  plan->unroll = 4;
  plan->chunks = tree_chunks(N, N < L_max ? N : L_max, (size_t)plan->nb * 16, 4);
  if (planes * plan->chunks > max_blocks(kBlock)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

}  // namespace sv
