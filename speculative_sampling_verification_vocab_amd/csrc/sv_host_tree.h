// Host half of the operators of a step with a tree of drafts: geometry and
// argument checks.  Plain C++ with no HIP types, like sv_host.h.
#pragma once

#include "sv_host_quant.h"

namespace sv {

constexpr int kMaxNodes = SPEC_MAX_NODES;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int32_t kMaxLength = 1 << 30;  // cache positions: sums with depths and windows stay in int32

// ---- attention ------------------------------------------------------------------

// Launch plan of spec_tree_attention and its quantised form.  The rows of one
// KV head are its G = Hq / Hkv query heads of every node, node by node; a block
// takes `rows` of them against some of their keys: one of `split` equal pieces,
// or one of `ranges` equal parts of the keys of the whole batch.
struct AttnPlan {
  int32_t R;       // rows per (sequence, KV head)
  int32_t dp;      // head size rounded up to 64, 128 or 256
  bool shared;     // the block's waves have rows of their own and share the keys; else keys of their own
  int32_t mt;      // tiles of 16 rows per wave
  int32_t rows;    // rows per block
  int32_t groups;  // blocks that share the rows of a KV head
  int32_t split;   // blocks (per group) that share the keys of a sequence's KV head
  int32_t ranges;  // blocks (per group) that share those of the whole batch, or 0
  int32_t least;   // tiles that a range has at least
  int32_t step;    // and whose multiple it has: a tile per wave, where these have keys of their own
  int32_t span;    // keys of a tile
  unsigned grid;
  int32_t join_rows;         // rows that a wave joins
  size_t slots;              // partial results of a group
  size_t stats, acc, total;  // workspace byte offsets
};

constexpr int kAttnStage = 64;          // keys that the waves of a block share at a time
constexpr int kAttnBlocksWanted = 512;  // 2 per CU
constexpr int kAttnLeastKeys = 256;     // keys of a piece or range at least
constexpr int kAttnMostKeys = 2048;     // keys of a piece at most, where sequences differ in length

constexpr size_t kAttnJoinWaves = 16384;  // of the launch that joins partial results, where there are so many rows

// How the keys are shared out, with times at 32 query heads on 8 KV heads of 128:
//  - a block per pair of sequence and KV head up to 1024 keys (B=1 N=4 L=1000: 15.7 us, in pieces 20.3), and from
//    4096 pairs on;
//  - pieces of each pair's own keys, all found from the block's number, while the longest piece is short: a batch of
//    sequences of half to all of L takes 35 us in pieces and 40 in ranges at B=8 N=16 L=4096, 8-bit B=4 N=32 L=16384
//    59 and 66 us;
//  - ranges of the batch's keys from there on, which every length fills alike: 8-bit B=64 N=1 L=8192 takes 185 us, a
//    block per pair 214; bf16 B=64 N=64 L=8192 636 and 680.  A block has to find its range first (2 to 3 us), and most
//    have parts of two pairs.
// 384 or 768 blocks in place of 512 are slower by 7 to 30 %.
//
// Which rows a block has, in the same terms:
//  - up to 64 rows: the waves have keys of their own (B=8 N=16 L=4096 35 us, shared 39; 8-bit B=1 N=16 L=131072 80 and
//    92 on one machine), 16 rows of them where there are no more.  One rule for both types, which the 8-bit cache's
//    figure decides: bf16 values at that length would gain 5 % by sharing (119 and 113 us);
//  - from there on shared keys (8-bit B=4 N=32 L=16384 58 us, own 84), 32 rows a wave: with 64 one wave per SIMD is left
//    and B=64 N=64 L=8192 takes 815 us, not 685 (both with a slower join).

inline spec_status_t check_attention(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t L_max,
                                     int32_t window, int32_t sinks, spec_dtype_t dtype, bool aligned, AttnPlan* p,
                                     bool* empty) {
  if (!valid_dtype(dtype) || B < 0 || N < 0 || Hq < 1 || Hkv < 1 || D < 1 || L_max < 0) return SPEC_ERR_INVALID_ARG;
  if (Hq % Hkv != 0 || N > kMaxNodes || D % 8 != 0 || D > 256 || L_max > kMaxLength) return SPEC_ERR_UNSUPPORTED;
  if ((long long)Hkv * D > (1 << 22) || Hq > (1 << 22)) return SPEC_ERR_UNSUPPORTED;  // 32 rows' offsets stay in uint32
  *empty = B == 0 || N == 0;
  if (*empty) return SPEC_OK;
  size_t n = 0;
  if (!mul_fits((size_t)B * (size_t)(L_max > N ? L_max : N), (size_t)Hq * (size_t)D * elem_size(dtype), kMaxBytes, &n))
    return SPEC_ERR_UNSUPPORTED;
  p->R = N * (Hq / Hkv);
  if ((size_t)p->R > max_blocks(kBlock) * kWavesPerBlock) return SPEC_ERR_UNSUPPORTED;  // the join's waves have one each
  p->dp = D <= 64 ? 64 : D <= 128 ? 128 : 256;
  p->shared = aligned && dtype == SPEC_BF16 && p->dp <= 128 && p->R > 64;
  p->mt = !p->shared && (p->R <= 16 || p->dp == 256) ? 1 : 2;
  p->rows = 16 * p->mt * (p->shared ? kWavesPerBlock : 1);
  p->groups = (p->R + p->rows - 1) / p->rows;
  p->span = p->shared ? kAttnStage : dtype == SPEC_F32 && p->dp == 256 ? 16 : 32;
  const size_t pairs = (size_t)B * (size_t)Hkv;
  if (pairs * (size_t)p->groups > max_blocks(kBlock) / 8) return SPEC_ERR_UNSUPPORTED;
  const size_t wanted = kAttnBlocksWanted > p->groups ? (size_t)(kAttnBlocksWanted / p->groups) : 1;
  const size_t keys = (size_t)L_max + (size_t)N;  // of a pair at most
  p->least = kAttnLeastKeys / p->span;
  p->step = p->shared ? 1 : kWavesPerBlock;
  p->split = 1;
  p->ranges = 0;
  p->slots = 0;
  if (pairs < 8 * wanted && keys > 4 * kAttnLeastKeys) {
    const size_t most = pairs * (keys / kAttnLeastKeys);
    const size_t ranges = wanted < most ? wanted : most;
    if (pairs * (keys / p->span + 4) > INT32_MAX) return SPEC_ERR_UNSUPPORTED;
    p->slots = 2 * ranges;  // whatever the window
    const size_t seen = window > 0 && (size_t)window + (size_t)sinks < (size_t)L_max ? (size_t)window + sinks + N : keys;
    size_t split = wanted / pairs;
    if (split > (seen + kAttnLeastKeys - 1) / kAttnLeastKeys) split = (seen + kAttnLeastKeys - 1) / kAttnLeastKeys;
    if (split < 1) split = 1;
    if (B == 1 || seen - (size_t)N <= split * kAttnMostKeys) p->split = (int32_t)split;
    else p->ranges = (int32_t)ranges;
  }
  const size_t rows_wave = pairs * (size_t)p->R / kAttnJoinWaves;
  p->join_rows = (int32_t)(rows_wave < 1 ? 1 : rows_wave > 8 ? 8 : rows_wave);
  const size_t items = p->ranges > 0 ? (size_t)p->ranges : pairs * (size_t)p->split;
  p->grid = (unsigned)((items + 7) / 8 * 8 * p->groups);
  p->stats = p->acc = p->total = 0;
  if (p->slots > 0) {
    const size_t rows = p->slots * (size_t)p->groups * (size_t)p->rows;
    if (rows > kMaxBytes / ((size_t)D * 4 + 8)) return SPEC_ERR_UNSUPPORTED;
    p->acc = align256(rows * 8);
    p->total = p->acc + align256(rows * (size_t)D * 4);
  }
  return SPEC_OK;
}

// Workspace bytes of a call on any buffers, with any window.
inline spec_status_t attention_workspace(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t L_max,
                                         spec_dtype_t dtype, size_t* bytes) {
  AttnPlan p{};
  bool empty = false;
  size_t most = 0;
  for (int aligned = 0; aligned < 2; ++aligned) {
    const spec_status_t sc = check_attention(B, N, Hq, Hkv, D, L_max, 0, 0, dtype, aligned != 0, &p, &empty);
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
  if (!(scale > 0.0f && isfinite(scale * kLog2e)) || window < 0 || sinks < 0) return SPEC_ERR_INVALID_ARG;
  const spec_status_t sc = check_attention(B, N, Hq, Hkv, D, L_max, window, sinks, dtype, aligned, p, empty);
  if (sc != SPEC_OK) return sc;
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

// What a call writes (its output, and its workspace where it has one) is apart from what it reads and from each other;
// the output may be the queries themselves.  Of a call that validate_attention took.
inline bool attention_overlaps(const AttnPointers& a, bool quantized, int32_t B, int32_t N, int32_t Hq, int32_t Hkv,
                               int32_t D, int32_t L_max, spec_dtype_t dtype, const AttnPlan& p, const void* workspace) {
  const size_t es = elem_size(dtype), rows = (size_t)B * N, entries = (size_t)B * L_max, heads = (size_t)Hkv * D;
  const size_t out = rows * Hq * D * es, own = rows * heads * es, cache = entries * heads * (quantized ? 1 : es);
  const size_t scales = quantized ? entries * quant_blocks((int32_t)heads) : 0;
  const struct {
    const void* at;
    size_t bytes;
  } in[] = {{a.k_cache, cache}, {a.v_cache, cache}, {a.k_scales, scales}, {a.v_scales, scales}, {a.k_new, own},
            {a.v_new, own}, {a.parents, rows * 4}, {a.cache_len, (size_t)B * 4}};
  for (const auto& i : in)
    if (overlap(a.out, out, i.at, i.bytes) || overlap(workspace, p.total, i.at, i.bytes)) return true;
  return (a.out != a.q && overlap(a.out, out, a.q, out)) || overlap(workspace, p.total, a.q, out) ||
         overlap(workspace, p.total, a.out, out);
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
  if (N > kMaxNodes || (size_t)B > max_blocks(kBlock) * kWavesPerBlock) return SPEC_ERR_UNSUPPORTED;  // a wave each
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

// The cache shares a byte with the staging, an input or an output, or the staging with an output: blocks would move
// what others have written already.  Of a call that a validate_tree_commit took and that has entries to move.
inline bool tree_commit_overlaps(const void* cache, size_t cache_bytes, const void* scales, size_t scale_bytes,
                                 const void* staging, size_t staging_bytes, const TreeCommitIO& io, int32_t B,
                                 int32_t N) {
  const struct {
    const void* at;
    size_t bytes;
  } lists[] = {{io.new_len, (size_t)B * 4}, {io.accepted_len, (size_t)B * 4}, {io.out_tokens, (size_t)B * N * 4},
               {io.path, io.path ? (size_t)B * N * 4 : 0}, {io.status, io.status ? (size_t)B * 4 : 0},
               {io.cache_len, (size_t)B * 4}, {io.tokens, (size_t)B * N * 4}, {io.parents, (size_t)B * N * 4},
               {io.sampled, (size_t)B * N * 4}};
  constexpr int kOutputs = 5;
  for (int i = 0; i < (int)(sizeof(lists) / sizeof(lists[0])); ++i) {
    if (overlap(cache, cache_bytes, lists[i].at, lists[i].bytes) || overlap(scales, scale_bytes, lists[i].at, lists[i].bytes))
      return true;
    if (i < kOutputs && overlap(staging, staging_bytes, lists[i].at, lists[i].bytes)) return true;
  }
  return overlap(cache, cache_bytes, staging, staging_bytes) || overlap(scales, scale_bytes, staging, staging_bytes) ||
         overlap(cache, cache_bytes, scales, scale_bytes);
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

// Planes that a block serves with one walk: several where a block has all of a
// path and there are blocks for it.  64 planes of 256 trees of 16, entries of 2 KB:
// two planes a block 28.5 us and 29.7 in 8 bits, one 33.4 and 35.6, six 32.1 and 33.3.
constexpr size_t kTreeBlocksWanted = 8192;
inline int32_t tree_planes(int32_t P, int32_t B, uint32_t chunks) {
  const size_t n = chunks == 1 ? (size_t)P * (size_t)B / kTreeBlocksWanted : 1;
  return (int32_t)(n < 1 ? 1 : n > 8 ? 8 : n);
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
