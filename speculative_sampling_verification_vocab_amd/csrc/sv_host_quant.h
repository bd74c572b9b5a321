// Host half of the 8-bit operators and the token log-probabilities: geometry
// and argument checks.  Plain C++ with no HIP types, like sv_host.h.
#pragma once

#include "sv_host.h"

namespace sv {

constexpr int kQuantBlock = SPEC_QUANT_BLOCK;  // values that share a scale

inline int32_t quant_blocks(int32_t d) { return d / kQuantBlock + (d % kQuantBlock != 0); }

// a * b and a + b in size_t with a flag for overflow (byte counts of buffers).
inline bool mul_fits(size_t a, size_t b, size_t limit, size_t* out) {
  if (b != 0 && a > limit / b) return false;
  *out = a * b;
  return true;
}

constexpr size_t kMaxBytes = SIZE_MAX / 4;  // byte counts of one buffer; offsets then fit 63 bits

// Blocks of `threads` threads that one launch can have: the grid's threads
// are counted in 32 bits.
constexpr size_t max_blocks(int threads) { return 0xffffffffu / (unsigned)threads; }

// [p, p + bytes) and [q, q + q_bytes) share a byte.
inline bool overlap(const void* p, size_t bytes, const void* q, size_t q_bytes) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return bytes != 0 && q_bytes != 0 && a < b + q_bytes && b < a + bytes;
}

// ---- rows -----------------------------------------------------------------------

// Blocks of the format that a block of threads quantises in a long launch, four
// per group of 16 lanes; short launches take fewer.
constexpr int kRowsPerBlock = kBlock / 16 * 4;

// Format blocks that one launch quantises: 2^30 - 64 at most, whose numbers
// stay in int32 with the grid's round-up.
inline bool rows_fit(size_t blocks) { return (blocks + kRowsPerBlock - 1) / kRowsPerBlock <= max_blocks(kBlock); }

// spec_quantize_rows; *empty when there is nothing to launch.
inline spec_status_t validate_quantize_rows(const void* x, int32_t R, int32_t d, spec_dtype_t dtype,
                                            const void* codes, const void* scales, bool* empty) {
  if (!valid_dtype(dtype) || R < 0 || d < 1) return SPEC_ERR_INVALID_ARG;
  *empty = R == 0;
  if (*empty) return SPEC_OK;
  if (!x || !codes || !scales) return SPEC_ERR_INVALID_ARG;
  if ((uintptr_t)x % elem_size(dtype) || (uintptr_t)codes % 16) return SPEC_ERR_INVALID_ARG;
  return rows_fit((size_t)R * (size_t)quant_blocks(d)) ? SPEC_OK : SPEC_ERR_UNSUPPORTED;
}

// ---- drafter head ---------------------------------------------------------------

// Launch plan of spec_draft_head_quantized: the tile that a block computes and
// the number of blocks that share a tile's sum.
struct HeadQPlan {
  int tile;    // index of the compiled tile (see launch_head_quantized)
  int mt, nt;  // its rows and columns
  int split;   // blocks per tile, each over a slice of the blocks of 128
  bool own_h;  // each block quantises its slice of h itself, with no launch before it
};

constexpr int kHeadQCUs = 256;     // compute units that a grid should reach
// Slices of d where there are fewer tiles than that: at most 8, of at least four
// blocks of 128.  d = 4096, us in 1, 2, 4, 8, 16 slices: M = 128, N = 8016 (plan:
// 4): 29.2, 24.3, 23.1, 31.2, 49.2; M = 64, N = 2000 (8): 21.5, 17.4, 15.1, 15.7,
// 19.9; M = 5, N = 500 (8): 8.4, 8.5, 8.1, 8.8, 11.2.  Few rows gain nothing and
// lose up to 1.2 (M = 16, d = 1024, N = 1000, 2 slices: 7.5 against 6.3 in one).
constexpr int kHeadQMaxSplit = 8;
// Bytes of h's codes that a block quantises for itself: 192 blocks of 128, six
// for each 16 lanes, whose values wait in registers (48 a thread) while the
// tile's rows are looked up.
constexpr int kHeadQOwn = 24 << 10;
// Tiles of 256 x 256 from which more than 128 rows are cut so, us against tiles
// of 128 x 128 at d = 4096: 64 tiles (M = 1000, N = 4000) 43.7 and 33.2; 126 (M =
// 300, N = 16000) 50.8 and 55.0; 188 (M = 300, N = 24000) 65.2 and 78.3; 256 (M =
// 300, N = 32768) 67.9 and 82.4, 512 rows computed for 300 or not; 2004 (M = 1000,
// N = 128256) 525 and 826.  The larger are ahead from about 100 tiles on.
constexpr int kHeadQSquares = 200;

inline HeadQPlan head_quantized_plan(int32_t M, int32_t d, int32_t N) {
  HeadQPlan p{};
  const long long nb = quant_blocks(d);
  auto tiles = [&](int mt, int nt) {
    return ((long long)M + mt - 1) / mt * (((long long)N + nt - 1) / nt);
  };
  // The largest tile that gives the chip enough of them: what bounds a block is
  // the bytes that its compute unit can have on their way, about 90 requests of
  // 128 bytes (34 bytes a nanosecond), and every tile reads its rows of h beside
  // its rows of W.  M = 128, d = 4096: N = 128256 takes 123 us in tiles of 128 x
  // 256 and 142 in 128 x 128; N = 32768, 128 and 256 of them, 42 and 34 us.  Up to
  // 64 rows, us at N = 8016, 32768, 128256: M = 16 in 16 x 32 tiles 11.4, 28.4, 100,
  // in 32 x 64 14.4, 26.6, 104; M = 32 in 32 x 64 14.9, 26.4, 106, in 16 x 32 12.5,
  // 41.3, 148, in 64 x 128 16.3, 27.0, 109; M = 64 in 64 x 128 17.7, 28.2, 118, in
  // 32 x 64 16.5, 44.2, 144, in 128 x 128 19.5, 31.3, 124.
  if (M <= 16) p.tile = 0, p.mt = 16, p.nt = 32;
  else if (M <= 32) p.tile = 1, p.mt = 32, p.nt = 64;
  else if (M <= 64) p.tile = 2, p.mt = 64, p.nt = 128;
  else if (M <= 128 && tiles(128, 256) >= kHeadQCUs) p.tile = 4, p.mt = 128, p.nt = 256;
  else if (M > 128 && tiles(256, 256) >= kHeadQSquares) p.tile = 5, p.mt = 256, p.nt = 256;
  else p.tile = 3, p.mt = 128, p.nt = 128;
  long long s = kHeadQCUs / (tiles(p.mt, p.nt) > 0 ? tiles(p.mt, p.nt) : 1);
  if (s > kHeadQMaxSplit) s = kHeadQMaxSplit;
  if (s > nb / 4) s = nb / 4;  // at least four blocks of 128 per slice
  p.split = s < 1 ? 1 : (int)s;
  const long long slice = (nb + p.split - 1) / p.split;
  // One launch less, where every CU has at most its first two blocks (N = 8016,
  // M = 1: 10.5 against 11.2 us on the GPU, M = 5: 11.8 against 11.4, and 9.9
  // against 12.8 us on the host); more
  // rounds of blocks would each quantise h again (M = 1, N = 32768: 28.4 and 27.3 us).
  p.own_h = p.tile == 0 && tiles(p.mt, p.nt) * p.split <= 2 * kHeadQCUs && (size_t)M * (size_t)(slice + 1) * kQuantBlock <= (size_t)kHeadQOwn;
  return p;
}

// Workspace of spec_draft_head_quantized: h's codes and scales, then the
// slices' fp32 partial tiles (split > 1).
struct HeadQWorkspace {
  size_t codes, scales, partial, total;  // byte offsets
};

inline bool head_quantized_layout(int32_t M, int32_t d, int32_t N, const HeadQPlan& p, HeadQWorkspace* w) {
  const size_t nb = (size_t)quant_blocks(d);
  size_t a = 0, b = 0, c = 0;
  if (!p.own_h && (!mul_fits((size_t)M, nb * kQuantBlock, kMaxBytes, &a) || !mul_fits((size_t)M, nb, kMaxBytes, &b)))
    return false;
  if (p.split > 1 && !mul_fits((size_t)M * (size_t)N, (size_t)p.split * sizeof(float), kMaxBytes, &c)) return false;
  w->codes = 0;
  w->scales = align256(a);
  w->partial = w->scales + align256(b);
  w->total = w->partial + align256(c);
  return true;
}

// The sizes of spec_draft_head_quantized (workspace sizing and the call).
inline spec_status_t check_head_quantized(int32_t M, int32_t d, int32_t V, int32_t cluster_size, int32_t n_sel,
                                          HeadQPlan* plan, HeadQWorkspace* w, bool* empty) {
  if (M < 0 || d < 1 || V < 1 || cluster_size < 1 || n_sel < 0) return SPEC_ERR_INVALID_ARG;
  if (V % cluster_size != 0) return SPEC_ERR_UNSUPPORTED;
  if (n_sel > V / cluster_size) return SPEC_ERR_INVALID_ARG;
  *empty = M == 0 || n_sel == 0;
  if (*empty) return SPEC_OK;
  const int32_t N = n_sel * cluster_size;  // at most V
  if (M > (1 << 30) || N > (1 << 30) || d > (1 << 30)) return SPEC_ERR_UNSUPPORTED;  // a tile past the end stays in int32
  *plan = head_quantized_plan(M, d, N);
  if (!head_quantized_layout(M, d, N, *plan, w)) return SPEC_ERR_UNSUPPORTED;
  size_t out = 0, wb = 0;
  if (!mul_fits((size_t)M * (size_t)N, 4, kMaxBytes, &out)) return SPEC_ERR_UNSUPPORTED;
  if (!mul_fits((size_t)V, (size_t)quant_blocks(d) * kQuantBlock, kMaxBytes, &wb)) return SPEC_ERR_UNSUPPORTED;
  const unsigned long long tiles = (((unsigned long long)M + plan->mt - 1) / plan->mt) *
                                   (((unsigned long long)N + plan->nt - 1) / plan->nt) * plan->split;
  if (tiles + 7 > max_blocks(512) || !rows_fit((size_t)M * (size_t)quant_blocks(d))) return SPEC_ERR_UNSUPPORTED;
  if (((size_t)M * (size_t)N + 1023) / 1024 > max_blocks(256)) return SPEC_ERR_UNSUPPORTED;  // the sum of partials
  return SPEC_OK;
}

// spec_draft_head_quantized.
inline spec_status_t validate_head_quantized(const void* h, const void* W_codes, const void* W_scales,
                                             const int32_t* cluster_ids, int32_t M, int32_t d, int32_t V,
                                             int32_t cluster_size, int32_t n_sel, const void* logits,
                                             spec_dtype_t out_dtype, const void* workspace, size_t workspace_bytes,
                                             HeadQPlan* plan, HeadQWorkspace* w, bool* empty) {
  if (!valid_dtype(out_dtype)) return SPEC_ERR_INVALID_ARG;
  const spec_status_t sc = check_head_quantized(M, d, V, cluster_size, n_sel, plan, w, empty);
  if (sc != SPEC_OK || *empty) return sc;
  if (!h || !W_codes || !W_scales || !cluster_ids || !logits) return SPEC_ERR_INVALID_ARG;
  if ((uintptr_t)h % 2 || (uintptr_t)W_codes % 16 || (uintptr_t)cluster_ids % 4 ||
      (uintptr_t)logits % elem_size(out_dtype))
    return SPEC_ERR_INVALID_ARG;
  if (w->total > 0 && (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < w->total))
    return SPEC_ERR_WORKSPACE;
  return SPEC_OK;
}

// ---- KV cache -------------------------------------------------------------------

// What both cache calls launch: 8-value units of a row, whole blocks of 16.
struct KvQPlan {
  bool copies;      // there is something to move
  bool vec;         // whole 8-value units at aligned addresses
  int32_t nb;       // blocks of 128 per row
  uint32_t chunks;  // blocks of threads per (plane, sequence)
  int32_t unroll;   // units per thread
};

// Sizes shared by the cache calls: rows is the longer row count of the two
// buffers, row_units the units that one (plane, sequence) can have.
inline spec_status_t check_kv_quantized(int32_t P, int32_t B, int32_t rows_move, int32_t rows_a, int32_t rows_b,
                                        int32_t E, spec_dtype_t dtype, bool single, KvQPlan* plan) {
  const size_t planes = (size_t)P * (size_t)B;
  if (planes > max_blocks(kBlock)) return SPEC_ERR_UNSUPPORTED;
  size_t rows = 0, bytes = 0;
  if (!mul_fits(planes, (size_t)(rows_a > rows_b ? rows_a : rows_b), kMaxBytes, &rows) ||
      !mul_fits(rows, (size_t)E * elem_size(dtype), kMaxBytes, &bytes))
    return SPEC_ERR_INVALID_ARG;
  plan->copies = P > 0 && rows_move > 0 && E > 0;
  plan->vec = false;
  plan->nb = quant_blocks(E);
  plan->chunks = 0;
  plan->unroll = 1;
  if (!plan->copies) return SPEC_OK;
  const size_t units = (size_t)rows_move * (size_t)plan->nb * 16;
  if (units > 0x7fffffffu / 2) return SPEC_ERR_UNSUPPORTED;  // unit numbers stay in int32
  // Four units per thread where that still gives every CU several blocks (64 x
  // 8192 entries read as bf16: 418 us, 472 with one); fp32 values are read back
  // by one (98 us for 16 x 4096 entries, 136 with four, whose stores then cut
  // lines in two).
  plan->unroll = single ? 1 : planes * ((units + 4 * kBlock - 1) / (4 * kBlock)) >= 4 * 256 ? 4 : 1;
  plan->chunks = (uint32_t)((units + (size_t)plan->unroll * kBlock - 1) / ((size_t)plan->unroll * kBlock));
  if (plan->chunks * planes > max_blocks(kBlock)) return SPEC_ERR_UNSUPPORTED;
  return SPEC_OK;
}

// spec_kv_commit_quantized; *empty when there is nothing to launch.
inline spec_status_t validate_kv_commit_quantized(const void* codes, const void* scales, const void* staging,
                                                  const int32_t* accepted_len, const int32_t* cache_len,
                                                  const int32_t* new_len, const int32_t* status, int32_t P,
                                                  int32_t B, int32_t K, int32_t L_max, int32_t E,
                                                  spec_dtype_t dtype, KvQPlan* plan, bool* empty) {
  if (!valid_dtype(dtype)) return SPEC_ERR_INVALID_ARG;
  if (P < 0 || B < 0 || K < 0 || L_max < 0 || E < 0) return SPEC_ERR_INVALID_ARG;
  *empty = B == 0;
  if (*empty) return SPEC_OK;
  if (!accepted_len || !cache_len || !new_len) return SPEC_ERR_INVALID_ARG;
  if ((uintptr_t)accepted_len % 4 || (uintptr_t)cache_len % 4 || (uintptr_t)new_len % 4 || (uintptr_t)status % 4)
    return SPEC_ERR_INVALID_ARG;
  // Blocks read accepted_len and cache_len while others write the outputs:
  // new_len is cache_len itself (the lengths then follow in a launch of their
  // own) or apart from every input.
  const size_t lens = (size_t)B * 4;
  if (new_len != cache_len && overlap(new_len, lens, cache_len, lens)) return SPEC_ERR_INVALID_ARG;
  if (overlap(new_len, lens, accepted_len, lens)) return SPEC_ERR_INVALID_ARG;
  if (status && (overlap(status, lens, accepted_len, lens) || overlap(status, lens, cache_len, lens) ||
                 overlap(status, lens, new_len, lens)))
    return SPEC_ERR_INVALID_ARG;
  // No more rows than the cache has are committed (none, and no buffers, with L_max == 0).
  const spec_status_t sc = check_kv_quantized(P, B, K < L_max ? K : L_max, K, L_max, E, dtype, false, plan);
  if (sc != SPEC_OK || !plan->copies) return sc;
  if (!codes || !scales || !staging || (uintptr_t)staging % elem_size(dtype)) return SPEC_ERR_INVALID_ARG;
  plan->vec = E % 8 == 0 && (uintptr_t)staging % 16 == 0 && (uintptr_t)codes % 8 == 0;
  return SPEC_OK;
}

// spec_kv_read_quantized; *empty when there is nothing to launch.
inline spec_status_t validate_kv_read_quantized(const void* codes, const void* scales, const int32_t* cache_len,
                                                const void* out, const int32_t* status, int32_t P, int32_t B,
                                                int32_t L_max, int32_t L_out, int32_t E, spec_dtype_t dtype,
                                                KvQPlan* plan, bool* empty) {
  if (!valid_dtype(dtype)) return SPEC_ERR_INVALID_ARG;
  if (P < 0 || B < 0 || L_max < 0 || L_out < 0 || E < 0) return SPEC_ERR_INVALID_ARG;
  *empty = B == 0;
  if (*empty) return SPEC_OK;
  if (!cache_len || (uintptr_t)cache_len % 4 || (uintptr_t)status % 4) return SPEC_ERR_INVALID_ARG;
  if (status && overlap(status, (size_t)B * 4, cache_len, (size_t)B * 4)) return SPEC_ERR_INVALID_ARG;
  const int32_t rows = L_max < L_out ? L_max : L_out;
  const spec_status_t sc = check_kv_quantized(P, B, rows, L_max, L_out, E, dtype, dtype == SPEC_F32, plan);
  if (sc != SPEC_OK || !plan->copies) return sc;
  if (!codes || !scales || !out || (uintptr_t)out % elem_size(dtype)) return SPEC_ERR_INVALID_ARG;
  plan->vec = E % 8 == 0 && (uintptr_t)out % 16 == 0 && (uintptr_t)codes % 8 == 0;
  return SPEC_OK;
}

// ---- token log-probabilities ----------------------------------------------------

// A row is cut into tiles, one wave's 8 chunks of 64 16-byte vectors.  Tiles
// and chunks lie on a row's 16-byte grid: a row that does not begin on a
// 16-byte boundary begins inside its first vector.
struct LogprobsShape {
  int N, V;
  int vec;         // values per 16 bytes
  int tile;        // values per tile
  int NT;          // tiles per row (enough for any alignment)
  int part_tiles;  // tiles per block of four waves, and
  int NP;          // parts per row; 0: a block does a whole row
  int top;
};

constexpr int kMaxTop = SPEC_MAX_TOP;
constexpr int kChunksPerTile = 8;
// Rows of up to 16 tiles are one block's, in one launch: 48 rows of 65536 bf16
// take 10.5 us so and 12.1 us in parts, 2048 of 32000 37.0 and 39.7, 1024 of
// 65536 30.5 and 34.6; 300 of 65536, the worst, 18.2 and 17.7.  Beyond that a
// compute unit is too slow for a row of its own: 48 rows of 128256 take 17 us
// in blocks of 16 waves and 15.3 in parts.
constexpr int kLpRowTiles = 16;
// Up to so many rows, one per CU, those blocks have 16 waves, else four: 256
// rows of 32000 take 11.4 us with 16; 512 take 21.3 with 16 and 16.1 with four.
constexpr int kLpWideRows = 256;
constexpr int kLpManyRows = 768;  // rows joined by blocks of four waves from here
// Parts of rows: as many as keep every CU in blocks, of up to 16 tiles (2048 to
// 8192 of them and 8 to 16 tiles measured within 3 %).
constexpr int kLpPartsWanted = 8192;
constexpr int kLpPartTiles = 16;

struct LogprobsPart {
  double R;  // reference, in units of log 2: sums are of 2^(x * s - R)
  double z;  // sum of e = 2^(x * s - R)
  double h;  // sum of e * (x * s - R)
};

struct LogprobsWorkspace {
  size_t parts, chunks, lanes, total;  // byte offsets
};

// aligned: every row begins on a 16-byte boundary (false: any may begin anywhere).
inline spec_status_t check_logprobs(int32_t N, int32_t V, spec_dtype_t dtype, int32_t top, bool aligned,
                                    LogprobsShape* s, LogprobsWorkspace* w) {
  if (!valid_dtype(dtype) || N < 0 || V < 1 || top < 0) return SPEC_ERR_INVALID_ARG;
  if (V > (1 << 30) || top > kMaxTop) return SPEC_ERR_UNSUPPORTED;
  s->N = N;
  s->V = V;
  s->vec = 16 / (int)elem_size(dtype);
  s->tile = kWave * s->vec * kChunksPerTile;
  s->NT = (V + (aligned ? 0 : s->vec - 1) + s->tile - 1) / s->tile;
  s->top = top;
  // The plan goes by the tiles that an aligned row has, so that the alignment
  // decides nothing but NT.
  const int full = (V + s->tile - 1) / s->tile;
  const bool one = full <= kLpRowTiles;
  long long tiles = (long long)N * full / kLpPartsWanted / kWavesPerBlock * kWavesPerBlock;
  tiles = tiles < kWavesPerBlock ? kWavesPerBlock : tiles > kLpPartTiles ? kLpPartTiles : tiles;
  s->part_tiles = (int)tiles;
  s->NP = one ? 0 : (s->NT + s->part_tiles - 1) / s->part_tiles;
  if ((size_t)N * (size_t)(one ? 1 : s->NP) > max_blocks(one && N <= kLpWideRows ? 1024 : kBlock))
    return SPEC_ERR_UNSUPPORTED;
  w->parts = 0;
  w->chunks = align256((size_t)N * s->NP * sizeof(LogprobsPart));
  w->lanes = w->chunks + (top > 0 && !one ? align256((size_t)N * s->NT * kChunksPerTile * sizeof(float)) : 0);
  w->total = w->lanes + (top > 0 && !one ? align256((size_t)N * s->NP * kWave * sizeof(float)) : 0);
  return SPEC_OK;
}

// spec_token_logprobs; *empty when there is nothing to launch.
inline spec_status_t validate_logprobs(const void* logits, const int32_t* tokens, int32_t N, int32_t V,
                                       spec_dtype_t dtype, float temperature, int32_t top, const float* logprobs,
                                       const float* entropy, const int32_t* top_ids, const float* top_logprobs,
                                       const void* workspace, size_t workspace_bytes, LogprobsShape* s,
                                       LogprobsWorkspace* w, bool* empty) {
  LogprobsShape any{};
  spec_status_t sc = check_logprobs(N, V, dtype, top, false, &any, w);
  if (sc != SPEC_OK) return sc;
  const size_t need = w->total;  // what the sizing function says
  const bool aligned = (uintptr_t)logits % 16 == 0 && ((size_t)V * elem_size(dtype)) % 16 == 0;
  sc = check_logprobs(N, V, dtype, top, aligned, s, w);
  if (sc != SPEC_OK) return sc;
  // log2(e) / T must be a finite float: T at or above the least normal one.
  if (!(temperature >= 1.17549435e-38f && isfinite(temperature))) return SPEC_ERR_INVALID_ARG;
  *empty = N == 0;
  if (*empty) return SPEC_OK;
  if (!logits || !tokens || !logprobs || (top > 0 && (!top_ids || !top_logprobs))) return SPEC_ERR_INVALID_ARG;
  if ((uintptr_t)logits % elem_size(dtype) || (uintptr_t)tokens % 4 || (uintptr_t)logprobs % 4 ||
      (uintptr_t)entropy % 4 || (uintptr_t)top_ids % 4 || (uintptr_t)top_logprobs % 4)
    return SPEC_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || (uintptr_t)workspace % 256 || workspace_bytes < need)) return SPEC_ERR_WORKSPACE;
  return SPEC_OK;
}

}  // namespace sv
