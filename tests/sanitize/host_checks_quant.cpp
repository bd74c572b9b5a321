// Exercises the host half of the 8-bit operators and the token log-probabilities
// (sv_host_quant.h: launch plans, workspace layouts and argument checks) for
// the AddressSanitizer / UndefinedBehaviorSanitizer build of the CPU test suite.
// Plain C++; no GPU, no HIP.  Prints "host checks ok" and exits 0 when every
// expectation holds.
#include <limits.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "../../speculative_sampling_verification_vocab_amd/csrc/sv_host_quant.h"

static int failures = 0;
#define EXPECT(cond)                                                                 \
  do {                                                                               \
    if (!(cond)) {                                                                   \
      fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, __LINE__, #cond); \
      ++failures;                                                                    \
    }                                                                                \
  } while (0)

static void* fake(uintptr_t a) { return reinterpret_cast<void*>(a); }

// Every part of a workspace, written to its end in a buffer of exactly the
// size that the sizing function says.
static void log_prob_workspaces() {
  const int Ns[] = {0, 1, 5, 48, 256, 257, 768, 769, 2048};
  const int Vs[] = {1, 7, 33, 4096, 32000, 32768, 50257, 65536, 65537, 131072, 131073, 262144, 600003, 1 << 20};
  for (int N : Ns)
    for (int V : Vs)
      for (int dt = 0; dt < 2; ++dt)
        for (int top = 0; top <= 32; top += 16) {
          sv::LogprobsShape any{}, s{};
          sv::LogprobsWorkspace w{};
          EXPECT(sv::check_logprobs(N, V, (spec_dtype_t)dt, top, false, &any, &w) == SPEC_OK);
          const size_t need = w.total;
          for (int aligned = 0; aligned < 2; ++aligned) {
            EXPECT(sv::check_logprobs(N, V, (spec_dtype_t)dt, top, aligned != 0, &s, &w) == SPEC_OK);
            EXPECT(w.total <= need);  // an aligned row never needs more
            EXPECT((long long)s.NT * s.tile >= V + (aligned ? 0 : s.vec - 1));
            EXPECT((s.NP == 0) == (any.NP == 0));
            if (s.NP > 0) EXPECT((long long)s.NP * s.part_tiles >= s.NT && s.part_tiles % sv::kWavesPerBlock == 0);
            if (s.NP == 0) EXPECT(s.NT <= sv::kLpRowTiles + 1);
            if (s.NP == 0 || need == 0 || need > ((size_t)32 << 20)) continue;
            unsigned char* b = static_cast<unsigned char*>(malloc(need));
            memset(b + w.parts, 1, (size_t)N * s.NP * sizeof(sv::LogprobsPart));
            if (top > 0) {
              EXPECT(w.chunks >= (size_t)N * s.NP * sizeof(sv::LogprobsPart));
              memset(b + w.chunks, 2, (size_t)N * s.NT * sv::kChunksPerTile * sizeof(float));
              EXPECT(w.lanes >= w.chunks + (size_t)N * s.NT * sv::kChunksPerTile * sizeof(float));
              memset(b + w.lanes, 3, (size_t)N * s.NP * sv::kWave * sizeof(float));
            }
            free(b);
          }
        }
  sv::LogprobsShape s{};
  sv::LogprobsWorkspace w{};
  EXPECT(sv::check_logprobs(INT32_MAX, 1 << 30, SPEC_BF16, 32, false, &s, &w) == SPEC_ERR_UNSUPPORTED);
  EXPECT(sv::check_logprobs(INT32_MAX, 1, SPEC_BF16, 0, false, &s, &w) == SPEC_ERR_UNSUPPORTED);
  EXPECT(sv::check_logprobs(1, INT32_MAX, SPEC_F32, 0, false, &s, &w) == SPEC_ERR_UNSUPPORTED);
  EXPECT(sv::check_logprobs(1, INT32_MIN, SPEC_F32, 0, false, &s, &w) == SPEC_ERR_INVALID_ARG);
}

static void head_plans() {
  const int Ms[] = {1, 2, 5, 16, 17, 32, 33, 64, 65, 128, 129, 256, 257, 1792, 5000};
  const int ds[] = {1, 127, 128, 129, 1000, 4096, 8192, 16512, 100000};
  const int Ns[] = {1, 31, 32, 33, 500, 8016, 32768, 65537, 128256};
  for (int M : Ms)
    for (int d : ds)
      for (int N : Ns) {
        sv::HeadQPlan p{};
        sv::HeadQWorkspace w{};
        bool empty = true;
        const spec_status_t sc = sv::check_head_quantized(M, d, N, 1, N, &p, &w, &empty);
        EXPECT(sc == SPEC_OK && !empty);
        const int nb = sv::quant_blocks(d);
        EXPECT(p.split >= 1 && p.split <= sv::kHeadQMaxSplit && (p.split == 1 || nb / p.split >= 4));
        EXPECT(p.mt >= 16 && p.nt >= 32);
        const int slice = (nb + p.split - 1) / p.split;
        if (p.own_h) EXPECT(M <= 16 && (size_t)M * (slice + 1) * 128 <= (size_t)sv::kHeadQOwn);
        if (!p.own_h) EXPECT(w.scales >= (size_t)M * nb * 128 && w.partial >= w.scales + (size_t)M * nb);
        if (p.split > 1) EXPECT(w.total >= w.partial + (size_t)p.split * M * N * sizeof(float));
        EXPECT(p.own_h == false || p.split > 1 || w.total == 0);
      }
  sv::HeadQPlan p{};
  sv::HeadQWorkspace w{};
  bool empty = false;
  EXPECT(sv::check_head_quantized(INT32_MAX, INT32_MAX, INT32_MAX, 1, INT32_MAX, &p, &w, &empty) != SPEC_OK);
  EXPECT(sv::check_head_quantized(INT32_MAX, 1, INT32_MAX, 1, INT32_MAX, &p, &w, &empty) != SPEC_OK);
  EXPECT(sv::check_head_quantized(1, 1 << 30, 1, 1, 1, &p, &w, &empty) == SPEC_OK);
  EXPECT(sv::check_head_quantized(1, INT32_MAX, 1, 1, 1, &p, &w, &empty) == SPEC_ERR_UNSUPPORTED);
  EXPECT(sv::check_head_quantized(-1, 1, 1, 1, 1, &p, &w, &empty) == SPEC_ERR_INVALID_ARG);
  EXPECT(sv::check_head_quantized(1, 1, 10, 3, 1, &p, &w, &empty) == SPEC_ERR_UNSUPPORTED);
}

static void caches() {
  sv::KvQPlan p{};
  bool empty = false;
  auto commit = [&](int P, int B, int K, int L, int E, spec_dtype_t dt) {
    return sv::validate_kv_commit_quantized(fake(0x1000), fake(0x2000), fake(0x3000), (int32_t*)fake(1ull << 40),
                                            (int32_t*)fake(1ull << 41), (int32_t*)fake(1ull << 42), nullptr, P, B, K, L,
                                            E, dt, &p, &empty);
  };
  EXPECT(commit(64, 256, 7, 64, 1024, SPEC_BF16) == SPEC_OK && p.vec && p.copies && p.nb == 8);
  EXPECT((size_t)p.chunks * p.unroll * 256 >= 7u * 8 * 16);
  EXPECT(commit(1, 1, 1, 1, 1, SPEC_F32) == SPEC_OK && !p.vec && p.chunks == 1);
  EXPECT(commit(2, 1, 0, 1, 1, SPEC_F32) == SPEC_OK && !p.copies);
  EXPECT(commit(INT32_MAX, INT32_MAX, 1, 1, 1, SPEC_F32) != SPEC_OK);
  EXPECT(commit(1, 1, INT32_MAX, INT32_MAX, INT32_MAX, SPEC_F32) != SPEC_OK);
  EXPECT(commit(1, 1, INT32_MAX, INT32_MAX, 1, SPEC_F32) == SPEC_ERR_UNSUPPORTED);
  EXPECT(commit(INT32_MIN, 1, 1, 1, 1, SPEC_F32) == SPEC_ERR_INVALID_ARG);
  auto read = [&](int P, int B, int L, int Lo, int E, spec_dtype_t dt) {
    return sv::validate_kv_read_quantized(fake(0x1000), fake(0x2000), (int32_t*)fake(1ull << 40), fake(0x3000), nullptr,
                                          P, B, L, Lo, E, dt, &p, &empty);
  };
  EXPECT(read(2, 64, 8192, 8192, 1024, SPEC_BF16) == SPEC_OK && p.unroll == 4);
  EXPECT(read(2, 64, 8192, 8192, 1024, SPEC_F32) == SPEC_OK && p.unroll == 1);
  EXPECT((size_t)p.chunks * 256 >= 8192u * 8 * 16);
  EXPECT(read(2, 1, INT32_MAX, INT32_MAX, 1024, SPEC_BF16) == SPEC_ERR_UNSUPPORTED);
  EXPECT(read(2, 1, INT32_MAX, 3, 1024, SPEC_BF16) == SPEC_OK);
  EXPECT(read(2, 1, 0, 3, 1024, SPEC_BF16) == SPEC_OK && !p.copies);

  size_t out = 0;
  EXPECT(!sv::mul_fits(SIZE_MAX, 2, SIZE_MAX, &out) && sv::mul_fits(SIZE_MAX, 0, 1, &out));
  EXPECT(sv::overlap(fake(100), 8, fake(107), 1) && !sv::overlap(fake(100), 8, fake(108), 8));
  EXPECT(!sv::overlap(fake(100), 0, fake(100), 8));
  EXPECT(sv::validate_quantize_rows(fake(0x10), INT32_MAX, INT32_MAX, SPEC_BF16, fake(0x100), fake(0x200), &empty) ==
         SPEC_ERR_UNSUPPORTED);
  EXPECT(sv::quant_blocks(INT32_MAX) == (1 << 24));
}

int main() {
  log_prob_workspaces();
  head_plans();
  caches();
  if (failures) return 1;
  puts("host checks ok");
  return 0;
}
