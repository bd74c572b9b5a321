// The largest sizes that the host half of the 8-bit operators and the token
// log-probabilities accepts: every launch of such a call has fewer than 2^32
// threads, and one size more is refused.  Plain C++; no GPU, no HIP.  Prints
// "launch limits ok" and exits 0 when every expectation holds.
#include <limits.h>
#include <stdio.h>

#include <initializer_list>

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
static bool launches(unsigned long long blocks, unsigned threads) { return blocks * threads < (1ull << 32); }

// The largest n in [1, INT32_MAX] that `accepts` takes (sizes below an accepted one are accepted).
template <typename F>
static int32_t largest(F accepts) {
  long long lo = 0, hi = (long long)INT32_MAX + 1;
  while (hi - lo > 1) {
    const long long mid = (lo + hi) / 2;
    if (accepts((int32_t)mid)) lo = mid;
    else hi = mid;
  }
  return (int32_t)lo;
}

// quantize_rows_kernel: 16 lanes per format block, four blocks per group of lanes.
static bool rows_launch(unsigned long long blocks) { return launches((blocks + 63) / 64, 256); }

int main() {
  bool empty = false;
  for (int d : {1, 128, 129, 4096, 100000}) {
    auto rows = [&](int32_t R) {
      return sv::validate_quantize_rows(fake(0x1000), R, d, SPEC_BF16, fake(0x2000), fake(0x3000), &empty) == SPEC_OK;
    };
    const int32_t R = largest(rows);
    EXPECT(R > 0 && rows_launch((unsigned long long)R * sv::quant_blocks(d)));
    EXPECT(R < INT32_MAX && !rows(R + 1));
    if (d == 1) EXPECT(R == (1 << 30) - 64);

    sv::HeadQPlan p{};
    sv::HeadQWorkspace w{};
    for (int N : {1, 33, 128256}) {
      auto head = [&](int32_t M) { return sv::check_head_quantized(M, d, N, 1, N, &p, &w, &empty) == SPEC_OK; };
      const int32_t M = largest(head);
      EXPECT(M > 0 && head(M));
      EXPECT(rows_launch((unsigned long long)M * sv::quant_blocks(d)));
      const unsigned long long tiles =
          (((unsigned long long)M + p.mt - 1) / p.mt) * (((unsigned long long)N + p.nt - 1) / p.nt) * p.split;
      EXPECT(launches((tiles + 7) / 8 * 8, 512));
      EXPECT(launches(((unsigned long long)M * N + 1023) / 1024, 256));
    }
  }
  for (int E : {1, 128, 1024}) {
    sv::KvQPlan p{};
    auto read = [&](int32_t L, spec_dtype_t dt) {
      return sv::validate_kv_read_quantized(fake(0x1000), fake(0x2000), (int32_t*)fake(1ull << 40), fake(0x3000), nullptr, 2,
                                            3, L, L, E, dt, &p, &empty) == SPEC_OK;
    };
    for (spec_dtype_t dt : {(spec_dtype_t)SPEC_BF16, (spec_dtype_t)SPEC_F32}) {
      const int32_t L = largest([&](int32_t n) { return read(n, dt); });
      EXPECT(L > 0 && read(L, dt) && launches(6ull * p.chunks, 256));
      EXPECT((unsigned long long)p.chunks * p.unroll * 256 >= (unsigned long long)L * p.nb * 16);
    }
  }
  for (int V : {1, 32000, 65537, 262144})
    for (int top : {0, 20})
      for (spec_dtype_t dt : {(spec_dtype_t)SPEC_BF16, (spec_dtype_t)SPEC_F32}) {
        sv::LogprobsShape s{};
        sv::LogprobsWorkspace w{};
        auto ok = [&](int32_t N) { return sv::check_logprobs(N, V, dt, top, false, &s, &w) == SPEC_OK; };
        const int32_t N = largest(ok);
        EXPECT(N > 0 && ok(N));
        if (s.NP == 0) EXPECT(launches(N, N <= sv::kLpWideRows ? 1024 : 256));
        else EXPECT(launches((unsigned long long)N * s.NP, 256) && launches(N, N <= 768 ? 512 : 256));
      }
  if (failures) return 1;
  puts("launch limits ok");
  return 0;
}
