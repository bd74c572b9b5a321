// Tokens drawn with request settings (gfx950, wave64).  A row's law after the
// temperature is w_v / sum w, w_v = exp((x_v - max x) / T).  Tokens are ranked
// by logit, equal ones by id, and kept up to the first of three cuts: the k-th
// token (top-k), the first whose cumulative weight reaches p of the top k's
// (top-p), the last with w >= m (min-p).  The token is the first kept one, by
// id, whose cumulative weight passes u times the kept weight.
//
// Weights are whole numbers: w 2^F rounded, with F such that a row's sum fits 62
// bits (44 for 262144 tokens), from an exponential in 64 bits.  Sums then do not
// depend on their order, so every pass over the row agrees with every other to the
// last bit, cuts and draws included, atomics or not; and the rounding, 2^-45 of
// the largest weight for each token, is far below the distance of a uniform
// from its nearest border but for one row in millions.
//
// A block of 16 waves does a row.  The cuts are found digit by digit in the
// ordered bits of the logits, a histogram of counts and weights per pass.

#include "sv_internal.h"
#include "sv_quant.h"

namespace sv {

namespace {

constexpr int kT = kSampleThreads;
constexpr int kSWaves = kT / kWave;
constexpr int kBins = 2048;    // bins of a digit, and chunks of a row
constexpr int kChunk = 512;    // tokens of a chunk, times a factor for rows beyond kBins chunks
constexpr float kNegInf = -__builtin_inff();

struct SampleArgs {
  const void* logits;      // [R][V]
  const float* uniforms;   // [R]
  SampleSettings set;
  int32_t* tokens;         // [R]
  int V;
  int F;                   // a weight of 1 is 2^F
};

// Bits of x in ascending order as unsigned numbers; both zeros are alike.
__device__ __forceinline__ uint32_t order_bits(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// The weight of logit x, w 2^F to the nearest whole number: 2^a in 64 bits with a =
// (x - max) log2(e) / T, by the exponential series of the fraction's
// natural logarithm (|t| <= 0.35, twelve terms: 6e-15).
struct Weight {
  double top, s;  // max x, log2(e) / T
  int F;
  __device__ __forceinline__ uint64_t operator()(float x) const {
    const double a = ((double)x - top) * s;
    if (!(a > -(double)(F + 2))) return 0;  // below half a unit
    const double n = __builtin_rint(a);
    const double t = (a - n) * 0.69314718055994530942;
    double y = 1.0 / 39916800.0;
    y = __builtin_fma(y, t, 1.0 / 3628800.0);
    y = __builtin_fma(y, t, 1.0 / 362880.0);
    y = __builtin_fma(y, t, 1.0 / 40320.0);
    y = __builtin_fma(y, t, 1.0 / 5040.0);
    y = __builtin_fma(y, t, 1.0 / 720.0);
    y = __builtin_fma(y, t, 1.0 / 120.0);
    y = __builtin_fma(y, t, 1.0 / 24.0);
    y = __builtin_fma(y, t, 1.0 / 6.0);
    y = __builtin_fma(y, t, 0.5);
    y = __builtin_fma(y, t, 1.0);
    y = __builtin_fma(y, t, 1.0);
    const double v = __builtin_ldexp(y, (int)n + F) + 4503599627370496.0;  // 2^52: the sum's low bits are v
    return (uint64_t)__double_as_longlong(v) - 0x4330000000000000ull;
  }
};

// What a block shares.
struct Shared {
  union {
    struct {
      uint32_t count[kBins];
      uint64_t mass[kBins];
    } bin;
    uint64_t sum[kBins];  // of a row's chunks
  };
  uint64_t wave[kSWaves];
  uint64_t found[4];
  float top[kSWaves];
  int bad;
};

__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor((unsigned long long)v, d);
  return v;
}

__device__ __forceinline__ uint64_t wave_scan64(uint64_t v, int lane) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint64_t w = __shfl_up((unsigned long long)v, d);
    if (lane >= d) v += w;
  }
  return v;
}

// Sum over the block; every thread gets it.
__device__ __forceinline__ uint64_t block_sum64(uint64_t v, Shared& sh) {
  v = wave_sum64(v);
  __syncthreads();
  if ((threadIdx.x & (kWave - 1)) == 0) sh.wave[threadIdx.x / kWave] = v;
  __syncthreads();
  uint64_t r = 0;
#pragma unroll
  for (int i = 0; i < kSWaves; ++i) r += sh.wave[i];
  return r;
}

// Sum of the threads before this one.
__device__ __forceinline__ uint64_t block_before64(uint64_t v, Shared& sh) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const uint64_t up_to = wave_scan64(v, lane);
  __syncthreads();
  if (lane == kWave - 1) sh.wave[w] = up_to;
  __syncthreads();
  uint64_t r = up_to - v;
  for (int i = 0; i < w; ++i) r += sh.wave[i];
  return r;
}

// The vector of tokens id .. id + n - 1 of a row; -inf past its end.
template <typename T>
__device__ __forceinline__ void load_row(const T* row, int V, int id, float (&x)[Elem<T>::kVec]) {
  constexpr int n = Elem<T>::kVec;
  if (id + n <= V) {
    const u32x4 w = load16<T, false, false>(row + id);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (sizeof(T) == 2) x[2 * q] = bf16_lo(w[q]), x[2 * q + 1] = bf16_hi(w[q]);
      else x[q] = __uint_as_float(w[q]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) x[i] = id + i < V ? to_f32(row[id + i]) : kNegInf;
  }
}

// f(x, id) for every token, a vector per thread at a time.
template <typename T, typename Fn>
__device__ __forceinline__ void for_row(const T* row, int V, Fn f) {
  constexpr int n = Elem<T>::kVec;
  for (int id = threadIdx.x * n; id < V; id += kT * n) {
    float x[n];
    load_row(row, V, id, x);
#pragma unroll
    for (int i = 0; i < n; ++i) f(x[i], id + i);
  }
}

// Sums of f(x, id) over the row's chunks of kChunk * factor tokens, in sh.sum, and over the row.
template <typename T, typename Fn>
__device__ __forceinline__ uint64_t chunk_sums(const T* row, int V, int factor, Shared& sh, Fn f) {
  constexpr int n = Elem<T>::kVec;
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int size = kChunk * factor, chunks = (V + size - 1) / size;
  __syncthreads();
  uint64_t total = 0;
  for (int c = w; c < chunks; c += kSWaves) {
    uint64_t s = 0;
    const int end = min((long long)V, (long long)(c + 1) * size);
    for (int id = c * size + lane * n; id < end; id += kWave * n) {
      float x[n];
      load_row(row, V, id, x);
#pragma unroll
      for (int i = 0; i < n; ++i) s += id + i < V ? f(x[i], id + i) : 0;
    }
    s = wave_sum64(s);
    if (lane == 0) sh.sum[c] = s;
    total += s;
  }
  return block_sum64(lane == 0 ? total : 0, sh);
}

// The smallest token up to which f sums to more than `target` (less than the row's sum), by the chunks' sums.
template <typename T, typename Fn>
__device__ __forceinline__ int locate(const T* row, int V, int factor, uint64_t target, Shared& sh, Fn f) {
  constexpr int n = Elem<T>::kVec;
  const int lane = threadIdx.x & (kWave - 1);
  const int size = kChunk * factor, chunks = (V + size - 1) / size;
  uint64_t own[kBins / kT], mine = 0;
#pragma unroll
  for (int i = 0; i < kBins / kT; ++i) {
    const int c = threadIdx.x * (kBins / kT) + i;
    own[i] = c < chunks ? sh.sum[c] : 0;
    mine += own[i];
  }
  uint64_t before = block_before64(mine, sh);
#pragma unroll
  for (int i = 0; i < kBins / kT; ++i) {
    if (before <= target && target < before + own[i]) {
      sh.found[0] = threadIdx.x * (kBins / kT) + i;
      sh.found[1] = before;
    }
    before += own[i];
  }
  __syncthreads();
  if (threadIdx.x < kWave) {
    const int c = (int)sh.found[0];
    uint64_t at = sh.found[1];
    for (int id0 = c * size; id0 < V; id0 += kWave * n) {
      const int id = id0 + lane * n;
      float x[n];
      uint64_t v[n], s = 0;
      load_row(row, V, min(id, V - 1), x);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        v[i] = id + i < V ? f(x[i], id + i) : 0;
        s += v[i];
      }
      const uint64_t up_to = at + wave_scan64(s, lane);
      const uint64_t hit = __ballot(up_to > target);
      if (hit != 0) {
        if (lane == __ffsll((unsigned long long)hit) - 1) {
          uint64_t y = up_to - s;
          int token = id;
#pragma unroll
          for (int i = 0; i < n; ++i) {
            y += v[i];
            if (y <= target) token = id + i + 1;
          }
          sh.found[2] = token;
        }
        break;
      }
      at = __shfl((unsigned long long)up_to, kWave - 1);
    }
  }
  __syncthreads();
  return (int)sh.found[2];
}

// A cut in the ranking: tokens above `key`, and the first `ties` by id at it.
struct Cut {
  uint32_t key;
  uint64_t ties;
  uint64_t mass;  // of the tokens kept
};

// The cut at which the ranked counts (by_mass false) or weights reach target.  Three
// passes over the row, each a digit of the keys that share the digits before.
// share >= 0: the target is that share of the row's weight, known after the first.
template <typename T>
__device__ __forceinline__ Cut find_cut(const T* row, int V, const Weight& weight, bool by_mass, uint64_t target,
                                        double share, Shared& sh) {
  uint32_t prefix = 0;
  uint64_t above_n = 0, above_m = 0;
  int shift = 21;
  uint32_t digits = 2048;
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kT) sh.bin.count[i] = 0, sh.bin.mass[i] = 0;
    __syncthreads();
    for_row(row, V, [&](float x, int id) {
      const uint32_t k = order_bits(x);
      if (id < V && (level == 0 || k >> (shift + (level == 1 ? 11 : 10)) == prefix)) {
        const uint32_t b = k >> shift & (digits - 1);
        const uint64_t w = weight(x);
        atomicAdd(&sh.bin.count[b], 1u);
        if (w != 0) atomicAdd((unsigned long long*)&sh.bin.mass[b], (unsigned long long)w);
      }
    });
    __syncthreads();
    // Thread t takes the bins kBins - 1 - 2 t and the one below: descending order.
    constexpr int kPer = kBins / kT;
    uint64_t n[kPer], m[kPer], n_all = 0, m_all = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int b = kBins - 1 - (int)threadIdx.x * kPer - i;
      n[i] = sh.bin.count[b];
      m[i] = sh.bin.mass[b];
      n_all += n[i];
      m_all += m[i];
    }
    if (level == 0 && share >= 0.0) {
      const double t = __builtin_ceil(share * (double)block_sum64(m_all, sh));
      target = t < 1.0 ? 1 : (uint64_t)t;
    }
    uint64_t n_before = above_n + block_before64(n_all, sh), m_before = above_m + block_before64(m_all, sh);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint64_t lo = by_mass ? m_before : n_before, hi = lo + (by_mass ? m[i] : n[i]);
      if (lo < target && target <= hi) {
        sh.found[0] = kBins - 1 - (int)threadIdx.x * kPer - i;
        sh.found[1] = n_before;
        sh.found[2] = m_before;
      }
      n_before += n[i];
      m_before += m[i];
    }
    __syncthreads();
    prefix = level == 2 ? prefix << 10 | (uint32_t)sh.found[0] : prefix << 11 | (uint32_t)sh.found[0];
    above_n = sh.found[1];
    above_m = sh.found[2];
    if (level == 0) shift = 10;
    else shift = 0, digits = 1024;
  }
  const uint64_t w = weight(order_value(prefix));
  Cut c;
  c.key = prefix;
  c.ties = by_mass ? (target - above_m + w - 1) / w : target - above_n;
  c.mass = above_m + c.ties * w;
  return c;
}

template <typename T>
__global__ void __launch_bounds__(kT) sample_tokens_kernel(SampleArgs a) {
  __shared__ Shared sh;
  const int r = blockIdx.x, V = a.V;
  const T* row = static_cast<const T*>(a.logits) + (size_t)r * (size_t)V;
  const float temperature = a.set.temperature.rows ? a.set.temperature.rows[r] : a.set.temperature.all;
  const int k = a.set.top_k.rows ? a.set.top_k.rows[r] : a.set.top_k.all;
  const float p = a.set.top_p.rows ? a.set.top_p.rows[r] : a.set.top_p.all;
  const float m = a.set.min_p.rows ? a.set.min_p.rows[r] : a.set.min_p.all;
  const float u = a.uniforms[r];
  const int factor = (int)(((long long)V + (long long)kChunk * kBins - 1) / ((long long)kChunk * kBins));

  if (threadIdx.x == 0) sh.bad = 0, sh.found[0] = sh.found[1] = sh.found[2] = 0;
  __syncthreads();
  float top = kNegInf;
  bool bad = false;
  for_row(row, V, [&](float x, int) {
    top = fmaxf(top, x);
    bad |= x != x;
  });
  top = wave_max(top);
  if ((threadIdx.x & (kWave - 1)) == 0) sh.top[threadIdx.x / kWave] = top;
  if (bad) sh.bad = 1;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kSWaves; ++i) top = fmaxf(top, sh.top[i]);
  // A fault of the row or of its settings: comparisons that NaN fails.
  if (sh.bad || !(fabsf(top) < __builtin_inff()) || !(temperature >= 0.0f && temperature < __builtin_inff()) || p != p ||
      m != m || !(u >= 0.0f && u < 1.0f)) {
    if (threadIdx.x == 0) a.tokens[r] = -1;
    return;
  }
  if (temperature == 0.0f) {
    auto is_top = [&](float x, int) -> uint64_t { return x == top; };
    chunk_sums(row, V, factor, sh, is_top);
    const int token = locate(row, V, factor, 0, sh, is_top);
    if (threadIdx.x == 0) a.tokens[r] = token;
    return;
  }
  Weight weight;
  weight.top = top;
  weight.s = 1.4426950408889634074 / (double)temperature;
  weight.F = a.F;
  const bool by_k = k >= 1 && k < V, by_p = p < 1.0f, by_m = m > 0.0f;
  Cut cut;
  cut.key = 0;
  cut.ties = ~0ull;
  auto narrow = [&](const Cut& c) {
    if (c.key > cut.key) cut = c;
    else if (c.key == cut.key && c.ties < cut.ties) cut.ties = c.ties;
  };
  uint64_t mass = 0;
  if (by_k) {
    const Cut c = find_cut(row, V, weight, false, (uint64_t)k, -1.0, sh);
    mass = c.mass;
    narrow(c);
  }
  if (by_p) {
    const double t = by_k ? __builtin_ceil((double)p * (double)mass) : 0.0;
    narrow(find_cut(row, V, weight, true, t < 1.0 ? 1 : (uint64_t)t, by_k ? -1.0 : p > 0.0f ? (double)p : 0.0, sh));
  }
  if (by_m) {
    // w >= m: x >= max + T ln m, as the least float that is.
    const double least = (double)top + (double)temperature * log((double)fminf(m, 1.0f));
    float f = (float)least;
    if ((double)f < least) f = order_value(order_bits(f) + 1);
    Cut c;
    c.key = order_bits(f);
    c.ties = ~0ull;
    c.mass = 0;
    narrow(c);
  }
  int last_tie = V;  // tokens at the cut's key are kept up to this one
  if (cut.ties != ~0ull) {
    auto tie = [&](float x, int) -> uint64_t { return order_bits(x) == cut.key; };
    const uint64_t n = chunk_sums(row, V, factor, sh, tie);
    if (cut.ties < n) last_tie = locate(row, V, factor, cut.ties - 1, sh, tie);
  }
  auto kept = [&](float x, int id) -> uint64_t {
    const uint32_t key = order_bits(x);
    return key > cut.key || (key == cut.key && id <= last_tie) ? weight(x) : 0;
  };
  const uint64_t total = chunk_sums(row, V, factor, sh, kept);
  const int token = locate(row, V, factor, (uint64_t)((double)u * (double)total), sh, kept);
  if (threadIdx.x == 0) a.tokens[r] = token;
}

}  // namespace

hipError_t launch_sample_tokens(const void* logits, const float* uniforms, int R, int V, int dtype,
                                const SampleSettings& set, int32_t* tokens, hipStream_t st) {
  SampleArgs a{};
  a.logits = logits;
  a.uniforms = uniforms;
  a.set = set;
  a.tokens = tokens;
  a.V = V;
  int bits = 0;
  while ((1ll << bits) < V) ++bits;
  a.F = 62 - bits < 50 ? 62 - bits : 50;
  if (dtype == 1) hipLaunchKernelGGL(sample_tokens_kernel<uint16_t>, dim3((unsigned)R), dim3(kT), 0, st, a);
  else hipLaunchKernelGGL(sample_tokens_kernel<float>, dim3((unsigned)R), dim3(kT), 0, st, a);
  return hipGetLastError();
}

}  // namespace sv
