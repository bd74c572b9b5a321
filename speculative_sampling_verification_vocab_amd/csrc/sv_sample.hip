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
// A block does a row, in one launch.  Its first pass over the row has the largest
// logit and what the settings ask for:
//  - top-k, or min-p alone: the tokens above a bound that at least k of them
//    reach (the k-th largest of disjoint sets of tokens), as a list in shared
//    memory, which is then ranked and cut;
//  - top-p over the whole row: bf16 logits as counts per value, in a table of 30
//    octaves of both signs, so that exact sums per value give the cut with no
//    second pass; fp32 ones as weights per upper half, and then those tokens
//    alone that share the cut's half;
//  - what neither holds (ties past the list, logits outside the octaves): the
//    cut digit by digit in the ordered bits, a histogram of counts and weights
//    per pass over the row.  One logit other than 0 but nearer to it than 2^-20
//    sends a row there, which costs bf16 rows several times the table's time
//    (below); logits of deviation 2.5 around 0 have one in 4 % of rows of 128256
//    and 8 % of 262144.  So does a temperature at which -2^10 has weight (from
//    about 30 on) where the row has values of -2^10 or below, or the last
//    vectors of its read are filled up with -inf behind its end.
// A last pass over the row (out of the L2 or the last level of cache, where a
// row fits) sums the kept weights in chunks, and the chunk that the uniform
// falls into is scanned for its token.  A list needs no such pass.
//
// Measured (event times of calls one after the other; floor: the logits' bytes
// at 6.4 TB/s):
//   2048 x 262144 bf16    greedy 178 us, top 50 195, top-p 430 to 490, all kept 373; floor 168.  The first pass runs at
//                         6 TB/s where nothing is counted; counting costs an LDS atomic per kept token, and the
//                         draw's pass reads the row again from memory
//   64 x 128256 bf16      greedy 9.6 us, top 50 21, top-p 42, all kept 29: a row per CU on a quarter of the CUs, bound
//                         by what one CU reads and by the barriers of the scans
//   1 x 32000 fp32        12 us for top 50: latency of a chain of 4 to 6 barriers and two reads
//   digit by digit        64 x 128256 bf16, top-p, 151 us if one row goes so and 157 if all do, where the table takes 40;
//                         2048 x 262144 460 us and 2260, by table 426.  fp32 top-p takes 160 to 165 us either way

#include "sv_internal.h"
#include "sv_quant.h"

namespace sv {

namespace {

constexpr int kBins = 2048;    // bins of a digit
constexpr int kChunk = 2048;   // tokens of a chunk, times a factor for rows of more than
constexpr int kChunks = 512;   // chunks
constexpr int kLoadsT = 4;     // 16-byte vectors of a thread's piece of a segment
constexpr int kList = 4096;    // candidates
// So many are ranked by counting, with every thread of a block of 16 waves, and the others sorted: top 200 with
// top-p on 64 rows of 128256 35 us and 41 sorted, top 50 21 and 28.  With eight waves counting pays for fewer: top
// 100 on 300 rows 43 us and 48 sorted, top 200 with top-p 70 counted and 57 sorted.
constexpr int kRanked = 512, kRankedFewer = 256;
// Where less than one token in so many is kept, weights are computed for those alone, and else taken from a table of
// the bf16 values' weights: 64 rows of 128256, all kept 29 us and 40 computed; top-p of 0.9 at T = 0.5 34 and 39.
constexpr int kSparse = 256;
// Values by sign and magnitude, in their upper 16 bits (a bf16 value itself): 30
// octaves, a bin for zero and what is smaller, and one for what is larger.
constexpr int kOctaves = 30, kOctave0 = 107;  // from 2^-20 to 2^10
constexpr int kLeast = kOctave0 * 128;        // upper bits of 2^-20
constexpr int kHuge = kOctaves * 128 + 1, kHalf = kHuge + 1, kTable = 2 * kHalf;
constexpr float kNegInf = -__builtin_inff();
template <typename T>
constexpr uint32_t kNinfOf = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;

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
// (x - max) log2(e) / T, as 2^n (1 + r q(r)), n the nearest whole number to a and q the
// polynomial that takes the values of (2^r - 1) / r at ten Chebyshev points of [-1/2, 1/2]
// (relative error of the power 5.7e-16; 1 at r = 0).  Equal logits have equal
// weights wherever they are computed, and the largest has 2^F exactly.
struct Weight {
  double top, s;  // max x, log2(e) / T
  int F;
  __device__ __forceinline__ uint64_t operator()(float x) const {
    const double a = ((double)x - top) * s;
    const double n = a + 6755399441055744.0;  // 1.5 * 2^52: the sum's low bits are the whole number
    const double r = a - (n - 6755399441055744.0);
    double y = 7.070977866508139e-09;
    y = __builtin_fma(y, r, 1.0205905413765595e-07);
    y = __builtin_fma(y, r, 1.3215451633221434e-06);
    y = __builtin_fma(y, r, 1.5252672924850737e-05);
    y = __builtin_fma(y, r, 1.5403530424776529e-04);
    y = __builtin_fma(y, r, 1.3333558200794592e-03);
    y = __builtin_fma(y, r, 9.618129107618665e-03);
    y = __builtin_fma(y, r, 5.550410866465167e-02);
    y = __builtin_fma(y, r, 2.4022650695910075e-01);
    y = __builtin_fma(y, r, 6.931471805599462e-01);
    y = __builtin_fma(y, r, 1.0);
    // Times 2^(n + F) in the exponent; added to 2^52, the low bits are the nearest whole number.
    const int hi = __double2hiint(y) + ((__double2loint(n) + F) << 20);
    const double v = __hiloint2double(hi, __double2loint(y)) + 4503599627370496.0;
    const uint64_t w = (uint64_t)(uint32_t)(__double2hiint(v) - 0x43300000) << 32 | (uint32_t)__double2loint(v);
    return a > -(double)(F + 2) ? w : 0;  // less than a quarter of a unit otherwise
  }
};

// A value that all lanes have, in scalar registers.
__device__ __forceinline__ float uniform(float x) { return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x))); }
__device__ __forceinline__ double uniform(double x) {
  return __hiloint2double(__builtin_amdgcn_readfirstlane(__double2hiint(x)), __builtin_amdgcn_readfirstlane(__double2loint(x)));
}

// What a block shares.
template <typename T>
struct Shared {
  union {
    struct {
      uint32_t count[kBins];
      uint64_t mass[kBins];
    } bin;
    uint64_t list[kList];    // candidates
    uint32_t table[kTable];
    uint64_t mass[kTable];   // fp32: the weights in the table's bins; bf16: the weights of its values
  };
  uint64_t chunk_sum[kChunks];   // weights above the cut
  uint32_t chunk_tie[kChunks];   // and tokens at it
  uint64_t wave[2][16];
  uint64_t found[4];
  uint64_t votes[2][16];
  float lanes[16][kWave];
  float top[2][16];
  uint64_t best;
  alignas(16) uint32_t end[4];
  int bad, tiny, low, count, cut;
};

template <int kCtrl, int kRowMask>
__device__ __forceinline__ uint64_t moved(uint64_t v) {
  return (uint64_t)(uint32_t)dpp::mov<kCtrl, kRowMask>(0, (int)(v >> 32)) << 32 | (uint32_t)dpp::mov<kCtrl, kRowMask>(0, (int)v);
}

// Inclusive sums over the lanes, as in wave_inclusive_scan, and their total.
__device__ __forceinline__ uint64_t wave_scan64(uint64_t v) {
  v += moved<dpp::kShr1, 0xf>(v);
  v += moved<dpp::kShr2, 0xf>(v);
  v += moved<dpp::kShr4, 0xf>(v);
  v += moved<dpp::kShr8, 0xf>(v);
  v += moved<dpp::kBcast15, 0xa>(v);
  v += moved<dpp::kBcast31, 0xc>(v);
  return v;
}
__device__ __forceinline__ uint64_t wave_sum64(uint64_t v) {
  v = wave_scan64(v);
  return (uint64_t)(uint32_t)dpp::lane63((int)(v >> 32)) << 32 | (uint32_t)dpp::lane63((int)v);
}

// Sum of the threads before this one, and of all.  The waves' sums alternate between two buffers (turn), so that one
// barrier is enough.
template <int kT, typename T>
__device__ __forceinline__ uint64_t block_scan64(uint64_t v, uint64_t& total, int& turn, Shared<T>& sh) {
  constexpr int kWaves = kT / kWave;
  const int lane = threadIdx.x & (kWave - 1), w = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const uint64_t up_to = wave_scan64(v);
  if (lane == kWave - 1) sh.wave[turn][w] = up_to;
  __syncthreads();
  const uint64_t all = wave_scan64(lane < kWaves ? sh.wave[turn][lane] : 0);
  turn ^= 1;
  auto at = [&](int i) {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(all >> 32), i) << 32 | (uint32_t)__builtin_amdgcn_readlane((int)all, i);
  };
  total = at(kWaves - 1);
  return (w > 0 ? at(w - 1) : 0) + up_to - v;
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
template <typename T, int kT, typename Fn>
__device__ __forceinline__ void for_row(const T* row, int V, Fn f) {
  constexpr int n = Elem<T>::kVec;
  for (int id = threadIdx.x * n; id < V; id += kT * n) {
    float x[n];
    load_row(row, V, id, x);
#pragma unroll
    for (int i = 0; i < n; ++i) f(x[i], id + i);
  }
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
template <typename T, int kT>
__device__ __forceinline__ Cut find_cut(const T* row, int V, const Weight& weight, bool by_mass, uint64_t target,
                                        double share, int& turn, Shared<T>& sh) {
  uint32_t prefix = 0;
  uint64_t above_n = 0, above_m = 0;
  int shift = 21;
  uint32_t digits = 2048;
#pragma unroll 1
  for (int level = 0; level < 3; ++level) {
    __syncthreads();
    for (int i = threadIdx.x; i < kBins; i += kT) sh.bin.count[i] = 0, sh.bin.mass[i] = 0;
    __syncthreads();
    for_row<T, kT>(row, V, [&](float x, int id) {
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
    uint64_t row_n, row_m;
    uint64_t n_before = above_n + block_scan64<kT>(n_all, row_n, turn, sh);
    uint64_t m_before = above_m + block_scan64<kT>(m_all, row_m, turn, sh);
    if (level == 0 && share >= 0.0) {
      const double t = __builtin_ceil(share * (double)row_m);
      target = t < 1.0 ? 1 : (uint64_t)t;
    }
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

// ---- the table ------------------------------------------------------------------

// Bin of a value by its upper 16 bits: zero first, then magnitudes, of either sign.
__device__ __forceinline__ int table_bin(uint32_t b) {
  const int m = (int)(b & 0x7fffu);
  return min(max(m, kLeast - 1), kLeast - 1 + kHuge) - (kLeast - 1) + (b & 0x8000u ? kHalf : 0);
}

// The same for two bf16 values at once, as byte offsets of bins of `size` bytes.
template <int size>
__device__ __forceinline__ uint32_t table_offsets(uint32_t w) {
  static_assert(size * kTable < 65536, "16 bits");
  typedef uint16_t halves __attribute__((ext_vector_type(2)));
  const halves m = __builtin_bit_cast(halves, w & 0x7fff7fffu), sign = __builtin_bit_cast(halves, w) >> 15;
  const halves lo = {kLeast - 1, kLeast - 1}, hi = {kLeast - 1 + kHuge, kLeast - 1 + kHuge};
  const halves half = {size * kHalf, size * kHalf}, bytes = {size, size};
  const halves t = __builtin_elementwise_min(__builtin_elementwise_max(m, lo), hi) - lo;
  return __builtin_bit_cast(uint32_t, (halves)(t * bytes + sign * half));
}

// The upper 16 bits that a bin stands for, and the bin at a place in descending order of values (zeros of both
// signs are counted in the first of their two).
__device__ __forceinline__ uint32_t table_value(int bin) {
  const int t = bin < kHalf ? bin : bin - kHalf;
  return (uint32_t)(t == 0 ? 0 : kLeast - 1 + t) | (bin < kHalf ? 0u : 0x8000u);
}
__device__ __forceinline__ int table_at(int place) { return place < kHalf ? kHuge - place : place; }

// A border in the table: its bin, what lies above it, and (by count or weight) the row's total.
struct Border {
  int bin;
  uint64_t above_n, above_m, total_m;
};

// The bin, from the highest down, at which counts (by_mass false) or weights reach target, or with share >=
// 0 that share of the total weight.  count(bin) and mass(bin, count) give a bin's; at most `target` must be there.
template <int kT, typename T, typename Bin, typename Mass>
__device__ __forceinline__ Border find_border(const Bin* table, bool by_mass, uint64_t target, double share, int& turn, Shared<T>& sh, Mass mass) {
  constexpr int kPer = (kTable + kT - 1) / kT;
  uint64_t n = 0, m = 0;
  const int first = (int)threadIdx.x * kPer;
#pragma unroll 1
  for (int i = 0; i < kPer; ++i) {
    const int bin = table_at(first + i);
    const auto c = first + i < kTable ? table[bin] : 0;
    n += c;
    m += c != 0 ? mass(bin, c) : 0;
  }
  Border b;
  uint64_t row_n;
  uint64_t n_before = block_scan64<kT>(n, row_n, turn, sh), m_before = block_scan64<kT>(m, b.total_m, turn, sh);
  if (share >= 0.0) {
    const double t = __builtin_ceil(share * (double)b.total_m);
    target = t < 1.0 ? 1 : (uint64_t)t;
  }
  const uint64_t lo = by_mass ? m_before : n_before, hi = lo + (by_mass ? m : n);
  if (lo < target && target <= hi) {
#pragma unroll 1
    for (int i = 0; i < kPer; ++i) {
      const int bin = table_at(first + i);
      const auto c = first + i < kTable ? table[bin] : 0;
      const uint64_t w = c != 0 ? mass(bin, c) : 0;
      if ((by_mass ? m_before + w : n_before + c) >= target) {
        sh.found[0] = bin;
        sh.found[1] = n_before;
        sh.found[2] = m_before;
        break;
      }
      n_before += c;
      m_before += w;
    }
  }
  __syncthreads();
  b.bin = (int)sh.found[0];
  b.above_n = sh.found[1];
  b.above_m = sh.found[2];
  __syncthreads();
  return b;
}

// ---- the draw -------------------------------------------------------------------

// The token of a row that a cut leaves: one pass for the chunks' weights above the cut and
// their ties at it, a scan, and one chunk again.  tabled (bf16, all values with weight in the table, the cut's not
// zero): many are kept, and the weights of values above the cut come from the table, others' as 0.
template <typename T, int kT>
__device__ __forceinline__ int draw(const T* row, int V, int factor, const Weight& weight, const Cut& cut, float u,
                                    bool tabled, int& turn, Shared<T>& sh) {
  constexpr int n = Elem<T>::kVec, kPer = kChunks > kT ? kChunks / kT : 1;
  constexpr uint32_t kNinf = kNinfOf<T>;
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  const int size = kChunk * factor, chunks = (V + size - 1) / size;
  const bool all = cut.key == 0;
  const float value = all ? kNegInf : order_value(cut.key);
  const uint64_t at_cut = all ? 0 : weight(value);
  __syncthreads();
  if constexpr (sizeof(T) == 2) {
    if (tabled) {
      for (int i = threadIdx.x; i < kTable; i += kT) {
        const float x = __uint_as_float(table_value(i) << 16);
        const bool in = i != kHuge && i != kTable - 1;  // beyond the table: none, or without weight
        sh.mass[i] = in && x > value && x <= (float)weight.top ? weight(x) : 0;
      }
      __syncthreads();
    }
  }
  // Ties' place in the table.  A min-p cut at no bf16 value has none, nor one beyond the octaves, whose bin is that of
  // zeros or of all that is larger.
  const uint32_t bits = __float_as_uint(value), octave = (bits >> 16 & 0x7fffu) - (uint32_t)kLeast;
  const uint32_t tie_at = all || (bits & 0xffffu) || octave >= kOctaves * 128u ? ~0u : 8u * (uint32_t)table_bin(bits >> 16);
  // A wave's chunks, two vectors at a time, the next ones on their way.
  constexpr int kGroup = 2;
  const int steps = (size + kWave * n * kGroup - 1) / (kWave * n * kGroup);  // of a chunk
  u32x4 next[kGroup];
  auto fetch = [&](int base) {
#pragma unroll
    for (int g = 0; g < kGroup; ++g) {
      const int id = base + (g * kWave + lane) * n;
      if (id + n <= V) next[g] = load16<T, false, false>(row + id);
      else next[g] = id < V ? *reinterpret_cast<const u32x4*>(sh.end) : u32x4{kNinf, kNinf, kNinf, kNinf};
    }
  };
  if (w < chunks) fetch(w * size);
  for (int c = w; c < chunks; c += kT / kWave) {
    uint64_t s = 0;
    uint32_t ties = 0;
    for (int step = 0; step < steps; ++step) {
      u32x4 raw[kGroup];
#pragma unroll
      for (int g = 0; g < kGroup; ++g) raw[g] = next[g];
      const bool more = step + 1 < steps;
      const long long base = more ? (long long)c * size + (step + 1) * (kWave * n * kGroup) : (long long)(c + kT / kWave) * size;
      if (more || base < V) fetch((int)base);
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        if constexpr (sizeof(T) == 2) {
          if (tabled) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint32_t at = table_offsets<8>(raw[g][q]), lo = at & 0xffffu, hi = at >> 16;
              const uint8_t* table = reinterpret_cast<const uint8_t*>(sh.mass);
              s += *reinterpret_cast<const uint64_t*>(table + lo) + *reinterpret_cast<const uint64_t*>(table + hi);
              ties += (lo == tie_at ? 1 : 0) + (hi == tie_at ? 1 : 0);
            }
            __builtin_amdgcn_sched_barrier(0);  // a vector at a time: registers
            continue;
          }
        }
        if (all) {
#pragma unroll
          for (int i = 0; i < n; ++i) {
            s += weight(raw_elem<T>(raw, g * n + i));
            if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);  // two weights at a time: registers
          }
          continue;
        }
        // Few are kept: the lanes' next ones together, until no lane has one.
        uint32_t hits = 0;
#pragma unroll
        for (int i = 0; i < n; ++i) hits |= raw_elem<T>(raw, g * n + i) >= value ? 1u << i : 0u;
#pragma unroll
        for (int q = 0; q < 4; ++q) asm("" : "+v"(raw[g][q]));  // unpacked again where one is picked: registers
        while (__any(hits != 0)) {
          const int at = __ffs(hits) - 1;
          float y = raw_elem<T>(raw, g * n);
#pragma unroll
          for (int i = 1; i < n; ++i) y = at == i ? raw_elem<T>(raw, g * n + i) : y;
          if (hits != 0) {
            if (y == value) ++ties;
            else s += weight(y);
          }
          hits &= hits - 1;
        }
      }
    }
    s = wave_sum64(s);
    ties = (uint32_t)wave_sum64(ties);
    if (lane == 0) sh.chunk_sum[c] = s, sh.chunk_tie[c] = ties;
  }
  __syncthreads();
  // Thread t has the chunks kPer t and on; ties are kept up to cut.ties of them.
  uint64_t own[kPer], tied[kPer], ties = 0, sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int c = (int)threadIdx.x * kPer + i;
    own[i] = c < chunks ? sh.chunk_sum[c] : 0;
    tied[i] = c < chunks ? sh.chunk_tie[c] : 0;
    ties += tied[i];
  }
  uint64_t row_ties, total;
  uint64_t ties_before = block_scan64<kT>(ties, row_ties, turn, sh);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const uint64_t room = cut.ties > ties_before ? cut.ties - ties_before : 0;
    own[i] += (tied[i] < room ? tied[i] : room) * at_cut;
    ties_before += tied[i];
    sum += own[i];
  }
  ties_before -= ties;
  uint64_t before = block_scan64<kT>(sum, total, turn, sh);
  const uint64_t target = (uint64_t)((double)u * (double)total);
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (before <= target && target < before + own[i]) {
      sh.found[0] = threadIdx.x * kPer + i;
      sh.found[1] = before;
      sh.found[2] = ties_before;
    }
    before += own[i];
    ties_before += tied[i];
  }
  __syncthreads();
  // That chunk's tokens, a vector per thread at a time.
  const int first = (int)sh.found[0] * size, end = (int)min((long long)V, (long long)first + size);
  uint64_t at = sh.found[1], ties_at = sh.found[2];
#pragma unroll 1
  for (int base = first; base < end; base += kT * n) {
    const int id = base + (int)threadIdx.x * n;
    const bool mine = id < end;
    float x[n];
    load_row(row, V, min(id, V - 1), x);
    uint64_t v[n], t = 0, s = 0, all_ties, all_mass;
#pragma unroll
    for (int i = 0; i < n; ++i) t += mine && id + i < V && x[i] == value ? 1 : 0;
    uint64_t rank = ties_at + block_scan64<kT>(t, all_ties, turn, sh);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const bool in = mine && id + i < V;
      v[i] = in && x[i] > value ? weight(x[i]) : in && x[i] == value && rank++ < cut.ties ? at_cut : 0;
      s += v[i];
      if (i % 2 == 1) __builtin_amdgcn_sched_barrier(0);  // two weights at a time: registers
    }
    uint64_t y = at + block_scan64<kT>(s, all_mass, turn, sh);
    if (y <= target && target < y + s) {
      int token = id;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        y += v[i];
        if (y <= target) token = id + i + 1;
      }
      sh.found[3] = token;
    }
    at += all_mass;
    ties_at += all_ties;
  }
  __syncthreads();
  return (int)sh.found[3];
}

// ---- candidates -----------------------------------------------------------------

// The largest 16-bit prefix p of ordered bits with at least k threads whose `own` has a prefix >= p (0
// if there are fewer than k).  Two bits at a time.
template <int kT, typename T>
__device__ __forceinline__ uint32_t kth_prefix(uint32_t own, uint32_t k, Shared<T>& sh) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  own >>= 16;
  uint32_t p = 0;
#pragma unroll 1
  for (int shift = 14; shift >= 0; shift -= 2) {
    uint64_t votes = 0;
#pragma unroll
    for (int i = 1; i <= 3; ++i)
      votes |= (uint64_t)__popcll(__ballot(own >= (p | (uint32_t)i << shift))) << (16 * (i - 1));
    uint64_t* at = sh.votes[shift >> 1 & 1];
    if (lane == 0) at[w] = votes;
    __syncthreads();
    votes = 0;
#pragma unroll
    for (int i = 0; i < kT / kWave; ++i) votes += at[i];
#pragma unroll
    for (int i = 3; i >= 1; --i)
      if ((votes >> (16 * (i - 1)) & 0xffff) >= k) {
        p |= (uint32_t)i << shift;
        break;
      }
  }
  return p;
}

// Up to so many, 64 disjoint sets of tokens give the bound: lane l's of every wave.  k
// of them that reach it are then among the first 64 ln(64 / (64 - k)) or so (k = 52: 107).
constexpr int kFewer = 52;

// The largest 16-bit prefix that at least k of those sets reach, one barrier and 16 votes of the wave.
template <int kT, typename T>
__device__ __forceinline__ uint32_t kth_of_lanes(float own, int k, Shared<T>& sh) {
  const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x / kWave;
  sh.lanes[w][lane] = own;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kT / kWave; ++i) own = fmaxf(own, sh.lanes[i][lane]);
  const uint32_t key = order_bits(own) >> 16;
  uint32_t p = 0;
#pragma unroll
  for (int shift = 15; shift >= 0; --shift)
    if (__popcll(__ballot(key >= (p | 1u << shift))) >= k) p |= 1u << shift;
  return p;
}

// Each of up to 512 listed tokens' ranks by (value, id) and by id, in the low and high half of ranks[i]: pairs of 64,
// a quarter of the pairs' second at a time.
template <int kT>
__device__ __forceinline__ void rank_list(const uint64_t* list, uint32_t* ranks, int n) {
  const int lane = threadIdx.x & (kWave - 1);
  const int groups = (n + kWave - 1) / kWave;
  for (int i = threadIdx.x; i < n; i += kT) ranks[i] = 0;
  __syncthreads();
  for (int unit = threadIdx.x / kWave; unit < groups * groups * 4; unit += kT / kWave) {
    const int mine = unit / (groups * 4) * kWave + lane, theirs = unit / 4 % groups * kWave + unit % 4 * 16;
    const uint64_t e = mine < n ? list[mine] : 0, f = theirs + (lane & 15) < n ? list[theirs + (lane & 15)] : ~0ull;
    uint32_t r = 0, by_id = 0;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const uint32_t lo = __builtin_amdgcn_readlane((int)f, j), hi = __builtin_amdgcn_readlane((int)(f >> 32), j);
      r += ((uint64_t)hi << 32 | lo) < e ? 1 : 0;
      by_id += lo < (uint32_t)e ? 1 : 0;
    }
    if (mine < n) atomicAdd(&ranks[mine], r | by_id << 16);
  }
  __syncthreads();
}

// The list's first n (a power of two) in ascending order.
template <int kT>
__device__ __forceinline__ void sort_list(uint64_t* list, int n) {
  for (int size = 2; size <= n; size *= 2)
    for (int step = size / 2; step > 0; step /= 2) {
      __syncthreads();
      for (int i = threadIdx.x; i < n / 2; i += kT) {
        const int lo = (i & ~(step - 1)) * 2 | (i & (step - 1)), hi = lo | step;
        const uint64_t x = list[lo], y = list[hi];
        if ((x > y) == ((lo & size) == 0)) list[lo] = y, list[hi] = x;
      }
    }
  __syncthreads();
}

template <typename T>
__device__ __forceinline__ T ninf_of() {
  if constexpr (sizeof(T) == 2) return 0xff80;
  else return kNegInf;
}

template <typename T>
__device__ __forceinline__ float raw_max(const u32x4 (&raw)[kLoadsT], int v) {
  constexpr int n = Elem<T>::kVec;
  float m = raw_elem<T>(raw, v * n);
#pragma unroll
  for (int i = 1; i < n; ++i) m = fmaxf(m, raw_elem<T>(raw, v * n + i));
  return m;
}

template <typename T, int kT>
__global__ void __launch_bounds__(kT, 4) sample_tokens_kernel(SampleArgs a) {
  constexpr int V8 = Elem<T>::kVec, kWaves = kT / kWave;
  __shared__ Shared<T> sh;
  const int r = blockIdx.x, V = a.V, lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  typedef uint16_t halves __attribute__((ext_vector_type(2)));
  const T* row = static_cast<const T*>(a.logits) + (size_t)r * (size_t)V;
  const float temperature = a.set.temperature.rows ? a.set.temperature.rows[r] : a.set.temperature.all;
  const int k = a.set.top_k.rows ? a.set.top_k.rows[r] : a.set.top_k.all;
  const float p = a.set.top_p.rows ? a.set.top_p.rows[r] : a.set.top_p.all;
  const float m = a.set.min_p.rows ? a.set.min_p.rows[r] : a.set.min_p.all;
  const float u = a.uniforms[r];
  const int factor = (int)(((long long)V + (long long)kChunk * kChunks - 1) / ((long long)kChunk * kChunks));
  const bool greedy = temperature == 0.0f, by_k = k >= 1 && k < V, by_p = p < 1.0f, by_m = m > 0.0f;
  const double s64 = uniform(1.4426950408889634074 / (double)temperature);
  // Few tokens and min-p alone: what a cut can keep is known while the row is read, and listed.  Other cuts
  // need the row's values first, in a table.
  const bool lists = !greedy && (by_k ? k <= kT : by_m && !by_p);
  const bool tables = !greedy && !lists;
  const bool counts = tables && (by_k || (by_p && sizeof(T) == 2));
  const double span_m = uniform(by_m ? (double)temperature * log((double)fminf(m, 1.0f)) : 0.0);
  // The least float at or above the min-p cut.
  auto least_kept = [&](float top) {
    const double least = (double)top + span_m;
    const float f = (float)least;
    return (double)f < least ? order_value(order_bits(f) + 1) : f;
  };

  if (threadIdx.x == 0) sh.bad = sh.tiny = sh.low = sh.count = 0, sh.best = ~0ull, sh.found[0] = sh.found[1] = sh.found[2] = sh.found[3] = 0;
  if (counts)
    for (int i = threadIdx.x; i < kTable; i += kT) sh.table[i] = 0;
  float top = kNegInf, bound = kNegInf, largest_own = kNegInf;
  uint32_t largest = 0, smallest = ~0u;  // magnitude bits; the least, less one, that are not zero
  // The row's last vector, where it is not whole, with -inf behind its end.
  constexpr uint32_t kNinf = kNinfOf<T>;
  if (threadIdx.x < V8) {
    const int id = V / V8 * V8 + (int)threadIdx.x;
    reinterpret_cast<T*>(sh.end)[threadIdx.x] = id < V ? row[id] : ninf_of<T>();
  }
  __syncthreads();
  u32x4 next[kLoadsT];
  auto fetch = [&](int base) {
#pragma unroll
    for (int v = 0; v < kLoadsT; ++v) {
      const int id = base + (v * kT + (int)threadIdx.x) * V8;
      if (id + V8 <= V) next[v] = load16<T, false, false>(row + id);
      else next[v] = id < V ? *reinterpret_cast<const u32x4*>(sh.end) : u32x4{kNinf, kNinf, kNinf, kNinf};
    }
  };
  constexpr int kSegment = kT * V8 * kLoadsT;
  // Tokens at or above the bound to the list.
  auto list_those = [&](const u32x4 (&raw)[kLoadsT], int v, int base, float most) {
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < V8; ++i) {
      const float x = raw_elem<T>(raw, v * V8 + i);
      hits |= x >= bound && x > kNegInf && x <= most ? 1u << i : 0u;
    }
    if (hits == 0) return;
    int at = atomicAdd(&sh.count, __popc(hits));
#pragma unroll
    for (int i = 0; i < V8; ++i)
      if (hits >> i & 1) {
        if (at < kList)
          sh.list[at] = (uint64_t)~order_bits(raw_elem<T>(raw, v * V8 + i)) << 32 |
                        (uint32_t)(base + (v * kT + (int)threadIdx.x) * V8 + i);
        ++at;
      }
  };
  fetch(0);
  int turn = 0, segment = 0;
#pragma unroll 1
  for (int base = 0; base < V; base += kSegment, turn ^= 1, ++segment) {
    u32x4 raw[kLoadsT];
    float most[kLoadsT], own = kNegInf;
#pragma unroll
    for (int v = 0; v < kLoadsT; ++v) raw[v] = next[v];
    if (V - base > kSegment) fetch(base + kSegment);
#pragma unroll
    for (int v = 0; v < kLoadsT; ++v) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (sizeof(T) == 2) {
          const halves m = __builtin_bit_cast(halves, raw[v][q] & 0x7fff7fffu);
          largest = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(halves, largest), m));
        } else {
          largest = max(largest, raw[v][q] & 0x7fffffffu);
        }
      }
    }
    if (tables) {
#pragma unroll
      for (int v = 0; v < kLoadsT; ++v) {
        const int id = base + (v * kT + (int)threadIdx.x) * V8;
        if (id >= V) continue;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (sizeof(T) == 2) {
            const halves one = {1, 1};
            smallest = __builtin_bit_cast(uint32_t, __builtin_elementwise_min(
                __builtin_bit_cast(halves, smallest), (halves)(__builtin_bit_cast(halves, raw[v][q] & 0x7fff7fffu) - one)));
            if (!counts) continue;
            const uint32_t at = table_offsets<4>(raw[v][q]);
            atomicAdd(reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(sh.table) + (at & 0xffffu)), 1u);
            atomicAdd(reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(sh.table) + (at >> 16)), 1u);
          } else {
            smallest = min(smallest, (raw[v][q] & 0x7fffffffu) - 1u);
            if (counts) atomicAdd(&sh.table[table_bin(raw[v][q] >> 16)], 1u);
          }
        }
        if (sizeof(T) == 4 || !counts) top = fmaxf(top, raw_max<T>(raw, v));
      }
      continue;
    }
#pragma unroll
    for (int v = 0; v < kLoadsT; ++v) {
      most[v] = raw_max<T>(raw, v);
      own = fmaxf(own, most[v]);
#pragma unroll
      for (int q = 0; q < 4; ++q) asm("" : "+v"(raw[v][q]));  // unpacked again where they are used again: registers
    }
    const float mine = wave_max(own);
    if (lane == 0) sh.top[turn][wave] = mine;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWaves; ++i) top = fmaxf(top, sh.top[turn][i]);
    if (top == kNegInf) continue;
    if (greedy) {
      // The lowest id of the largest value: the least of (value's complement, id).
      if (own == top) {
        int id = 0;
#pragma unroll
        for (int v = kLoadsT - 1; v >= 0; --v)
#pragma unroll
          for (int i = V8 - 1; i >= 0; --i)
            id = raw_elem<T>(raw, v * V8 + i) == top ? base + (v * kT + (int)threadIdx.x) * V8 + i : id;
        atomicMin((unsigned long long*)&sh.best, (unsigned long long)~order_bits(top) << 32 | (uint32_t)id);
      }
    } else if (lists) {
      // k threads' largest so far are k tokens of the row; taken anew when as much again was read.
      largest_own = fmaxf(largest_own, own);
      if (by_k && (segment & (segment + 1)) == 0)
        bound = fmaxf(bound, order_value(max(k <= kFewer ? kth_of_lanes<kT>(largest_own, k, sh)
                                                         : kth_prefix<kT>(order_bits(largest_own), (uint32_t)k, sh), 0x80u) << 16));
      if (by_m && !(by_k && by_p)) bound = fmaxf(bound, least_kept(top));  // top-p of the top k: all of their weight
#pragma unroll
      for (int v = 0; v < kLoadsT; ++v)
        if (__any(most[v] >= bound)) list_those(raw, v, base, __builtin_inff());
    }
  }
  // A fault of the row or of its settings: comparisons that NaN fails.
  const bool nan = sizeof(T) == 2 ? (largest & 0xffffu) > 0x7f80u || largest >> 16 > 0x7f80u : largest > 0x7f800000u;
  if (nan) sh.bad = 1;
  const bool tiny = sizeof(T) == 2 ? (smallest & 0xffffu) < kLeast - 1 || smallest >> 16 < kLeast - 1
                                   : smallest < ((uint32_t)kLeast << 16) - 1;
  if (tables && tiny) sh.tiny = 1;
  if (tables && (sizeof(T) == 2 ? (largest & 0xffffu) >= 0x4480u || largest >> 16 >= 0x4480u : largest >= 0x44800000u))
    sh.low = 1;  // a magnitude of 2^10 or more: of the largest, of one below, or of the fill behind the row's end
  if (counts) {
    __syncthreads();
    if (threadIdx.x == 0) sh.table[0] += sh.table[kHalf], sh.table[kHalf] = 0;
    __syncthreads();
    // The largest value of bf16 rows.
    for (int i = (int)threadIdx.x; sizeof(T) == 2 && i < kTable && top == kNegInf; i += kT)
      if (sh.table[table_at(i)] != 0) top = __uint_as_float(table_value(table_at(i)) << 16);
    if (sizeof(T) == 2 && (sh.table[kHuge] != 0 || sh.tiny || sh.table[kTable - 1] >= (uint32_t)V)) {
      // A value that the table does not tell.
      top = kNegInf;
      for_row<T, kT>(row, V, [&](float x, int) { top = fmaxf(top, x); });
    }
  }
  top = wave_max(top);
  if (lane == 0) sh.top[turn][wave] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kWaves; ++i) top = fmaxf(top, sh.top[turn][i]);
  if (sh.bad || !(fabsf(top) < __builtin_inff()) || !(temperature >= 0.0f && temperature < __builtin_inff()) || p != p ||
      m != m || !(u >= 0.0f && u < 1.0f)) {
    if (threadIdx.x == 0) a.tokens[r] = -1;
    return;
  }
  if (greedy) {
    if (threadIdx.x == 0) a.tokens[r] = (int)(uint32_t)sh.best;
    return;
  }
  top = uniform(top);
  const Weight weight{uniform((double)top), s64, a.F};
  const float least = uniform(by_m ? least_kept(top) : kNegInf);
  Cut cut;
  cut.key = 0;
  cut.ties = ~0ull;
  auto narrow = [&](const Cut& c) {
    if (c.key > cut.key) cut = c;
    else if (c.key == cut.key && c.ties < cut.ties) cut.ties = c.ties;
  };
  bool done = !by_k && !by_p, listed = lists, tabled = false;
  uint64_t row_mass = 0;
  if (tables) {
    // Values outside the table that have weight, or that a cut may meet, leave the row to its digits.
    const bool weightless = top > -1024.0f && weight(-1024.0f) == 0;
    // Values of -2^10 and below: masked ones, and what fills the last vector behind the row's end.
    const int low = counts ? (int)sh.table[kTable - 1] : sh.low;
    const bool plain = top < 1024.0f && !sh.tiny && (low == 0 || weightless) && (!by_k || k <= V - low);
    uint64_t kept = (uint64_t)V;  // at most
    if (plain && sizeof(T) == 2 && !done) {
      // A bin is a value: the cuts are known.
      auto mass = [&](int bin, uint32_t c) { return (uint64_t)c * weight(__uint_as_float(table_value(bin) << 16)); };
      uint64_t all = 0;
      if (by_k) {
        const Border b = find_border<kT>(sh.table, false, (uint64_t)k, -1.0, turn, sh, mass);
        Cut c;
        const float x = __uint_as_float(table_value(b.bin) << 16);
        c.key = order_bits(x);
        c.ties = (uint64_t)k - b.above_n;
        kept = (uint64_t)k;
        all = c.mass = b.above_m + c.ties * weight(x);
        narrow(c);
      }
      if (by_p) {
        const double t = __builtin_ceil((double)p * (double)all);
        const Border b = find_border<kT>(sh.table, true, t < 1.0 ? 1 : (uint64_t)t, by_k ? -1.0 : p > 0.0f ? (double)p : 0.0, turn, sh, mass);
        Cut c;
        const float x = __uint_as_float(table_value(b.bin) << 16);
        const uint64_t w = weight(x);
        const double tt = by_k ? t : __builtin_ceil((p > 0.0f ? (double)p : 0.0) * (double)b.total_m);
        const uint64_t goal = tt < 1.0 ? 1 : (uint64_t)tt;
        c.key = order_bits(x);
        c.ties = (goal - b.above_m + w - 1) / w;
        c.mass = 0;
        kept = b.above_n + c.ties < kept ? b.above_n + c.ties : kept;
        narrow(c);
      }
      done = true;
    }
    tabled = plain && sizeof(T) == 2 && kept > (uint64_t)V / kSparse;
    if (plain && sizeof(T) == 4 && !done) {
      // A bin's values share 16 bits: the cut's bin is known, and its tokens, or with the ones above all that can be
      // kept, are listed.
      auto least_of = [&](int bin) { return __uint_as_float(table_value(bin) << 16 | (bin >= kHalf ? 0xffffu : 0u)); };
      auto most_of = [&](int bin) { return __uint_as_float(table_value(bin) << 16 | (bin < kHalf && bin != 0 ? 0xffffu : 0u)); };
      auto list_between = [&](float lo, float hi) {
        __syncthreads();
        if (threadIdx.x == 0) sh.count = 0;
        __syncthreads();
        bound = lo;
        fetch(0);
#pragma unroll 1
        for (int base = 0; base < V; base += kSegment) {
          u32x4 raw[kLoadsT];
#pragma unroll
          for (int v = 0; v < kLoadsT; ++v) raw[v] = next[v];
          if (V - base > kSegment) fetch(base + kSegment);
#pragma unroll
          for (int v = 0; v < kLoadsT; ++v)
            if (__any(raw_max<T>(raw, v) >= lo)) list_those(raw, v, base, hi);
        }
        __syncthreads();
        return sh.count;
      };
      Border b;
      uint64_t goal = (uint64_t)k;
      if (by_k) {
        b = find_border<kT>(sh.table, false, goal, -1.0, turn, sh, [](int, uint32_t) { return (uint64_t)0; });
      } else {
        __syncthreads();
        for (int i = threadIdx.x; i < kTable; i += kT) sh.mass[i] = 0;
        __syncthreads();
        fetch(0);
#pragma unroll 1
        for (int base = 0; base < V; base += kSegment) {
          u32x4 raw[kLoadsT];
#pragma unroll
          for (int v = 0; v < kLoadsT; ++v) raw[v] = next[v];
          if (V - base > kSegment) fetch(base + kSegment);
#pragma unroll
          for (int v = 0; v < kLoadsT; ++v)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const uint64_t w = weight(__uint_as_float(raw[v][q]));
              if (w != 0) atomicAdd((unsigned long long*)&sh.mass[table_bin(raw[v][q] >> 16)], (unsigned long long)w);
            }
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.mass[0] += sh.mass[kHalf], sh.mass[kHalf] = 0;
        __syncthreads();
        const double share = p > 0.0f ? (double)p : 0.0;
        b = find_border<kT>(sh.mass, true, 1, share, turn, sh, [](int, uint64_t m) { return m; });
        row_mass = b.total_m;
        const double t = __builtin_ceil(share * (double)row_mass);
        goal = t < 1.0 ? 1 : (uint64_t)t;
      }
      __syncthreads();
      if (list_between(least_of(b.bin), __builtin_inff()) <= kList) {
        listed = true;
      } else if (!(by_k && by_p)) {
        const int in_bin = list_between(least_of(b.bin), most_of(b.bin));
        if (in_bin <= kList) {
          int size = 2;
          while (size < in_bin) size *= 2;
          for (int i = in_bin + (int)threadIdx.x; i < size; i += kT) sh.list[i] = ~0ull;
          sort_list<kT>(sh.list, size);
          const int per = (size + kT - 1) / kT;
          uint64_t own[kList / kT], sum = 0;
#pragma unroll
          for (int i = 0; i < kList / kT; ++i) {
            const int at = (int)threadIdx.x * per + i;
            own[i] = i < per && at < in_bin ? by_k ? 1 : weight(order_value(~(uint32_t)(sh.list[at] >> 32))) : 0;
            sum += own[i];
          }
          uint64_t in_all;
          uint64_t before = (by_k ? b.above_n : b.above_m) + block_scan64<kT>(sum, in_all, turn, sh);
#pragma unroll
          for (int i = 0; i < kList / kT; ++i) {
            if (before < goal && goal <= before + own[i]) sh.cut = (int)threadIdx.x * per + i;
            before += own[i];
          }
          __syncthreads();
          const int at = sh.cut;
          Cut c;
          c.key = ~(uint32_t)(sh.list[at] >> 32);
          int ties = 1;
          while (ties <= at && ~(uint32_t)(sh.list[at - ties] >> 32) == c.key) ++ties;
          c.ties = (uint64_t)ties;
          c.mass = 0;
          narrow(c);
          done = true;
        }
      }
    }
  }
  const int n = sh.count;
  if (listed && n <= kList) {
    // Ranked: the bits' complements ascend where the logits descend.  Few are ranked by counting, more are sorted.
    const bool few = n <= (kT == kSampleThreads ? kRanked : kRankedFewer);
    int size = n;
    uint64_t own_entry = 0;
    uint32_t own_ranks = 0;
    if (few) {
      uint32_t* ranks = reinterpret_cast<uint32_t*>(sh.list + kRanked);
      rank_list<kT>(sh.list, ranks, n);
      if ((int)threadIdx.x < n) own_entry = sh.list[threadIdx.x], own_ranks = ranks[threadIdx.x];
      __syncthreads();
      if ((int)threadIdx.x < n) sh.list[own_ranks & 0xffffu] = own_entry;
      __syncthreads();
    } else {
      size = 2;
      while (size < n) size *= 2;
      for (int i = n + (int)threadIdx.x; i < size; i += kT) sh.list[i] = ~0ull;
      sort_list<kT>(sh.list, size);
    }
    const int per = (size + kT - 1) / kT;  // 8 at most
    constexpr int kPer = kList / kT;
    uint64_t own[kPer], sum = 0;
    float value[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = (int)threadIdx.x * per + i;
      const uint64_t e = i < per && at < n ? sh.list[at] : ~0ull;
      value[i] = e == ~0ull ? kNegInf : order_value(~(uint32_t)(e >> 32));
      own[i] = e == ~0ull ? 0 : weight(value[i]);
      sum += own[i];
      __builtin_amdgcn_sched_barrier(0);  // one at a time: registers
    }
    if (threadIdx.x == 0) sh.cut = n, sh.found[0] = row_mass;
    uint64_t all;
    const uint64_t before = block_scan64<kT>(sum, all, turn, sh);
    uint64_t up_to = before;
    const int nk = by_k ? min(k, n) : n;
    if (by_k && by_p) {
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        up_to += own[i];
        if (i < per && (int)threadIdx.x * per + i == nk - 1) sh.found[0] = up_to;
      }
    }
    __syncthreads();
    const double share = __builtin_ceil((double)fmaxf(p, 0.0f) * (double)sh.found[0]);
    const uint64_t target = share < 1.0 ? 1 : (uint64_t)share;
    // The first index that is not kept.
    up_to = before;
    int mine = nk;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = (int)threadIdx.x * per + i;
      up_to += own[i];
      if (i >= per || at >= n) continue;
      if (by_p && up_to >= target) mine = min(mine, at + 1);
      if (by_m && value[i] < least) mine = min(mine, at);
    }
    mine = wave_min(mine);
    if (lane == 0) atomicMin(&sh.cut, mine);
    __syncthreads();
    const int kept = sh.cut;
    {
      // The kept ones by id.
      __syncthreads();
      int count = kept;
      if (few) {
        if ((int)threadIdx.x < n)
          sh.list[own_ranks >> 16] = (int)(own_ranks & 0xffffu) < kept ? own_entry << 32 | own_entry >> 32 : ~0ull;
        count = size = n;
        __syncthreads();
      } else {
        size = 2;
        while (size < kept) size *= 2;
        for (int i = threadIdx.x; i < size; i += kT) {
          const uint64_t e = sh.list[i];
          sh.list[i] = i < kept ? e << 32 | e >> 32 : ~0ull;
        }
        sort_list<kT>(sh.list, size);
      }
      const int per = (size + kT - 1) / kT;
      sum = 0;
      uint32_t id[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int at = (int)threadIdx.x * per + i;
        const uint64_t e = i < per && at < count ? sh.list[at] : ~0ull;
        id[i] = (uint32_t)(e >> 32);
        own[i] = e == ~0ull ? 0 : weight(order_value(~(uint32_t)e));
        sum += own[i];
        __builtin_amdgcn_sched_barrier(0);
      }
      uint64_t total;
      uint64_t from = block_scan64<kT>(sum, total, turn, sh);
      const uint64_t goal = (uint64_t)((double)u * (double)total);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (from <= goal && goal < from + own[i]) a.tokens[r] = (int)id[i];
        from += own[i];
      }
      return;
    }
  }

  // Cuts that neither the list nor the table gave: digit by digit.
  uint64_t mass = 0;
  if (by_k && !done) {
    const Cut c = find_cut<T, kT>(row, V, weight, false, (uint64_t)k, -1.0, turn, sh);
    mass = c.mass;
    narrow(c);
  }
  if (by_p && !done) {
    const double t = by_k ? __builtin_ceil((double)p * (double)mass) : 0.0;
    narrow(find_cut<T, kT>(row, V, weight, true, t < 1.0 ? 1 : (uint64_t)t, by_k ? -1.0 : p > 0.0f ? (double)p : 0.0, turn, sh));
  }
  if (by_m) {
    Cut c;
    c.key = order_bits(least);
    c.ties = ~0ull;
    c.mass = 0;
    narrow(c);
  }
  if (cut.key == order_bits(0.0f)) tabled = false;  // zeros of both signs are its ties
  const int token = draw<T, kT>(row, V, factor, weight, cut, u, tabled, turn, sh);
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
  const dim3 grid((unsigned)R);
  if (R <= kSampleWideRows) {
    if (dtype == 1) hipLaunchKernelGGL((sample_tokens_kernel<uint16_t, 1024>), grid, dim3(1024), 0, st, a);
    else hipLaunchKernelGGL((sample_tokens_kernel<float, 1024>), grid, dim3(1024), 0, st, a);
  } else {
    if (dtype == 1) hipLaunchKernelGGL((sample_tokens_kernel<uint16_t, 512>), grid, dim3(512), 0, st, a);
    else hipLaunchKernelGGL((sample_tokens_kernel<float, 512>), grid, dim3(512), 0, st, a);
  }
  return hipGetLastError();
}

}  // namespace sv
