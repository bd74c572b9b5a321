// Log-probabilities of given tokens, the rows' entropies and their likeliest
// alternatives.  With a_v = x_v * s - ref, s = log2(e) / T and any reference:
//   Z = sum 2^a_v,  H = sum 2^a_v a_v,
//   ln P(t) = ln 2 (a_t - log2 Z),  entropy = ln 2 (log2 Z - H / Z).
// Waves take tiles of 64 16-byte vectors x 8 (4096 bf16 or 2048 fp32 logits),
// each logit once, against a running reference, and keep the maximum of every
// chunk of 512 (256) consecutive logits.  The alternatives then cost a few of
// the row's chunks: the n-th largest maximum of 64 disjoint sets of tokens is
// a bound that n tokens reach, so only chunks whose maximum reaches it are
// read again, and what reaches it there (little more than n tokens) is ranked
// by counting.  Rows whose ties make that many (all logits equal) take the n
// chunks with the largest maxima one by one instead: those hold the n best
// tokens, for their maxima alone come before everything in any other chunk.
//
// Short rows take one launch, a block per row (lp_row_kernel); the others two:
// blocks of four waves take parts of rows (lp_part_kernel), so that every
// compute unit has the same to do, and a block per row joins them
// (lp_pick_kernel).
//
// Long batches are bound by reading the rows, with the vector ALU close behind:
// about nine operations per bf16 logit (unpack, half a maximum, FMA, a
// quarter-rate exponential, add, FMA) against the eleven that pass in the time
// of its two bytes.  1152 rows of 262144 with 20 alternatives: parts 93 us
// (604 MB, 6.5 TB/s; the read stream reaches 7.1), join 12.5 us.  Single rows
// are bound by their chain of loads: 5 rows of 32000 fp32 take 7.6 us, about
// 0.6 to the token, 0.5 to the first tile, 2.5 to the sums, 2.5 to the pick.

#include <type_traits>

#include "sv_common.h"
#include "sv_host_quant.h"
#include "sv_internal.h"

namespace sv {

namespace {

struct LpArgs {
  const void* logits;      // [N][V]
  const int32_t* tokens;   // [N]
  LogprobsPart* parts;     // [N][NP]
  float* chunks;           // [N][NT * 8] chunk maxima; null without alternatives
  float* lanes;            // [N][NP][64] the lanes' maxima over a part; null without alternatives
  float* logprobs;         // [N]
  float* entropy;          // [N] or null
  int32_t* top_ids;        // [N][top]
  float* top_logprobs;     // [N][top]
  int V, NT, top;
  int NP, part_tiles;      // parts of a row and their tiles (a multiple of 4)
  float s;                 // log2(e) / T
};

// Position q on a row's 16-byte grid holds token q - pre.
template <typename T>
__device__ __forceinline__ int row_lead(const T* row) {
  return (int)(((uintptr_t)row & 15) / sizeof(T));
}

// The vector at position q of the grid; tokens outside the row read as -inf.
// Only whole vectors inside the row are loaded as such.
template <typename T>
__device__ __forceinline__ u32x4 load_vec(const T* row, int V, int pre, int q) {
  constexpr int V8 = Elem<T>::kVec;
  const int id = q - pre;
  if (id >= 0 && id + V8 <= V) return stream16(row + id);
  constexpr uint32_t kNinf = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  u32x4 w{kNinf, kNinf, kNinf, kNinf};
  if (id + V8 <= 0 || id >= V) return w;
#pragma unroll
  for (int k = 0; k < V8; ++k) {
    if (id + k < 0 || id + k >= V) continue;
    if constexpr (sizeof(T) == 2)
      w[k / 2] = (k & 1) ? (w[k / 2] & 0xffffu) | ((uint32_t)row[id + k] << 16)
                         : (w[k / 2] & 0xffff0000u) | (uint32_t)row[id + k];
    else
      w[k] = __float_as_uint(row[id + k]);
  }
  return w;
}

// Maxima over the wave of eight values per lane: lane l ends with that of
// value l % 8.  Three exchanges halve the values a lane carries, each over
// lanes that differ in one more of the three low lane bits (a mirror of eight
// lanes flips all three, so it comes first, while a lane still holds every
// value); three more go over the eight groups of eight lanes.
__device__ __forceinline__ float wave_max8(const float (&c)[8], int lane) {
  float d[4], e[2];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float keep = lane & 4 ? c[j + 4] : c[j], send = lane & 4 ? c[j] : c[j + 4];
    d[j] = fmaxf(keep, dpp::mov<dpp::kHalfMirror, 0xf>(0.0f, send));
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float keep = lane & 2 ? d[j + 2] : d[j], send = lane & 2 ? d[j] : d[j + 2];
    e[j] = fmaxf(keep, dpp::mov<dpp::kQuadSwap2, 0xf>(0.0f, send));
  }
  const float keep = lane & 1 ? e[1] : e[0], send = lane & 1 ? e[0] : e[1];
  float v = fmaxf(keep, dpp::mov<dpp::kQuadSwap1, 0xf>(0.0f, send));
  v = fmaxf(v, dpp::mov<0x128, 0xf>(0.0f, v));  // row_ror:8
#if defined(__HIP_DEVICE_COMPILE__)
  const auto r16 = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r16[0]), __uint_as_float(r16[1]));
  const auto r32 = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r32[0]), __uint_as_float(r32[1]));
#endif
  return v;
}

// fp32 bits in the order of the values (-0 as 0).
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }

constexpr int kList = 1024;        // candidates held at a time; a chunk adds at most 512
constexpr int kSelect = 128;       // chunks that a row reads again before it goes one by one
constexpr int kBatch = 8;          // chunks loaded together
constexpr int kNone = (int)0x80000000;

// The best entry of a lane's share (i = lane, lane + 64, ..) of a list in LDS
// or device memory.
template <typename P, typename F>
__device__ __forceinline__ void best_of_lane(const P* list, int count, int lane, F order, int* best, int* at) {
  int b = kNone, w = 0x7fffffff;
#pragma unroll 8
  for (int i = lane; i < count; i += kWave) {
    const int o = order(list[i]);
    if (o > b) b = o, w = i;
  }
  *best = b;
  *at = w;
}

struct Candidate {
  int order, id;
};

__device__ __forceinline__ bool before(int o1, int i1, int o2, int i2) { return o1 > o2 || (o1 == o2 && i1 < i2); }

// LDS accesses of one wave are done in order; this keeps the compiler to it.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// The n best of `count` (> 64) candidates to the front of the list, in order.
// Every lane calls this; the list is in LDS and belongs to this wave.
__device__ __forceinline__ void keep_best(Candidate* list, int count, int n, int lane) {
  Candidate mine{kNone, 0x7fffffff};
  int bo = kNone, bi = 0x7fffffff, at = -1;
  auto rescan = [&]() {
    bo = kNone, bi = 0x7fffffff, at = -1;
    for (int i = lane; i < count; i += kWave)
      if (before(list[i].order, list[i].id, bo, bi)) bo = list[i].order, bi = list[i].id, at = i;
  };
  rescan();
  for (int r = 0; r < n; ++r) {
    const int o = wave_max(bo);
    const int id = wave_min(bo == o ? bi : 0x7fffffff);
    if (lane == r) mine = Candidate{o, id};
    if (bo == o && bi == id && at >= 0) {
      list[at] = Candidate{kNone, 0x7fffffff};
      rescan();
    }
  }
  wave_sync();
  if (lane < n) list[lane] = mine;
  wave_sync();
}

__device__ __forceinline__ double wave_max64(double v) {
  return dpp::reduce(v, -__builtin_inf(), [](double x, double y) { return x > y ? x : y; });
}

constexpr double kLn2 = 0.69314718055994530942;

// A row's law: ln P(x) = ln 2 ((x s - ref) - log2 Z), in that order, for ref may
// dwarf log2 Z.  Where one token has all of the probability, the roundings of
// its own term in Z are left (6e-8): they carry no result past its bound, a
// logarithm of a probability past 0 or an entropy below it.
struct RowLaw {
  double ref, log2Z, s;
};
__device__ __forceinline__ float log_prob(const RowLaw& w, float x) {
  const double v = kLn2 * ((double)x * w.s - w.ref - w.log2Z);
  return v > 0.0 ? 0.0f : (float)v;
}

// A row without a law: NaN, and no alternatives.
__device__ __forceinline__ void write_nothing(const LpArgs& a, size_t row_i, int lane) {
  const float nan = __builtin_nanf("");
  if (lane == 0) {
    a.logprobs[row_i] = nan;
    if (a.entropy) a.entropy[row_i] = nan;
  }
  if (lane < a.top) {
    a.top_ids[row_i * a.top + lane] = -1;
    a.top_logprobs[row_i * a.top + lane] = nan;
  }
}

// A candidate as a number: later is larger, equal values with lower ids first.
__device__ __forceinline__ uint64_t key_of(const Candidate& c) {
  return ((uint64_t)((uint32_t)c.order ^ 0x80000000u) << 32) | (uint32_t)~c.id;
}

// Rank of one candidate per lane among `have` <= 64 of them.
__device__ __forceinline__ int rank_in_wave(const Candidate& mine, int have) {
  const uint64_t key = key_of(mine);
  const int lo = (int)(uint32_t)key, hi = (int)(uint32_t)(key >> 32);
  int rank = 0;
  for (int j = 0; j < have; ++j) {
    const uint64_t other = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane(hi, j) << 32) |
                           (uint32_t)__builtin_amdgcn_readlane(lo, j);
    rank += other > key ? 1 : 0;
  }
  return rank;
}

// The n-th largest of 64 lanes' maxima of disjoint sets of tokens: n tokens reach it.
__device__ __forceinline__ int bound_of(float lane_max, int n, int lane) {
  const int mine = order_of(lane_max);
  int reach = 0;  // lanes at or above this one
#pragma unroll 8
  for (int j = 0; j < kWave; ++j) reach += __builtin_amdgcn_readlane(mine, j) >= mine ? 1 : 0;
  const int o = wave_max(reach >= n ? mine : kNone);
  return max(o, order_of(-__builtin_inff()) + 1);  // -inf is no alternative
}

__device__ __forceinline__ void write_top(const LpArgs& a, size_t row_i, const RowLaw& w, const Candidate& c, int rank) {
  a.top_ids[row_i * a.top + rank] = c.id;
  a.top_logprobs[row_i * a.top + rank] = log_prob(w, value_of(c.order));
}

// Entries have .. top - 1: no token left.
__device__ __forceinline__ void write_rest(const LpArgs& a, size_t row_i, int have, int lane) {
  if (lane >= have && lane < a.top) {
    a.top_ids[row_i * a.top + lane] = -1;
    a.top_logprobs[row_i * a.top + lane] = -__builtin_inff();
  }
}

// The alternatives from the chunks with the a.top largest maxima, by one wave.
// maxima: the row's chunk maxima (in LDS or in the workspace; the chunks taken
// are overwritten).  list, count: LDS of this wave's own.
template <typename T, typename P>
__device__ __forceinline__ void pick_by_chunks(const LpArgs& a, size_t row_i, const T* row, P* maxima, Candidate* list,
                                               int* count, const RowLaw& law, int lane) {
  constexpr int V8 = Elem<T>::kVec, kChunk = kWave * V8;
  const int NC = a.NT * kChunksPerTile, n = a.top, pre = row_lead(row);
  const int ninf = order_of(-__builtin_inff());
  if (lane == 0) *count = 0;

  // Lane r holds the r-th chunk.
  auto order = [](float x) { return order_of(x); };
  int best, at, chosen = 0, chunks = 0, last = kNone;
  best_of_lane(maxima, NC, lane, order, &best, &at);
  for (; chunks < n; ++chunks) {
    const int o = wave_max(best);
    if (o <= ninf) break;
    const int c = wave_min(best == o ? at : 0x7fffffff);
    if (lane == chunks) chosen = c;
    last = o;
    if (at == c) {
      maxima[c] = -__builtin_inff();
      best_of_lane(maxima, NC, lane, order, &best, &at);
    }
  }
  // Candidates come before or are `bound_o`, `bound_id`.
  int bound_o = max(chunks == n ? last : kNone, ninf + 1), bound_id = 0x7fffffff;

  auto load_batch = [&](int first, u32x4 (&w)[kBatch]) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (first + k < chunks)
        w[k] = load_vec(row, a.V, pre, __builtin_amdgcn_readlane(chosen, first + k) * kChunk + lane * V8);
  };
  if (chunks < n) {
    // Too few chunks for a bound from their maxima: the n-th largest of the
    // lanes' maxima, which are as many different tokens.
    float lm = -__builtin_inff();
    for (int first = 0; first < chunks; first += kBatch) {
      u32x4 w[kBatch];
      load_batch(first, w);
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (first + k < chunks) {
          const u32x4 one[1] = {w[k]};
          lm = fmaxf(lm, raw_lane_max<T>(one));
        }
    }
    bound_o = max(bound_o, bound_of(lm, n, lane));
  }
  wave_sync();
  int have = 0;
  for (int first = 0; first < chunks; first += kBatch) {
    u32x4 w[kBatch];
    load_batch(first, w);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (first + k >= chunks) break;
      if (have > kList - kChunk) {
        keep_best(list, have, n, lane);
        bound_o = list[n - 1].order;
        bound_id = list[n - 1].id;
        wave_sync();
        if (lane == 0) *count = n;
        wave_sync();
      }
      const u32x4 one[1] = {w[k]};
      const int base = __builtin_amdgcn_readlane(chosen, first + k) * kChunk + lane * V8 - pre;
      if (order_of(raw_lane_max<T>(one)) >= bound_o) {
#pragma unroll
        for (int e = 0; e < V8; ++e) {
          const int o = order_of(raw_elem<T>(one, e));
          if (before(o, base + e, bound_o, bound_id)) list[atomicAdd(count, 1)] = Candidate{o, base + e};
        }
      }
      wave_sync();
      have = __builtin_amdgcn_readfirstlane(*count);
    }
  }
  if (have > kWave) {
    keep_best(list, have, n, lane);
    have = n;
  }
  const Candidate mine = lane < have ? list[lane] : Candidate{kNone, 0x7fffffff};
  const int rank = rank_in_wave(mine, have);
  if (lane < have && rank < n) write_top(a, row_i, law, mine, rank);
  write_rest(a, row_i, have, lane);
}

// A wave's sums over its tiles.  lane_max: the lane's largest logit.
struct WaveSums {
  double R, z, h;
  float lane_max;
};

// How a tile's exponents t = x s - ref are formed: by one FMA; the same, with
// the factor of the entropy's products kept above -1e4, for 0 * -inf of a logit
// of -inf; and, kept so too, from the difference, for a reference that cannot
// be taken out of the FMA (see kExpRefWide).
enum { kPlain = 0, kClamped = 1, kWide = 2 };

// Tiles first, first + step, .. below `end` of a row.  A lane's sums are
// against the wave's reference R (in units of log 2): fp32 within a tile, 64
// (32) terms in four chains, fp64 over the tiles.  Any reference will do that
// no logit passes by 2^20 (exponents then lose no more than their rounding near
// 20): the row's own token, x0, likely within that of the largest logit, else
// a tile's maximum, taken where one does pass (a first tile's, where x0 is not
// finite).  Chunk maxima go to `maxima` (a row's, in LDS or memory).
template <typename T, bool kTop>
__device__ __forceinline__ WaveSums sum_tiles(const T* row, int V, float s, float x0, int first, int end, int step,
                                              int lane, float* maxima) {
  constexpr int V8 = Elem<T>::kVec, kTileN = kTile<T>;
  const int pre = row_lead(row);
  WaveSums w{-__builtin_inf(), 0.0, 0.0, -__builtin_inff()};
  float m_ref = -__builtin_inff(), hi = __builtin_inff();
  int mode = kPlain;
  if (__builtin_fabsf(x0) < __builtin_inff()) {
    m_ref = x0, hi = exp_ref_hi(x0, s);
    mode = exp_ref_wide(x0, s) ? kWide : kPlain;
    w.R = mode == kWide ? (double)x0 * (double)s : (double)hi;
  }
  for (int tile = first; tile < end; tile += step) {
    const int q0 = tile * kTileN;
    u32x4 raw[kLoads];
    if (q0 >= pre && q0 - pre + kTileN <= V) {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) raw[j] = stream16(row + (q0 - pre) + j * (kWave * V8) + lane * V8);
    } else {
#pragma unroll
      for (int j = 0; j < kLoads; ++j) raw[j] = load_vec(row, V, pre, q0 + j * (kWave * V8) + lane * V8);
    }
    if (tile == first && mode == kPlain) {
      // Where a mask is in sight, not first the plain way.
      bool masked = false;
#pragma unroll
      for (int k = 0; k < V8; ++k) masked |= raw_elem<T>(raw, k) == -__builtin_inff();
      if (__any(masked)) mode = kClamped;
    }
    float c[kLoads], z4[4], h4[4];
    // The tile's chunk maxima (a lane's share) and with kSums its sums.
    auto pass = [&](auto sums_c, auto mode_c) {
      constexpr bool kSums = decltype(sums_c)::value;
      constexpr int kMode = decltype(mode_c)::value;
#pragma unroll
      for (int i = 0; i < 4; ++i) z4[i] = h4[i] = 0.0f;
      // Unpacked by each pass for itself: shared between passes, a tile's
      // floats would stay in 64 registers.
      uint32_t high = 0xffff0000u, half = 16;
      asm volatile("" : "+s"(high), "+s"(half));
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
#pragma unroll
        for (int k = 0; k < V8; ++k) {
          float x;
          if constexpr (sizeof(T) == 2)
            x = __uint_as_float(k & 1 ? raw[j][k / 2] & high : raw[j][k / 2] << half);
          else
            x = __uint_as_float(raw[j][k]);
          c[j] = k == 0 ? x : fmaxf(c[j], x);
          if constexpr (kSums) {
            const float t = kMode == kWide ? (x - m_ref) * s : __builtin_fmaf(x, s, -hi);
            const float p = exp2_fast(t);
            z4[k & 3] += p;
            h4[k & 3] = __builtin_fmaf(p, kMode == kPlain ? t : fmaxf(t, -1.0e4f), h4[k & 3]);
          }
        }
      }
    };
    auto all_sums = [&]() {
      if (mode == kPlain) pass(std::true_type{}, std::integral_constant<int, kPlain>{});
      else if (mode == kClamped) pass(std::true_type{}, std::integral_constant<int, kClamped>{});
      else pass(std::true_type{}, std::integral_constant<int, kWide>{});
    };
    float lm;
    auto reduce_max = [&]() {
      lm = c[0];
#pragma unroll
      for (int j = 1; j < kLoads; ++j) lm = fmaxf(lm, c[j]);
    };
    auto renew = [&](float m) {  // m becomes the reference
      const bool w2 = exp_ref_wide(m, s);
      const double R2 = w2 ? (double)m * (double)s : (double)exp_ref_hi(m, s), dr = w.R - R2;
      if (w.R > -__builtin_inf()) {
        const double f = exp2_fast((float)dr);  // dr < -20: what it scales is the smaller part
        w.h = f * (w.h + dr * w.z);
        w.z *= f;
      }
      w.R = R2, m_ref = m, hi = exp_ref_hi(m, s);
      mode = w2 ? kWide : mode == kWide ? kClamped : mode;
    };
    if (m_ref == -__builtin_inff()) {
      pass(std::false_type{}, std::integral_constant<int, kPlain>{});
      reduce_max();
      const float m = wave_max(lm);
      if (m > m_ref) renew(m);
    }
    all_sums();
    reduce_max();
    if (__any((lm - m_ref) * s > 20.0f)) {  // where there is no reference yet, lm is -inf and this NaN
      renew(wave_max(lm));
      all_sums();
    }
    w.lane_max = fmaxf(w.lane_max, lm);
    if constexpr (kTop) {
      const float cm = wave_max8(c, lane);
      if (lane < 8) maxima[tile * kChunksPerTile + lane] = cm;
    }
    const float z = (z4[0] + z4[1]) + (z4[2] + z4[3]);
    float h = (h4[0] + h4[1]) + (h4[2] + h4[3]);
    if (mode == kPlain && __any(h != h)) {
      // A logit of -inf: this tile's products again, and the tiles after it,
      // with exponents kept finite.  A NaN logit or +inf stays visible in z.
      mode = kClamped;
      all_sums();
      h = (h4[0] + h4[1]) + (h4[2] + h4[3]);
    }
    w.z += (double)z;
    w.h += (double)h;
  }
  w.z = wave_sum(w.z);
  w.h = wave_sum(w.h);
  return w;
}

// Sums of up to 64 lanes, one part each, against the largest reference.
// False: the row has no law (its largest logit is not finite, or a NaN).
__device__ __forceinline__ void join_parts(double& R, double& z, double& h) {
  const bool any = !(z == 0.0);  // a part of nothing but -inf adds nothing
  const double Ra = wave_max64(any ? R : -__builtin_inf()), dr = R - Ra;
  double f = 1.0;
  if (__any(any && dr != 0.0)) f = exp2_fast((float)dr);  // mostly all have the token's reference
  const double Z = wave_sum(any ? f * z : 0.0), H = wave_sum(any ? f * (h + dr * z) : 0.0);
  R = Ra, z = Z, h = H;
}
__device__ __forceinline__ bool has_law(double R, double Z) {
  return Z > 0.0 && Z < __builtin_inf() && R > -__builtin_inf() && R < __builtin_inf();
}

struct PickShared {
  Candidate list[kList];
  int chosen[kSelect];
  int rank[kWave];
  int chunks, count, bound;
};

// The chunks whose maximum reaches the bound, by one wave.  lane_max: of the
// tokens that this lane of any wave has seen.  (Sets of whole chunks would
// give a bound too, a poor one where the likely tokens have neighbouring ids.)
template <typename P>
__device__ __forceinline__ void select_chunks(const P* maxima, int NC, int n, float lane_max, PickShared& sh,
                                              int lane) {
  constexpr int kKeep = 8;  // chunk maxima of a lane in registers
  float v[kKeep];
#pragma unroll
  for (int k = 0; k < kKeep; ++k) v[k] = lane + k * kWave < NC ? maxima[lane + k * kWave] : -__builtin_inff();
  const int bound = bound_of(lane_max, n, lane);
  int found = 0;
  auto keep = [&](float x, int i) {
    const bool in = order_of(x) >= bound;
    const uint64_t all = __ballot(in);
    const int at = found + __builtin_amdgcn_mbcnt_hi((uint32_t)(all >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)all, 0));
    if (in && at < kSelect) sh.chosen[at] = i;
    found += __popcll(all);
  };
#pragma unroll
  for (int k = 0; k < kKeep; ++k) keep(v[k], lane + k * kWave);
  for (int i0 = kKeep * kWave; i0 < NC; i0 += kWave)
    keep(i0 + lane < NC ? maxima[i0 + lane] : -__builtin_inff(), i0 + lane);
  sh.rank[lane] = 0;
  if (lane == 0) sh.chunks = found, sh.count = 0, sh.bound = bound;
}

// A row's alternatives, by a block of NW waves: the selected chunks' tokens
// that reach the bound, and their ranks.  What select_chunks left, and the
// law, are visible to the block.
template <typename T, int NW>
__device__ __forceinline__ void pick(const LpArgs& a, size_t row_i, const T* row, float* maxima, PickShared& sh,
                                     const RowLaw& law, int wave, int lane) {
  constexpr int V8 = Elem<T>::kVec, kChunk = kWave * V8;
  const int n = a.top, pre = row_lead(row), sel = sh.chunks, bound = sh.bound;
  if (sel <= kSelect) {
    for (int k0 = wave; k0 < sel; k0 += NW * kBatch) {
      u32x4 w[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (k0 + k * NW < sel) w[k] = load_vec(row, a.V, pre, sh.chosen[k0 + k * NW] * kChunk + lane * V8);
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        if (k0 + k * NW >= sel) break;
        const u32x4 one[1] = {w[k]};
        const int base = sh.chosen[k0 + k * NW] * kChunk + lane * V8 - pre;
        if (order_of(raw_lane_max<T>(one)) >= bound) {
#pragma unroll
          for (int e = 0; e < V8; ++e) {
            const int o = order_of(raw_elem<T>(one, e));
            if (o >= bound) {
              const int at = atomicAdd(&sh.count, 1);
              if (at < kList) sh.list[at] = Candidate{o, base + e};
            }
          }
        }
      }
    }
  }
  __syncthreads();
  const int have = sh.count;
  if (sel > kSelect || have > kList) {
    __syncthreads();  // every wave has read the counts before one of them is used again
    if (wave == 0) pick_by_chunks<T>(a, row_i, row, maxima, sh.list, &sh.count, law, lane);
    return;
  }
  if (have <= kWave) {
    // Each wave counts against every NW-th candidate.
    const Candidate mine = lane < have ? sh.list[lane] : Candidate{kNone, 0x7fffffff};
    const uint64_t key = key_of(mine);
    int rank = 0;
    for (int j = wave; j < have; j += NW) rank += key_of(sh.list[j]) > key ? 1 : 0;
    if (rank) atomicAdd(&sh.rank[lane], rank);
    __syncthreads();
    if (wave != 0) return;
    rank = sh.rank[lane];
    if (lane < have && rank < n) write_top(a, row_i, law, mine, rank);
  } else {
    for (int i = threadIdx.x; i < have; i += kWave * NW) {
      const Candidate mine = sh.list[i];
      const uint64_t key = key_of(mine);
      int rank = 0;
      for (int j = 0; j < have; ++j) rank += key_of(sh.list[j]) > key ? 1 : 0;
      if (rank < n) write_top(a, row_i, law, mine, rank);
    }
  }
  if (wave == 0) write_rest(a, row_i, have, lane);
}

// A row's law from its joined sums, by one wave: writes what does not need the
// alternatives.  Returns whether there is a law.
template <typename T>
__device__ __forceinline__ bool write_law(const LpArgs& a, size_t row_i, float xt, double R, double Z, double H,
                                          RowLaw* law, int lane) {
  if (!has_law(R, Z)) {
    write_nothing(a, row_i, lane);
    return false;
  }
  *law = RowLaw{R, log2(Z), (double)a.s};
  if (lane == 0) {
    a.logprobs[row_i] = log_prob(*law, xt);
    const double entropy = kLn2 * (law->log2Z - H / Z);
    if (a.entropy) a.entropy[row_i] = entropy < 0.0 ? 0.0f : (float)entropy;
  }
  return true;
}

struct RowShared {
  PickShared pick;
  RowLaw law;
  int ok;
};

// One block per row, NW waves.
template <typename T, int NW, bool kTop>
__global__ void __launch_bounds__(kWave * NW) lp_row_kernel(LpArgs a) {
  __shared__ float maxima[kTop ? (kLpRowTiles + 1) * kChunksPerTile : 1];  // an unaligned row may reach into one more
  __shared__ float lane_maxima[kTop ? NW : 1][kWave];
  __shared__ double part[NW][3];
  __shared__ RowShared sh;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const size_t row_i = blockIdx.x;
  const int token = a.tokens[row_i];
  if ((uint32_t)token >= (uint32_t)a.V) {
    if (wave == 0) write_nothing(a, row_i, lane);
    return;
  }
  const T* row = static_cast<const T*>(a.logits) + row_i * (size_t)a.V;
  const float xt = to_f32(row[token]);
  const WaveSums w = sum_tiles<T, kTop>(row, a.V, a.s, xt, wave, a.NT, NW, lane, maxima);
  if (lane == 0) part[wave][0] = w.R, part[wave][1] = w.z, part[wave][2] = w.h;
  if constexpr (kTop) lane_maxima[wave][lane] = w.lane_max;
  __syncthreads();
  if (wave == 0) {
    double R = lane < NW ? part[lane % NW][0] : -__builtin_inf();
    double Z = lane < NW ? part[lane % NW][1] : 0.0, H = lane < NW ? part[lane % NW][2] : 0.0;
    join_parts(R, Z, H);
    RowLaw law{};
    const bool ok = write_law<T>(a, row_i, xt, R, Z, H, &law, lane);
    if (kTop && lane == 0) sh.ok = ok, sh.law = law;
  } else if (kTop && wave == 1) {
    float lm = lane_maxima[0][lane];
#pragma unroll
    for (int i = 1; i < (kTop ? NW : 1); ++i) lm = fmaxf(lm, lane_maxima[i][lane]);
    select_chunks(maxima, a.NT * kChunksPerTile, a.top, lm, sh.pick, lane);
  }
  if constexpr (kTop) {
    __syncthreads();
    if (sh.ok) pick<T, NW>(a, row_i, row, maxima, sh.pick, sh.law, wave, lane);
  }
}

// Block (row, part): a.part_tiles tiles of a live row.
template <typename T, bool kTop>
__global__ void __launch_bounds__(kBlock) lp_part_kernel(LpArgs a) {
  __shared__ double part[kWavesPerBlock][3];
  __shared__ float lane_maxima[kTop ? kWavesPerBlock : 1][kWave];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  // Blocks go to the eight XCDs in turn; a batch's dead rows come at the same
  // places of every sequence.  Each 64 blocks are turned by one more place, so
  // that no XCD gets the same rows of all sequences.
  uint32_t v = blockIdx.x;
  if ((v | 63u) < gridDim.x) v = (v & ~63u) | ((v + (v >> 6)) & 63u);
  const uint32_t row_i = v / (uint32_t)a.NP;
  const int p = (int)(v - row_i * (uint32_t)a.NP);
  if ((uint32_t)a.tokens[row_i] >= (uint32_t)a.V) return;
  const T* row = static_cast<const T*>(a.logits) + (size_t)row_i * (size_t)a.V;
  const int first = p * a.part_tiles;
  const WaveSums w =
      sum_tiles<T, kTop>(row, a.V, a.s, to_f32(row[a.tokens[row_i]]), first + wave, min(first + a.part_tiles, a.NT), kWavesPerBlock, lane,
                         kTop ? a.chunks + (size_t)row_i * (size_t)(a.NT * kChunksPerTile) : nullptr);
  if (lane == 0) part[wave][0] = w.R, part[wave][1] = w.z, part[wave][2] = w.h;
  if constexpr (kTop) lane_maxima[wave][lane] = w.lane_max;
  __syncthreads();
  if (kTop && wave == 1)
    a.lanes[((size_t)row_i * a.NP + p) * kWave + lane] =
        fmaxf(fmaxf(lane_maxima[0][lane], lane_maxima[kTop ? 1 : 0][lane]),
              fmaxf(lane_maxima[kTop ? 2 : 0][lane], lane_maxima[kTop ? 3 : 0][lane]));
  if (wave != 0) return;
  double R = lane < kWavesPerBlock ? part[lane & 3][0] : -__builtin_inf();
  double Z = lane < kWavesPerBlock ? part[lane & 3][1] : 0.0, H = lane < kWavesPerBlock ? part[lane & 3][2] : 0.0;
  join_parts(R, Z, H);
  if (lane == 0) a.parts[(size_t)row_i * a.NP + p] = LogprobsPart{R, Z, H};
}

template <typename T, int NW>
__global__ void __launch_bounds__(kWave * NW) lp_pick_kernel(LpArgs a) {
  __shared__ RowShared sh;
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const size_t row_i = blockIdx.x;
  const int token = a.tokens[row_i];
  if ((uint32_t)token >= (uint32_t)a.V) {
    if (wave == 0) write_nothing(a, row_i, lane);
    return;
  }
  const T* row = static_cast<const T*>(a.logits) + row_i * (size_t)a.V;
  float* maxima = a.top > 0 ? a.chunks + row_i * (size_t)(a.NT * kChunksPerTile) : nullptr;
  if (wave == 0) {
    const float xt = to_f32(row[token]);
    const LogprobsPart* parts = a.parts + row_i * a.NP;
    double R = -__builtin_inf(), Z = 0.0, H = 0.0;
    for (int p0 = 0; p0 < a.NP; p0 += kWave) {
      // 64 parts with what is joined so far
      const LogprobsPart p = p0 + lane < a.NP ? parts[p0 + lane] : LogprobsPart{-__builtin_inf(), 0.0, 0.0};
      double r = p.R, z = p.z, h = p.h;
      join_parts(r, z, h);
      if (p0 == 0) {
        R = r, Z = z, H = h;
      } else {
        double r2 = lane == 0 ? R : lane == 1 ? r : -__builtin_inf();
        double z2 = lane == 0 ? Z : lane == 1 ? z : 0.0, h2 = lane == 0 ? H : lane == 1 ? h : 0.0;
        join_parts(r2, z2, h2);
        R = r2, Z = z2, H = h2;
      }
    }
    RowLaw law{};
    const bool ok = write_law<T>(a, row_i, xt, R, Z, H, &law, lane);
    if (lane == 0) sh.ok = ok, sh.law = law;
  } else if (wave == 1 && a.top > 0) {
    const float* lanes = a.lanes + row_i * (size_t)a.NP * kWave + lane;
    float lm = lanes[0];
#pragma unroll 8
    for (int p = 1; p < a.NP; ++p) lm = fmaxf(lm, lanes[(size_t)p * kWave]);
    select_chunks(maxima, a.NT * kChunksPerTile, a.top, lm, sh.pick, lane);
  }
  if (a.top == 0) return;
  __syncthreads();
  if (sh.ok) pick<T, NW>(a, row_i, row, maxima, sh.pick, sh.law, wave, lane);
}

template <typename T>
hipError_t launch_typed(const LpArgs& a, int N, hipStream_t st) {
  const dim3 rows((unsigned)N);
  if (a.NP == 0) {
    const bool wide = N <= kLpWideRows;
    if (a.top > 0) {
      if (wide) hipLaunchKernelGGL((lp_row_kernel<T, 16, true>), rows, dim3(kWave * 16), 0, st, a);
      else hipLaunchKernelGGL((lp_row_kernel<T, 4, true>), rows, dim3(kWave * 4), 0, st, a);
    } else {
      if (wide) hipLaunchKernelGGL((lp_row_kernel<T, 16, false>), rows, dim3(kWave * 16), 0, st, a);
      else hipLaunchKernelGGL((lp_row_kernel<T, 4, false>), rows, dim3(kWave * 4), 0, st, a);
    }
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((size_t)N * (size_t)a.NP));
  if (a.top > 0) hipLaunchKernelGGL((lp_part_kernel<T, true>), grid, dim3(kBlock), 0, st, a);
  else hipLaunchKernelGGL((lp_part_kernel<T, false>), grid, dim3(kBlock), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Eight waves join a row sooner (512 rows of 151936: 9.2 against 10.7 us);
  // with more rows than the chip has blocks of eight at a time four do (1152
  // rows of 262144: 12.8 against 17.8 us).
  if (N <= kLpManyRows) hipLaunchKernelGGL((lp_pick_kernel<T, 8>), rows, dim3(kWave * 8), 0, st, a);
  else hipLaunchKernelGGL((lp_pick_kernel<T, 4>), rows, dim3(kWave * 4), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobsShape& s, const LogprobsWorkspace& w, const void* logits,
                           const int32_t* tokens, int dtype, float temperature, float* logprobs, float* entropy,
                           int32_t* top_ids, float* top_logprobs, void* workspace, hipStream_t st) {
  LpArgs a{};
  a.logits = logits;
  a.tokens = tokens;
  a.parts = reinterpret_cast<LogprobsPart*>(static_cast<char*>(workspace) + w.parts);
  a.chunks = s.top > 0 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + w.chunks) : nullptr;
  a.lanes = s.top > 0 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + w.lanes) : nullptr;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.V = s.V;
  a.NT = s.NT;
  a.NP = s.NP;
  a.part_tiles = s.part_tiles;
  a.top = s.top;
  a.s = (float)(1.4426950408889634073599 / (double)temperature);
  return dtype == 1 ? launch_typed<uint16_t>(a, s.N, st) : launch_typed<float>(a, s.N, st);
}

}  // namespace sv
