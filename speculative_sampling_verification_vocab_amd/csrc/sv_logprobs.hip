// Log-probabilities of given tokens, the rows' entropies and their likeliest
// alternatives.  With a_v = x_v * s - ref, s = log2(e) / T and any reference:
//   Z = sum 2^a_v,  H = sum 2^a_v a_v,
//   ln P(t) = ln 2 (a_t - log2 Z),  entropy = ln 2 (log2 Z - H / Z).
// Two launches:
//   * lp_tiles_kernel reads each live row once, one wave per tile of 64
//     16-byte vectors x 8 (4096 bf16 or 2048 fp32 logits): the tile's
//     reference (its maximum), Z and H, and the maxima of its 8 chunks of 512
//     (256) consecutive logits.
//   * lp_pick_kernel, one wave per row, adds the tiles in fp64 and finds the
//     alternatives: the n chunks with the largest maxima (equal ones by lower
//     position) hold the n best tokens, for the n maxima themselves come
//     before everything in any other chunk; so it reads n chunks again, keeps
//     what is not below the n-th maximum, and ranks that.
// The first launch is bound by HBM: about ten VALU operations per bf16 logit
// (unpack, half a maximum, FMA, a quarter-rate exponential, add, FMA) against
// the eleven that pass in the time of its two bytes.

#include "sv_common.h"
#include "sv_host_quant.h"
#include "sv_internal.h"

namespace sv {

namespace {

struct LpArgs {
  const void* logits;      // [N][V]
  const int32_t* tokens;   // [N]
  LogprobsTile* tiles;     // [N][NT]
  float* chunks;           // [N][NT * 8]; null without alternatives
  float* logprobs;         // [N]
  float* entropy;          // [N] or null
  int32_t* top_ids;        // [N][top]
  float* top_logprobs;     // [N][top]
  int V, NT, groups, top;
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

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

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

template <typename T, bool kTop>
__global__ void __launch_bounds__(kBlock) lp_tiles_kernel(LpArgs a) {
  constexpr int V8 = Elem<T>::kVec, kTileN = kTile<T>;
  const int lane = threadIdx.x & (kWave - 1);
  const uint32_t row_i = blockIdx.x / (uint32_t)a.groups;
  const int tile = (int)(blockIdx.x - row_i * (uint32_t)a.groups) * kWavesPerBlock + threadIdx.x / kWave;
  if (tile >= a.NT || (uint32_t)a.tokens[row_i] >= (uint32_t)a.V) return;
  const T* row = static_cast<const T*>(a.logits) + (size_t)row_i * (size_t)a.V;
  const int pre = row_lead(row);
  const int q0 = tile * kTileN;
  u32x4 raw[kLoads];
  if (q0 >= pre && q0 - pre + kTileN <= a.V) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) raw[j] = stream16(row + (q0 - pre) + j * (kWave * V8) + lane * V8);
  } else {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) raw[j] = load_vec(row, a.V, pre, q0 + j * (kWave * V8) + lane * V8);
  }

  float c[kLoads];
#pragma unroll
  for (int j = 0; j < kLoads; ++j) {
    c[j] = raw_elem<T>(raw, j * V8);
#pragma unroll
    for (int k = 1; k < V8; ++k) c[j] = fmaxf(c[j], raw_elem<T>(raw, j * V8 + k));
  }
  float m;
  if constexpr (kTop) {
    m = wave_max8(c, lane);
    if (lane < 8) a.chunks[((size_t)row_i * a.NT + tile) * kChunksPerTile + lane] = m;
    m = fmaxf(m, dpp::mov<dpp::kQuadSwap1, 0xf>(0.0f, m));
    m = fmaxf(m, dpp::mov<dpp::kQuadSwap2, 0xf>(0.0f, m));
    m = fmaxf(m, dpp::mov<dpp::kHalfMirror, 0xf>(0.0f, m));
    m = dpp::lane63(m);
  } else {
    m = wave_max(lane_max(c));
  }

  // Sums of a tile against its own maximum, in fp32: 64 terms per lane in
  // four chains, then across lanes.  A reference that cannot be taken out of
  // the FMA (see kExpRefWide) subtracts first.
  const float s = a.s, hi = exp_ref_hi(m, s);
  const bool wide = exp_ref_wide(m, s);
  float z4[4] = {0.f, 0.f, 0.f, 0.f}, h4[4] = {0.f, 0.f, 0.f, 0.f};
  if (!wide) {
#pragma unroll
    for (int e = 0; e < kLoads * V8; ++e) {
      const float t = __builtin_fmaf(raw_elem<T>(raw, e), s, -hi), p = exp2_fast(t);
      z4[e & 3] += p;
      h4[e & 3] = __builtin_fmaf(p, t, h4[e & 3]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kLoads * V8; ++e) {
      const float t = (raw_elem<T>(raw, e) - m) * s, p = exp2_fast(t);
      z4[e & 3] += p;
      h4[e & 3] = __builtin_fmaf(p, t, h4[e & 3]);
    }
  }
  const float z = (z4[0] + z4[1]) + (z4[2] + z4[3]);
  float h = (h4[0] + h4[1]) + (h4[2] + h4[3]);
  if (__any(h != h)) {
    // A logit of -inf (0 * -inf): the products again, with exponents that
    // give 0 either way kept finite.  A NaN logit or +inf stays visible in z.
    h = 0.0f;
#pragma unroll
    for (int e = 0; e < kLoads * V8; ++e) {
      const float x = raw_elem<T>(raw, e);
      const float t = fmaxf(wide ? (x - m) * s : __builtin_fmaf(x, s, -hi), -1.0e4f);
      h = __builtin_fmaf(exp2_fast(t), t, h);
    }
  }
  const float zs = wave_sum(z), hs = wave_sum(h);
  if (lane == 0) {
    LogprobsTile r;
    r.ref = m == -__builtin_inff() ? -__builtin_inf() : wide ? (double)m * (double)s : (double)hi;
    r.z = zs;
    r.h = hs;
    a.tiles[(size_t)row_i * a.NT + tile] = r;
  }
}

// fp32 bits in the order of the values (-0 as 0).
__device__ __forceinline__ int order_of(float x) {
  const int b = __float_as_int(x + 0.0f);
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float value_of(int o) { return __int_as_float(o ^ ((o >> 31) & 0x7fffffff)); }

constexpr int kList = 1024;        // candidates held at a time; a chunk adds at most 512
constexpr int kChunksLds = 1024;   // chunk maxima held in LDS (V up to 524288 bf16, 262144 fp32)
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
  __syncthreads();
  if (lane < n) list[lane] = mine;
  __syncthreads();
}

__device__ __forceinline__ double wave_max64(double v) {
  return dpp::reduce(v, -__builtin_inf(), [](double x, double y) { return x > y ? x : y; });
}

template <typename T>
__global__ void __launch_bounds__(kWave) lp_pick_kernel(LpArgs a) {
  constexpr int V8 = Elem<T>::kVec, kChunk = kWave * V8;
  constexpr double kLn2 = 0.69314718055994530942;
  __shared__ float maxima[kChunksLds];
  __shared__ Candidate list[kList];
  __shared__ int count;
  const int lane = threadIdx.x;
  const size_t row_i = blockIdx.x;
  const float nan = __builtin_nanf("");
  const int token = a.tokens[row_i];
  const T* row = static_cast<const T*>(a.logits) + row_i * (size_t)a.V;
  bool ok = (uint32_t)token < (uint32_t)a.V;
  double R = -__builtin_inf(), Z = 0.0, H = 0.0, log2Z = 0.0;
  if (ok) {
    const float xt = to_f32(row[token]);
    const LogprobsTile* tiles = a.tiles + row_i * a.NT;
    for (int t = lane; t < a.NT; t += kWave) R = fmax(R, tiles[t].ref);
    R = wave_max64(R);
    for (int t = lane; t < a.NT; t += kWave) {
      const LogprobsTile r = tiles[t];
      if (r.z == 0.0f) continue;  // nothing but -inf
      const double dr = r.ref - R, w = exp2(dr);
      Z += w * (double)r.z;
      H += w * ((double)r.h + dr * (double)r.z);
    }
    Z = wave_sum(Z);
    H = wave_sum(H);
    ok = Z > 0.0 && Z < __builtin_inf() && R > -__builtin_inf() && R < __builtin_inf();
    log2Z = log2(Z);
    if (ok && lane == 0) {
      a.logprobs[row_i] = (float)(kLn2 * ((double)xt * (double)a.s - R - log2Z));
      if (a.entropy) a.entropy[row_i] = (float)(kLn2 * (log2Z - H / Z));
    }
  }
  if (!ok) {
    if (lane == 0) {
      a.logprobs[row_i] = nan;
      if (a.entropy) a.entropy[row_i] = nan;
    }
    if (lane < a.top) {
      a.top_ids[row_i * a.top + lane] = -1;
      a.top_logprobs[row_i * a.top + lane] = nan;
    }
    return;
  }
  if (a.top == 0) return;

  // The chunks with the a.top largest maxima: lane r holds the r-th.
  const int NC = a.NT * kChunksPerTile, n = a.top;
  float* stored = a.chunks + row_i * (size_t)NC;
  const bool in_lds = NC <= kChunksLds;
  if (in_lds)
    for (int i = lane; i < NC; i += kWave) maxima[i] = stored[i];
  if (lane == 0) count = 0;
  __syncthreads();
  auto take_chunks = [&](float* v, int* chosen) {
    int best, at, found = 0;
    auto order = [](float x) { return order_of(x); };
    best_of_lane(v, NC, lane, order, &best, &at);
    const int ninf = order_of(-__builtin_inff());
    int last = kNone;
    for (; found < n; ++found) {
      const int o = wave_max(best);
      if (o <= ninf) break;
      const int c = wave_min(best == o ? at : 0x7fffffff);
      if (lane == found) *chosen = c;
      last = o;
      if (at == c) {
        v[c] = -__builtin_inff();
        best_of_lane(v, NC, lane, order, &best, &at);
      }
    }
    // fewer chunks than n: no bound yet
    return found == n ? Candidate{last, found} : Candidate{kNone, found};
  };
  int chosen = 0;
  const Candidate got = in_lds ? take_chunks(maxima, &chosen) : take_chunks(stored, &chosen);
  const int chunks = got.id;
  const int pre = row_lead(row);
  // Candidates come before or are `bound_o`, `bound_id`.
  int bound_o = max(got.order, order_of(-__builtin_inff()) + 1), bound_id = 0x7fffffff;

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
    const int lo = order_of(lm);
    int rank = 0;
    for (int j = 0; j < kWave; ++j) {
      const int o = __builtin_amdgcn_readlane(lo, j);
      rank += o > lo || (o == lo && j < lane) ? 1 : 0;
    }
    bound_o = max(bound_o, wave_max(rank == n - 1 ? lo : kNone));
  }
  for (int first = 0; first < chunks; first += kBatch) {
    u32x4 w[kBatch];
    load_batch(first, w);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (first + k >= chunks) break;
      if (count > kList - kChunk) {  // uniform: count is read after a barrier
        keep_best(list, count, n, lane);
        bound_o = list[n - 1].order;
        bound_id = list[n - 1].id;
        __syncthreads();
        if (lane == 0) count = n;
        __syncthreads();
      }
      const u32x4 one[1] = {w[k]};
      const int base = __builtin_amdgcn_readlane(chosen, first + k) * kChunk + lane * V8 - pre;
      if (order_of(raw_lane_max<T>(one)) >= bound_o) {
#pragma unroll
        for (int e = 0; e < V8; ++e) {
          const int o = order_of(raw_elem<T>(one, e));
          if (before(o, base + e, bound_o, bound_id)) list[atomicAdd(&count, 1)] = Candidate{o, base + e};
        }
      }
      __syncthreads();
    }
  }
  int have = count;
  if (have > kWave) {
    keep_best(list, have, n, lane);
    have = n;
  }
  const Candidate mine = lane < have ? list[lane] : Candidate{kNone, 0x7fffffff};
  int rank = 0;
  for (int j = 0; j < have; ++j)
    rank += before(__builtin_amdgcn_readlane(mine.order, j), __builtin_amdgcn_readlane(mine.id, j), mine.order, mine.id)
                ? 1 : 0;
  if (lane < have && rank < n) {
    a.top_ids[row_i * n + rank] = mine.id;
    a.top_logprobs[row_i * n + rank] = (float)(kLn2 * ((double)value_of(mine.order) * (double)a.s - R - log2Z));
  }
  if (lane >= have && lane < n) {
    a.top_ids[row_i * n + lane] = -1;
    a.top_logprobs[row_i * n + lane] = -__builtin_inff();
  }
}

template <typename T>
hipError_t launch_typed(const LpArgs& a, int N, hipStream_t st) {
  const dim3 grid((unsigned)((size_t)N * (size_t)a.groups));
  if (a.top > 0) hipLaunchKernelGGL((lp_tiles_kernel<T, true>), grid, dim3(kBlock), 0, st, a);
  else hipLaunchKernelGGL((lp_tiles_kernel<T, false>), grid, dim3(kBlock), 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((lp_pick_kernel<T>), dim3((unsigned)N), dim3(kWave), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_logprobs(const LogprobsShape& s, const LogprobsWorkspace& w, const void* logits,
                           const int32_t* tokens, int dtype, float temperature, float* logprobs, float* entropy,
                           int32_t* top_ids, float* top_logprobs, void* workspace, hipStream_t st) {
  LpArgs a{};
  a.logits = logits;
  a.tokens = tokens;
  a.tiles = reinterpret_cast<LogprobsTile*>(static_cast<char*>(workspace) + w.tiles);
  a.chunks = s.top > 0 ? reinterpret_cast<float*>(static_cast<char*>(workspace) + w.chunks) : nullptr;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.V = s.V;
  a.NT = s.NT;
  a.groups = s.groups;
  a.top = s.top;
  a.s = (float)(1.4426950408889634073599 / (double)temperature);
  return dtype == 1 ? launch_typed<uint16_t>(a, s.N, st) : launch_typed<float>(a, s.N, st);
}

}  // namespace sv
