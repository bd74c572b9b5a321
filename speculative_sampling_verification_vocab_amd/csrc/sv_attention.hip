// Attention of a tree of drafted tokens over a KV cache and the tree's own
// entries (gfx950, wave64).  For node i and query head h of KV head k:
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(c q.k_j - m),  c = scale * log2(e),
// over the entries j that node i sees, with m a running reference, each row's
// own: when a tile's largest c q.k_j passes m by more than 8, m becomes that
// maximum and what was summed is scaled down; otherwise p_j <= 2^8 and nothing is.
//
// The rows of a KV head are its G query heads of every node.  Four waves of a
// block take 16 MT rows each against keys of their own, 32 at a time, and a
// tile never leaves the wave's registers:
//   S^T = K Q^T   matrix products with the keys as rows: a lane reads KW
//                 consecutive values of its key straight from memory;
//   P             stays where S^T's result is: lane (g, m) holds keys 16 u + 4 g + r
//                 (u < 2, r < 4) of row m, and the second product takes its
//                 inner index in just that order;
//   O^T += V^T P^T  a lane reads CW consecutive values of the same keys' rows,
//                 whole rows of V at a time; in bf16, value j of eight keys is
//                 brought into one operand by byte permutes.
// So keys and values are read once, with no shared memory and no barrier in
// the loop, and a tile's keys are asked for while the one before is worked on.
// The waves' results meet in shared memory, 16 rows at a time, and those of
// blocks that share the keys in a second launch (tree_join_kernel); sv_host_tree.h
// says how the keys are shared out.
//
// More than 64 rows of a KV head are bound by the products and not by memory:
// then each wave has 32 rows of its own and all four take the same keys,
// 64 at a time from shared memory, in two buffers, bf16 values by direct loads
// and codes decoded once for all waves.
//
// Measured (32 query heads on 8 KV heads of 128, half to all of L cached):
//   B=64 N=1 L=8192 bf16      299 us  5.4 TB/s: the cache's bytes, of 6.0 to 6.4 that reads alone reach
//   B=32 N=8 L=8192 bf16      184 us  4.4 TB/s, and 8-bit 122 us, 3.4 TB/s
//   B=1 N=16 L=131072 bf16    119 us  4.5 TB/s, and 8-bit 78 to 92 us by machine, 2.9 to 3.5 TB/s: the registers leave
//                             two waves per SIMD, and the loads that those have in flight bound it
//   B=64 N=64 L=8192 bf16     636 us  655 TFLOP/s of 1130 that a large product reaches: softmax and permutes
//                             share the issue slots with the matrix instructions
//
// Sums, maxima and both products' accumulators are fp32.  The weights p are
// rounded to bf16 for the bf16 product, half a step of 2^-8 each at random,
// like the values they multiply.
//
// Entries that a row does not see weigh exactly 0 whatever they hold: their
// score is replaced, and where a tile with such entries has a value that is not
// finite, that value is left out of the product and its own product with the
// weight added to the rows that see it: an infinity or a NaN, and NaN for an
// infinity of weight 0, as the matrix product has it for tiles seen whole.

#include <type_traits>

#include "sv_dma.h"
#include "sv_internal.h"
#include "sv_quant.h"
#include "sv_tree.h"

namespace sv {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

struct AttnArgs {
  const void *q, *k_new, *v_new;              // [B][N][Hq][D], [B][N][Hkv][D]
  const uint8_t *k_cache, *v_cache;           // [B][L][Hkv][D] values or codes
  const uint8_t *k_scales, *v_scales;         // [B][L][nb]
  const int32_t *parents, *cache_len;         // [B][N], [B]
  void* out;                                  // [B][N][Hq][D]
  float2* stats;                              // [slots][groups][rows] reference and sum
  float* acc;                                 // [slots][groups][rows][D]
  int B, N, Hq, Hkv, G, D, L, nb, R, groups;
  int split, ranges, least, step, span;       // see AttnPlan
  int window, sinks;
  float c;
};

constexpr int kStage = kAttnStage;  // keys that the waves of a block share
constexpr float kSlack = 8.0f;      // how far a weight's exponent may pass its reference
constexpr float kNinf = -__builtin_inff(), kMost = 3.402823466e38f;  // the largest float

__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- operands -------------------------------------------------------------------

// n consecutive values of a row as the matrix product takes them: dwords of two
// bf16, or floats.
template <typename T, int n>
struct Frag {
  static constexpr int kWords = std::is_same<T, float>::value ? n : n / 2;
  uint32_t w[kWords];
};

template <typename T, int n>
__device__ __forceinline__ void load_values(const uint8_t* p, Frag<T, n>& f) {
  constexpr int W = Frag<T, n>::kWords;
#pragma unroll
  for (int i = 0; i + 4 <= W; i += 4) {
    const u32x4 v = *reinterpret_cast<const typename AnyVector<typename std::conditional<
        std::is_same<T, float>::value, float, uint16_t>::type>::type*>(p + 4 * i);
#pragma unroll
    for (int q = 0; q < 4; ++q) f.w[i + q] = v[q];
  }
  if constexpr (W % 4 == 2) {
    typedef uint32_t pair __attribute__((ext_vector_type(2), aligned(2)));
    const pair v = *reinterpret_cast<const pair*>(p + 4 * (W - 2));
    f.w[W - 2] = v[0];
    f.w[W - 1] = v[1];
  }
}

template <typename T, int n>
__device__ __forceinline__ void clear(Frag<T, n>& f) {
#pragma unroll
  for (int i = 0; i < Frag<T, n>::kWords; ++i) f.w[i] = 0;
}

// n codes with their scale to a fragment.
template <typename T, int n>
__device__ __forceinline__ void decode(const uint32_t (&q)[n / 4], const float* scale, Frag<T, n>& f) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
  for (int i = 0; i < n / 4; ++i) {
    const float s = scale[i / 2];
    if constexpr (std::is_same<T, float>::value) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[i], true);
      f.w[4 * i] = __float_as_uint(lo[0] * s);
      f.w[4 * i + 1] = __float_as_uint(lo[1] * s);
      f.w[4 * i + 2] = __float_as_uint(hi[0] * s);
      f.w[4 * i + 3] = __float_as_uint(hi[1] * s);
    } else {
      f.w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], s, false));
      f.w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[i], s, true));
    }
  }
#endif
}

// 2^(byte - 127) by its bits; 255 stands for NaN and 0 for 2^-127.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

template <typename T>
constexpr int kEs = std::is_same<T, float>::value ? 4 : 2;

// Rows of keys or values: base is the first one's address for the block's head,
// and rows are `stride` bytes apart.
struct Rows {
  const uint8_t* base;
  const uint8_t* scales;  // its first row's scale byte 0
  uint32_t stride;
};

// The shape of a kernel's operands.
template <typename T, bool kQ, int DP, int MT, bool kWhole>
struct Shape {
  static constexpr bool kF32 = std::is_same<T, float>::value;
  static constexpr bool kAll = kWhole;                   // heads of DP values, no less
  static constexpr int U = kF32 && DP == 256 ? 1 : 2;    // keys / 16 of a tile (registers)
  static constexpr int kKeys = 16 * U;
  static constexpr int kSlots = 4 * U;                   // keys of a tile that a lane holds weights of
  static constexpr int KW = kQ ? 16 : kF32 ? 4 : 8;      // consecutive values of a key per lane
  static constexpr int KS = DP / (4 * KW);               // such pieces per key
  static constexpr int CW = DP == 64 || (kF32 && !kQ) ? 4 : 8;  // consecutive values of a value row per lane
  static constexpr int VS = DP / (16 * CW);              // such pieces per row
  static constexpr int OT = DP / 16;                     // result tiles of 16 values: (piece, value)
  typedef Frag<T, KW> Keys[U][KS];
  typedef Frag<T, CW> Values[kSlots][VS];
};

// The tile's key of a lane's slot i: 16 u + 4 g + r.
__device__ __forceinline__ int key_of(int i, int lane) { return i / 4 * 16 + (lane >> 4) * 4 + i % 4; }

// Keys u * 16 + lane % 16 of a tile whose last key is `last`.
template <typename S, typename T>
__device__ __forceinline__ void load_keys(const Rows& r, int last, int D, int lane, typename S::Keys& k) {
  constexpr int n = S::KW > 8 ? 8 : S::KW;  // D is a multiple of 8
#pragma unroll
  for (int u = 0; u < S::U; ++u) {
    const uint32_t row = (uint32_t)min(u * 16 + (lane & 15), last) * r.stride;
#pragma unroll
    for (int s = 0; s < S::KS; ++s)
#pragma unroll
      for (int e = 0; e < S::KW; e += n) {
        const int d = s * 4 * S::KW + (lane >> 4) * S::KW + e;
        Frag<T, n> f;
        load_values<T, n>(r.base + (row + (uint32_t)((S::kAll || d < D ? d : 0) * kEs<T>)), f);
#pragma unroll
        for (int i = 0; i < Frag<T, n>::kWords; ++i) k[u][s].w[e * kEs<T> / 4 + i] = f.w[i];
      }
  }
}

// Values of the lane's slots: whole rows, CW consecutive values per lane and piece.
template <typename S, typename T>
__device__ __forceinline__ void load_rows(const Rows& r, int last, int D, int lane, typename S::Values& v) {
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    const uint32_t row = (uint32_t)min(key_of(i, lane), last) * r.stride;
#pragma unroll
    for (int s = 0; s < S::VS; ++s) {
      const int d = s * 16 * S::CW + (lane & 15) * S::CW;
      load_values<T, S::CW>(r.base + (row + (uint32_t)((S::kAll || d < D ? d : 0) * kEs<T>)), v[i][s]);
    }
  }
}

// Keys as codes, KW per piece, and a scale for each 8.
template <typename S>
struct KeyCodes {
  uint32_t w[S::U][S::KS][S::KW / 4];
  uint32_t scale[S::U][S::KS][S::KW / 8];
};
template <typename S>
struct ValueCodes {
  uint32_t w[S::kSlots][S::VS][S::CW / 4];
  uint32_t scale[S::kSlots][S::VS];
};

template <int n>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[n / 4]) {
  if constexpr (n == 8) {
    const u32x2_any v = *reinterpret_cast<const u32x2_any*>(p);
    w[0] = v[0];
    w[1] = v[1];
  } else {
    typedef uint32_t word __attribute__((aligned(1)));
    w[0] = *reinterpret_cast<const word*>(p);
  }
}

// one: the head lies in whole blocks of 128, or inside one, so that a scale
// serves 128 values (or all of them).
template <typename S>
__device__ __forceinline__ void load_key_codes(const Rows& r, int nb, int head, int last, int D, bool one, int lane,
                                               KeyCodes<S>& c) {
  constexpr int kPer128 = 128 / (4 * S::KW);  // pieces of 128 values
#pragma unroll
  for (int u = 0; u < S::U; ++u) {
    const uint32_t key = (uint32_t)min(u * 16 + (lane & 15), last);
    const uint32_t row = key * r.stride;
#pragma unroll
    for (int s = 0; s < S::KS; ++s) {
      const int d = (s * 4 + (lane >> 4)) * S::KW;
      if (S::KW == 16 && (S::kAll || D % 16 == 0)) {
        const u32x4 v = *reinterpret_cast<const u32x4_any1*>(r.base + (row + (uint32_t)(S::kAll || d < D ? d : 0)));
#pragma unroll
        for (int q = 0; q < S::KW / 4; ++q) c.w[u][s][q] = v[q];
      } else {
#pragma unroll
        for (int e = 0; e < S::KW / 8; ++e) {
          uint32_t v[2];
          load_codes<8>(r.base + (row + (uint32_t)(S::kAll || d + 8 * e < D ? d + 8 * e : 0)), v);
          c.w[u][s][2 * e] = v[0];
          c.w[u][s][2 * e + 1] = v[1];
        }
      }
      if (one) {
        if (s % kPer128 == 0) c.scale[u][s][0] = r.scales[key * (uint32_t)nb + (uint32_t)((head + s * 4 * S::KW) >> 7)];
        else c.scale[u][s][0] = c.scale[u][s - s % kPer128][0];
        if constexpr (S::KW == 16) c.scale[u][s][1] = c.scale[u][s][0];
      } else {
#pragma unroll
        for (int e = 0; e < S::KW / 8; ++e) {
          const int at = d + 8 * e < D ? d + 8 * e : 0;
          c.scale[u][s][e] = r.scales[key * (uint32_t)nb + (uint32_t)((head + at) >> 7)];
        }
      }
    }
  }
}

template <typename S>
__device__ __forceinline__ void load_row_codes(const Rows& r, int nb, int head, int last, int D, int lane,
                                               ValueCodes<S>& c) {
#pragma unroll
  for (int i = 0; i < S::kSlots; ++i) {
    const uint32_t key = (uint32_t)min(key_of(i, lane), last);
#pragma unroll
    for (int s = 0; s < S::VS; ++s) {
      const int d = s * 16 * S::CW + (lane & 15) * S::CW;
      const int at = S::kAll || d < D ? d : 0;
      load_codes<S::CW>(r.base + (key * r.stride + (uint32_t)at), c.w[i][s]);
      c.scale[i][s] = r.scales[key * (uint32_t)nb + (uint32_t)((head + at) >> 7)];
    }
  }
}

// ---- products -------------------------------------------------------------------

__device__ __forceinline__ f32x4 mfma(const uint32_t (&a)[4], const uint32_t (&b)[4], f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
      0, 0, 0);
#else
  return c;
#endif
}
__device__ __forceinline__ f32x4 mfma(float a, float b, f32x4 c) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
#else
  return c;
#endif
}

// c += the products of n values of 16 keys with those of 16 rows.
template <typename T, int n>
__device__ __forceinline__ f32x4 product(const Frag<T, n>& a, const Frag<T, n>& b, f32x4 c) {
  if constexpr (std::is_same<T, float>::value) {
#pragma unroll
    for (int i = 0; i < n; ++i) c = mfma(__uint_as_float(a.w[i]), __uint_as_float(b.w[i]), c);
  } else {
#pragma unroll
    for (int i = 0; i < n / 2; i += 4) {
      const uint32_t x[4] = {a.w[i], a.w[i + 1], a.w[i + 2], a.w[i + 3]};
      const uint32_t y[4] = {b.w[i], b.w[i + 1], b.w[i + 2], b.w[i + 3]};
      c = mfma(x, y, c);
    }
  }
  return c;
}

// The two halves of dwords a and b that hold value `odd` of each.
__device__ __forceinline__ uint32_t halves(uint32_t a, uint32_t b, int odd) {
  return __builtin_amdgcn_perm(b, a, odd ? 0x07060302u : 0x05040100u);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// What a wave keeps of its 16 MT rows.
template <typename S, int MT>
struct Sums {
  f32x4 o[MT][S::OT];  // tile (piece s, value j): rows 4 g + r are values s * 16 CW + (4 g + r) * CW + j
  float m[MT];         // reference, the same in the four lanes of a row
  float l[MT];         // the lane's part of the sum
};

// Values past the head stand for zeros: the queries' are, but 0 times an infinity is not 0.
template <typename S, typename T>
__device__ __forceinline__ void cut_key(int D, int s, int lane, Frag<T, S::KW>& k) {
#pragma unroll
  for (int i = 0; i < Frag<T, S::KW>::kWords; ++i) {
    const int d = s * 4 * S::KW + (lane >> 4) * S::KW + i * 4 / kEs<T>;
    k.w[i] = d < D ? k.w[i] : 0u;
  }
}

// Scores to weights: x[t][u][r] is row t * 16 + lane % 16's product with key 16 u + 4 g + r.  seen: null, or
// bit i says whether the row sees the lane's slot i.  A row's reference moves where its largest score passes it by
// more than the slack.
template <typename S, int MT, bool kMasked>
__device__ __forceinline__ void weigh(f32x4 (&x)[MT][S::U], const uint32_t (&seen)[MT], float c, Sums<S, MT>& z) {
  float top[MT];
  bool move = false;
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    top[t] = kNinf;
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i) {
      if constexpr (kMasked) x[t][i / 4][i % 4] = seen[t] >> i & 1 ? x[t][i / 4][i % 4] : kNinf;
      top[t] = fmaxf(top[t], x[t][i / 4][i % 4]);
    }
    top[t] *= c;
    move |= top[t] > z.m[t] + kSlack;
  }
  if (__any(move)) {
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float w = fmaxf(top[t], __shfl_xor(top[t], 16));
      w = fmaxf(w, __shfl_xor(w, 32));
      // Each row by its own scores: others' are not seen.  A score that c takes out of range leaves a finite reference,
      // so that its weight is infinite and the row NaN; with an infinite one its weight would be 0.
      const float m = w > z.m[t] + kSlack ? fminf(w, kMost) : z.m[t];
      const float f = m == z.m[t] ? 1.0f : exp2_of(z.m[t] - m);
      z.m[t] = m;
      z.l[t] *= f;
#pragma unroll
      for (int i = 0; i < S::OT; ++i) z.o[t][i] *= f;
    }
  }
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const float m = z.m[t] == kNinf ? 0.0f : z.m[t];
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i) {
      x[t][i / 4][i % 4] = exp2_of(__builtin_fmaf(x[t][i / 4][i % 4], c, -m));
      z.l[t] += x[t][i / 4][i % 4];
    }
  }
}

// z += V^T P^T for one piece of the tile's values.
template <typename S, typename T, int MT>
__device__ __forceinline__ void add_piece(const Frag<T, S::CW> (&v)[S::kSlots], int s, const f32x4 (&p)[MT][S::U],
                                          Sums<S, MT>& z) {
  if constexpr (S::kF32) {
#pragma unroll
    for (int i = 0; i < S::kSlots; ++i)
#pragma unroll
      for (int j = 0; j < S::CW; ++j)
#pragma unroll
        for (int t = 0; t < MT; ++t)
          z.o[t][s * S::CW + j] = mfma(__uint_as_float(v[i].w[j]), p[t][i / 4][i % 4], z.o[t][s * S::CW + j]);
  } else {
    uint32_t w[MT][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[t][i] = pack2(p[t][i / 2][2 * i % 4], p[t][i / 2][2 * i % 4 + 1]);
#pragma unroll
    for (int j = 0; j < S::CW; ++j) {
      uint32_t a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = halves(v[2 * i].w[j / 2], v[2 * i + 1].w[j / 2], j & 1);
#pragma unroll
      for (int t = 0; t < MT; ++t) z.o[t][s * S::CW + j] = mfma(a, w[t], z.o[t][s * S::CW + j]);
    }
  }
}

// Bits of w that an infinity or NaN has, and w without such values.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  if constexpr (std::is_same<T, float>::value) return (w & 0x7f800000u) == 0x7f800000u ? 0xffffffffu : 0u;
  else return ((w & 0x7f80u) == 0x7f80u ? 0xffffu : 0u) | ((w & 0x7f800000u) == 0x7f800000u ? 0xffff0000u : 0u);
}

// ---- the kernel -----------------------------------------------------------------

// The keys of a sequence with `length` cached entries: those that every node sees before the window (none
// without one), those from the first that the window of any node reaches, and the tree's own, each in tiles of
// `span` keys.
struct Keys {
  int n, low, first;                   // cached entries; 0 .. first and low .. n are read
  int tiles_first, tiles_cache, tiles; // ends of the three parts
  bool valid;
};

__device__ __forceinline__ Keys keys_of(const AttnArgs& a, int span, int length) {
  Keys k;
  k.valid = length >= 0 && length <= a.L;
  k.n = k.valid ? length : 0;
  k.low = k.first = 0;
  if (a.window > 0) {
    k.low = max(0, k.n - a.window + 1);
    k.first = min(a.sinks, k.low);
    if (k.first == k.low) k.first = k.low = 0;
  }
  k.tiles_first = (k.first + span - 1) / span;
  k.tiles_cache = k.tiles_first + (k.n - k.low + span - 1) / span;
  k.tiles = k.tiles_cache + (a.N + span - 1) / span;
  return k;
}

// The batch's tiles are numbered through, sequence by sequence and KV head by KV head, and cut into a.ranges equal
// ranges (a.least tiles at least), one per block: every block has the same to do, whatever the lengths.
__device__ __forceinline__ int lanes_scan(int v) {  // inclusive, over the lanes
  v += dpp::mov<dpp::kShr1, 0xf>(0, v);
  v += dpp::mov<dpp::kShr2, 0xf>(0, v);
  v += dpp::mov<dpp::kShr4, 0xf>(0, v);
  v += dpp::mov<dpp::kShr8, 0xf>(0, v);
  v += dpp::mov<dpp::kBcast15, 0xa>(0, v);
  v += dpp::mov<dpp::kBcast31, 0xc>(0, v);
  return v;
}

// Tiles of a range.  The whole batch has at most 2^31 - 1 tiles (checked on the host).
__device__ __forceinline__ int range_of(const AttnArgs& a, int total) {
  const int per = max((int)(((uint32_t)total + (uint32_t)a.ranges - 1) / (uint32_t)a.ranges), a.least);
  return (per + a.step - 1) / a.step * a.step;
}

// Tiles of range i (0: there is no such range), and where it begins: sequence, KV head and the tile's number there.
__device__ __forceinline__ int find_range(const AttnArgs& a, uint32_t range, int lane, int& b, int& h, int& tile) {
  const int t0 = lane < a.B ? keys_of(a, a.span, a.cache_len[lane]).tiles : 0;
  int all = t0;
  for (int i = lane + kWave; i < a.B; i += kWave) all += keys_of(a, a.span, a.cache_len[i]).tiles;
  const int total = dpp::lane63(lanes_scan(all)) * a.Hkv, per = range_of(a, total);
  if (range >= (uint32_t)a.ranges || (uint64_t)range * (uint32_t)per >= (uint64_t)total) return 0;
  const int p = (int)range * per;
  int before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kWave) {
    const int t = b0 == 0 ? t0 : b0 + lane < a.B ? keys_of(a, a.span, a.cache_len[b0 + lane]).tiles : 0;
    const int up_to = before + lanes_scan(t) * a.Hkv;
    const uint64_t hit = __ballot(p < up_to);
    if (hit != 0) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int of_b = __builtin_amdgcn_readlane(t, l), rem = p - (__builtin_amdgcn_readlane(up_to, l) - of_b * a.Hkv);
      b = b0 + l;
      h = rem / of_b;
      tile = rem - h * of_b;
      return min(per, total - p);
    }
    before = dpp::lane63(up_to);
  }
  return 0;
}

// Result of a row in shared memory: DP values, padded so that the sixteen rows
// of a tile start in different banks.
template <int DP>
constexpr int kPad = DP + 4;

// kShared: every wave has 16 MT rows of its own, and all take the same keys, 64 at a time from shared memory.
template <typename T, bool kQ, int DP, int MT, bool kWhole, bool kShared>
__global__ void __launch_bounds__(kBlock, DP == 256 || (DP == 128 && std::is_same<T, float>::value) ? 1 : 2)
    tree_attention_kernel(AttnArgs a) {
  typedef Shape<T, kQ && !kShared, DP, MT, kWhole> S;
  __shared__ uint64_t line_of[kMaxNodes];
  __shared__ int depth_of[kMaxNodes];
  __shared__ float2 stat[kWavesPerBlock][16 * MT];
  __shared__ float part[kShared ? 1 : kWavesPerBlock][kShared ? 4 : 16 * kPad<DP>];
  constexpr int kSpan = kShared ? kStage : S::kKeys;  // keys of a tile
  __shared__ __align__(256) uint8_t stage[kShared ? 2 : 1][2][kShared ? kStage * DP * 2 : 16];  // keys, values

  // Blocks that share keys, one per group of rows, are eight apart: the same XCD.
  const uint32_t eight = blockIdx.x / (8u * a.groups), rest = blockIdx.x % (8u * a.groups);
  const uint32_t item = eight * 8 + rest % 8;
  const int group = (int)(rest / 8);
  // scalar, and with it the tiles' addresses
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const size_t heads = (size_t)a.Hkv * a.D;                                   // values per entry
  constexpr int kKeys = S::kKeys;

  int b = 0, h = 0, begin = 0;
  int left = 0;  // tiles of the block's range
  if (a.ranges == 0) {
    const uint32_t pair = item / (uint32_t)a.split;
    if (pair >= (uint32_t)a.B * (uint32_t)a.Hkv) return;
    b = (int)(pair / (uint32_t)a.Hkv);
    h = (int)(pair % (uint32_t)a.Hkv);
    const uint32_t tiles = (uint32_t)keys_of(a, kSpan, a.cache_len[b]).tiles, piece = item - pair * (uint32_t)a.split;
    const uint32_t each = tiles / (uint32_t)a.split, more = tiles - each * (uint32_t)a.split;
    begin = (int)(piece * each + min(piece, more));
    left = (int)(each + (piece < more ? 1 : 0));
  } else {
    left = find_range(a, item, threadIdx.x & (kWave - 1), b, h, begin);
    if (left == 0) return;
  }
  // The pieces of the block's range, one pair's after the other.
#pragma unroll 1
  for (int nth = 0;; ++nth) {
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));  // or the lane's offsets would be kept from one piece to the next, in scratch
    const int lane = tid & (kWave - 1), g = lane >> 4;
    b = __builtin_amdgcn_readfirstlane(b);
    h = __builtin_amdgcn_readfirstlane(h);
    const Keys keys = keys_of(a, kSpan, a.cache_len[b]);
    const int n = keys.n, low = keys.low, first = keys.first;
    const int tiles_first = keys.tiles_first, tiles_cache = keys.tiles_cache;
    const bool valid = keys.valid;
    const int from = __builtin_amdgcn_readfirstlane(begin);
    const int to = __builtin_amdgcn_readfirstlane(min(keys.tiles, from + left));
    const bool alone = from == 0 && to == keys.tiles && a.split == 1;  // no other block has keys of these rows
    const size_t slot0 = a.ranges == 0 ? (size_t)item : 2 * (size_t)item + (nth > 0);

    if (wave == 0) {
      const TreeNode t = tree_node(lane < a.N ? a.parents[(size_t)b * a.N + lane] : -2, lane, a.N);
      line_of[lane] = t.line;
      depth_of[lane] = t.depth;
    }

    // The rows' queries: row m is node m / G, head m % G of the KV head's G.  Rows past the last have zeros: any query
    // read in their place would be another block's row, which that block may be writing (out is q).
    const int row0 = (kShared ? group * kWavesPerBlock + wave : group) * 16 * MT;
    Frag<T, S::KW> q[MT][S::KS];
    int node[MT];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      const int m = row0 + t * 16 + (lane & 15);
      const bool is_row = m < a.R;
      node[t] = is_row ? m / a.G : 0;
      const int head = h * a.G + (is_row ? m - node[t] * a.G : 0);
      const size_t row = ((size_t)b * a.N + node[t]) * a.Hq + head;
      const uint8_t* p = static_cast<const uint8_t*>(a.q) + row * (size_t)a.D * kEs<T>;
#pragma unroll
      for (int s = 0; s < S::KS; ++s)
#pragma unroll
        for (int e = 0; e < S::KW; e += (S::KW > 8 ? 8 : S::KW)) {
          constexpr int w = S::KW > 8 ? 8 : S::KW;
          const int d = s * 4 * S::KW + g * S::KW + e;
          Frag<T, w> f;
          if (is_row && (kWhole || d < a.D)) load_values<T, w>(p + d * kEs<T>, f);
          else clear(f);
#pragma unroll
          for (int i = 0; i < Frag<T, w>::kWords; ++i) q[t][s].w[e * kEs<T> / 4 + i] = f.w[i];
        }
    }

    const int edge = a.window > 0 ? n + a.N - 1 - a.window : -1;  // no window hides a later entry from any node
    const int head = h * a.D;
    const bool one_scale = a.D % 128 == 0 ? head % 128 == 0 : head % 128 + a.D <= 128;

    Sums<S, MT> z;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      z.m[t] = kNinf;
      z.l[t] = 0.0f;
#pragma unroll
      for (int i = 0; i < S::OT; ++i) z.o[t][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();

    // A tile of the cache: its first entry, and the tile's last key.
    auto place = [&](int tile, int& j0) {
      j0 = tile < tiles_first ? tile * kSpan : low + (tile - tiles_first) * kSpan;
      return min(kSpan, (tile < tiles_first ? first : n) - j0) - 1;
    };
    auto rows_at = [&](const uint8_t* base, const uint8_t* scales, int j0) {
      const size_t row = (size_t)b * a.L + j0;
      Rows r;
      r.base = base + (row * heads + head) * (kQ ? 1 : kEs<T>);
      r.scales = kQ ? scales + row * (size_t)a.nb : nullptr;
      r.stride = (uint32_t)heads * (kQ ? 1 : kEs<T>);
      return r;
    };
    typedef typename std::conditional<kQ, KeyCodes<S>, typename S::Keys>::type CacheKeys;
    CacheKeys k;
    auto fetch_keys = [&](int tile) {
      int j0;
      // a constant leaves the offsets in registers
      const int last = kWhole ? (place(tile, j0), kKeys - 1) : place(tile, j0);
      const Rows r = rows_at(a.k_cache, a.k_scales, j0);
      if constexpr (kQ) load_key_codes<S>(r, a.nb, head, last, a.D, one_scale, lane, k);
      else load_keys<S, T>(r, last, a.D, lane, k);
    };
    auto add_key = [&](Frag<T, S::KW>& f, int u, int s, f32x4 (&x)[MT][S::U], int lane) {
      if constexpr (!kWhole) cut_key<S, T>(a.D, s, lane, f);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        x[t][u] = product<T, S::KW>(f, q[t][s], s == 0 ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : x[t][u]);
    };
    // Tiles that some row does not see all of: values that are not finite are taken out of the product (bits of the
    // slots that had some), and their products with the weights added to the rows that see them: an infinity or NaN
    // itself, but NaN for an infinity whose weight is 0.  marks: bit i where the row sees slot i, bit 16 + i where its
    // weight is 0.  value(key, d): the CW values from d on.
    auto take_out = [&](typename S::Values& v) {
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < S::kSlots; ++i)
#pragma unroll
        for (int s = 0; s < S::VS; ++s)
#pragma unroll
          for (int w = 0; w < Frag<T, S::CW>::kWords; ++w) {
            const uint32_t f = not_finite<T>(v[i][s].w[w]);
            v[i][s].w[w] &= ~f;
            bad |= f != 0 ? 1u << i : 0u;
          }
      return bad;
    };
    auto add_others = [&](uint32_t bad, const uint32_t (&marks)[MT], int lane, auto value) {
      const int g = lane >> 4;
      if (!__any(bad != 0)) return;
#pragma unroll 1
      for (int key = 0; key < kKeys; ++key) {
        const int group16 = (key >> 2) & 3, slot = (key >> 4) * 4 + (key & 3);
        if (!__any((lane >> 4) == group16 && (bad >> slot & 1))) continue;
#pragma unroll
        for (int s = 0; s < S::VS; ++s)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int d = s * 16 * S::CW + (g * 4 + r) * S::CW;
            const Frag<T, S::CW> f = value(key, d < a.D ? d : 0);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              const uint32_t mark = __shfl(marks[t], group16 * 16 + (lane & 15)) >> slot;
#pragma unroll
              for (int j = 0; j < S::CW; ++j) {
                uint32_t w;
                if constexpr (S::kF32) w = f.w[j];
                else w = j & 1 ? f.w[j / 2] & 0xffff0000u : f.w[j / 2] << 16;
                const bool add = (mark & 1) && (w & 0x7f800000u) == 0x7f800000u;
                w |= mark >> 16 & 1 ? 0x7fc00000u : 0u;  // 0 times an infinity
                z.o[t][s * S::CW + j][r] += add ? __uint_as_float(w) : -0.0f;  // -0 leaves every sum as it is
              }
            }
            __builtin_amdgcn_sched_barrier(0);  // one load at a time: registers
          }
      }
    };

    // Tiles that every row sees whole: of the first entries, and behind the window's edge.
    const int edge_tiles = edge >= low ? (edge - low) / kSpan + 1 : 0;
    const int first_end = max(from, min(to, first / kSpan));
    const int later = min(max(from, tiles_first + edge_tiles), to);
    const int later_end = max(later, min(to, tiles_first + (n - low) / kSpan));
    const int count = first_end - from + later_end - later;
    auto whole_tile = [&](int i) { return i < first_end - from ? from + i : later + i - (first_end - from); };
    if constexpr (kShared) {
      // A row of shared memory has its 16-byte pieces in an order of its own, so that sixteen keys' pieces of one place
      // lie in different banks.
      constexpr int kRow = DP * 2, kPieces = kRow / 16;
      auto turned = [](int row, int piece) { return piece ^ (kPieces == 16 ? row & 15 : row >> 1 & 7); };
      // One stage: keys and values of 64 entries, a quarter by each wave.
      constexpr int kRowsD = kWave / kPieces, kDmas = kStage / kRowsD / kWavesPerBlock;  // rows of a DMA
      auto issue = [&](int i, int buffer) {
        int j0;
        place(whole_tile(i), j0);
        const Rows kr = rows_at(a.k_cache, a.k_scales, j0), vr = rows_at(a.v_cache, a.v_scales, j0);
#pragma unroll
        for (int d = 0; d < kDmas; ++d) {
          const int row0 = (wave * kDmas + d) * kRowsD, row = row0 + lane / kPieces, slot = lane % kPieces;
          const int kd = turned(row, slot) * 8, vd = slot * 8;
          const uint32_t k_at = (uint32_t)row * kr.stride + (uint32_t)((kWhole || kd < a.D ? kd : 0) * 2);
          const uint32_t v_at = (uint32_t)row * vr.stride + (uint32_t)((kWhole || vd < a.D ? vd : 0) * 2);
          dma16(kr.base + k_at, &stage[buffer][0][row0 * kRow]);
          dma16(vr.base + v_at, &stage[buffer][1][row0 * kRow]);
        }
      };
      // The same from codes, by way of registers: 16 per lane and load.
      constexpr int kLanesC = DP / 16, kRowsC = kWave / kLanesC, kLoadsC = kStage / kRowsC / kWavesPerBlock;
      uint32_t codes[2][kLoadsC][4], scales[2][kLoadsC][2];
      auto fetch = [&](int i) {
        int j0;
        place(whole_tile(i), j0);
        const Rows both[2] = {rows_at(a.k_cache, a.k_scales, j0), rows_at(a.v_cache, a.v_scales, j0)};
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int c = 0; c < kLoadsC; ++c) {
            const uint32_t row = (uint32_t)((wave * kLoadsC + c) * kRowsC + lane / kLanesC);
            const int d = lane % kLanesC * 16;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int at = kWhole || d + 8 * e < a.D ? d + 8 * e : 0;
              if (!kWhole || e == 0) {
                if constexpr (kWhole) {
                  const uint8_t* p = both[v].base + (row * both[v].stride + (uint32_t)at);
                  const u32x4 w = *reinterpret_cast<const u32x4_any1*>(p);
#pragma unroll
                  for (int q = 0; q < 4; ++q) codes[v][c][q] = w[q];
                } else {
                  uint32_t w[2];
                  load_codes<8>(both[v].base + (row * both[v].stride + (uint32_t)at), w);
                  codes[v][c][2 * e] = w[0];
                  codes[v][c][2 * e + 1] = w[1];
                }
                scales[v][c][e] = both[v].scales[row * (uint32_t)a.nb + (uint32_t)((head + at) >> 7)];
              }
              if (kWhole && e == 1)  // 16 codes of a whole head are in one block where the head begins on 16
                scales[v][c][1] = scales[v][c][0];
            }
          }
      };
      auto put = [&](int buffer) {
#pragma unroll
        for (int v = 0; v < 2; ++v)
#pragma unroll
          for (int c = 0; c < kLoadsC; ++c) {
            const int row = (wave * kLoadsC + c) * kRowsC + lane / kLanesC;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int piece = lane % kLanesC * 2 + e;
              const float sc = scale_of(scales[v][c][e]);
              const uint32_t w[2] = {codes[v][c][2 * e], codes[v][c][2 * e + 1]};
              Frag<T, 8> f;
              decode<T, 8>(w, &sc, f);
              *reinterpret_cast<u32x4*>(&stage[buffer][v][row * kRow + (v == 0 ? turned(row, piece) : piece) * 16]) =
                  u32x4{f.w[0], f.w[1], f.w[2], f.w[3]};
            }
          }
      };
      if constexpr (kQ) {
        if (count > 0) fetch(0);
      } else {
        if (count > 0) issue(0, 0);
      }
      for (int i = 0; i < count; ++i) {
        const int buffer = i & 1;
        // The stage is there, and every wave is done with the other buffer.
        if constexpr (kQ) {
          put(buffer);
          if (i + 1 < count) fetch(i + 1);
          block_barrier();
        } else {
          wait_vmcnt<0>();
          block_barrier();
          if (i + 1 < count) issue(i + 1, buffer ^ 1);
        }
#pragma unroll
        for (int half = 0; half < kStage / kKeys; ++half) {
          f32x4 x[MT][S::U];
#pragma unroll
          for (int u = 0; u < S::U; ++u)
#pragma unroll
            for (int s = 0; s < S::KS; ++s) {
              const int row = half * kKeys + u * 16 + (lane & 15);
              const uint8_t* p = &stage[buffer][0][row * kRow + turned(row, 4 * s + g) * 16];
              const u32x4 w = *reinterpret_cast<const u32x4*>(p);
              Frag<T, S::KW> f;
#pragma unroll
              for (int q = 0; q < 4; ++q) f.w[q] = w[q];
              add_key(f, u, s, x, lane);
            }
          const uint32_t none[MT] = {};
          weigh<S, MT, false>(x, none, a.c, z);
#pragma unroll
          for (int s = 0; s < S::VS; ++s) {
            Frag<T, S::CW> piece[S::kSlots];
#pragma unroll
            for (int slot = 0; slot < S::kSlots; ++slot) {
              typedef uint32_t words __attribute__((ext_vector_type(S::CW / 2)));
              const words w = *reinterpret_cast<const words*>(
                  &stage[buffer][1][(half * kKeys + key_of(slot, lane)) * kRow + (s * 16 + (lane & 15)) * S::CW * 2]);
#pragma unroll
              for (int q = 0; q < S::CW / 2; ++q) piece[slot].w[q] = w[q];
            }
            add_piece<S, T, MT>(piece, s, x, z);
          }
        }
      }
    } else {
      if (wave < count) fetch_keys(whole_tile(wave));
      for (int i = wave; i < count; i += kWavesPerBlock) {
        int j0;
        const int last = kWhole ? (place(whole_tile(i), j0), kKeys - 1) : place(whole_tile(i), j0);
        const Rows rows = rows_at(a.v_cache, a.v_scales, j0);
        typedef typename std::conditional<kQ, ValueCodes<S>, typename S::Values>::type CacheValues;
        CacheValues raw;
        if constexpr (kQ) load_row_codes<S>(rows, a.nb, head, last, a.D, lane, raw);
        else load_rows<S, T>(rows, last, a.D, lane, raw);
        f32x4 x[MT][S::U];
#pragma unroll
        for (int u = 0; u < S::U; ++u)
#pragma unroll
          for (int s = 0; s < S::KS; ++s) {
            if constexpr (kQ) {
              const float sc[2] = {scale_of(k.scale[u][s][0]), scale_of(k.scale[u][s][S::KW / 8 - 1])};
              Frag<T, S::KW> f;
              decode<T, S::KW>(k.w[u][s], sc, f);
              add_key(f, u, s, x, lane);
            } else {
              add_key(k[u][s], u, s, x, lane);
            }
          }
        __builtin_amdgcn_sched_barrier(0);
        if (i + kWavesPerBlock < count) fetch_keys(whole_tile(i + kWavesPerBlock));
        const uint32_t none[MT] = {};
        weigh<S, MT, false>(x, none, a.c, z);
#pragma unroll
        for (int s = 0; s < S::VS; ++s) {
          Frag<T, S::CW> piece[S::kSlots];
#pragma unroll
          for (int i8 = 0; i8 < S::kSlots; ++i8) {
            if constexpr (kQ) {
              const float sc = scale_of(raw.scale[i8][s]);
              decode<T, S::CW>(raw.w[i8][s], &sc, piece[i8]);
            } else {
              piece[i8] = raw[i8][s];
            }
          }
          add_piece<S, T, MT>(piece, s, x, z);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // The others: ends, entries at the window's edge, and the tree's own, of which a node sees its ancestors and
    // itself.  A tile's 32 keys at a time.
    constexpr int kParts = kSpan / kKeys;
    const int before = later - first_end, careful = before + to - later_end;
#pragma unroll 1
    for (int i = kShared ? 0 : wave; i < careful * kParts; i += kShared ? 1 : kWavesPerBlock) {
      const int part_of = i % kParts * kKeys, at = i / kParts;
      const int tile = at < before ? first_end + at : later_end + at - before;
      int my = tid;
      asm volatile("" : "+v"(my));  // these few tiles' offsets are not kept through the loop above
      const int lane = my & (kWave - 1);
      const bool own = tile >= tiles_cache;
      int j0, last;
      typename S::Keys key;
      typename S::Values v;
      f32x4 x[MT][S::U];
      Rows vr;
      if (own) {
        j0 = (tile - tiles_cache) * kSpan + part_of;
        last = min(kKeys, a.N - j0) - 1;
        if (last < 0) continue;
        const size_t at = (((size_t)b * a.N + j0) * heads + head) * kEs<T>;
        const Rows kr{static_cast<const uint8_t*>(a.k_new) + at, nullptr, (uint32_t)heads * kEs<T>};
        vr = Rows{static_cast<const uint8_t*>(a.v_new) + at, nullptr, (uint32_t)heads * kEs<T>};
        load_keys<S, T>(kr, last, a.D, lane, key);
        if constexpr (!kQ) load_rows<S, T>(vr, last, a.D, lane, v);
      } else {
        last = min(place(tile, j0) - part_of, kKeys - 1);
        j0 += part_of;
        if (last < 0) continue;
        const Rows kr = rows_at(a.k_cache, a.k_scales, j0);
        vr = rows_at(a.v_cache, a.v_scales, j0);
        if constexpr (kQ) {
          KeyCodes<S> kc;
          load_key_codes<S>(kr, a.nb, head, last, a.D, one_scale, lane, kc);
#pragma unroll
          for (int u = 0; u < S::U; ++u)
#pragma unroll
            for (int s = 0; s < S::KS; ++s) {
              const float sc[2] = {scale_of(kc.scale[u][s][0]), scale_of(kc.scale[u][s][S::KW / 8 - 1])};
              decode<T, S::KW>(kc.w[u][s], sc, key[u][s]);
            }
        } else {
          load_keys<S, T>(kr, last, a.D, lane, key);
          load_rows<S, T>(vr, last, a.D, lane, v);
        }
      }
#pragma unroll
      for (int u = 0; u < S::U; ++u)
#pragma unroll
        for (int s = 0; s < S::KS; ++s) add_key(key[u][s], u, s, x, lane);
      __builtin_amdgcn_sched_barrier(0);
      uint32_t seen[MT];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        const uint64_t line = line_of[node[t]];
        const int hidden = a.window > 0 ? n + depth_of[node[t]] - a.window : -1;  // up to here, but for the first
        seen[t] = 0;
#pragma unroll
        for (int i = 0; i < S::kSlots; ++i) {
          const int off = key_of(i, lane), j = min(j0 + off, own ? kMaxNodes - 1 : n);
          const int position = own ? n + depth_of[j & (kMaxNodes - 1)] : j;
          const bool sees = off <= last && (!own || (line >> (j & 63) & 1)) &&
              (position > hidden || position < a.sinks);
          seen[t] |= sees ? 1u << i : 0u;
        }
      }
      weigh<S, MT, true>(x, seen, a.c, z);
      if constexpr (kQ) {
        if (!own) {  // now, when the keys' registers are free
          ValueCodes<S> vc;
          load_row_codes<S>(vr, a.nb, head, last, a.D, lane, vc);
#pragma unroll
          for (int i = 0; i < S::kSlots; ++i)
#pragma unroll
            for (int s = 0; s < S::VS; ++s) {
              const float sc = scale_of(vc.scale[i][s]);
              decode<T, S::CW>(vc.w[i][s], &sc, v[i][s]);
            }
        } else {
          load_rows<S, T>(vr, last, a.D, lane, v);
        }
      }
      const uint32_t bad = take_out(v);
      if (__any(bad != 0)) {
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t zero = 0;
#pragma unroll
          for (int i = S::kSlots - 1; i >= 0; --i) {
            zero = zero << 1 | (x[t][i / 4][i % 4] == 0.0f ? 1u : 0u);
            asm("" : "+v"(zero));  // as shifts: a constant for each bit would be kept in a register through the loop
          }
          seen[t] |= zero << 16;
        }
      }
#pragma unroll
      for (int s = 0; s < S::VS; ++s) {
        Frag<T, S::CW> piece[S::kSlots];
#pragma unroll
        for (int i = 0; i < S::kSlots; ++i) piece[i] = v[i][s];
        add_piece<S, T, MT>(piece, s, x, z);
      }
      __builtin_amdgcn_sched_barrier(0);
      add_others(bad, seen, lane, [&](int key_at, int d) {
        const uint32_t at = (uint32_t)min(key_at, last);
        Frag<T, S::CW> f;
        if constexpr (kQ) {
          if (!own) {
            uint32_t w[S::CW / 4];
            load_codes<S::CW>(vr.base + (at * vr.stride + (uint32_t)d), w);
            const float sc = scale_of(vr.scales[at * (uint32_t)a.nb + (uint32_t)((head + d) >> 7)]);
            decode<T, S::CW>(w, &sc, f);
            return f;
          }
        }
        load_values<T, S::CW>(vr.base + (at * vr.stride + (uint32_t)(d * kEs<T>)), f);
        return f;
      });
    }

    if constexpr (kShared) {
      // A wave's rows are its own: lane (g, m) has values (4 g + r) CW .. of each piece of row m.
      const size_t slot = (slot0 * a.groups + group) * (kWavesPerBlock * 16 * MT) + wave * 16 * MT;
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        float l = z.l[t] + __shfl_xor(z.l[t], 16);
        l += __shfl_xor(l, 32);
        const int r = t * 16 + (lane & 15), m = row0 + r;
        if (m >= a.R) continue;
        if (line_of[node[t]] == 0) l = 0.0f;
        if (!valid) l = __builtin_nanf("");
        const float inv = 1.0f / l;
        const size_t to = (((size_t)b * a.N + node[t]) * a.Hq + h * a.G + (m - node[t] * a.G)) * (size_t)a.D;
        if (!alone && g == 0) a.stats[slot + r] = float2{l == 0.0f ? kNinf : z.m[t], l};
#pragma unroll
        for (int s = 0; s < S::VS; ++s)
#pragma unroll
          for (int r4 = 0; r4 < 4; ++r4)
#pragma unroll
            for (int j = 0; j < S::CW; j += 4) {
              const int d = s * 16 * S::CW + (g * 4 + r4) * S::CW + j;
              if (!kWhole && d >= a.D) continue;
              f32x4 y;
#pragma unroll
              for (int e = 0; e < 4; ++e) y[e] = z.o[t][s * S::CW + j + e][r4];
              if (!alone) {
                *reinterpret_cast<f32x4*>(a.acc + (slot + r) * (size_t)a.D + d) = y;
              } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] = l == 0.0f ? 0.0f : y[e] * inv;
                typedef uint32_t pair __attribute__((ext_vector_type(2), aligned(2)));
                *reinterpret_cast<pair*>(static_cast<uint16_t*>(a.out) + to + d) =
                    pair{pack2(y[0], y[1]), pack2(y[2], y[3])};
              }
            }
      }
    } else {
      // The waves' results, 16 rows at a time.
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        z.l[t] += __shfl_xor(z.l[t], 16);
        z.l[t] += __shfl_xor(z.l[t], 32);
        if (g == 0) stat[wave][t * 16 + (lane & 15)] = float2{z.m[t], z.l[t]};
      }
      __syncthreads();
      const size_t slot = (slot0 * a.groups + group) * (16 * MT);
#pragma unroll
      for (int t = 0; t < MT; ++t) {
        {
          const int r = t * 16 + (lane & 15);
          float m = stat[0][r].x;
#pragma unroll
          for (int w = 1; w < kWavesPerBlock; ++w) m = fmaxf(m, stat[w][r].x);
          const float f = z.m[t] == kNinf ? 0.0f : exp2_of(z.m[t] - m);
          float* to = &part[wave][(lane & 15) * kPad<DP>];
#pragma unroll
          for (int s = 0; s < S::VS; ++s)
#pragma unroll
            for (int r4 = 0; r4 < 4; ++r4)
#pragma unroll
              for (int j = 0; j < S::CW; j += 4) {
                f32x4 y;
#pragma unroll
                for (int i = 0; i < 4; ++i) y[i] = z.o[t][s * S::CW + j + i][r4] * f;
                *reinterpret_cast<f32x4*>(to + s * 16 * S::CW + (g * 4 + r4) * S::CW + j) = y;
              }
        }
        __syncthreads();
        constexpr int kQuads = DP / 4;
#pragma unroll
        for (int k = 0; k < 16 * kQuads / kBlock; ++k) {
          const int at = k * kBlock + tid, r = at / kQuads, d = at % kQuads * 4;
          const int m = row0 + t * 16 + r;
          if (m >= a.R || d >= a.D) continue;
          f32x4 y = *reinterpret_cast<const f32x4*>(&part[0][r * kPad<DP> + d]);
#pragma unroll
          for (int w = 1; w < kWavesPerBlock; ++w) y += *reinterpret_cast<const f32x4*>(&part[w][r * kPad<DP> + d]);
          float ref = stat[0][t * 16 + r].x;
#pragma unroll
          for (int w = 1; w < kWavesPerBlock; ++w) ref = fmaxf(ref, stat[w][t * 16 + r].x);
          float l = 0.0f;
#pragma unroll
          for (int w = 0; w < kWavesPerBlock; ++w) {
            const float2 s = stat[w][t * 16 + r];
            l += s.x == kNinf ? s.y : s.y * exp2_of(s.x - ref);
          }
          const int nd = m / a.G;
          if (line_of[nd] == 0) l = 0.0f;
          if (!valid) l = __builtin_nanf("");
          if (!alone) {
            *reinterpret_cast<f32x4*>(a.acc + (slot + t * 16 + r) * (size_t)a.D + d) = y;
            if (d == 0) a.stats[slot + t * 16 + r] = float2{l == 0.0f ? kNinf : ref, l};
            continue;
          }
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = l == 0.0f ? 0.0f : y[i] * inv;
          const size_t at_out = (((size_t)b * a.N + nd) * a.Hq + h * a.G + (m - nd * a.G)) * (size_t)a.D + d;
          if constexpr (S::kF32) {
            typedef float quad __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<quad*>(static_cast<float*>(a.out) + at_out) = quad{y[0], y[1], y[2], y[3]};
          } else {
            typedef uint32_t pair __attribute__((ext_vector_type(2), aligned(2)));
            *reinterpret_cast<pair*>(static_cast<uint16_t*>(a.out) + at_out) =
                pair{pack2(y[0], y[1]), pack2(y[2], y[3])};
          }
        }
        __syncthreads();
      }
    }
    left -= to - from;
    if (left <= 0) return;
    begin = 0;
    if (++h == a.Hkv) h = 0, ++b;
    __syncthreads();  // the tree's lines and the waves' results give way to the next ones
  }
}

// The rows of a KV head whose keys several blocks have: a range's first piece is in its first slot, another in its
// second.  A wave has `rows` rows, one after the other.  Its lanes have 16-byte parts of the pieces' results: as many
// pieces at a time as a row's parts leave lanes for, and several such loads in flight.  A wave per row spends more on
// finding the pieces than on joining them where rows are many: B=64 N=64 L=8192 85 us, 38 with eight rows a wave.
template <typename T>
__global__ void __launch_bounds__(kBlock) tree_join_kernel(AttnArgs a, int rows_per_block, int rows) {
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
  const int m0 = ((int)blockIdx.x * kWavesPerBlock + wave) * rows;
  const int b = (int)blockIdx.y / a.Hkv, h = (int)blockIdx.y % a.Hkv;
  if (m0 >= a.R) return;
  int first = (int)blockIdx.y * a.split, next = first + 1, count = a.split, step = 1;  // the pieces' slots
  if (a.ranges > 0) {
    int before = 0, all = 0;
    for (int i = lane; i < a.B; i += kWave) {
      const int t = keys_of(a, a.span, a.cache_len[i]).tiles;
      all += t;
      before += i < b ? t : 0;
    }
    const int per = range_of(a, dpp::lane63(lanes_scan(all)) * a.Hkv);
    const int tiles = keys_of(a, a.span, a.cache_len[b]).tiles;
    const int begin = dpp::lane63(lanes_scan(before)) * a.Hkv + h * tiles;
    const int range = begin / per;
    count = (begin + tiles - 1) / per - range + 1;
    if (count == 1) return;
    first = 2 * range + (begin != range * per ? 1 : 0);  // not its range's first piece?
    next = 2 * range + 2;
    step = 2;
  }
  const int parts = a.D > 128 ? 64 : a.D > 64 ? 32 : 16, at_once = kWave / parts;
  const int d = (lane & (parts - 1)) * 4;
  auto join = [&](int m, auto loads) {
    constexpr int kLoads = decltype(loads)::value;
    const int group = m / rows_per_block, r = m % rows_per_block;
    float ref = kNinf, l = 0.0f;
    f32x4 y{0.0f, 0.0f, 0.0f, 0.0f};
    for (int i0 = lane / parts; i0 < count; i0 += at_once * kLoads) {
      float2 w[kLoads];
      f32x4 v[kLoads];
      bool in[kLoads];
      float top = ref;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const int i = min(i0 + j * at_once, count - 1);
        const size_t at = ((size_t)(i == 0 ? first : next + (i - 1) * step) * a.groups + group) * rows_per_block + r;
        w[j] = a.stats[at];
        v[j] = *reinterpret_cast<const f32x4*>(a.acc + at * (size_t)a.D + (d < a.D ? d : 0));
      }
      __builtin_amdgcn_sched_barrier(0);  // all loads first: B=1 N=16 L=131072 4.8 us, 6.4 one after the other
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        in[j] = i0 + j * at_once < count;  // with a sum of 0 too: its results are zeros, or NaN by 0 times an infinity
        if (in[j]) top = fmaxf(top, w[j].x);
      }
      const float old = ref == kNinf ? 0.0f : exp2_of(ref - top);
      ref = top;
      l *= old;
      y *= old;
#pragma unroll
      for (int j = 0; j < kLoads; ++j) {
        const float f = w[j].x == kNinf ? 1.0f : exp2_of(w[j].x - ref);
        l += in[j] ? w[j].y * f : 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += in[j] ? v[j][e] * f : 0.0f;
      }
    }
    float top = ref;
    for (int o = parts; o < kWave; o *= 2) top = fmaxf(top, __shfl_xor(top, o));
    const float f = ref == kNinf ? 1.0f : exp2_of(ref - top);  // -inf: nothing, or a sum that is NaN
    l *= f;
    y *= f;
    for (int o = parts; o < kWave; o *= 2) {
      l += __shfl_xor(l, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) y[i] += __shfl_xor(y[i], o);
    }
    if (lane >= parts || d >= a.D) return;
    const float inv = 1.0f / l;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = l == 0.0f ? 0.0f : l != l ? l : y[i] * inv;
    const int nd = m / a.G;
    const size_t to = (((size_t)b * a.N + nd) * a.Hq + h * a.G + (m - nd * a.G)) * (size_t)a.D + d;
    if constexpr (std::is_same<T, float>::value) {
      typedef float quad __attribute__((ext_vector_type(4), aligned(4)));
      *reinterpret_cast<quad*>(static_cast<float*>(a.out) + to) = quad{y[0], y[1], y[2], y[3]};
    } else {
      typedef uint32_t pair2 __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<pair2*>(static_cast<uint16_t*>(a.out) + to) = pair2{pack2(y[0], y[1]), pack2(y[2], y[3])};
    }
  };
  const int m1 = min(a.R, m0 + rows);
  if (count > 4 * at_once) {
    for (int m = m0; m < m1; ++m) join(m, std::integral_constant<int, 8>{});
  } else {
    for (int m = m0; m < m1; ++m) join(m, std::integral_constant<int, 2>{});
  }
}

template <typename T, bool kQ, int DP, int MT, bool kShared>
void start(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (a.D == DP)
    hipLaunchKernelGGL((tree_attention_kernel<T, kQ, DP, MT, true, kShared>), dim3(p.grid), dim3(kBlock), 0, st, a);
  else
    hipLaunchKernelGGL((tree_attention_kernel<T, kQ, DP, MT, false, kShared>), dim3(p.grid), dim3(kBlock), 0, st, a);
}

template <typename T, bool kQ, int DP>
void start_rows(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if constexpr (!std::is_same<T, float>::value && DP <= 128) {
    if (p.shared) {
      start<T, kQ, DP, 2, true>(a, p, st);
      return;
    }
  }
  if (p.mt == 1) start<T, kQ, DP, 1, false>(a, p, st);
  else if constexpr (DP <= 128) start<T, kQ, DP, 2, false>(a, p, st);
}

template <typename T, bool kQ>
hipError_t run(const AttnArgs& a, const AttnPlan& p, hipStream_t st) {
  if (p.dp == 64) start_rows<T, kQ, 64>(a, p, st);
  else if (p.dp == 128) start_rows<T, kQ, 128>(a, p, st);
  else start_rows<T, kQ, 256>(a, p, st);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (p.ranges == 0 && p.split == 1)) return e;
  const int per_block = p.join_rows * kWavesPerBlock;
  const dim3 grid((unsigned)((a.R + per_block - 1) / per_block), (unsigned)(a.B * a.Hkv));
  hipLaunchKernelGGL((tree_join_kernel<T>), grid, dim3(kBlock), 0, st, a, p.rows, p.join_rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tree_attention(const AttnPointers& io, bool quantized, int B, int N, int Hq, int Hkv, int D, int L,
                                 float scale, int window, int sinks, int dtype, const AttnPlan& plan, void* workspace,
                                 hipStream_t st) {
  AttnArgs a{};
  a.q = io.q;
  a.k_new = io.k_new;
  a.v_new = io.v_new;
  a.k_cache = static_cast<const uint8_t*>(io.k_cache);
  a.v_cache = static_cast<const uint8_t*>(io.v_cache);
  a.k_scales = static_cast<const uint8_t*>(io.k_scales);
  a.v_scales = static_cast<const uint8_t*>(io.v_scales);
  a.parents = io.parents;
  a.cache_len = io.cache_len;
  a.out = const_cast<void*>(io.out);
  if (plan.slots > 0) {
    a.stats = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + plan.stats);
    a.acc = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + plan.acc);
  }
  a.B = B;
  a.N = N;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  a.D = D;
  a.L = L;
  a.nb = quant_blocks(Hkv * D);
  a.R = plan.R;
  a.groups = plan.groups;
  a.split = plan.split;
  a.ranges = plan.ranges;
  a.least = plan.least;
  a.step = plan.step;
  a.span = plan.span;
  a.window = window;
  a.sinks = sinks;
  a.c = scale * kLog2e;
  if (dtype == 1) return quantized ? run<uint16_t, true>(a, plan, st) : run<uint16_t, false>(a, plan, st);
  return quantized ? run<float, true>(a, plan, st) : run<float, false>(a, plan, st);
}

}  // namespace sv
