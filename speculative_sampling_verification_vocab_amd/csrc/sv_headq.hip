// Drafter head on a weight in the 8-bit block format: C[M, N] = hq[M, d] *
// Wq[N, d]^T over a shortlist of N tokens, both operands e4m3 with a
// power-of-two scale per block of 128 dims (sv_quant.h).
//
// One v_mfma_scale_f32_16x16x128_f8f6f4 covers exactly one block of the
// format: lane l gives 32 of the 128 codes of row l % 16 of each operand and
// that row's scale byte, and the matrix core applies both scales and adds to
// the fp32 accumulator, so scales cost no arithmetic of their own.  Which 32
// codes a lane gives is free as long as both operands agree, for the four
// 32-code groups share the scale: lane group g gives the 16-byte pieces g and
// g + 4 of the row.
//
// That instruction adds each group of 8 consecutive dims' products with what
// lies below 2^-13 of the largest one's power of two cut off, toward zero
// (measured; a product has 8 significant bits, so the largest one and those
// down to 2^-5 of it stay whole, and the groups' sums and the accumulator lose
// fp32 roundings only).  A group is off by at most 7 * 2^-13 of its largest
// product: 1.4e-5 of the result for normal data (rms), a hundredth of the
// rounding to bf16, and less than that rounding for any data whose large
// products do not cancel each other.  bf16 outputs take it, for half the matrix
// time.  fp32 outputs take v_mfma_f32_16x16x32_bf16 on the codes' values, which
// bf16 holds exactly (6e-9): one conversion per two codes, which applies the
// scale, and twice the matrix time.
//
// For few rows the product is bound by the stream of W's codes (d bytes per
// token, 2 M flops per byte); for many rows by the matrix cores.  Both
// operands go from memory to LDS by DMA (global_load_lds, 16 bytes per lane,
// several stages in flight), 128-byte rows with their eight 16-byte pieces
// XOR-swizzled so that fragment reads meet no bank conflicts; scale bytes are
// put in LDS once per 64 blocks of d, four to a dword.  WK wave groups take
// every WK-th block of 128, their sums added through LDS at the end.
// Narrow shortlists split d over several blocks of threads; their fp32 tiles
// are added in a fixed order by a second launch.
//
// Measured at d = 4096, bf16 out (GPU time; see head_quantized_plan for the
// tiles): N = 32768: M = 1, 16, 64, 128: 27, 28, 29, 34 us (134 MB of W: 19 us
// at the read stream's rate); N = 128256: M = 8, 128: 100, 123 us; M = 1792:
// 880-930 us by the card, 2.0-2.1 PFLOP/s, where a library's product of 8192^3
// reaches 3.1 (the 256 x 256 tile's stages meet at one barrier with two
// buffers; the matrix cores are busy in 45 % of the cycles, the LDS in 25 %).
// fp32 out: M = 128, N = 32768: 49 us; M = 1792, N = 32768: 414 us, 1.16 PFLOP/s
// (a library's bf16 product of 8192^3: 1.40).

#include "sv_common.h"
#include "sv_dma.h"
#include "sv_host_quant.h"
#include "sv_internal.h"
#include "sv_quant.h"

namespace sv {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct HeadQArgs {
  const uint16_t* h;      // bf16 [M][d], where the blocks quantise it themselves
  int d, vec_h;           // vec_h: d % 8 == 0 and 16-byte aligned rows
  const uint8_t* hq;      // [M][D]
  const uint8_t* hs;      // [M][nb]
  const uint8_t* wq;      // [V][D]
  const uint8_t* ws;      // [V][nb]
  const int32_t* cids;    // [n_sel], any order
  int M, N, cs, nclusters;
  int nb;                 // blocks of 128 in a row; D = 128 * nb
  int m_tiles;
  int total, per_xcd;     // tiles (times slices), and how many each XCD takes in turn
  int split, split_nb;    // blocks of threads per tile; blocks of 128 per slice
  int dword_scales;       // scale rows begin on 4-byte boundaries
  void* out;              // [M][N] fp32 or bf16
  int out_bf16;
  float* partial;         // split > 1: fp32 [split][M][N]
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

// Four consecutive outputs at o.
__device__ __forceinline__ void store4(void* dst, bool bf16, size_t o, const float (&v)[4]) {
  if (bf16)
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dst) + o) = uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
  else
    *reinterpret_cast<float4*>(static_cast<float*>(dst) + o) = float4{v[0], v[1], v[2], v[3]};
}
__device__ __forceinline__ void store1(void* dst, bool bf16, size_t o, float v) {
  if (bf16) static_cast<uint16_t*>(dst)[o] = __builtin_bit_cast(uint16_t, (__bf16)v);
  else static_cast<float*>(dst)[o] = v;
}

// kOwnH: few enough values of h that every block quantises its slice of them
// into LDS (kHeadQOwn bytes), with no launch before it; only W rows are staged.
template <int WM, int WN, int WK, int TM, int TN, int NBUF, bool kOwnH>
struct HeadQTile {
  static constexpr int kMt = 16 * WM * TM, kNt = 16 * WN * TN, kRows = kOwnH ? kNt : kMt + kNt;  // rows staged
  static constexpr int kH = kOwnH ? 0 : kMt;           // of those, rows of h
  static constexpr int NW = WM * WN * WK, kThreads = kWave * NW;
  static constexpr int kOwn = kOwnH ? kHeadQOwn + kHeadQOwn / kQuantBlock : 0;  // codes and scale bytes of h
  static constexpr int kGroup = kRows / 8;             // DMA instructions per block of 128
  static constexpr int kIW = WK * kGroup / NW;         // per wave and stage of WK blocks
  static constexpr int kStage = WK * kRows * 128;      // bytes
  static constexpr int kSeg = kRows > 256 ? 32 : 64;   // blocks of 128 whose scales are in LDS at a time
  static_assert(!kOwnH || (kMt == 16 && kHeadQOwn / kQuantBlock * kLanesPerBlock <= 6 * kThreads), "own h");
  static_assert(kRows % 8 == 0 && WK * kGroup % NW == 0, "DMA split");
  static_assert(NBUF >= 2 && (NBUF - 2) * kIW < 64, "pipeline depth");
  static_assert(kSeg % WK == 0 && WK <= 4, "scale groups");
  static_assert((WK - 1) * WM * WN * kWave * TN * 4 * 4 <= NBUF * kStage, "reduction space");
  static_assert(16 * WM * (kNt + 4) * 4 <= NBUF * kStage, "epilogue space");
  static_assert(kThreads % (kNt / 4) == 0, "epilogue rows per pass");
};

// Eight codes as bf16, times a power of two.
__device__ __forceinline__ bf16x8 codes_to_bf16(int lo, int hi, float scale) {
#if defined(__HIP_DEVICE_COMPILE__)
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#else
  return bf16x8{};
#endif
}
__device__ __forceinline__ float scale_float(uint32_t byte) { return __uint_as_float((byte << 23) & 0x7f800000u); }

// kF32: the products of fp32 outputs (see above).
template <int WM, int WN, int WK, int TM, int TN, int NBUF, bool kOwnH, bool kF32>
__global__ void __launch_bounds__(kWave * WM * WN * WK) headq_kernel(HeadQArgs a) {
  using C = HeadQTile<WM, WN, WK, TM, TN, NBUF, kOwnH>;
  constexpr int kH = C::kH;
  constexpr int kMt = C::kMt, kNt = C::kNt, kRows = C::kRows, NW = C::NW, kIW = C::kIW, kSeg = C::kSeg;
  // One LDS object: beside a second one the compiler waits for every DMA in
  // flight before each read of this one.
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NBUF * C::kStage + kSeg * kRows + 4 * kRows + C::kOwn];
  uint32_t* const sc = reinterpret_cast<uint32_t*>(lds + NBUF * C::kStage);  // [kSeg / 4][kRows]: four scale bytes
  int* const token = reinterpret_cast<int*>(lds + NBUF * C::kStage + kSeg * kRows);  // W or h row of a tile row, or -1

  uint8_t* const own = lds + NBUF * C::kStage + kSeg * kRows + 4 * kRows;  // h's codes, then its scale bytes
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  const int wk = wave / (WM * WN), wmn = wave % (WM * WN);
  const int wm = wmn / WN, wn = wmn % WN;
  // Blocks go to the eight XCDs in turn: each takes a run of tiles, row tiles
  // first, so that the row tiles of a column tile read its W rows from one L2.
  const int v0 = (int)(blockIdx.x & 7) * a.per_xcd + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= a.per_xcd || v0 >= a.total) return;
  int v = v0;
  const int tiles = a.total / a.split;
  const int slice = v / tiles;
  v -= slice * tiles;
  const int n0 = (v / a.m_tiles) * kNt, m0 = (v % a.m_tiles) * kMt;
  const int b0 = slice * a.split_nb, blocks = min(a.nb - b0, a.split_nb);

  constexpr int kOwnUnits = kOwnH ? 6 : 1;
  float ox[kOwnUnits][kPerLaneQ];
  int om[kOwnUnits], ob[kOwnUnits];  // row and block of this slice
  if constexpr (kOwnH) {
    // h's values, on their way while the tile's rows are looked up.
#pragma unroll
    for (int k = 0; k < kOwnUnits; ++k) {
      const int i = min((int)threadIdx.x / kLanesPerBlock + k * (C::kThreads / kLanesPerBlock), a.M * blocks - 1);
      om[k] = i / blocks, ob[k] = i - om[k] * blocks;
      const int at = (b0 + ob[k]) * kQuantBlock + (int)(threadIdx.x % kLanesPerBlock) * kPerLaneQ;
      const uint16_t* p = a.h + (size_t)om[k] * (size_t)a.d + at;
      if (a.vec_h) load8<uint16_t, true, false>(p, a.d - at, ox[k]);
      else load8<uint16_t, false, false>(p, a.d - at, ox[k]);
    }
  }

  for (int r = threadIdx.x; r < kRows; r += C::kThreads) {
    int t = -1;
    if (r < kH) {
      if (m0 + r < a.M) t = m0 + r;
    } else if (n0 + r - kH < a.N) {
      const int n = n0 + r - kH, c = n / a.cs, cl = a.cids[c];
      if (cl >= 0 && cl < a.nclusters) t = cl * a.cs + (n - c * a.cs);
    }
    token[r] = t;
  }
  __syncthreads();

  // DMA instruction j of this wave: block `sub` of the stage, tile rows 8 * g ..
  // Rows that are none load the first one of h or W; their outputs are not
  // stored, or stored as zeros.
  const size_t D = (size_t)a.nb * kQuantBlock;
  const uint8_t* src[kIW];
#pragma unroll
  for (int j = 0; j < kIW; ++j) {
    const int g = (j * NW + wave) % C::kGroup, r = 8 * g + (lane >> 3);
    const int t = token[r];
    src[j] = (r < kH ? a.hq : a.wq) + (size_t)max(t, 0) * D + 16 * ((lane & 7) ^ ((r >> 1) & 7));
  }
  // Scales of blocks first .. first + seg - 1 of the rows, word i of [group][row].
  auto scale_word = [&](int i, int first) {
    const int g = i / kRows, r = i - g * kRows, b = first + 4 * g;
    const uint8_t* p = (r < kH ? a.hs : a.ws) + (size_t)max(token[r], 0) * a.nb + b;
    if (a.dword_scales) return *reinterpret_cast<const uint32_t*>(p);
    uint32_t w = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (b + e < a.nb) w |= (uint32_t)p[e] << (8 * e);
    return w;
  };

  f32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int frow = lane & 15, fc = lane >> 4;
  const int arow0 = wm * 16 * TM + frow, brow0 = kH + wn * 16 * TN + frow;
  auto fragment = [&](const uint8_t* buf, int r) {
    const int x = (r >> 1) & 7;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(buf + r * 128 + 16 * (fc ^ x));
    const u32x4 hi = *reinterpret_cast<const u32x4*>(buf + r * 128 + 16 * ((fc + 4) ^ x));
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };
  // h's slice in LDS: a row's blocks one after the other, rows 128 bytes further
  // apart than that, so that neighbours meet other banks; pieces swizzled as
  // in a stage.  Rows past M read the last one's.
  const int own_row = (blocks + 1) * kQuantBlock;
  auto quantize_own = [&]() {
#pragma unroll
    for (int k = 0; k < kOwnUnits; ++k) {
      if (k * (C::kThreads / kLanesPerBlock) >= a.M * blocks) break;
      int byte;
      const uint2 q = quantize8(ox[k], &byte);  // the last unit again in spare lanes: the same codes
      const int sub = threadIdx.x % kLanesPerBlock;
      *reinterpret_cast<uint2*>(own + om[k] * own_row + ob[k] * kQuantBlock +
                                16 * ((sub / 2) ^ ((om[k] >> 1) & 7)) + 8 * (sub & 1)) = q;
      if (sub == 0) own[kHeadQOwn + ob[k] * a.M + om[k]] = (uint8_t)byte;
    }
  };
  const int own_m = min(frow, a.M - 1);
  auto own_fragment = [&](int b) {
    const uint8_t* p = own + own_m * own_row + b * kQuantBlock;
    const int x = (own_m >> 1) & 7;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(p + 16 * (fc ^ x));
    const u32x4 hi = *reinterpret_cast<const u32x4*>(p + 16 * ((fc + 4) ^ x));
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
  };

  // Segments of up to kSeg blocks: their scales go to LDS, then the stages run
  // with no other memory loads between the DMAs that the waits count.
  for (int first = b0; first < b0 + blocks; first += kSeg) {
    const int seg = min(b0 + blocks - first, kSeg), stages = (seg + WK - 1) / WK;
    // Rows lie a multiple of 128 bytes apart, mostly of 4096, and the memory's
    // channels take turns every 256: the pieces that a stage reads of its rows
    // are all on one channel or two.  So that not all blocks wait for the same
    // ones, each begins at another stage and goes round (M = 128, N = 128256, d =
    // 4096: 157 -> 142 us).  Where several row tiles read the same W rows they
    // stay in step instead, for their L2's sake (M = 1792: 880 against 950 us).
    const int rot = kMt < 256 && a.m_tiles == 1 ? (int)((unsigned)(v0 % a.per_xcd) % (unsigned)stages) : 0;
    auto stage_of = [&](int s) { return s + rot < stages ? s + rot : s + rot - stages; };
    auto issue = [&](int s) {
      uint8_t* dst = lds + s % NBUF * C::kStage;
      const int sk = stage_of(s);
#pragma unroll
      for (int j = 0; j < kIW; ++j) {
        const int sub = (j * NW + wave) / C::kGroup;
        const int b = first + min(sk * WK + sub, seg - 1);  // past the segment: its last block again, not used
        dma16(src[j] + (size_t)b * kQuantBlock, dst + 1024 * (j * NW + wave));
      }
    };
    __syncthreads();  // every wave has finished the segment before
#pragma unroll
    for (int s = 0; s < NBUF - 1; ++s)
      if (s < stages) issue(s);
    const int words = (seg + 3) / 4 * kRows;
    if constexpr (kOwnH) {
      static_assert(kSeg / 4 * kRows <= C::kThreads, "one word each");
      uint32_t w = 0;
      if ((int)threadIdx.x < words) w = scale_word(threadIdx.x, first);
      if (first == b0) quantize_own();
      if ((int)threadIdx.x < words) sc[threadIdx.x] = w;
    } else {
      for (int i = threadIdx.x; i < words; i += C::kThreads) sc[i] = scale_word(i, first);
    }
    __syncthreads();

    uint32_t sa[TM], sb[TN];
    for (int s = 0; s < stages; ++s) {
      // Stage s has landed once only the later stages' DMAs can be in flight.
      if (s + NBUF - 2 < stages) wait_vmcnt<(NBUF - 2) * kIW>();
      else wait_vmcnt<0>();
      block_barrier();
      // Every wave has finished stage s - 1, whose buffer the next DMA refills.
      if (s + NBUF - 1 < stages) issue(s + NBUF - 1);
      const int kb = stage_of(s) * WK + wk;  // this wave's block of the segment
      if ((kb & 3) < WK || s == 0) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
          if (!kOwnH) sa[i] = sc[kb / 4 * kRows + arow0 + 16 * i] >> (8 * (kb & 3));
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] = sc[kb / 4 * kRows + brow0 + 16 * j] >> (8 * (kb & 3));
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i)
          if (!kOwnH) sa[i] >>= 8 * (WK % 4);  // with WK = 4 each stage reads its word
#pragma unroll
        for (int j = 0; j < TN; ++j) sb[j] >>= 8 * (WK % 4);
      }
      if (WK > 1 && kb >= seg) continue;  // the last stage is short
      if (kOwnH) sa[0] = own[kHeadQOwn + (first - b0 + kb) * a.M + own_m];
      const uint8_t* buf = lds + s % NBUF * C::kStage + wk * kRows * 128;
      i32x8 bf[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) bf[j] = fragment(buf, brow0 + 16 * j);
#if defined(__HIP_DEVICE_COMPILE__)
      if constexpr (kF32) {
        bf16x8 bv[TN][4];
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int p = 0; p < 4; ++p) bv[j][p] = codes_to_bf16(bf[j][2 * p], bf[j][2 * p + 1], scale_float(sb[j]));
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const i32x8 af = kOwnH ? own_fragment(first - b0 + kb) : fragment(buf, arow0 + 16 * i);
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const bf16x8 av = codes_to_bf16(af[2 * p], af[2 * p + 1], scale_float(sa[i]));
#pragma unroll
            for (int j = 0; j < TN; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, bv[j][p], acc[i][j], 0, 0, 0);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
          const i32x8 af = kOwnH ? own_fragment(first - b0 + kb) : fragment(buf, arow0 + 16 * i);
#pragma unroll
          for (int j = 0; j < TN; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(af, bf[j], acc[i][j], 0, 0, 0, (int)sa[i], 0,
                                                                         (int)sb[j]);
        }
      }
#endif
    }
  }
  // Every DMA has landed (the last stages waited for vmcnt 0).
  __syncthreads();
  float* stage = reinterpret_cast<float*>(lds);

  if (WK > 1) {
    // One row chunk at a time, groups 1 .. park their sums and group 0 adds
    // them in order.
    constexpr int kE = TN * 4;
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      if (wk > 0) {
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            stage[(((wk - 1) * WM * WN + wmn) * kE + j * 4 + r) * kWave + lane] = acc[i][j][r];
      }
      __syncthreads();
      if (wk == 0) {
#pragma unroll
        for (int k2 = 1; k2 < WK; ++k2)
#pragma unroll
          for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              acc[i][j][r] += stage[(((k2 - 1) * WM * WN + wmn) * kE + j * 4 + r) * kWave + lane];
      }
      __syncthreads();
    }
  }

  // Through LDS to whole rows, one chunk of 16 rows per wave row at a time:
  // lane l holds D[4 * (l / 16) + r][l % 16] of each 16 x 16 chunk; then every
  // thread stores 4 consecutive columns.
  constexpr int kLd = kNt + 4, kTpr = kNt / 4;
  const int c4 = (int)(threadIdx.x % kTpr) * 4;
  void* dst = a.split == 1 ? a.out : static_cast<void*>(a.partial + (size_t)slice * a.M * a.N);
  const bool bf16 = a.split == 1 && a.out_bf16;
  const bool vec = a.N % 4 == 0 && (uintptr_t)dst % (bf16 ? 8 : 16) == 0;
  bool none[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) none[e] = token[kH + c4 + e] < 0;
#pragma unroll
  for (int i = 0; i < TM; ++i) {
    if (i > 0) __syncthreads();
    if (wk == 0) {
#pragma unroll
      for (int j = 0; j < TN; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          stage[(wm * 16 + 4 * fc + r) * kLd + wn * 16 * TN + 16 * j + frow] = acc[i][j][r];
    }
    __syncthreads();
    for (int r = threadIdx.x / kTpr; r < 16 * WM; r += C::kThreads / kTpr) {
      const int m = m0 + (r / 16) * 16 * TM + 16 * i + r % 16;
      if (m >= a.M) continue;
      float w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = none[e] ? 0.0f : stage[r * kLd + c4 + e];
      const size_t o = (size_t)m * a.N + n0 + c4;
      if (vec) {
        if (n0 + c4 < a.N) store4(dst, bf16, o, w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n0 + c4 + e < a.N) store1(dst, bf16, o + e, w[e]);
      }
    }
  }
}

// out[m, n] = sum over slices 0 .. split - 1 of partial[s][m][n], in order.
__global__ void __launch_bounds__(kBlock) headq_reduce_kernel(HeadQArgs a) {
  const size_t MN = (size_t)a.M * (size_t)a.N;
  const size_t q = ((size_t)blockIdx.x * kBlock + threadIdx.x) * 4;
  if (q >= MN) return;
  const bool whole = MN % 4 == 0;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int s = 0; s < a.split; ++s) {
    const float* p = a.partial + (size_t)s * MN + q;
    if (whole) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (q + e < MN) v[e] += p[e];
    }
  }
  if (whole && (uintptr_t)a.out % (a.out_bf16 ? 8 : 16) == 0) {
    store4(a.out, a.out_bf16, q, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (q + e < MN) store1(a.out, a.out_bf16, q + e, v[e]);
  }
}

template <int WM, int WN, int WK, int TM, int TN, int NBUF, bool kOwnH = false>
hipError_t launch_tile(HeadQArgs a, const HeadQPlan& plan, hipStream_t st) {
  using C = HeadQTile<WM, WN, WK, TM, TN, NBUF, kOwnH>;
  if (plan.mt != C::kMt || plan.nt != C::kNt) return hipErrorInvalidValue;
  a.m_tiles = (a.M + C::kMt - 1) / C::kMt;
  const long long tiles = ((long long)a.N + C::kNt - 1) / C::kNt * a.m_tiles;
  a.split_nb = (a.nb + plan.split - 1) / plan.split;
  a.split = (a.nb + a.split_nb - 1) / a.split_nb;  // no empty slice
  const long long total = tiles * a.split;
  a.total = (int)total;
  a.per_xcd = (int)((total + 7) / 8);
  a.dword_scales = a.nb % 4 == 0 && a.split_nb % 4 == 0 && (uintptr_t)a.hs % 4 == 0 && (uintptr_t)a.ws % 4 == 0;
  const dim3 grid((unsigned)a.per_xcd * 8), block(C::kThreads);
  if (a.out_bf16) hipLaunchKernelGGL((headq_kernel<WM, WN, WK, TM, TN, NBUF, kOwnH, false>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((headq_kernel<WM, WN, WK, TM, TN, NBUF, kOwnH, true>), grid, block, 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.split == 1) return e;
  const size_t quads = ((size_t)a.M * (size_t)a.N + 3) / 4;
  hipLaunchKernelGGL(headq_reduce_kernel, dim3((unsigned)((quads + kBlock - 1) / kBlock)), dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_head_quantized(const void* h, const void* W_codes, const void* W_scales, const int32_t* cluster_ids,
                                 int M, int d, int V, int cluster_size, int n_sel, void* out, int out_dtype,
                                 const HeadQPlan& plan, const HeadQWorkspace& w, void* workspace, hipStream_t st) {
  char* base = static_cast<char*>(workspace);
  HeadQArgs a{};
  a.hq = reinterpret_cast<const uint8_t*>(base + w.codes);
  a.hs = reinterpret_cast<const uint8_t*>(base + w.scales);
  a.wq = static_cast<const uint8_t*>(W_codes);
  a.ws = static_cast<const uint8_t*>(W_scales);
  a.cids = cluster_ids;
  a.M = M;
  a.N = n_sel * cluster_size;
  a.cs = cluster_size;
  a.nclusters = V / cluster_size;
  a.nb = quant_blocks(d);
  a.out = out;
  a.out_bf16 = out_dtype == 1;
  a.partial = reinterpret_cast<float*>(base + w.partial);
  if (plan.own_h) {
    a.h = static_cast<const uint16_t*>(h);
    a.d = d;
    a.vec_h = d % 8 == 0 && (uintptr_t)h % 16 == 0;
    return launch_tile<1, 2, 4, 1, 1, 3, true>(a, plan, st);
  }
  const hipError_t e = launch_quantize_rows(h, M, d, 1, base + w.codes, base + w.scales, st);
  if (e != hipSuccess) return e;
  switch (plan.tile) {
    case 0: return launch_tile<1, 2, 4, 1, 1, 3>(a, plan, st);
    case 1: return launch_tile<1, 4, 1, 2, 1, 3>(a, plan, st);
    case 2: return launch_tile<2, 4, 1, 2, 2, 3>(a, plan, st);
    case 3: return launch_tile<2, 4, 1, 4, 2, 3>(a, plan, st);
    case 4: return launch_tile<2, 4, 1, 4, 4, 3>(a, plan, st);
    default: return launch_tile<2, 4, 1, 8, 4, 2>(a, plan, st);
  }
}

}  // namespace sv
