// Rows and KV caches in the 8-bit block format (sv_quant.h): quantising rows,
// the KV commit that quantises as it writes, and reading a cache back.
// All three only move data: a value is read once, a code written once (or the
// reverse), about one operation per byte in between, so each is bound by HBM.
// One lane holds 8 values: 16 bytes of bf16 or 32 of fp32 on one side, 8 of
// codes on the other, and the 16 lanes of a DPP row hold a block, whose
// maximum then takes four lane moves and no LDS.
// Measured: a weight of 128256 x 4096 bf16 quantised in 247 us (1.58 GB, 6.4
// TB/s read and written; a device copy reaches 5.0); 256 x 7 drafts of 64
// planes of 1024, half of them accepted, committed in 45 us (177 MB, 3.9 TB/s,
// in runs of 2 KB to 14 KB); 2 planes of 64 x 8192 entries of 1024 read back in
// 401 us (2.43 GB, 6.0 TB/s).

#include "sv_internal.h"
#include "sv_quant.h"

namespace sv {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ---- rows -----------------------------------------------------------------------

// Blocks of the format are numbered through all rows: block i's codes are
// bytes 128 * i .., its scale is byte i.  Each thread takes part in U of them,
// 16 apart, whose loads are issued together.
template <typename T, bool kVec, int U>
__global__ void __launch_bounds__(kBlock) quantize_rows_kernel(const T* __restrict__ x, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales, uint32_t blocks,
                                                               uint32_t nb, int d) {
  constexpr int kPer = kBlock / kLanesPerBlock;
  const int sub = threadIdx.x % kLanesPerBlock;
  const uint32_t first = blockIdx.x * (uint32_t)(kPer * U) + threadIdx.x / kLanesPerBlock;
  float v[U][kPerLaneQ];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = min(first + (uint32_t)(k * kPer), blocks - 1);  // past the end: the last one again, not stored
    const uint32_t row = i / nb;
    const int at = (int)(i - row * nb) * kQuantBlock + sub * kPerLaneQ;
    load8<T, kVec>(x + (size_t)row * (size_t)d + at, d - at, v[k]);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const uint32_t i = first + (uint32_t)(k * kPer);
    int sb;
    const uint2 q = quantize8(v[k], &sb);
    if (i >= blocks) continue;
    store_codes<true>(codes + (size_t)i * kQuantBlock + sub * kPerLaneQ, kPerLaneQ, q);
    if (sub == 0) scales[i] = (uint8_t)sb;
  }
}

template <typename T, bool kVec>
hipError_t launch_rows(const void* x, void* codes, void* scales, uint32_t blocks, uint32_t nb, int d, hipStream_t st) {
  constexpr int kPer = kBlock / kLanesPerBlock;
  const T* p = static_cast<const T*>(x);
  uint8_t *c = static_cast<uint8_t*>(codes), *s = static_cast<uint8_t*>(scales);
  static_assert(kRowsPerBlock == kPer * 4, "the grid that rows_fit checks");
  if (blocks >= (uint32_t)(kRowsPerBlock * 1024))
    hipLaunchKernelGGL((quantize_rows_kernel<T, kVec, 4>), dim3((blocks + kRowsPerBlock - 1) / kRowsPerBlock),
                       dim3(kBlock), 0, st, p, c, s, blocks, nb, d);
  else
    hipLaunchKernelGGL((quantize_rows_kernel<T, kVec, 1>), dim3((blocks + kPer - 1) / kPer), dim3(kBlock), 0, st, p, c,
                       s, blocks, nb, d);
  return hipGetLastError();
}

// ---- KV cache -------------------------------------------------------------------

struct KvQArgs {
  uint8_t* codes;       // [P][B][Lmax][E]
  uint8_t* scales;      // [P][B][Lmax][nb]
  const void* in;       // commit: staging [P][B][K][E]
  void* out;            // read: [P][B][Lout][E]
  const int32_t* acc;   // commit: [B]
  const int32_t* len;   // [B]
  int32_t* new_len;     // commit: [B]
  int32_t* status;      // [B] or null
  int B, K, Lmax, Lout, E, nb;
  uint32_t chunks;      // thread blocks per (plane, sequence)
};

// Status of sequence b's commit: 0 commit n entries, 1 no room, 2 n outside [0, K].
__device__ __forceinline__ int commit_status(const KvQArgs& a, int b, int& n, int& len) {
  n = a.acc[b];
  len = a.len[b];
  if (n < 0 || n > a.K) return 2;
  if (len < 0 || len > a.Lmax - n) return 1;
  return 0;
}

// One (plane, sequence) per a.chunks blocks; its n accepted rows of nb format
// blocks are numbered through.  lens: the first block of each sequence also
// writes its new length and status (new_len is not cache_len, so no block
// reads what another writes).
template <typename T, bool kVec, int U, bool kStream>
__global__ void __launch_bounds__(kBlock) kvq_commit_kernel(KvQArgs a, int lens) {
  const uint32_t pb = blockIdx.x / a.chunks, chunk = blockIdx.x - pb * a.chunks;
  const int b = (int)(pb % (uint32_t)a.B);
  int n, len;
  const int st = commit_status(a, b, n, len);
  if (lens && chunk == 0 && pb < (uint32_t)a.B && threadIdx.x == 0) {
    a.new_len[b] = st == 0 ? len + n : len;
    if (a.status) a.status[b] = st;
  }
  if (st != 0) return;
  constexpr int kPer = kBlock / kLanesPerBlock;
  const int total = n * a.nb;
  const int base = (int)chunk * (kPer * U), first = base + threadIdx.x / kLanesPerBlock;
  if (base >= total) return;
  const int sub = threadIdx.x % kLanesPerBlock;
  const T* src = static_cast<const T*>(a.in) + (size_t)pb * (size_t)a.K * (size_t)a.E;
  const size_t row0 = (size_t)pb * (size_t)a.Lmax + (size_t)len;
  float v[U][kPerLaneQ];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (base + k * kPer >= total) break;  // few drafts fill a part of the block: 60 us without, 48 with
    const int i = min(first + k * kPer, total - 1);
    const int r = i / a.nb;
    const int at = (i - r * a.nb) * kQuantBlock + sub * kPerLaneQ;
    load8<T, kVec, kStream>(src + (size_t)r * (size_t)a.E + at, a.E - at, v[k]);
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    if (base + k * kPer >= total) break;
    const int i = first + k * kPer;
    int sb;
    const uint2 q = quantize8(v[k], &sb);
    if (i >= total) continue;
    const int r = i / a.nb, blk = i - r * a.nb;
    const int at = blk * kQuantBlock + sub * kPerLaneQ;
    store_codes<kVec>(a.codes + (row0 + (size_t)r) * (size_t)a.E + at, a.E - at, q);
    if (sub == 0) a.scales[(row0 + (size_t)r) * (size_t)a.nb + blk] = (uint8_t)sb;
  }
}

__global__ void __launch_bounds__(kBlock) kvq_lengths_kernel(KvQArgs a) {
  const int b = blockIdx.x * kBlock + threadIdx.x;
  if (b >= a.B) return;
  int n, len;
  const int st = commit_status(a, b, n, len);
  a.new_len[b] = st == 0 ? len + n : len;
  if (a.status) a.status[b] = st;
}

// 2^(byte - 127); byte 255 is e8m0's NaN.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : byte == 255 ? 0x7fc00000u : byte << 23);
}

// Eight codes to values.  The product with a power of two is exact (subnormal
// results aside), and has four significant bits: bf16 holds it as it is.
__device__ __forceinline__ void decode8(uint2 q, float s, float (&x)[kPerLaneQ]) {
#if defined(__HIP_DEVICE_COMPILE__)
  const auto a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.x, true);
  const auto c = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8((int)q.y, true);
  x[0] = a[0] * s, x[1] = a[1] * s, x[2] = b[0] * s, x[3] = b[1] * s;
  x[4] = c[0] * s, x[5] = c[1] * s, x[6] = d[0] * s, x[7] = d[1] * s;
#endif
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)lo, (__bf16)hi});
}

template <bool kVec>
__device__ __forceinline__ void store8(uint16_t* p, const float (&x)[kPerLaneQ]) {
  const u32x4 w{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
  if (kVec) __builtin_nontemporal_store(w, reinterpret_cast<u32x4*>(p));  // 64 x 8192 entries: 420 -> 403 us
  else *reinterpret_cast<u32x4_any2*>(p) = w;
}
template <bool kVec>
__device__ __forceinline__ void store8(float* p, const float (&x)[kPerLaneQ]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const u32x4 w{__float_as_uint(x[4 * q]), __float_as_uint(x[4 * q + 1]), __float_as_uint(x[4 * q + 2]),
                  __float_as_uint(x[4 * q + 3])};
    if (kVec) *reinterpret_cast<u32x4*>(p + 4 * q) = w;
    else *reinterpret_cast<u32x4_any4*>(p + 4 * q) = w;
  }
}
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }

template <typename T, bool kVec, int U>
__global__ void __launch_bounds__(kBlock) kvq_read_kernel(KvQArgs a) {
  const uint32_t pb = blockIdx.x / a.chunks, chunk = blockIdx.x - pb * a.chunks;
  const int b = (int)(pb % (uint32_t)a.B);
  const int n = a.len[b];
  const int st = n < 0 || n > a.Lmax || n > a.Lout ? 1 : 0;
  if (a.status && chunk == 0 && pb < (uint32_t)a.B && threadIdx.x == 0) a.status[b] = st;
  if (st != 0) return;
  constexpr int kPer = kBlock / kLanesPerBlock;
  const int total = n * a.nb;
  const int base = (int)chunk * (kPer * U), first = base + threadIdx.x / kLanesPerBlock;
  if (base >= total) return;
  const int sub = threadIdx.x % kLanesPerBlock;
  const size_t row0 = (size_t)pb * (size_t)a.Lmax;
  const uint8_t* src = a.codes + row0 * (size_t)a.E;
  const uint8_t* sc = a.scales + row0 * (size_t)a.nb;
  T* dst = static_cast<T*>(a.out) + (size_t)pb * (size_t)a.Lout * (size_t)a.E;
  uint2 q[U];
  uint32_t sb[U];
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int i = min(first + k * kPer, total - 1);  // nearly all are there: no branch
    const int r = i / a.nb;
    const int at = (i - r * a.nb) * kQuantBlock + sub * kPerLaneQ;
    const uint8_t* p = src + (size_t)r * (size_t)a.E + at;
    q[k] = uint2{0u, 0u};
    sb[k] = sc[i];
    if (at + kPerLaneQ <= a.E) {
      if (kVec) {
        q[k] = *reinterpret_cast<const uint2*>(p);
      } else {
        const u32x2_any w = *reinterpret_cast<const u32x2_any*>(p);
        q[k] = uint2{w[0], w[1]};
      }
    } else if (!kVec) {
#pragma unroll
      for (int e = 0; e < kPerLaneQ; ++e) {
        const uint32_t c = at + e < a.E ? (uint32_t)p[e] : 0u;
        if (e < 4) q[k].x |= c << (8 * e);
        else q[k].y |= c << (8 * (e - 4));
      }
    }
  }
#pragma unroll
  for (int k = 0; k < U; ++k) {
    const int i = first + k * kPer;
    if (i >= total) continue;
    const int r = i / a.nb;
    const int at = (i - r * a.nb) * kQuantBlock + sub * kPerLaneQ;
    T* p = dst + (size_t)r * (size_t)a.E + at;
    float x[kPerLaneQ];
    decode8(q[k], scale_value(sb[k]), x);
    if (at + kPerLaneQ <= a.E) {
      store8<kVec>(p, x);
    } else if (!kVec) {
#pragma unroll
      for (int e = 0; e < kPerLaneQ; ++e)
        if (at + e < a.E) store1(p + e, x[e]);
    }
  }
}

__global__ void __launch_bounds__(kBlock) kvq_read_status_kernel(KvQArgs a) {
  const int b = blockIdx.x * kBlock + threadIdx.x;
  if (b < a.B) a.status[b] = a.len[b] < 0 || a.len[b] > a.Lmax || a.len[b] > a.Lout ? 1 : 0;
}

template <typename T, bool kVec, int U>
void start_commit(const KvQArgs& a, unsigned grid, int lens, bool stream, hipStream_t st) {
  if (stream) hipLaunchKernelGGL((kvq_commit_kernel<T, kVec, U, true>), dim3(grid), dim3(kBlock), 0, st, a, lens);
  else hipLaunchKernelGGL((kvq_commit_kernel<T, kVec, U, false>), dim3(grid), dim3(kBlock), 0, st, a, lens);
}
template <typename T, bool kVec, int U>
void start_read(const KvQArgs& a, unsigned grid, hipStream_t st) {
  hipLaunchKernelGGL((kvq_read_kernel<T, kVec, U>), dim3(grid), dim3(kBlock), 0, st, a);
}

}  // namespace

hipError_t launch_quantize_rows(const void* x, int R, int d, int dtype, void* codes, void* scales, hipStream_t st) {
  const uint32_t nb = (uint32_t)quant_blocks(d), blocks = (uint32_t)R * nb;
  const size_t row = (size_t)d * (dtype == 1 ? 2 : 4);
  const bool vec = row % 16 == 0 && d % 8 == 0 && (uintptr_t)x % 16 == 0;
  if (dtype == 1)
    return vec ? launch_rows<uint16_t, true>(x, codes, scales, blocks, nb, d, st)
               : launch_rows<uint16_t, false>(x, codes, scales, blocks, nb, d, st);
  return vec ? launch_rows<float, true>(x, codes, scales, blocks, nb, d, st)
             : launch_rows<float, false>(x, codes, scales, blocks, nb, d, st);
}

hipError_t launch_kv_commit_quantized(void* codes, void* scales, const void* staging, const int32_t* accepted_len,
                                      const int32_t* cache_len, int32_t* new_len, int32_t* status, int P, int B, int K,
                                      int Lmax, int E, int dtype, const KvQPlan& plan, hipStream_t st) {
  KvQArgs a{};
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.in = staging;
  a.acc = accepted_len;
  a.len = cache_len;
  a.new_len = new_len;
  a.status = status;
  a.B = B;
  a.K = K;
  a.Lmax = Lmax;
  a.E = E;
  a.nb = plan.nb;
  a.chunks = plan.chunks;
  const int lens = new_len != cache_len;
  if (plan.copies) {
    const unsigned grid = (unsigned)((size_t)P * (size_t)B * plan.chunks);
    const int pick = (dtype == 1 ? 4 : 0) + (plan.vec ? 2 : 0) + (plan.unroll == 4 ? 1 : 0);
    // Staging that fits in the memory-side cache is likely still there (64
    // planes x 64 x 7 entries of 1024 fp32: 26 us nontemporal, 17 plain); more
    // than that streams (2 x 2000 bf16 entries: 42 and 48 us).
    const bool stream = (size_t)P * B * K * E * (dtype == 1 ? 2 : 4) > ((size_t)256 << 20);
    switch (pick) {
      case 0: start_commit<float, false, 1>(a, grid, lens, stream, st); break;
      case 1: start_commit<float, false, 4>(a, grid, lens, stream, st); break;
      case 2: start_commit<float, true, 1>(a, grid, lens, stream, st); break;
      case 3: start_commit<float, true, 4>(a, grid, lens, stream, st); break;
      case 4: start_commit<uint16_t, false, 1>(a, grid, lens, stream, st); break;
      case 5: start_commit<uint16_t, false, 4>(a, grid, lens, stream, st); break;
      case 6: start_commit<uint16_t, true, 1>(a, grid, lens, stream, st); break;
      default: start_commit<uint16_t, true, 4>(a, grid, lens, stream, st); break;
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || lens) return e;
  }
  hipLaunchKernelGGL(kvq_lengths_kernel, dim3(((unsigned)B + kBlock - 1) / kBlock), dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_kv_read_quantized(const void* codes, const void* scales, const int32_t* cache_len, void* out,
                                    int32_t* status, int P, int B, int Lmax, int Lout, int E, int dtype,
                                    const KvQPlan& plan, hipStream_t st) {
  KvQArgs a{};
  a.codes = static_cast<uint8_t*>(const_cast<void*>(codes));
  a.scales = static_cast<uint8_t*>(const_cast<void*>(scales));
  a.out = out;
  a.len = cache_len;
  a.status = status;
  a.B = B;
  a.Lmax = Lmax;
  a.Lout = Lout;
  a.E = E;
  a.nb = plan.nb;
  a.chunks = plan.chunks;
  if (!plan.copies) {
    if (!status) return hipSuccess;
    hipLaunchKernelGGL(kvq_read_status_kernel, dim3(((unsigned)B + kBlock - 1) / kBlock), dim3(kBlock), 0, st, a);
    return hipGetLastError();
  }
  const unsigned grid = (unsigned)((size_t)P * (size_t)B * plan.chunks);
  if (dtype != 1) {  // one unit per thread (see check_kv_quantized)
    if (plan.vec) start_read<float, true, 1>(a, grid, st);
    else start_read<float, false, 1>(a, grid, st);
  } else if (plan.unroll == 4) {
    if (plan.vec) start_read<uint16_t, true, 4>(a, grid, st);
    else start_read<uint16_t, false, 4>(a, grid, st);
  } else {
    if (plan.vec) start_read<uint16_t, true, 1>(a, grid, st);
    else start_read<uint16_t, false, 1>(a, grid, st);
  }
  return hipGetLastError();
}

}  // namespace sv
