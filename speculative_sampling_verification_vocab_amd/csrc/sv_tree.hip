// Commit of a tree's path.  From the root (node 0) the walk goes on to the
// first child whose token is the one that was drawn at the node, until there is
// none: the drawn tokens along the path are the step's output, whatever the
// drafts were, and the path's entries move from staging to the cache.
//
// The walk is one wave's, a node per lane: a ballot finds the child, so a path
// of d nodes costs d ballots after three loads.  Every block walks for itself
// (a few hundred nanoseconds beside loads that it must wait for anyway), so the
// copy needs no launch before it; the entries of a path are scattered in
// staging and contiguous in the cache.
//
// Measured (64 planes, entries of 1024 bf16 values, staging from memory): 256
// trees of 16 34 us, 3.9 TB/s read and written of a large copy's 4.9, and in 8 bits
// 34 us too, 3.0 TB/s, where the walk's chain of loads and the codes' arithmetic
// show (28 and 29 us where the memory-side cache has the staging); one tree of 8
// 3.5 and 4.5 us, two dependent loads and a launch.

#include <type_traits>

#include "sv_internal.h"
#include "sv_quant.h"
#include "sv_tree.h"

namespace sv {

namespace {

struct TreeCommitArgs {
  TreeCommitIO io;
  int P, B, N, L;
  uint32_t chunks;
  int planes;  // of a block
  // values
  uint8_t* cache;          // [P][B][L][units]
  const uint8_t* staging;  // [P][B][N][units]
  int units;               // vectors or elements of an entry
  // 8-bit
  uint8_t *codes, *scales;  // [P][B][L][E], [P][B][L][nb]
  const void* in;           // [P][B][N][E]
  int E, nb;
};

struct Walk {
  int count;   // nodes of the path, 0 for a faulty sequence
  int len;     // cache_len
  int status;  // 0 committed, 1 no room, 2 faulty
};

// Where piece i of a block's planes is, with n pieces per entry and `count`
// entries per plane: at most 512 entries, so that a quotient by a reciprocal is
// off by one at most.  Whole divisions here cost a fifth of the copy's time.
struct Pieces {
  int n, count;
  float per_n, per_count;
  __device__ __forceinline__ Pieces(int n_, int count_) : n(n_), count(count_), per_n(1.0f / n_), per_count(1.0f / count_) {}
  // The plane, and the path's node r; the piece of that entry.
  __device__ __forceinline__ int place(int i, int& plane, int& r) const {
    int q = (int)((float)i * per_n), u = i - q * n;
    if (u < 0) --q, u += n;
    else if (u >= n) ++q, u -= n;
    plane = (int)(((float)q + 0.5f) * per_count);
    r = q - plane * count;
    return u;
  }
};

// The walk of sequence b, by the 64 lanes of a wave; path[i] is its node i.
// out: the lane writes what it knows of the outputs too.
__device__ __forceinline__ Walk walk_tree(const TreeCommitArgs& a, int b, int lane, int* path, bool out) {
  const size_t at = (size_t)b * a.N + lane;
  const bool in = lane < a.N;
  const int parent = in ? a.io.parents[at] : -2, token = in ? a.io.tokens[at] : 0, drawn = in ? a.io.sampled[at] : 0;
  Walk w;
  w.len = a.io.cache_len[b];
  w.count = 0;
  int mine = -1, emitted = -1;  // the path's node `lane`, and the token drawn there
  bool fault = __builtin_amdgcn_readlane(parent, 0) != -1;
  int cur = 0;
  while (!fault) {
    const int t = __builtin_amdgcn_readlane(drawn, cur);
    if (t < 0) {
      fault = true;
      break;
    }
    if (lane == w.count) mine = cur, emitted = t;
    ++w.count;
    const uint64_t next = __ballot(in && lane > cur && parent == cur && token == t);
    if (next == 0) break;
    cur = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)next) - 1);
  }
  if (fault) w.count = 0, mine = -1, emitted = -1;
  w.status = fault ? 2 : w.len < 0 || w.len > a.L - w.count ? 1 : 0;
  if (path) path[lane] = mine;
  if (out) {
    if (in) {
      a.io.out_tokens[at] = emitted;
      if (a.io.path) a.io.path[at] = mine;
    }
    if (lane == 0) {
      a.io.accepted_len[b] = w.count - 1;
      if (a.io.status) a.io.status[b] = w.status;
      a.io.new_len[b] = w.status == 0 ? w.len + w.count : w.len;
    }
  }
  return w;
}

// Block (planes, sequence, chunk): the path's units, chunk by chunk of four per
// thread.  out: the first block of a sequence writes its outputs.
template <int kUnit>
__global__ void __launch_bounds__(kBlock) tree_commit_kernel(TreeCommitArgs a, int out) {
  __shared__ int path[kMaxNodes];
  __shared__ int head[3];
  const uint32_t gb = blockIdx.x / a.chunks, chunk = blockIdx.x - gb * a.chunks;
  const int b = (int)(gb % (uint32_t)a.B), plane0 = (int)(gb / (uint32_t)a.B) * a.planes;
  if (threadIdx.x < kWave) {
    const Walk w = walk_tree(a, b, threadIdx.x, path, out && chunk == 0 && plane0 == 0);
    if (threadIdx.x == 0) head[0] = w.count, head[1] = w.len, head[2] = w.status;
  }
  __syncthreads();
  if (head[2] != 0) return;
  constexpr int kU = 4;
  const int total = head[0] * a.units * min(a.planes, a.P - plane0);
  using U = typename std::conditional<kUnit == 16, u32x4, typename std::conditional<kUnit == 4, uint32_t, uint16_t>::type>::type;
  const U* s = reinterpret_cast<const U*>(a.staging);
  U* d = reinterpret_cast<U*>(a.cache);
  const Pieces pieces(a.units, head[0]);
  for (int i0 = (int)chunk * kBlock * kU + threadIdx.x; i0 < total; i0 += (int)a.chunks * kBlock * kU) {
    U v[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int i = i0 + k * kBlock;
      if (i < total) {
        int p, r;
        const int u = pieces.place(i, p, r);
        const size_t pb = (size_t)(plane0 + p) * a.B + b;
        v[k] = s[(pb * a.N + path[r]) * a.units + u];
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int i = i0 + k * kBlock;
      if (i < total) {
        int p, r;
        const int u = pieces.place(i, p, r);
        const size_t pb = (size_t)(plane0 + p) * a.B + b;
        U* to = d + (pb * a.L + head[1] + r) * a.units + u;
        // Nontemporal whole vectors: 512 and 256 trees whose staging comes from memory 60 and 34 us, else 72 and 40; 64
        // trees and fewer the same.
        if constexpr (kUnit == 16) __builtin_nontemporal_store(v[k], to);
        else *to = v[k];
      }
    }
  }
}

template <typename T, bool kVec>
__global__ void __launch_bounds__(kBlock) tree_commit_quantized_kernel(TreeCommitArgs a, int out) {
  __shared__ int path[kMaxNodes];
  __shared__ int head[3];
  const uint32_t gb = blockIdx.x / a.chunks, chunk = blockIdx.x - gb * a.chunks;
  const int b = (int)(gb % (uint32_t)a.B), plane0 = (int)(gb / (uint32_t)a.B) * a.planes;
  if (threadIdx.x < kWave) {
    const Walk w = walk_tree(a, b, threadIdx.x, path, out && chunk == 0 && plane0 == 0);
    if (threadIdx.x == 0) head[0] = w.count, head[1] = w.len, head[2] = w.status;
  }
  __syncthreads();
  if (head[2] != 0) return;
  constexpr int kU = 4, kPer = kBlock / kLanesPerBlock;
  // Blocks of the format, 16 lanes each.
  const int total = head[0] * a.nb * min(a.planes, a.P - plane0);
  const int sub = threadIdx.x % kLanesPerBlock;
  const T* src = static_cast<const T*>(a.in);
  const Pieces pieces(a.nb, head[0]);
  for (int base = (int)chunk * kPer * kU; base < total; base += (int)a.chunks * kPer * kU) {
    const int first = base + threadIdx.x / kLanesPerBlock;
    float v[kU][kPerLaneQ];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (base + k * kPer >= total) break;
      const int i = min(first + k * kPer, total - 1);
      int p, r;
      const int at = pieces.place(i, p, r) * kQuantBlock + sub * kPerLaneQ;
      const size_t pb = (size_t)(plane0 + p) * a.B + b;
      load8<T, kVec, false>(src + (pb * a.N + path[r]) * (size_t)a.E + at, a.E - at, v[k]);
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (base + k * kPer >= total) break;
      const int i = first + k * kPer;
      int sb;
      const uint2 q = quantize8(v[k], &sb);
      if (i >= total) continue;
      int p, r;
      const int blk = pieces.place(i, p, r), at = blk * kQuantBlock + sub * kPerLaneQ;
      const size_t row = ((size_t)(plane0 + p) * a.B + b) * a.L + head[1] + r;
      store_codes<kVec>(a.codes + row * (size_t)a.E + at, a.E - at, q);
      if (sub == 0) a.scales[row * (size_t)a.nb + blk] = (uint8_t)sb;
    }
  }
}

// The outputs alone: a wave per sequence.
__global__ void __launch_bounds__(kBlock) tree_walk_kernel(TreeCommitArgs a) {
  const int b = blockIdx.x * kWavesPerBlock + threadIdx.x / kWave;
  if (b < a.B) walk_tree(a, b, threadIdx.x & (kWave - 1), nullptr, true);
}

hipError_t finish(const TreeCommitArgs& a, bool copied, hipStream_t st) {
  if (copied) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.io.new_len != a.io.cache_len) return e;
  }
  hipLaunchKernelGGL(tree_walk_kernel, dim3(((unsigned)a.B + kWavesPerBlock - 1) / kWavesPerBlock), dim3(kBlock), 0, st, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tree_commit(void* cache, const void* staging, const TreeCommitIO& io, int P, int B, int N, int L,
                              const TreeCopyPlan& plan, hipStream_t st) {
  TreeCommitArgs a{};
  a.io = io;
  a.P = P;
  a.B = B;
  a.N = N;
  a.L = L;
  a.chunks = plan.chunks;
  a.planes = tree_planes(P, B, plan.chunks);
  a.cache = static_cast<uint8_t*>(cache);
  a.staging = static_cast<const uint8_t*>(staging);
  a.units = plan.units;
  const bool copies = plan.chunks > 0;
  if (copies) {
    const dim3 grid((unsigned)((size_t)((P + a.planes - 1) / a.planes) * (size_t)B * plan.chunks));
    const int out = io.new_len != io.cache_len;
    if (plan.unit_bytes == 16) hipLaunchKernelGGL(tree_commit_kernel<16>, grid, dim3(kBlock), 0, st, a, out);
    else if (plan.unit_bytes == 4) hipLaunchKernelGGL(tree_commit_kernel<4>, grid, dim3(kBlock), 0, st, a, out);
    else hipLaunchKernelGGL(tree_commit_kernel<2>, grid, dim3(kBlock), 0, st, a, out);
  }
  return finish(a, copies, st);
}

hipError_t launch_tree_commit_quantized(void* codes, void* scales, const void* staging, const TreeCommitIO& io, int P,
                                        int B, int N, int L, int E, int dtype, const KvQPlan& plan, hipStream_t st) {
  TreeCommitArgs a{};
  a.io = io;
  a.P = P;
  a.B = B;
  a.N = N;
  a.L = L;
  a.chunks = plan.chunks;
  a.planes = tree_planes(P, B, plan.chunks);
  a.codes = static_cast<uint8_t*>(codes);
  a.scales = static_cast<uint8_t*>(scales);
  a.in = staging;
  a.E = E;
  a.nb = plan.nb;
  if (plan.copies) {
    const dim3 grid((unsigned)((size_t)((P + a.planes - 1) / a.planes) * (size_t)B * plan.chunks));
    const int out = io.new_len != io.cache_len;
    if (dtype == 1) {
      if (plan.vec) hipLaunchKernelGGL((tree_commit_quantized_kernel<uint16_t, true>), grid, dim3(kBlock), 0, st, a, out);
      else hipLaunchKernelGGL((tree_commit_quantized_kernel<uint16_t, false>), grid, dim3(kBlock), 0, st, a, out);
    } else {
      if (plan.vec) hipLaunchKernelGGL((tree_commit_quantized_kernel<float, true>), grid, dim3(kBlock), 0, st, a, out);
      else hipLaunchKernelGGL((tree_commit_quantized_kernel<float, false>), grid, dim3(kBlock), 0, st, a, out);
    }
  }
  return finish(a, plan.copies, st);
}

}  // namespace sv
