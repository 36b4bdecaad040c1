// libtrace routed rows for gfx950: the sort of (token, expert) pairs by
// expert, the gather of the tokens' rows into that order, the weighted sum of
// the experts' rows back to the tokens, and that sum's gradients.
//
// Sort: a stable counting sort.  A workgroup owns a chunk of pairs, its four
// waves consecutive quarters of it; a wave ranks 64 pairs at a time
// by comparing expert numbers bit by bit (one ballot per bit), so the order
// inside an expert is the pairs' own and no result depends on the order of
// atomics.  One chunk is one launch.  More chunks take a counting launch and a
// scatter launch, whose workgroups each sum the counts of the chunks before
// theirs; past kSumChunks a scan over the chunks' counts (one workgroup, one
// lane per expert) runs between the two (128 experts, with the sums and with
// the scan: 131072 pairs 15 and 19 us, 2097152 pairs 83 and 123 us, but the
// sums grow with the square).
//
// Dispatch, combine and combine's gradients move rows and are bound by
// memory: 16 bytes per lane, sums in fp32 in the order of a token's pairs.
// 16384 tokens of 2048, 8 experts each: dispatch 144 us (537 MB written and,
// since a token's rows lie far apart, as much read, most of it from the
// last-level cache: 7.5 TB/s), combine 116 us (5.2 TB/s; of fp32 rows 217, 5.3
// TB/s), its gradients 220 us (5.2 TB/s).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_mx.h"

namespace trace_dev {

constexpr uint32_t kSortChunk = 2048;  // at most
constexpr uint32_t kSortWaves = kThreads / 64;
constexpr uint32_t kSortRounds = kSortChunk / kThreads;
constexpr uint32_t kSumChunks = 1024;

// Expert of a pair as a bin: experts that are not held share the last bin.
__device__ __forceinline__ uint32_t expert_bin(const int64_t* __restrict__ ids, uint64_t pair, uint32_t experts) {
  const int64_t e = ids[pair];
  return (e >= 0 && e < (int64_t)experts) ? (uint32_t)e : experts;
}

// Lanes of the wave, among those with `active`, that hold the same bin.
__device__ __forceinline__ uint64_t same_bin(uint32_t bin, bool active, uint32_t bits) {
  uint64_t peers = __ballot(active);
  for (uint32_t b = 0; b < bits; ++b) {
    const uint64_t set = __ballot((bin >> b) & 1u);
    peers &= ((bin >> b) & 1u) ? set : ~set;
  }
  return peers;
}

// Counts of a chunk's bins: counts[chunk][experts + 1].
__global__ __launch_bounds__(kThreads) void expert_count_kernel(const int64_t* __restrict__ ids, uint64_t pairs,
                                                                uint32_t experts, uint32_t chunk,
                                                                uint32_t* __restrict__ counts) {
  __shared__ uint32_t hist[trace_host::kMaxExperts + 1];
  for (uint32_t e = threadIdx.x; e <= experts; e += kThreads) hist[e] = 0;
  __syncthreads();
  const uint64_t base = (uint64_t)blockIdx.x * chunk;
#pragma unroll
  for (uint32_t r = 0; r < kSortRounds; ++r) {
    const uint64_t pair = base + r * kThreads + threadIdx.x;
    if (r * kThreads < chunk && pair < pairs) atomicAdd(&hist[expert_bin(ids, pair, experts)], 1u);
  }
  __syncthreads();
  for (uint32_t e = threadIdx.x; e <= experts; e += kThreads)
    counts[(uint64_t)blockIdx.x * (experts + 1) + e] = hist[e];
}

// Exclusive prefix over v of the workgroup's lanes, in lane order; *total is
// the sum.  `part` holds one word per wave.
template <int kWaves>
__device__ __forceinline__ uint32_t block_prefix(uint32_t v, uint32_t* part, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = (uint32_t)__shfl_up((int)s, d);
    if (lane >= (uint32_t)d) s += up;
  }
  if (lane == 63) part[wave] = s;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += (uint32_t)w < wave ? part[w] : 0u;
    all += part[w];
  }
  __syncthreads();
  *total = all;
  return before + s - v;
}

// One workgroup: counts[chunk][bin] become the first position of the bin's
// pairs of that chunk in the sorted order; offsets are written.
__global__ __launch_bounds__(1024) void expert_scan_kernel(uint32_t* __restrict__ counts, uint32_t chunks,
                                                           uint32_t experts, int64_t* __restrict__ offsets) {
  __shared__ uint32_t part[16];
  uint32_t carry = 0;
  for (uint32_t e0 = 0; e0 <= experts; e0 += 1024) {
    const uint32_t e = e0 + threadIdx.x;
    uint32_t sum = 0;
    if (e <= experts) {
#pragma unroll 8
      for (uint32_t c = 0; c < chunks; ++c) sum += counts[(uint64_t)c * (experts + 1) + e];
    }
    uint32_t total;
    uint32_t at = carry + block_prefix<16>(sum, part, &total);
    carry += total;
    if (e <= experts) {
      offsets[e] = (int64_t)at;  // the last bin starts where the held experts' rows end
#pragma unroll 8
      for (uint32_t c = 0; c < chunks; ++c) {
        uint32_t* p = &counts[(uint64_t)c * (experts + 1) + e];
        const uint32_t n = *p;
        *p = at;
        at += n;
      }
    }
  }
}

// Where expert_place_kernel has the first positions of its chunk's bins from:
// its own counts, the only chunk's; all chunks' counts; or their scan.
enum SortFirst { kOnlyChunk, kSumCounts, kScanned };

// Places a chunk's pairs; all but kScanned write the offsets.
template <SortFirst kFirst>
__global__ __launch_bounds__(kThreads) void expert_place_kernel(const int64_t* __restrict__ ids, uint64_t pairs,
                                                                uint32_t topk, uint32_t experts, uint32_t bits,
                                                                uint32_t chunk, const uint32_t* __restrict__ counts,
                                                                int64_t* __restrict__ offsets,
                                                                int64_t* __restrict__ row_index,
                                                                int64_t* __restrict__ slot) {
  __shared__ uint32_t next[kSortWaves][trace_host::kMaxExperts + 1];  // next free position, per wave and bin
  __shared__ uint32_t part[kSortWaves];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t share = chunk / kSortWaves;
  const uint64_t base = (uint64_t)blockIdx.x * chunk + wave * share;
  const auto in_share = [&](uint32_t r) { return r * 64 < share && base + r * 64 < pairs; };
  for (uint32_t w = 0; w < kSortWaves; ++w)
    for (uint32_t e = threadIdx.x; e <= experts; e += kThreads) next[w][e] = 0;
  __syncthreads();
  uint32_t bin[kSortRounds];
#pragma unroll
  for (uint32_t r = 0; r < kSortRounds; ++r) {
    const uint64_t pair = base + r * 64 + lane;
    bin[r] = in_share(r) && pair < pairs ? expert_bin(ids, pair, experts) : 0u;
  }
#pragma unroll
  for (uint32_t r = 0; r < kSortRounds; ++r)
    if (in_share(r) && base + r * 64 + lane < pairs) atomicAdd(&next[wave][bin[r]], 1u);
  __syncthreads();
  uint32_t carry = 0;
  for (uint32_t e0 = 0; e0 <= experts; e0 += kThreads) {
    const uint32_t e = e0 + threadIdx.x;
    uint32_t at = 0;
    if (kFirst == kScanned) {
      if (e <= experts) at = counts[(uint64_t)blockIdx.x * (experts + 1) + e];
    } else {
      uint32_t sum = 0, before = 0, total;  // of all chunks, and of those before this one
      if (e <= experts) {
        if (kFirst == kOnlyChunk) {
          for (uint32_t w = 0; w < kSortWaves; ++w) sum += next[w][e];
        } else {
          constexpr uint32_t kAtOnce = 16;
          for (uint32_t c0 = 0; c0 < gridDim.x; c0 += kAtOnce) {
            uint32_t n[kAtOnce];
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) {
              const uint32_t c = c0 + i < gridDim.x ? c0 + i : gridDim.x - 1;
              n[i] = counts[(uint64_t)c * (experts + 1) + e];
            }
#pragma unroll
            for (uint32_t i = 0; i < kAtOnce; ++i) {
              if (c0 + i < gridDim.x) sum += n[i];
              if (c0 + i < blockIdx.x) before += n[i];
            }
          }
        }
      }
      at = carry + block_prefix<kSortWaves>(sum, part, &total);
      carry += total;
      if (blockIdx.x == 0 && e <= experts) offsets[e] = (int64_t)at;  // the last bin starts where the held rows end
      at += before;
    }
    if (e <= experts)
      for (uint32_t w = 0; w < kSortWaves; ++w) {
        const uint32_t n = next[w][e];
        next[w][e] = at;
        at += n;
      }
  }
  __syncthreads();
#pragma unroll
  for (uint32_t r = 0; r < kSortRounds; ++r) {
    if (!in_share(r)) break;
    const uint64_t pair = base + r * 64 + lane;
    const bool active = pair < pairs;
    const uint64_t peers = same_bin(bin[r], active, bits);
    const uint32_t rank = (uint32_t)__popcll(peers & ((1ull << lane) - 1));
    uint32_t at = 0;
    if (active) at = next[wave][bin[r]] + rank;
    // every lane has read before the first of a bin's lanes moves the position on
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (active && rank == 0) next[wave][bin[r]] = at + (uint32_t)__popcll(peers);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (active) {
      const bool held = bin[r] < experts;
      row_index[at] = held ? (int64_t)(pair / topk) : -1;
      slot[pair] = held ? (int64_t)at : -1;
    }
  }
}

// out row r = x row row_index[r]; zeros for an index outside [0, tokens).
// One lane per 8-element vector.
template <bool kNT>
__global__ __launch_bounds__(kThreads) void expert_dispatch_kernel(const uint4* __restrict__ x, uint64_t tokens,
                                                                   uint32_t row_vecs,
                                                                   const int64_t* __restrict__ row_index,
                                                                   uint64_t nvec, uint4* __restrict__ out) {
  const uint64_t stride = (uint64_t)gridDim.x * kThreads;
  for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < nvec; g += stride) {
    const uint64_t r = g / row_vecs;
    const uint32_t c = (uint32_t)(g - r * row_vecs);
    const int64_t t = row_index[r];
    uint4 v = make_uint4(0, 0, 0, 0);
    if (t >= 0 && t < (int64_t)tokens) v = x[(uint64_t)t * row_vecs + c];
    store_vec<kNT>(&out[g], v);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 p = __builtin_convertvector((f32x2){a, b}, bf16x2);
  uint32_t u;
  __builtin_memcpy(&u, &p, 4);
  return u;
}

__device__ __forceinline__ void add_scaled(float (&acc)[8], const uint4& v, float w) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, bf16_lo(u[i]), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, bf16_hi(u[i]), acc[2 * i + 1]);
  }
}

__device__ __forceinline__ void add_scaled(float (&acc)[8], const uint4& lo, const uint4& hi, float w) {
  const uint32_t u[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = fmaf(w, __uint_as_float(u[i]), acc[i]);
}

// out[t] = sum over j of weights[t][j] * y[slot[t][j]] in fp32, j ascending;
// slots outside [0, rows) are left out.  One lane per 8-element vector, of y in
// bf16 or (kF32) fp32.  kNT: y in bf16 is past the last-level cache (131072 rows
// of 2048: 116 us against 125; fp32 rows, 1.07 GB of them, take 217 us without
// the hint and 230 with it).
template <bool kF32, bool kNT>
__global__ __launch_bounds__(kThreads) void expert_combine_kernel(const uint4* __restrict__ y, uint64_t rows,
                                                                  uint32_t row_vecs, const int64_t* __restrict__ slot,
                                                                  const float* __restrict__ weights, uint32_t topk,
                                                                  uint64_t nvec, uint4* __restrict__ out) {
  const uint64_t stride = (uint64_t)gridDim.x * kThreads;
  for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < nvec; g += stride) {
    const uint64_t t = g / row_vecs;
    const uint32_t c = (uint32_t)(g - t * row_vecs);
    float acc[8] = {};
#pragma unroll 8
    for (uint32_t j = 0; j < topk; ++j) {
      const int64_t s = slot[t * topk + j];
      const float w = weights ? weights[t * topk + j] : 1.f;
      if (s >= 0 && s < (int64_t)rows) {
        const uint64_t at = (uint64_t)s * row_vecs + c;
        if constexpr (kF32)
          add_scaled(acc, load_vec<kNT>(&y[2 * at]), load_vec<kNT>(&y[2 * at + 1]), w);
        else
          add_scaled(acc, load_vec<kNT>(&y[at]), w);
      }
    }
    out[g] = make_uint4(pack_bf16(acc[0], acc[1]), pack_bf16(acc[2], acc[3]), pack_bf16(acc[4], acc[5]),
                        pack_bf16(acc[6], acc[7]));
  }
}

// Rows of grad_y that no slot names become zeros.  Up to kScanPairs pairs,
// workgroups of the gradients' own launch take kScanRows rows each and look
// through all slots for their rows (192 pairs of 2048: 5.9 us a call, 10.3 with
// the two launches below; 8192 of 512: 9.0 and 11).  Past them every row's first
// vector is marked, the gradients overwrite what they name, and the rows that
// kept the mark are cleared (131072 rows of 2048, all named: 10 us, where
// clearing all of them first takes 78).  The mark is eight signalling NaNs, which
// no result can be: rounding to bf16 makes every NaN a quiet one.
constexpr uint64_t kScanPairs = 8192;
constexpr uint32_t kScanRows = 8;
constexpr uint32_t kMark = 0x7f817f81u;
constexpr uint32_t kClearRows = 16;  // rows to a wave

__global__ __launch_bounds__(kThreads) void expert_mark_kernel(uint64_t rows, uint32_t row_vecs,
                                                               uint4* __restrict__ grad_y) {
  const uint64_t stride = (uint64_t)gridDim.x * kThreads;
  for (uint64_t r = (uint64_t)blockIdx.x * kThreads + threadIdx.x; r < rows; r += stride)
    grad_y[r * row_vecs] = make_uint4(kMark, kMark, kMark, kMark);
}

__global__ __launch_bounds__(kThreads) void expert_clear_kernel(uint64_t rows, uint32_t row_vecs,
                                                                uint4* __restrict__ grad_y) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t stride = (uint64_t)gridDim.x * kSortWaves * kClearRows;
  for (uint64_t r0 = ((uint64_t)blockIdx.x * kSortWaves + (threadIdx.x >> 6)) * kClearRows; r0 < rows; r0 += stride) {
    bool marked = false;
    if (lane < kClearRows && r0 + lane < rows) {
      const uint4 v = grad_y[(r0 + lane) * row_vecs];
      marked = v.x == kMark && v.y == kMark && v.z == kMark && v.w == kMark;
    }
    for (uint64_t left = __ballot(marked); left; left &= left - 1) {
      uint4* row = grad_y + (r0 + (uint32_t)__ffsll((long long)left) - 1) * row_vecs;
      for (uint32_t c = lane; c < row_vecs; c += 64) row[c] = make_uint4(0, 0, 0, 0);
    }
  }
}

// Gradients of the weighted sum, one workgroup per token: grad_y[slot] =
// bf16(w * grad_out[t]) and grad_weights[t][j] = <grad_out[t], y[slot]> in
// fp32, summed lane by lane, then over lanes and waves in a fixed order.
// `scans` workgroups before the tokens' clear rows without a slot.  kNT: y and
// grad_y are past the last-level cache (16384 tokens, 8 rows of 2048 each: 220 us
// against 239).
template <bool kNT>
__global__ __launch_bounds__(kThreads) void expert_combine_bwd_kernel(
    const uint4* __restrict__ grad_out, const uint4* __restrict__ y, uint64_t rows, uint32_t row_vecs,
    const int64_t* __restrict__ slot, const float* __restrict__ weights, uint64_t tokens, uint32_t topk,
    uint64_t scans, uint4* __restrict__ grad_y, float* __restrict__ grad_weights) {
  __shared__ uint32_t named;  // bit r: a slot names row r of the workgroup's
  __shared__ float part[kThreads / 64][trace_host::kMaxTopk];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (uint64_t unit = blockIdx.x; unit < scans + tokens; unit += gridDim.x) {
    if (unit < scans) {
      const uint64_t r0 = unit * kScanRows;
      if (threadIdx.x == 0) named = 0;
      __syncthreads();
#pragma unroll 8
      for (uint32_t i = threadIdx.x; i < (uint32_t)tokens * topk; i += kThreads) {
        const uint64_t at = (uint64_t)slot[i] - r0;  // a negative slot, or one before r0, is past every row
        if (at < kScanRows) atomicOr(&named, 1u << at);
      }
      __syncthreads();
      for (uint32_t r = 0; r < kScanRows && r0 + r < rows; ++r) {
        if (named >> r & 1) continue;
        for (uint32_t c = threadIdx.x; c < row_vecs; c += kThreads) grad_y[(r0 + r) * row_vecs + c] = make_uint4(0, 0, 0, 0);
      }
      __syncthreads();
      continue;
    }
    const uint64_t u = unit - scans;
    for (uint32_t j = 0; j < topk; ++j) {
      const int64_t s = slot[u * topk + j];
      const float w = weights ? weights[u * topk + j] : 1.f;
      float dot = 0.f;
      if (s >= 0 && s < (int64_t)rows) {
        for (uint32_t c = threadIdx.x; c < row_vecs; c += kThreads) {
          const uint4 gv = grad_out[u * row_vecs + c], yv = load_vec<kNT>(&y[(uint64_t)s * row_vecs + c]);
          const uint32_t a[4] = {gv.x, gv.y, gv.z, gv.w}, b[4] = {yv.x, yv.y, yv.z, yv.w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = bf16_lo(a[i]), hi = bf16_hi(a[i]);
            dot = fmaf(lo, bf16_lo(b[i]), dot);
            dot = fmaf(hi, bf16_hi(b[i]), dot);
            o[i] = pack_bf16(w * lo, w * hi);
          }
          store_vec<kNT>(&grad_y[(uint64_t)s * row_vecs + c], make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) dot += __shfl_xor(dot, d);
      if (lane == 0) part[wave][j] = dot;
    }
    __syncthreads();
    if (threadIdx.x < topk) {
      float sum = 0.f;
#pragma unroll
      for (uint32_t v = 0; v < kThreads / 64; ++v) sum += part[v][threadIdx.x];
      grad_weights[u * topk + threadIdx.x] = sum;
    }
    __syncthreads();
  }
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

static unsigned rows_grid(uint64_t units, uint32_t per) {
  const uint64_t g = (units + per - 1) / per;
  return (unsigned)(g < kMaxGroups ? g : kMaxGroups);
}

// Pairs to a chunk.  The only one is cut to fit (192 pairs: 3.4 us, 6.2 uncut;
// 1600 pairs: 7.5 us, 9.0 in two chunks); then 1024 (4096 pairs: 8.5 us, 12 with
// 2048; 131072: 13.6 and 14.9) until their number tells (524288: 35 us, 23 with
// 2048).
static uint32_t sort_chunk(uint64_t pairs) {
  if (pairs <= kSortChunk) return pairs ? (uint32_t)((pairs + kThreads - 1) / kThreads) * kThreads : kThreads;
  return pairs <= 262144 ? 1024 : kSortChunk;
}

static uint64_t sort_chunks(uint64_t pairs) { return (pairs + sort_chunk(pairs) - 1) / sort_chunk(pairs); }

uint64_t expert_sort_workspace_words(uint64_t pairs, uint32_t experts) {
  const uint64_t chunks = sort_chunks(pairs);
  return chunks > 1 ? chunks * (experts + 1) : 0;
}

hipError_t launch_expert_sort(const int64_t* ids, uint64_t pairs, uint32_t topk, uint32_t experts, uint32_t* workspace,
                              int64_t* offsets, int64_t* row_index, int64_t* slot, hipStream_t stream) {
  uint32_t bits = 0;
  while ((experts >> bits) != 0) ++bits;  // bins 0..experts
  const uint32_t chunk = sort_chunk(pairs);
  const uint64_t chunks = sort_chunks(pairs);
  const dim3 grid((unsigned)(chunks > 1 ? chunks : 1)), block(kThreads);
  if (chunks <= 1) {
    hipLaunchKernelGGL(expert_place_kernel<kOnlyChunk>, grid, block, 0, stream, ids, pairs, topk, experts, bits, chunk,
                       static_cast<const uint32_t*>(nullptr), offsets, row_index, slot);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(expert_count_kernel, grid, block, 0, stream, ids, pairs, experts, chunk, workspace);
  const uint32_t* counts = workspace;
  if (chunks <= kSumChunks) {
    hipLaunchKernelGGL(expert_place_kernel<kSumCounts>, grid, block, 0, stream, ids, pairs, topk, experts, bits, chunk,
                       counts, offsets, row_index, slot);
  } else {
    hipLaunchKernelGGL(expert_scan_kernel, dim3(1), dim3(1024), 0, stream, workspace, (uint32_t)chunks, experts, offsets);
    hipLaunchKernelGGL(expert_place_kernel<kScanned>, grid, block, 0, stream, ids, pairs, topk, experts, bits, chunk,
                       counts, offsets, row_index, slot);
  }
  return hipGetLastError();
}

hipError_t launch_expert_dispatch(const uint16_t* x, uint64_t tokens, uint64_t cols, const int64_t* row_index,
                                  uint64_t rows, uint16_t* out, hipStream_t stream) {
  const uint64_t nvec = rows * (cols / 8);
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  uint4* ov = reinterpret_cast<uint4*>(out);
  if (past_cache(nvec * 16))
    hipLaunchKernelGGL(expert_dispatch_kernel<true>, dim3(rows_grid(nvec, kThreads)), dim3(kThreads), 0, stream, xv,
                       tokens, (uint32_t)(cols / 8), row_index, nvec, ov);
  else
    hipLaunchKernelGGL(expert_dispatch_kernel<false>, dim3(rows_grid(nvec, kThreads)), dim3(kThreads), 0, stream, xv,
                       tokens, (uint32_t)(cols / 8), row_index, nvec, ov);
  return hipGetLastError();
}

hipError_t launch_expert_combine(const void* y, bool f32, uint64_t rows, uint64_t cols, const int64_t* slot,
                                 const float* weights, uint64_t tokens, uint32_t topk, uint16_t* out,
                                 hipStream_t stream) {
  const uint64_t nvec = tokens * (cols / 8);
  const bool nt = past_cache(2 * rows * cols);
  const auto kernel = f32 ? expert_combine_kernel<true, false>
                          : (nt ? expert_combine_kernel<false, true> : expert_combine_kernel<false, false>);
  hipLaunchKernelGGL(kernel, dim3(rows_grid(nvec, kThreads)), dim3(kThreads), 0, stream, static_cast<const uint4*>(y),
                     rows, (uint32_t)(cols / 8), slot, weights, topk, nvec, reinterpret_cast<uint4*>(out));
  return hipGetLastError();
}

hipError_t launch_expert_combine_bwd(const uint16_t* grad_out, const uint16_t* y, uint64_t rows, uint64_t cols,
                                     const int64_t* slot, const float* weights, uint64_t tokens, uint32_t topk,
                                     bool clear, uint16_t* grad_y, float* grad_weights, hipStream_t stream) {
  const uint32_t row_vecs = (uint32_t)(cols / 8);
  uint4* gv = reinterpret_cast<uint4*>(grad_y);
  clear = clear && rows > 0 && row_vecs > 0;
  const bool scan = clear && tokens * topk <= kScanPairs;
  const uint64_t scans = scan ? (rows + kScanRows - 1) / kScanRows : 0;
  if (clear && !scan)
    hipLaunchKernelGGL(expert_mark_kernel, dim3(rows_grid(rows, kThreads)), dim3(kThreads), 0, stream, rows, row_vecs, gv);
  const auto kernel = past_cache(2 * rows * cols) ? expert_combine_bwd_kernel<true> : expert_combine_bwd_kernel<false>;
  if (tokens + scans > 0)
    hipLaunchKernelGGL(kernel, dim3(rows_grid(tokens + scans, 1)), dim3(kThreads), 0, stream,
                       reinterpret_cast<const uint4*>(grad_out), reinterpret_cast<const uint4*>(y), rows, row_vecs, slot,
                       weights, tokens, topk, scans, gv, grad_weights);
  if (clear && !scan)
    hipLaunchKernelGGL(expert_clear_kernel, dim3(rows_grid(rows, kSortWaves * kClearRows)), dim3(kThreads), 0, stream,
                       rows, row_vecs, gv);
  return hipGetLastError();
}

}  // namespace trace_host
