// libtrace quantiser for gfx950: bf16 activations or weights to the operands
// of the microscaled products (mx_product.hip) in one pass -- MXFP4 or MXFP8
// codes, one E8M0 scale byte per 32-element block, and, for the
// straight-through backward, the clip mask.  Scales and codes are those of
// mx_capture and mx8_capture, the mask that of the RNE fake-quant forwards.
//
// One lane per 8-element vector (a quarter block: one 128-bit load); the four
// lanes of a block agree on its largest magnitude by two DPP moves.  Dividing
// by a power of two is a multiplication by its exact inverse.  The kernel is
// bound by memory: 2 bytes in, 0.53 (MXFP4) or 1.03 (MXFP8) out per element
// (16384 x 4096 to MXFP8: 32 us, 6.5 TB/s, part of it from the last-level cache).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_math.h"
#include "fp4_block.h"
#include "launch.h"
#include "launch_mx.h"
#include "mx_quantize_dev.h"

namespace trace_dev {

template <int kFmt, bool kNT>
__global__ __launch_bounds__(kThreads) void mx_quantize_kernel(const uint4* __restrict__ x, uint64_t nvec,
                                                               uint8_t* __restrict__ scales,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ mask,
                                                               const int64_t* __restrict__ used, uint32_t row_vecs) {
  if (used) {  // rows from *used on are left out
    const int64_t n = *used;
    nvec = n <= 0 ? 0 : ((uint64_t)n >= nvec / row_vecs ? nvec : (uint64_t)n * row_vecs);
  }
  const uint64_t stride = (uint64_t)gridDim.x * kThreads;
  for (uint64_t g = (uint64_t)blockIdx.x * kThreads + threadIdx.x; g < nvec; g += stride) {
    const uint4 v = load_vec<kNT>(&x[g]);  // nvec is a multiple of 4: a block's four lanes are active together
    uint32_t sb, keep;
    const uint2 c = quantize_vector<kFmt == trace_host::kE2M1>(v, sb, keep);
    if ((g & 3) == 0) scales[g >> 2] = (uint8_t)sb;
    if (kFmt == trace_host::kE2M1)
      store_word<kNT>(reinterpret_cast<uint32_t*>(codes) + g, c.x);
    else
      store_pair<kNT>(reinterpret_cast<uint2*>(codes) + g, c);
    if (mask) store_word<kNT>(&mask[g], (uint8_t)keep);
  }
}

}  // namespace trace_dev

namespace trace_host {

using namespace trace_dev;

hipError_t launch_mx_quantize(MxFormat fmt, const uint16_t* x, uint64_t nblocks, uint8_t* scales, uint8_t* codes,
                              uint8_t* mask, const int64_t* used, uint32_t row_blocks, hipStream_t stream) {
  if (nblocks == 0) return hipSuccess;  // an empty grid is not a valid launch
  const uint64_t nvec = 4 * nblocks;
  const uint64_t need = (nvec + kThreads - 1) / kThreads;
  const dim3 grid((unsigned)(need < kMaxGroups ? need : kMaxGroups)), block(kThreads);
  const uint4* xv = reinterpret_cast<const uint4*>(x);
  const bool nt = past_cache(nblocks * 64);
  if (fmt == kE2M1 && nt)
    hipLaunchKernelGGL((mx_quantize_kernel<kE2M1, true>), grid, block, 0, stream, xv, nvec, scales, codes, mask,
                       used, 4 * row_blocks);
  else if (fmt == kE2M1)
    hipLaunchKernelGGL((mx_quantize_kernel<kE2M1, false>), grid, block, 0, stream, xv, nvec, scales, codes, mask,
                       used, 4 * row_blocks);
  else if (nt)
    hipLaunchKernelGGL((mx_quantize_kernel<kE4M3, true>), grid, block, 0, stream, xv, nvec, scales, codes, mask,
                       used, 4 * row_blocks);
  else
    hipLaunchKernelGGL((mx_quantize_kernel<kE4M3, false>), grid, block, 0, stream, xv, nvec, scales, codes, mask,
                       used, 4 * row_blocks);
  return hipGetLastError();
}

}  // namespace trace_host
