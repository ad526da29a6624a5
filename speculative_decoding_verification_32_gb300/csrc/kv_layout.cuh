// kv_layout.cuh -- the KV cache's number formats, shared by the kernels that
// write it, read it back and attend over it.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "specverify.h"

namespace sv {

template <int CT>
struct CacheType;
template <>
struct CacheType<SPEC_BF16> {
  using type = __nv_bfloat16;
};
template <>
struct CacheType<SPEC_F16> {
  using type = __half;
};

// Scale byte of a head vector whose largest magnitude has the fp32 bits `a`:
// the smallest c >= 1 with a / 2^(c - 127) <= 448 = 1.75 * 2^8; 255 if `a` is
// not finite.  Bits compare like the magnitudes they stand for.
__device__ __forceinline__ uint32_t e4m3_scale_byte(uint32_t a) {
  if (a >= 0x7f800000u) return 255u;
  const int c = static_cast<int>(a >> 23) - 8 + ((a & 0x7fffffu) > 0x600000u);
  return static_cast<uint32_t>(c < 1 ? 1 : c);
}

// The scale 2^(c - 127) a byte stands for.
__device__ __forceinline__ float e4m3_scale(uint32_t c) {
  if (c == 255u) return __uint_as_float(0x7fc00000u);
  return __uint_as_float(c ? c << 23 : 0x00400000u);
}

}  // namespace sv
