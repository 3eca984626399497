// fa_host.h -- host-side helpers shared by the library's translation units
// (forward entry points in fa_fwd.cu, backward in fa_bwd.cu, decoding in
// fa_decode.cu, the paged caches in fa_cache.cu and fa_cache4.cu, page tables in
// fa_pages.cu, rotary positions in fa_rope.cu).  Internal: not
// part of the C ABI (the library is built with hidden visibility).
#pragma once

#include <cuda.h>

#include <cstddef>
#include <cstdint>

#include "fa.h"

namespace fa_host {

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

constexpr int kMaxDevices = 64;

inline bool overlaps(uintptr_t a, size_t na, uintptr_t b, size_t nb) { return a < b + nb && b < a + na; }

// The current device's TMA encoder and SM count (initialised once per device;
// fails with FA_ERR_UNSUPPORTED on anything but sm_103).
fa_status_t encoder(EncodeTiledFn *fn, int *num_sms);

// 3-D view [BH, N, d] of a contiguous [B, H, N, d] 16-bit tensor; box = 64
// columns x 128 rows x 1 head, SWIZZLE_128B, rows past N read as zeros (and
// are not written by stores).
fa_status_t encode_qkv_map(EncodeTiledFn encode, CUtensorMap *map, const void *ptr, int BH, int N,
                           int d, fa_dtype_t dtype);

// Argument checks shared by the forward entry points (no CUDA calls).  Sets
// *empty for a problem with nothing to compute.
fa_status_t check_args(const void *q, const void *k, const void *v, const void *o, const float *lse,
                       int B, int H, int N, int d, float scale, int causal, fa_dtype_t dtype,
                       bool *empty);

// Addresses of the backward / decoding / cache / pages units' status words on the
// current device (bit 0: a bounded wait expired; bit 2: an index outside its range;
// 0 when nothing was recorded); NULL if there is none to be had.
unsigned int *bwd_status_word();
unsigned int *decode_status_word();
unsigned int *cache_status_word();
unsigned int *cache4_status_word();
unsigned int *pages_status_word();

}  // namespace fa_host
