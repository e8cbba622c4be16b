// Sizes and launchers of latent attention (internal to libbfp8; arguments are validated by the C-ABI
// layer before any launcher is called).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bfp8 {

constexpr int kLatentDim = 512;                            // latents of a token
constexpr int kRopeDim = 64;                               // its rotary key
constexpr int kLatentRow = kLatentDim + 2 * kRopeDim;      // bytes of a cache row
constexpr uint32_t kLatentMinCode = 127 - 42, kLatentMaxCode = 127 + 40;  // scale codes the writer makes

// A paged cache and (for readers) its page table.
struct LatentCache {
  const uint8_t* rows;    // row r of page p at p * page_stride + r * kLatentRow
  const uint8_t* scales;  // its scale code at p * scale_stride + r
  int64_t page_stride, scale_stride;
  int pages, page_size;
  const int32_t* table;  // [B][table_stride] pages of a sequence in order, the first table_width entries
  int64_t table_stride;
  int table_width;
};

hipError_t launch_latent_write(const uint16_t* kv, int64_t T, int64_t ld_kv, const uint16_t* w, float eps,
                               const int64_t* slots, const LatentCache& cache, uint8_t* rows, uint8_t* scales,
                               hipStream_t stream);
hipError_t launch_latent_read(const LatentCache& cache, const int32_t* cu, int64_t B, int64_t T, uint16_t* out,
                              int64_t ld_out, hipStream_t stream);
hipError_t launch_latent_gather(const LatentCache& cache, const int32_t* cu, int64_t B, int64_t T, uint8_t* q,
                                int64_t ldq, uint8_t* e, int64_t ld_e, uint16_t* rope, int64_t ld_rope,
                                hipStream_t stream);

}  // namespace bfp8
