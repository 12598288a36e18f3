// Kernels behind the paged attention call (internal to the library).
#pragma once

#include "dims.h"
#include "paged.h"

namespace cobs {

struct PagedArgs;

// float32 on the CUDA cores, chunks: rows of a record, blocks launched.
int paged_simt_rec_rows(const PagedDims& m);
int paged_simt_workers(const PagedDims& m);
cudaError_t launch_paged_simt(const PagedDims& m, const PagedArgs& a, const float* Q, const float* kc,
                              const float* vc, cudaStream_t s);

// bf16 on the tensor cores, chunks.
int paged_chunk_rec_rows(const PagedDims& m);
int paged_chunk_workers(const PagedDims& m);
cudaError_t launch_paged_chunk(const PagedDims& m, const PagedArgs& a, const void* Q, const void* kc, const void* vc,
                               cudaStream_t s);

// One new token per request.
int paged_decode_rec_rows(const PagedDims& m);
int paged_decode_workers(const PagedDims& m);
cudaError_t launch_paged_decode(const PagedDims& m, const PagedArgs& a, const void* Q, const void* kc, const void* vc,
                                cudaStream_t s);
cudaError_t launch_paged_decode_f32(const PagedDims& m, const PagedArgs& a, const float* Q, const float* kc, const float* vc,
                                    cudaStream_t s);

}  // namespace cobs
