// host_common.h -- host-side helpers that the translation units of the
// library share (defined in api.cu): per-device set-up, tensor-map encoding,
// error mapping.  Not part of the C ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace ajvp {
namespace host {

constexpr int kMaxDevices = 64;

int fail(cudaError_t e);          // remembers e for attn_jvp_last_cuda_error, returns AJVP_ERR_CUDA
int device(int *dev);             // checks the current device and sets the kernels up on it
int sm_count(int dev);            // of a device that device() accepted
int encoder();                    // resolves cuTensorMapEncodeTiled
uint64_t wait_bound_ns();
// [BH][L][d] bf16 tensor, boxes of 64 columns x box_rows rows, 128-byte swizzle
int encode(CUtensorMap *m, const void *ptr, int64_t d, int64_t L, int64_t BH, uint32_t box_rows);
// [rows][128] bytes, boxes of 128 columns x box_rows rows, 128-byte swizzle
int encode_codes(CUtensorMap *m, const void *ptr, int64_t rows, uint32_t box_rows);
uint64_t stats_bytes(int64_t BH, int64_t Lq);
uint64_t partial_bytes(int64_t BH, int64_t Lk, int64_t parts);

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// device status words of the other translation units (each holds its own):
// read into *word (ORed), cleared when set
cudaError_t scored_status(int *word);
cudaError_t cache_status(int *word);
// a bounded wait in them that runs out and sets that word (scored: the sleeping form)
cudaError_t scored_selftest(uint64_t bound_ns, cudaStream_t stream);
cudaError_t cache_selftest(uint64_t bound_ns, cudaStream_t stream);

}  // namespace host
}  // namespace ajvp
