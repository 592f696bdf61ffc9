// moe_dropout: kept elements scaled, the others 0, the mask computed from a
// counter and never stored.
//
// HBM-bound: 2 bytes in and 2 out an element; the generator's 128 bits serve
// the 8 elements of a thread's 16-byte load. 32768 x 2880: 62 to 65 us, 5.8 to 6.1
// TB/s (64 to 68 us with stores through the caches); 64 x 256: 2.6 us.
#include "dropout_util.h"
#include "params.h"

namespace moe {

constexpr int kDropThreads = 256;
constexpr int64_t kDropMaxBlocks = 65536;  // a grid-stride loop does the rest

__global__ __launch_bounds__(kDropThreads) void dropout_kernel(const uint16_t* x, int64_t x_ld, int64_t pieces,
                                                               int32_t row_pieces, Dropout d, uint16_t* y,
                                                               int64_t y_ld) {
  const uint64_t seed = d.threshold ? d.rng[0] : 0, offset = d.threshold ? d.rng[1] : 0;
  for (int64_t i = (int64_t)blockIdx.x * kDropThreads + threadIdx.x; i < pieces;
       i += (int64_t)gridDim.x * kDropThreads) {
    const int64_t row = i / row_pieces;
    const int64_t col = (i - row * row_pieces) * 8;
    float f[8];
    unpack8(*reinterpret_cast<const u32x4_t*>(x + row * x_ld + col), f);
    drop8(d, seed, offset, (uint64_t)i, f);
    __builtin_nontemporal_store(pack8(f), reinterpret_cast<u32x4_t*>(y + row * y_ld + col));
  }
}

hipError_t launch_dropout(const uint16_t* x, int64_t x_ld, int64_t rows, int64_t n, float p, const uint64_t* rng,
                          uint16_t* y, int64_t y_ld, hipStream_t stream) {
  const int64_t pieces = rows * (n / 8);
  if (pieces == 0) return hipSuccess;
  const int64_t want = (pieces + kDropThreads - 1) / kDropThreads;
  hipLaunchKernelGGL(dropout_kernel, dim3((uint32_t)(want < kDropMaxBlocks ? want : kDropMaxBlocks)),
                     dim3(kDropThreads), 0, stream, x, x_ld, pieces, (int32_t)(n / 8), make_dropout(p, rng), y, y_ld);
  return hipGetLastError();
}

}  // namespace moe
