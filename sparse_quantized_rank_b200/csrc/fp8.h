// Block-scaled FP8 matrices: memory layout, and the launch entry points
// shared by the host ABI (fp8.cu) and the product kernels (fp8_decode.cu,
// fp8_gemm.cu).
#pragma once
#include "kernels.h"

namespace cql {

// [rows][cols] values: codes [blocks][rows][128], then scales [quads][rows][4 bytes].
struct Fp8Shape {
  int64_t rows;
  int cols, blocks, quads;                   // blocks = ceil(cols / 128), quads = ceil(blocks / 4)
  uint64_t codes_len, scales_off, scales_len, total;
};
inline Fp8Shape fp8_shape(int64_t rows, int cols) {
  Fp8Shape s;
  s.rows = rows;
  s.cols = cols;
  s.blocks = (cols + kGroup - 1) / kGroup;
  s.quads = (s.blocks + 3) / 4;
  s.codes_len = (uint64_t)rows * s.blocks * kGroup;
  s.scales_off = align256(s.codes_len);
  s.scales_len = (uint64_t)rows * s.quads * 4;
  s.total = s.scales_off + align256(s.scales_len);
  return s;
}

// dst = the block-scaled form of src [rows][ld].  In a forward the kernel is
// launched programmatically dependent on the one before it and lets the product
// kernel start: at once, or (where that reads offsets) when those before are done.
// err: where the checked build records an index out of range, or null.
enum Fp8Launch { kFp8Plain = 0, kFp8Early = 1, kFp8Offsets = 2 };
cudaError_t launch_fp8_quantize(const Fp8Shape& s, const void* src, int dt, int64_t ld, uint8_t* dst, Fp8Launch pdl,
                                uint32_t* err, cudaStream_t st);
cudaError_t launch_fp8_dequantize(const Fp8Shape& s, const uint8_t* src, void* out, int dt, int64_t ld,
                                  cudaStream_t st);

// y[t][n] = sum_k X[t][k] W[e N + n][k] for the tokens t of expert e.
struct Fp8Product {
  Fp8Shape w, x;                             // W: experts * n rows; X: tokens rows
  const uint8_t* w_base;
  const uint8_t* x_base;                     // the block-scaled X, or null: it is quantised from `raw`
  const void* raw;                           // [tokens][ldx] of xdt
  int xdt;
  int64_t ldx;
  int n, experts;
  bool early;                                // weights (and offsets) may be read before the kernel before is done
  const int32_t* offsets;                    // [experts + 1] on the device, or null: one expert, every token
  void* y;
  int ydt;
  int64_t ldy;
  uint32_t* status;
  bool debug;                                // x is withheld, the waits for it run out after ~10 ms
};
// Elements from a matrix's first to behind its last, rows ld apart.
CQL_HD uint64_t fp8_extent(int64_t rows, int64_t ld, int cols) { return (uint64_t)((rows - 1) * ld + cols); }
// Few tokens an expert (fp8_decode.cu).  With very few, X is quantised on the
// way, from `raw`; else it is block-scaled already.
bool fp8_decodes(int tokens, int experts, int64_t weights);           // weights: n_out * k_in of an expert
bool fp8_decode_quantizes(int tokens, int experts);
cudaError_t ready_fp8_decode();               // what the launch asks of the runtime succeeds
cudaError_t launch_fp8_decode(const Fp8Product& p, cudaStream_t st);
// Any number, X block-scaled (fp8_gemm.cu).
cudaError_t ready_fp8_gemm();
cudaError_t launch_fp8_gemm(const Fp8Product& p, cudaStream_t st);

}  // namespace cql
