// Block-scaled FP8 (e4m3) matrices: quantising, reading back, and the host
// ABI of the FP8 linear layers (include/cql.h, "BLOCK-SCALED FP8").
//
// A block is 128 consecutive columns of one row.  Its scale is the smallest
// power of two 2^e with max|v| <= 448 * 2^e (e at least -126), so v / 2^e is
// an exact exponent shift, the rounding to e4m3 is the only one, and the
// scale byte e + 127 is what the block-scaled tensor-core product reads.
#include <string.h>

#include "fp8.cuh"

namespace cql {
namespace {

constexpr int Q_WARPS = 8;

CQL_DEV float load_as_f32(const void* p, int dt, int64_t i) {
  if (dt == CQL_DT_F32) return reinterpret_cast<const float*>(p)[i];
  return to_f32_act(p, dt, (uint64_t)i);
}

// How a warp takes the four blocks (512 columns) of a row's quad, so that every
// access of it is to consecutive addresses.  A pass covers 32 * PER columns:
//   VEC, fp32    4 passes of a block, a lane 4 columns (16 bytes)
//   VEC, 16-bit  2 passes of two blocks, a lane 8 columns (16 bytes)
//   else         4 passes of a block, a lane columns lane, lane + 32, + 64, + 96
template <int DT, bool VEC>
struct Pass {
  static constexpr int PER = VEC && DT != CQL_DT_F32 ? 8 : 4;        // columns a lane
  static constexpr int N = 16 / PER;                                 // passes a quad
  // first column within the quad, and distance to the lane's next one
  CQL_DEV static int col(int pass, int lane) { return pass * 32 * PER + (VEC ? PER * lane : lane); }
  static constexpr int STEP = VEC ? 1 : 32;
};

// Bound by memory: reads the source once and writes 1 + 1/128 bytes a value.  A
// warp has a row's quad to itself, so that the block's largest magnitude is a
// reduction inside it, the source is read in one go and the four scale bytes are
// one store.  11008 x 4096 in fp32, quantised and read back (451 MB): 75 us,
// 92 % of the measured copy bandwidth; with 16 columns a lane, whose stores lie
// 16 bytes apart within a block, it took 93 us.
template <int DT, bool VEC>
__global__ void __launch_bounds__(Q_WARPS * 32) k_fp8_quantize(Fp8Shape s, const void* src, int64_t ld, uint8_t* dst,
                                                               int pdl, uint32_t* err) {
  [[maybe_unused]] const uint64_t in_src = fp8_extent(s.rows, ld, s.cols);       // checked build
  using P = Pass<DT, VEC>;
  // The product kernel may start on its weights at once; where it reads offsets
  // too (kFp8Offsets), when the kernels before, which may have written them, are done.
  if (pdl == kFp8Early) pdl_launch_dependents();
  if (pdl != kFp8Plain) pdl_wait();
  if (pdl == kFp8Offsets) pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * Q_WARPS + (threadIdx.x >> 5);
  const int quad = blockIdx.y;
  if (blockIdx.x == 0 && quad == 0) {             // the padding behind the two planes
    for (uint64_t i = s.codes_len + threadIdx.x; i < s.scales_off; i += blockDim.x) dst[i] = 0;
    for (uint64_t i = s.scales_off + s.scales_len + threadIdx.x; i < s.total; i += blockDim.x) dst[i] = 0;
  }
  if (row >= s.rows) return;
  float v[P::N][P::PER];
#pragma unroll
  for (int i = 0; i < P::N; ++i) {
    const int c = quad * 4 * kGroup + P::col(i, lane);
    const int64_t at = row * ld + c;
    if (VEC && c + P::PER <= s.cols && CQL_IN(err, at + P::PER - 1, in_src, 402)) {
      if constexpr (DT == CQL_DT_F32) {
        const float4 f = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(src) + at);
        v[i][0] = f.x;
        v[i][1] = f.y;
        v[i][2] = f.z;
        v[i][3] = f.w;
      } else if constexpr (VEC) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(src) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][2 * j] = DT == CQL_DT_BF16 ? bf16_bits_to_f32(w[j] & 0xFFFFu) : f16_bits_to_f32(w[j] & 0xFFFFu);
          v[i][2 * j + 1] = DT == CQL_DT_BF16 ? bf16_bits_to_f32(w[j] >> 16) : f16_bits_to_f32(w[j] >> 16);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < P::PER; ++j)
        v[i][j] = c + j * P::STEP < s.cols && CQL_IN(err, at + j * P::STEP, in_src, 402)
                      ? load_as_f32(src, DT, at + j * P::STEP)
                      : 0.0f;
    }
  }
  // magnitudes compare as integers, infinities and NaNs above every finite one
  uint32_t top[P::N];
#pragma unroll
  for (int i = 0; i < P::N; ++i) {
    top[i] = 0;
#pragma unroll
    for (int j = 0; j < P::PER; ++j) top[i] = max(top[i], __float_as_uint(v[i][j]) & 0x7FFFFFFFu);
  }
  if (P::N == 4) {
#pragma unroll
    for (int i = 0; i < P::N; ++i) top[i] = __reduce_max_sync(0xffffffffu, top[i]);
  } else {
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < P::N; ++i) top[i] = max(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    }
  }
  uint32_t word = 0;                              // the quad's scale bytes
#pragma unroll
  for (int i = 0; i < P::N; ++i) {
    const uint32_t amax = top[i];
    const int sub = P::N == 4 ? i : 2 * i + (lane >> 4);             // block of the quad
    const int blk = 4 * quad + sub;
    const bool bad = amax >= 0x7F800000u;
    const uint32_t byte = bad ? kFp8ScaleNaN : fp8_scale_byte(amax);
    const float inv = __uint_as_float((254u - (bad ? 127u : byte)) << 23);   // 2^-e
    if (blk < s.blocks) {
      word |= byte << (8 * sub);
      const int64_t code = ((int64_t)blk * s.rows + row) * kGroup + (P::col(i, lane) & (kGroup - 1));
      if (!CQL_IN(err, code + (VEC ? P::PER - 1 : 96), s.codes_len, 403)) continue;
      uint8_t* to = dst + code;
      uint32_t w[P::PER / 4];
#pragma unroll
      for (int j = 0; j < P::PER / 4; ++j)
        w[j] = bad ? 0x7F7F7F7Fu
                   : e4m3_pair(v[i][4 * j] * inv, v[i][4 * j + 1] * inv) |
                         (e4m3_pair(v[i][4 * j + 2] * inv, v[i][4 * j + 3] * inv) << 16);
      if constexpr (!VEC) {
#pragma unroll
        for (int j = 0; j < 4; ++j) to[32 * j] = (uint8_t)(w[0] >> (8 * j));
      } else if constexpr (P::PER == 8) {
        *reinterpret_cast<uint2*>(to) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t*>(to) = w[0];
      }
    }
  }
  if (P::N == 2) word |= __shfl_xor_sync(0xffffffffu, word, 16);
  const int64_t scale = ((int64_t)quad * s.rows + row) * 4;
  if (lane == 0 && CQL_IN(err, scale + 3, s.scales_len, 404))
    *reinterpret_cast<uint32_t*>(dst + s.scales_off + scale) = word;
  // A forward that follows directly may read this matrix as its weight before its
  // own wait.  Its CTAs start when all of this kernel's have ended, each behind
  // these fences: every byte is in L2 by then.  It reads codes (through the async
  // proxy) and weight scales there, past L1, which it must not trust before the wait.
  if (pdl == kFp8Plain) {
    asm volatile("fence.proxy.async.global;" ::: "memory");
    __threadfence();
  }
}

// The same passes, the other way round.  e4m3 to fp16 and the power-of-two scale
// in fp32 are exact; a 16-bit output is rounded once, from that.
template <int DT, bool VEC>
__global__ void __launch_bounds__(Q_WARPS * 32) k_fp8_dequantize(Fp8Shape s, const uint8_t* src, void* out, int64_t ld) {
  using P = Pass<DT, VEC>;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * Q_WARPS + (threadIdx.x >> 5);
  const int quad = blockIdx.y;
  if (row >= s.rows) return;
  [[maybe_unused]] uint32_t* const err = nullptr; // the checked build skips, and has no word to record in
  [[maybe_unused]] const uint64_t in_out = fp8_extent(s.rows, ld, s.cols);
  const int64_t from_scale = ((int64_t)quad * s.rows + row) * 4;
  const uint32_t word = CQL_IN(err, from_scale + 3, s.scales_len, 405)
                            ? *reinterpret_cast<const uint32_t*>(src + s.scales_off + from_scale)
                            : 0u;
  uint32_t w[P::N][P::PER / 4];
#pragma unroll
  for (int i = 0; i < P::N; ++i) {
    const int blk = 4 * quad + (P::N == 4 ? i : 2 * i + (lane >> 4));
    const int64_t code = ((int64_t)blk * s.rows + row) * kGroup + (P::col(i, lane) & (kGroup - 1));
    const uint8_t* from = src + code;
    if (blk >= s.blocks || !CQL_IN(err, code + (VEC ? P::PER - 1 : 96), s.codes_len, 406)) {
#pragma unroll
      for (int j = 0; j < P::PER / 4; ++j) w[i][j] = 0u;
    } else if constexpr (!VEC) {
      w[i][0] = from[0] | ((uint32_t)from[32] << 8) | ((uint32_t)from[64] << 16) | ((uint32_t)from[96] << 24);
    } else if constexpr (P::PER == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(from);
      w[i][0] = u.x;
      w[i][1] = u.y;
    } else {
      w[i][0] = *reinterpret_cast<const uint32_t*>(from);
    }
  }
#pragma unroll
  for (int i = 0; i < P::N; ++i) {
    const uint32_t byte = (word >> (8 * (P::N == 4 ? i : 2 * i + (lane >> 4)))) & 0xFFu;
    // 2^(byte - 127); byte 0 is 2^-127, a subnormal
    const float scale = byte == kFp8ScaleNaN ? __uint_as_float(0x7FC00000u)
                                             : __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
    float v[P::PER];
#pragma unroll
    for (int j = 0; j < P::PER / 2; ++j) {
      uint32_t h;
      const uint16_t two = (uint16_t)(w[i][j >> 1] >> (16 * (j & 1)));
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(two));
      v[2 * j] = f16_bits_to_f32(h & 0xFFFFu) * scale;
      v[2 * j + 1] = f16_bits_to_f32(h >> 16) * scale;
    }
    const int c = quad * 4 * kGroup + P::col(i, lane);
    const int64_t at = row * ld + c;
    if (VEC && c + P::PER <= s.cols && CQL_IN(err, at + P::PER - 1, in_out, 407)) {
      if constexpr (DT == CQL_DT_F32) {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(out) + at) = make_float4(v[0], v[1], v[2], v[3]);
      } else if constexpr (VEC) {
        *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(out) + at) =
            make_uint4(pack16(v[0], v[1], DT), pack16(v[2], v[3], DT), pack16(v[4], v[5], DT), pack16(v[6], v[7], DT));
      }
    } else {
#pragma unroll
      for (int j = 0; j < P::PER; ++j)
        if (c + j * P::STEP < s.cols && CQL_IN(err, at + j * P::STEP, in_out, 407)) store_out(out, DT, (uint64_t)(at + j * P::STEP), v[j]);
    }
  }
}

int esize(int dt) { return dt == CQL_DT_F32 ? 4 : 2; }
bool aligned_to(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool vectors_ok(const void* p, int dt, int64_t ld) { return aligned_to(p, 16) && (ld * esize(dt)) % 16 == 0; }

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8Shape& s, const void* src, int dt, int64_t ld, uint8_t* dst, Fp8Launch pdl,
                                uint32_t* err, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((s.rows + Q_WARPS - 1) / Q_WARPS), (unsigned)s.quads);
  cfg.blockDim = dim3(Q_WARPS * 32);
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = pdl != kFp8Plain ? 1 : 0;
  const bool vec = vectors_ok(src, dt, ld);
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, s, src, ld, dst, (int)pdl, err); };
  if (dt == CQL_DT_F32) return vec ? go(k_fp8_quantize<CQL_DT_F32, true>) : go(k_fp8_quantize<CQL_DT_F32, false>);
  if (dt == CQL_DT_F16) return vec ? go(k_fp8_quantize<CQL_DT_F16, true>) : go(k_fp8_quantize<CQL_DT_F16, false>);
  return vec ? go(k_fp8_quantize<CQL_DT_BF16, true>) : go(k_fp8_quantize<CQL_DT_BF16, false>);
}

cudaError_t launch_fp8_dequantize(const Fp8Shape& s, const uint8_t* src, void* out, int dt, int64_t ld,
                                  cudaStream_t st) {
  const dim3 grid((unsigned)((s.rows + Q_WARPS - 1) / Q_WARPS), (unsigned)s.quads);
  const bool vec = vectors_ok(out, dt, ld);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(Q_WARPS * 32);
  cfg.stream = st;
  auto go = [&](auto kernel) { return cudaLaunchKernelEx(&cfg, kernel, s, src, out, ld); };
  if (dt == CQL_DT_F32) return vec ? go(k_fp8_dequantize<CQL_DT_F32, true>) : go(k_fp8_dequantize<CQL_DT_F32, false>);
  if (dt == CQL_DT_F16) return vec ? go(k_fp8_dequantize<CQL_DT_F16, true>) : go(k_fp8_dequantize<CQL_DT_F16, false>);
  return vec ? go(k_fp8_dequantize<CQL_DT_BF16, true>) : go(k_fp8_dequantize<CQL_DT_BF16, false>);
}

}  // namespace cql

// ---------------------------------------------------------------------------
// host ABI
// ---------------------------------------------------------------------------
using namespace cql;

namespace {

bool shape_ok(int64_t rows, int32_t cols) {
  return rows >= 0 && rows <= (int64_t)CQL_FP8_MAX_ROWS && cols >= 1 && cols <= CQL_FP8_MAX_COLS;
}
bool plain_dt(int dt) { return dt == CQL_DT_F32 || dt == CQL_DT_F16 || dt == CQL_DT_BF16; }
cql_status of_cuda(cudaError_t e) { return e == cudaSuccess ? CQL_OK : CQL_ERR_CUDA; }

cql_status forward(int32_t n_out, int32_t k_in, int32_t experts, const void* weight, const void* x, cql_dtype x_dt,
                   int64_t ldx, const int32_t* offsets, void* y, cql_dtype y_dt, int64_t ldy, int32_t tokens,
                   void* workspace, uint64_t ws_bytes, uint32_t* status, cql_stream_t stream) {
  if (n_out < 1 || n_out > CQL_FP8_MAX_OUT || k_in < 1 || k_in > CQL_FP8_MAX_COLS) return CQL_ERR_ARG;
  if (experts < 1 || experts > CQL_FP8_MAX_EXPERTS || (int64_t)experts * n_out > (int64_t)CQL_FP8_MAX_ROWS)
    return CQL_ERR_ARG;
  if (tokens < 0 || tokens > CQL_FP8_MAX_TOKENS) return CQL_ERR_ARG;
  const bool debug = ((uint32_t)x_dt & CQL_FLAG_DEBUG_SKIP_X) != 0;
  x_dt = (cql_dtype)((uint32_t)x_dt & ~CQL_FLAG_DEBUG_SKIP_X);
  const bool kept = x_dt == CQL_DT_FP8_BLOCK;
  if (!kept && !plain_dt(x_dt)) return CQL_ERR_ARG;
  if (!plain_dt(y_dt)) return CQL_ERR_ARG;
  if (kept ? ldx != 0 : ldx < k_in) return CQL_ERR_ARG;
  if (ldy < n_out) return CQL_ERR_ARG;
  if (weight == nullptr || status == nullptr) return CQL_ERR_ARG;
  if (!aligned_to(weight, 256) || !aligned_to(status, 8)) return CQL_ERR_ALIGN;
  if (tokens == 0) return CQL_OK;
  if (x == nullptr || y == nullptr) return CQL_ERR_ARG;
  if (!aligned_to(x, kept ? 256 : esize(x_dt)) || !aligned_to(y, esize(y_dt))) return CQL_ERR_ALIGN;
  Fp8Product p{};
  p.w = fp8_shape((int64_t)experts * n_out, k_in);
  p.x = fp8_shape(tokens, k_in);
  p.w_base = static_cast<const uint8_t*>(weight);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool few = fp8_decodes(tokens, experts, (int64_t)n_out * k_in);
  if (kept) {
    p.x_base = static_cast<const uint8_t*>(x);
  } else {
    if (fp8_decode_quantizes(tokens, experts)) {
      p.raw = x;
      p.xdt = (int)x_dt;
      p.ldx = ldx;
    } else {
      if (workspace == nullptr) return CQL_ERR_ARG;
      if (!aligned_to(workspace, 256)) return CQL_ERR_ALIGN;
      if (ws_bytes < p.x.total) return CQL_ERR_SIZE;
      cudaError_t e = few ? ready_fp8_decode() : ready_fp8_gemm();    // before anything is launched
      if (e != cudaSuccess) return CQL_ERR_CUDA;
      e = launch_fp8_quantize(p.x, x, x_dt, ldx, static_cast<uint8_t*>(workspace),
                                                offsets == nullptr ? kFp8Early : kFp8Offsets, status, st);
      if (e != cudaSuccess) return CQL_ERR_CUDA;
      p.x_base = static_cast<const uint8_t*>(workspace);
    }
  }
  p.early = offsets == nullptr || (!kept && p.raw == nullptr);
  p.n = n_out;
  p.experts = experts;
  p.offsets = offsets;
  p.y = y;
  p.ydt = (int)y_dt;
  p.ldy = ldy;
  p.status = status;
  p.debug = debug;
  // an x that is quantised on the way is one of fp8_decodes' too
  return of_cuda(few ? launch_fp8_decode(p, st) : launch_fp8_gemm(p, st));
}

}  // namespace

extern "C" {

cql_status cql_fp8_matrix_layout(int64_t rows, int32_t cols, cql_fp8_layout* out) {
  if (out == nullptr || !shape_ok(rows, cols)) return CQL_ERR_ARG;
  const Fp8Shape s = fp8_shape(rows, cols);
  out->total_bytes = s.total;
  out->codes_off = 0;
  out->codes_len = s.codes_len;
  out->scales_off = s.scales_off;
  out->scales_len = s.scales_len;
  return CQL_OK;
}

cql_status cql_fp8_quantize(const void* src, cql_dtype dt, int64_t rows, int32_t cols, int64_t ld, void* matrix,
                            uint64_t matrix_bytes, cql_stream_t stream) {
  if (!shape_ok(rows, cols) || !plain_dt(dt) || ld < cols) return CQL_ERR_ARG;
  if (rows == 0) return CQL_OK;
  if (src == nullptr || matrix == nullptr) return CQL_ERR_ARG;
  if (!aligned_to(src, esize(dt)) || !aligned_to(matrix, 256)) return CQL_ERR_ALIGN;
  const Fp8Shape s = fp8_shape(rows, cols);
  if (matrix_bytes < s.total) return CQL_ERR_SIZE;
  return of_cuda(launch_fp8_quantize(s, src, dt, ld, static_cast<uint8_t*>(matrix), kFp8Plain, nullptr,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

cql_status cql_fp8_dequantize(const void* matrix, uint64_t matrix_bytes, int64_t rows, int32_t cols, void* out,
                              cql_dtype dt, int64_t ld, cql_stream_t stream) {
  if (!shape_ok(rows, cols) || !plain_dt(dt) || ld < cols) return CQL_ERR_ARG;
  if (rows == 0) return CQL_OK;
  if (matrix == nullptr || out == nullptr) return CQL_ERR_ARG;
  if (!aligned_to(out, esize(dt)) || !aligned_to(matrix, 256)) return CQL_ERR_ALIGN;
  const Fp8Shape s = fp8_shape(rows, cols);
  if (matrix_bytes < s.total) return CQL_ERR_SIZE;
  return of_cuda(launch_fp8_dequantize(s, static_cast<const uint8_t*>(matrix), out, dt, ld,
                                       reinterpret_cast<cudaStream_t>(stream)));
}

cql_status cql_fp8_workspace_size(int32_t k_in, int32_t experts, int32_t tokens, uint64_t* bytes) {
  if (bytes == nullptr || k_in < 1 || k_in > CQL_FP8_MAX_COLS || experts < 1 || experts > CQL_FP8_MAX_EXPERTS ||
      tokens < 0 || tokens > CQL_FP8_MAX_TOKENS)
    return CQL_ERR_ARG;
  *bytes = fp8_decode_quantizes(tokens, experts) ? 0 : fp8_shape(tokens, k_in).total;
  return CQL_OK;
}

cql_status cql_fp8_linear_forward(int32_t n_out, int32_t k_in, const void* weight, const void* x, cql_dtype x_dt,
                                  int64_t ldx, void* y, cql_dtype y_dt, int64_t ldy, int32_t tokens, void* workspace,
                                  uint64_t ws_bytes, uint32_t* status, cql_stream_t stream) {
  return forward(n_out, k_in, 1, weight, x, x_dt, ldx, nullptr, y, y_dt, ldy, tokens, workspace, ws_bytes, status,
                 stream);
}

cql_status cql_fp8_grouped_forward(int32_t n_out, int32_t k_in, int32_t experts, const void* weight, const void* x,
                                   cql_dtype x_dt, int64_t ldx, const int32_t* offsets, void* y, cql_dtype y_dt,
                                   int64_t ldy, int32_t tokens, void* workspace, uint64_t ws_bytes, uint32_t* status,
                                   cql_stream_t stream) {
  if (offsets == nullptr) return CQL_ERR_ARG;
  if (!aligned_to(offsets, 4)) return CQL_ERR_ALIGN;
  return forward(n_out, k_in, experts, weight, x, x_dt, ldx, offsets, y, y_dt, ldy, tokens, workspace, ws_bytes,
                 status, stream);
}

}  // extern "C"
