// Quantisation to microscaled 4-bit floating point and back (the format and
// the rounding are in mx4.cuh), in the rows' own order or straight into the
// dispatch's sorted order.
//
// Bound by memory: bf16 rows are read once (2 bytes a value) and written once
// (17/32 of a byte). In quantisation a lane takes a block of 32 values: its
// largest magnitude needs no other lane, its codes are one 16-byte store beside
// its neighbours', the warp's scales 32 bytes together, and four (fp32: eight)
// 16-byte loads are in flight (45056 x 2048 bf16: 41 us, 5.7 TB/s; with eight
// values a lane, four lanes to a block and 4-byte stores, 45 us, and into six
// sorted rows a token, 8192 x 4096, 38 us instead of 30). Dequantisation, which
// mostly stores, keeps eight values a lane, whose stores are then 16 bytes
// beside one another.
#include <cuda_runtime.h>

#include "kernels.h"
#include "moe.h"
#include "mx4.cuh"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace stm {
namespace {

using namespace mx4;

constexpr int QTHREADS = 256;
constexpr int kPasses = 4;             // eight values of a lane
constexpr int kChunk = kPasses * 256;  // values per warp

// Eight values as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

// The values at p, or zeros: selected, not branched round, so that the loads of
// a thread go out together.
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p, bool inside) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) / 2); ++i)
    r.v[i] = inside ? __ldcs(reinterpret_cast<const uint4*>(p) + i) : make_uint4(0u, 0u, 0u, 0u);
  return r;
}

template <typename T>
__device__ __forceinline__ void values8(const Raw8<T>& r, float* f) {
  if constexpr (sizeof(T) == 4) {
    unpack16(r.v[0], f, static_cast<float*>(nullptr));
    unpack16(r.v[1], f + 4, static_cast<float*>(nullptr));
  } else {
    unpack16_bf16(r.v[0], f);
  }
}

constexpr int kSlots = 8;  // a token's sorted rows that are looked up at once

// Sorted positions of the first slots; -1 for one past k, without a row or outside [0, P).
__device__ __forceinline__ void load_slots(const int32_t* __restrict__ pp, int k, int64_t P, int (&p)[kSlots]) {
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    p[j] = j < k ? __ldg(pp + j) : -1;
    if (p[j] >= P) p[j] = -1;
  }
}

// SORTED: row t's codes go to the rows pair_pos[t*k + j] of `data` and
// `scale`, and the rows at or past offsets[E] are zeroed; else to row t.
template <typename T, bool SORTED>
__global__ void __launch_bounds__(QTHREADS) quantize_kernel(const T* __restrict__ x, int64_t rows, int K,
                                                            uint32_t* __restrict__ data, uint8_t* __restrict__ scale,
                                                            int pitch, int chunks,
                                                            const int32_t* __restrict__ pair_pos,
                                                            const int32_t* __restrict__ offsets, int k, int E) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = (int64_t)blockIdx.x * (QTHREADS / 32) + (threadIdx.x >> 5);
  const int64_t warps = (int64_t)gridDim.x * (QTHREADS / 32);
  const int64_t P = rows * k;
  for (int64_t it = warp0; it < rows * chunks; it += warps) {
    const int64_t row = it / chunks;
    const int c0 = (int)(it - row * chunks) * kChunk;
    int p[kSlots];
    if constexpr (SORTED) load_slots(pair_pos + row * k, k, P, p);
    const int col = c0 + lane * kBlock;
    Raw8<T> raw[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) raw[u] = load8(x + row * K + col + u * 8, col < K);
    float f[kBlock];
#pragma unroll
    for (int u = 0; u < 4; ++u) values8(raw[u], f + 8 * u);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kBlock; ++i) m = max(m, __float_as_uint(f[i]) & 0x7fffffffu);
    const uint32_t b = scale_byte(m);
    const float inv = inverse_scale(b);
#pragma unroll
    for (int i = 0; i < kBlock; ++i) f[i] *= inv;
    const uint4 code = b == kScaleNaN ? make_uint4(0u, 0u, 0u, 0u)
                                      : make_uint4(pack8(f), pack8(f + 8), pack8(f + 16), pack8(f + 24));
    const int pad0 = K / kBlock;  // the row's last chunk also writes the padding
    auto store = [&](int64_t r) {
      uint8_t* s = scale + r * pitch;
      if (col < K) {
        *reinterpret_cast<uint4*>(data + r * (K / 8) + col / 8) = code;
        s[col / kBlock] = (uint8_t)b;
      }
      if (K - c0 <= kChunk && pad0 + lane < pitch) s[pad0 + lane] = 0;
    };
    if constexpr (SORTED) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (p[j] >= 0) store(p[j]);
      for (int j = kSlots; j < k; ++j) {
        const int q = __ldg(pair_pos + row * k + j);
        if (q >= 0 && q < P) store(q);
      }
    } else {
      store(row);
    }
  }
  if constexpr (SORTED) {
    for (int64_t r = max(0, __ldg(offsets + E)) + warp0; r < P; r += warps) {
      for (int i = lane; i < K / 8; i += 32) data[r * (K / 8) + i] = 0u;
      for (int i = lane; i < pitch; i += 32) scale[r * pitch + i] = 0;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(QTHREADS) dequantize_kernel(const uint32_t* __restrict__ data,
                                                              const uint8_t* __restrict__ scale, int64_t rows, int K,
                                                              int pitch, int chunks, T* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = (int64_t)blockIdx.x * (QTHREADS / 32) + (threadIdx.x >> 5);
  const int64_t warps = (int64_t)gridDim.x * (QTHREADS / 32);
  for (int64_t it = warp0; it < rows * chunks; it += warps) {
    const int64_t row = it / chunks;
    const int c0 = (int)(it - row * chunks) * kChunk;
    uint32_t w[kPasses], b[kPasses];
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int col = c0 + u * 256 + lane * 8;
      w[u] = col < K ? __ldcs(data + row * (K / 8) + col / 8) : 0u;
      b[u] = col < K ? __ldg(scale + row * pitch + col / kBlock) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int col = c0 + u * 256 + lane * 8;
      if (col >= K) break;
      float f[8];
      unpack8(w[u], f);
      const float s = scale_value(b[u]);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] *= s;
      T* o = out + row * K + col;
      if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(o)[0] = make_float4(f[0], f[1], f[2], f[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(f[4], f[5], f[6], f[7]);
      } else {
        *reinterpret_cast<uint4*>(o) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      }
    }
  }
}

bool ok_ptr(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Blocks for `items` warps' work, at most `most`.
unsigned warp_grid(int64_t items, int64_t most = 148 * 8) {
  return (unsigned)std::max<int64_t>(1, std::min<int64_t>(ceil_div(items, QTHREADS / 32), most));
}

// Dequantisation, which mostly stores, runs with blocks that are replaced as
// they end (45056 x 2048 to bf16: 39 us, with resident blocks 46).
constexpr int64_t kManyBlocks = 148 * 8 * 64;

moe_status check_rows(int64_t rows, int64_t K, int32_t dtype) {
  if (rows < 0 || K <= 0 || K % kBlock != 0 || K >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31))
    return MOE_ERR_INVALID_ARGUMENT;
  if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace
}  // namespace stm

using namespace stm;

MOE_API moe_status moe_mx4_quantize(int64_t rows, int64_t K, int32_t dtype, const void* x, void* data, void* scale,
                                    moe_stream_t stream) {
  const moe_status st = check_rows(rows, K, dtype);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(data) || !ok_ptr(scale)) return MOE_ERR_INVALID_ARGUMENT;
  const int chunks = (int)ceil_div(K, kChunk), pitch = (int)scale_pitch(K);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t* d = static_cast<uint32_t*>(data);
  uint8_t* sc = static_cast<uint8_t*>(scale);
  if (dtype == MOE_DTYPE_F32)
    quantize_kernel<float, false><<<warp_grid(rows * chunks), QTHREADS, 0, s>>>(
        static_cast<const float*>(x), rows, (int)K, d, sc, pitch, chunks, nullptr, nullptr, 1, 0);
  else
    quantize_kernel<__nv_bfloat16, false><<<warp_grid(rows * chunks), QTHREADS, 0, s>>>(
        static_cast<const __nv_bfloat16*>(x), rows, (int)K, d, sc, pitch, chunks, nullptr, nullptr, 1, 0);
  return status(cudaGetLastError());
}

MOE_API moe_status moe_mx4_dequantize(int64_t rows, int64_t K, int32_t dtype, const void* data, const void* scale,
                                      void* out, moe_stream_t stream) {
  const moe_status st = check_rows(rows, K, dtype);
  if (st != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  if (!ok_ptr(data) || !ok_ptr(scale) || !ok_ptr(out)) return MOE_ERR_INVALID_ARGUMENT;
  const int chunks = (int)ceil_div(K, kChunk), pitch = (int)scale_pitch(K);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const uint32_t* d = static_cast<const uint32_t*>(data);
  const uint8_t* sc = static_cast<const uint8_t*>(scale);
  if (dtype == MOE_DTYPE_F32)
    dequantize_kernel<float><<<warp_grid(rows * chunks, kManyBlocks), QTHREADS, 0, s>>>(
        d, sc, rows, (int)K, pitch, chunks, static_cast<float*>(out));
  else
    dequantize_kernel<__nv_bfloat16><<<warp_grid(rows * chunks, kManyBlocks), QTHREADS, 0, s>>>(
        d, sc, rows, (int)K, pitch, chunks, static_cast<__nv_bfloat16*>(out));
  return status(cudaGetLastError());
}

MOE_API moe_status moe_mx4_permute_rows(const moe_problem* p, const void* x, const int32_t* pair_pos,
                                        const int32_t* offsets, void* data, void* scale, moe_stream_t stream) {
  size_t bytes = 0;
  const moe_status st = moe_workspace_size(p, &bytes);  // validates the problem
  if (st != MOE_OK) return st;
  if (p->H % kBlock != 0) return MOE_ERR_INVALID_ARGUMENT;
  if (p->T == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(pair_pos) || !ok_ptr(offsets) || !ok_ptr(data) || !ok_ptr(scale))
    return MOE_ERR_INVALID_ARGUMENT;
  const int chunks = (int)ceil_div(p->H, kChunk), pitch = (int)scale_pitch(p->H);
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint32_t* d = static_cast<uint32_t*>(data);
  uint8_t* sc = static_cast<uint8_t*>(scale);
  if (p->dtype == MOE_DTYPE_F32)
    quantize_kernel<float, true><<<warp_grid(p->T * chunks), QTHREADS, 0, s>>>(
        static_cast<const float*>(x), p->T, (int)p->H, d, sc, pitch, chunks, pair_pos, offsets, (int)p->k, (int)p->E);
  else
    quantize_kernel<__nv_bfloat16, true><<<warp_grid(p->T * chunks), QTHREADS, 0, s>>>(
        static_cast<const __nv_bfloat16*>(x), p->T, (int)p->H, d, sc, pitch, chunks, pair_pos, offsets, (int)p->k,
        (int)p->E);
  return status(cudaGetLastError());
}
