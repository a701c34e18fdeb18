// Token rows sorted by expert and back in token order, with the routing
// weights applied, and the gradients of both.
//
// The plan is the dispatch's (dispatch.cu): pair q = t*k + j sits at sorted
// position pos(q) = pair_pos[q], or nowhere (-1); positions at or past
// offsets[E] hold no pair. With P = T*k sorted rows of H columns:
//   permute            xs[pos(q)] = x[t], rows without a pair 0
//   its gradient       dx[t] = sum_j dxs[pos(t,j)]
//   unpermute          out[t] = sum_j w[t,j] ys[pos(t,j)] (+ shared[t])
//   its gradient       dys[pos(q)] = w[q] dout[t], rows without a pair 0,
//                      dw[q] = sum_h dout[t,h] ys[pos(q),h]
// Sums run in fp32 in a fixed order (no atomics); each result is rounded once
// to its type.
//
// All four are bound by memory: every row is read once and written once, and
// there is at most one multiply-add per element read. They are therefore cut
// by token: a token's own row (x, dout, out) is read or written once, in
// registers, and only its k sorted rows are touched besides it, each with
// 16-byte accesses that cover whole lines. A thread first issues the loads of
// up to eight sorted rows and then uses them in slot order.
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace stm {
namespace {

constexpr int RTHREADS = 256;
constexpr int kSlots = 8;  // sorted rows of a token in flight at once

// 16 bytes of a row as fp32: 4 fp32 or 8 bf16 values.
template <typename T>
__device__ __forceinline__ void load16(const T* p, float* f) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  if constexpr (sizeof(T) == 4) unpack16(v, f, static_cast<float*>(nullptr));
  else unpack16_bf16(v, f);
}

// The N values at p as fp32: 16 bytes, or 8 (four bf16 beside four fp32).
template <int N, typename T>
__device__ __forceinline__ void loadn(const T* p, float* f) {
  if constexpr (N * sizeof(T) == 16) {
    load16(p, f);
  } else {
    static_assert(N == 4 && sizeof(T) == 2, "four bf16");
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
  }
}

template <int N, typename T>
__device__ __forceinline__ void storen(T* p, const float* f) {
  if constexpr (sizeof(T) == 4) {
    static_assert(N == 4, "four fp32");
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else if constexpr (N == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  }
}

// Sorted positions of a token's slots j0 .. j0+7; -1 for a slot past k, one
// without a row, or (a plan that is not the dispatch's) one outside [0, P).
__device__ __forceinline__ void load_slots(const int32_t* __restrict__ pp, int j0, int k, int64_t P, int (&p)[kSlots]) {
#pragma unroll
  for (int j = 0; j < kSlots; ++j) {
    p[j] = j0 + j < k ? __ldg(pp + j0 + j) : -1;
    if (p[j] >= P) p[j] = -1;
  }
}

// Zeroes the rows [offsets[E], P) of `rows` (nvec 16-byte vectors each).
__device__ __forceinline__ void zero_unused_rows(uint4* __restrict__ rows, const int32_t* __restrict__ offsets, int E,
                                                 int64_t P, int nvec) {
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t nb = (int64_t)gridDim.x * gridDim.y;
  for (int64_t r = max(0, __ldg(offsets + E)) + b; r < P; r += nb)
    for (int v = threadIdx.x; v < nvec; v += RTHREADS) rows[r * nvec + v] = make_uint4(0u, 0u, 0u, 0u);
}

// A block is 256 >> lg token lanes of 1 << lg threads: a thread handles one
// vector column of one token at a time, so no index needs a division.
__global__ void __launch_bounds__(RTHREADS) permute_rows_kernel(const uint4* __restrict__ x,
                                                                const int32_t* __restrict__ pair_pos,
                                                                const int32_t* __restrict__ offsets,
                                                                uint4* __restrict__ xs, int64_t Tn, int nvec, int k,
                                                                int E, int lg) {
  const int64_t P = Tn * k;
  const int tpb = RTHREADS >> lg, col = threadIdx.x & ((1 << lg) - 1);
  for (int64_t t = (int64_t)blockIdx.x * tpb + (threadIdx.x >> lg); t < Tn; t += (int64_t)gridDim.x * tpb) {
    const int32_t* pp = pair_pos + t * k;
    int p[kSlots];
    load_slots(pp, 0, k, P, p);
    for (int v = (blockIdx.y << lg) + col; v < nvec; v += gridDim.y << lg) {
      const uint4 val = x[t * nvec + v];
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (p[j] >= 0) xs[(int64_t)p[j] * nvec + v] = val;
      for (int j = kSlots; j < k; ++j) {
        const int q = __ldg(pp + j);
        if (q >= 0 && q < P) xs[(int64_t)q * nvec + v] = val;
      }
    }
  }
  zero_unused_rows(xs, offsets, E, P, nvec);
}

template <typename TY, typename TO, bool WEIGHTED>
__global__ void __launch_bounds__(RTHREADS) unpermute_rows_kernel(const TY* __restrict__ ys,
                                                                  const int32_t* __restrict__ pair_pos,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ shared_out,
                                                                  TO* __restrict__ out, int64_t Tn, int H, int k,
                                                                  int lg) {
  constexpr int N = 16 / sizeof(TY);
  const int64_t P = Tn * k;
  const int nvec = H / N;
  const int tpb = RTHREADS >> lg, col = threadIdx.x & ((1 << lg) - 1);
  for (int64_t t = (int64_t)blockIdx.x * tpb + (threadIdx.x >> lg); t < Tn; t += (int64_t)gridDim.x * tpb) {
    int p0[kSlots];
    float w0[kSlots];
    load_slots(pair_pos + t * k, 0, k, P, p0);
    if constexpr (WEIGHTED) {
#pragma unroll
      for (int j = 0; j < kSlots; ++j) w0[j] = j < k ? __ldg(w + t * k + j) : 0.f;
    }
    for (int v = (blockIdx.y << lg) + col; v < nvec; v += gridDim.y << lg) {
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      auto add = [&](const int (&p)[kSlots], const float (&ww)[kSlots]) {
        uint4 raw[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
          if (p[j] >= 0) raw[j] = __ldcs(reinterpret_cast<const uint4*>(ys + (int64_t)p[j] * H) + v);
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          if (p[j] < 0) continue;  // a slot without a row adds nothing, whatever its weight
          float f[N];
          if constexpr (sizeof(TY) == 4) unpack16(raw[j], f, static_cast<float*>(nullptr));
          else unpack16_bf16(raw[j], f);
#pragma unroll
          for (int i = 0; i < N; ++i) acc[i] = WEIGHTED ? fmaf(ww[j], f[i], acc[i]) : acc[i] + f[i];
        }
      };
      add(p0, w0);
      for (int j0 = kSlots; j0 < k; j0 += kSlots) {
        int p[kSlots];
        float ww[kSlots];
        load_slots(pair_pos + t * k, j0, k, P, p);
        if constexpr (WEIGHTED) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j) ww[j] = j0 + j < k ? __ldg(w + t * k + j0 + j) : 0.f;
        }
        add(p, ww);
      }
      if (shared_out != nullptr) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
          const float4 s = __ldcs(reinterpret_cast<const float4*>(shared_out + t * H + v * N + i));
          acc[i] += s.x;
          acc[i + 1] += s.y;
          acc[i + 2] += s.z;
          acc[i + 3] += s.w;
        }
      }
      storen<N>(out + t * H + (int64_t)v * N, acc);
    }
  }
}

// Sums eight values over a warp: afterwards the lanes with (lane & 3) == 0
// hold the whole sum of value (lane >> 2). Each step halves what a lane
// keeps, so eight sums take 9 shuffles instead of 40.
__device__ __forceinline__ float warp_sum8(float (&a)[kSlots], int lane) {
#pragma unroll
  for (int n = 4, o = 16; n >= 1; n >>= 1, o >>= 1) {
    const bool upper = lane & o;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = upper ? a[i] : a[i + n];
      const float keep = upper ? a[i + n] : a[i];
      a[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
  }
  a[0] += __shfl_xor_sync(0xffffffffu, a[0], 2);
  a[0] += __shfl_xor_sync(0xffffffffu, a[0], 1);
  return a[0];
}

// 1 << lw warps share one token's columns, and its slots are taken eight at a
// time. dys and dw may each be absent.
template <typename TY, typename TD>
__global__ void __launch_bounds__(RTHREADS) unpermute_rows_backward_kernel(
    const TD* __restrict__ dout, const TY* __restrict__ ys, const int32_t* __restrict__ pair_pos,
    const int32_t* __restrict__ offsets, const float* __restrict__ w, TY* __restrict__ dys, float* __restrict__ dw,
    int64_t Tn, int H, int k, int E, int lw) {
  constexpr int N = 16 / sizeof(TY);
  __shared__ float part[RTHREADS / 32][kSlots];
  const int64_t P = Tn * k;
  const int nvec = H / N;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int tpb = (RTHREADS / 32) >> lw, team = 32 << lw;
  for (int64_t tb = (int64_t)blockIdx.x * tpb; tb < Tn; tb += (int64_t)gridDim.x * tpb) {
    const int64_t t = tb + (warp >> lw);
    const bool live = t < Tn;
    for (int j0 = 0; j0 < k; j0 += kSlots) {
      int p[kSlots];
      float ww[kSlots], acc[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        p[j] = -1;
        ww[j] = 1.f;
        acc[j] = 0.f;
      }
      if (live) {
        load_slots(pair_pos + t * k, j0, k, P, p);
        if (w != nullptr) {
#pragma unroll
          for (int j = 0; j < kSlots; ++j) ww[j] = j0 + j < k ? __ldg(w + t * k + j0 + j) : 0.f;
        }
        for (int v = threadIdx.x & (team - 1); v < nvec; v += team) {
          float d[N];
          loadn<N>(dout + t * H + (int64_t)v * N, d);
          uint4 raw[kSlots];
          if (dw != nullptr) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
              if (p[j] >= 0) raw[j] = __ldcs(reinterpret_cast<const uint4*>(ys + (int64_t)p[j] * H) + v);
          }
          if (dys != nullptr) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
              if (p[j] < 0) continue;
              float g[N];
#pragma unroll
              for (int i = 0; i < N; ++i) g[i] = ww[j] * d[i];
              storen<N>(dys + (int64_t)p[j] * H + (int64_t)v * N, g);
            }
          }
          if (dw != nullptr) {
#pragma unroll
            for (int j = 0; j < kSlots; ++j) {
              if (p[j] < 0) continue;
              float f[N];
              if constexpr (sizeof(TY) == 4) unpack16(raw[j], f, static_cast<float*>(nullptr));
              else unpack16_bf16(raw[j], f);
#pragma unroll
              for (int i = 0; i < N; ++i) acc[j] = fmaf(d[i], f[i], acc[j]);
            }
          }
        }
      }
      if (dw != nullptr) {  // the same for the whole block
        const float s = warp_sum8(acc, lane);
        const int j = lane >> 2;
        if (lw == 0) {
          if (live && (lane & 3) == 0 && j0 + j < k) dw[t * k + j0 + j] = s;
        } else {
          if ((lane & 3) == 0) part[warp][j] = s;
          __syncthreads();
          const int first = warp & ~((1 << lw) - 1);
          if (live && warp == first && lane < kSlots && j0 + lane < k) {
            float sum = 0.f;
            for (int i = 0; i < (1 << lw); ++i) sum += part[first + i][lane];
            dw[t * k + j0 + lane] = sum;
          }
          __syncthreads();
        }
      }
    }
  }
  if (dys != nullptr) zero_unused_rows(reinterpret_cast<uint4*>(dys), offsets, E, P, nvec);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok_ptr(const void* p) { return p != nullptr && aligned16(p); }
bool ok_opt(const void* p) { return p == nullptr || aligned16(p); }

moe_status check_problem(const moe_problem* p) {
  size_t bytes = 0;
  return moe_workspace_size(p, &bytes);  // validates the problem
}

// log2 of the threads a token lane gets: the most (up to 256) that leave at
// most a quarter of them idle on the last pass over nvec vectors, and never
// fewer than 4.
int lane_log2(int64_t nvec) {
  int lg = 8;
  while (lg > 2 && round_up(nvec, int64_t(1) << lg) * 4 > nvec * 5) --lg;
  return lg;
}

// Blocks for T tokens in lanes of 1 << lg threads: full residency (eight
// blocks of 256 threads on each of 148 SMs), split over the columns too when
// the tokens alone give fewer.
dim3 lane_grid(int64_t T, int64_t nvec, int lg) {
  const int64_t full = 148 * 8;
  const int64_t bx = ceil_div(T, RTHREADS >> lg);
  const int64_t by = std::max<int64_t>(1, std::min<int64_t>(ceil_div(nvec, int64_t(1) << lg), full / std::max<int64_t>(1, bx)));
  return dim3((unsigned)std::min(bx, full), (unsigned)by);
}

template <typename TY, typename TO>
cudaError_t launch_unpermute(const void* ys, const int32_t* pair_pos, const float* w, const float* shared_out,
                             void* out, int64_t T, int64_t H, int64_t k, cudaStream_t s) {
  const int64_t nvec = H * sizeof(TY) / 16;
  const int lg = lane_log2(nvec);
  const dim3 grid = lane_grid(T, nvec, lg);
  if (w != nullptr)
    unpermute_rows_kernel<TY, TO, true><<<grid, RTHREADS, 0, s>>>(
        static_cast<const TY*>(ys), pair_pos, w, shared_out, static_cast<TO*>(out), T, (int)H, (int)k, lg);
  else
    unpermute_rows_kernel<TY, TO, false><<<grid, RTHREADS, 0, s>>>(
        static_cast<const TY*>(ys), pair_pos, w, shared_out, static_cast<TO*>(out), T, (int)H, (int)k, lg);
  return cudaGetLastError();
}

template <typename TY, typename TD>
cudaError_t launch_unpermute_backward(const void* dout, const void* ys, const int32_t* pair_pos,
                                      const int32_t* offsets, const float* w, void* dys, float* dw, int64_t T,
                                      int64_t H, int64_t k, int64_t E, cudaStream_t s) {
  const int64_t nvec = H * sizeof(TY) / 16;
  // One warp per token while that alone fills the GPU (64 warps on each of
  // 148 SMs); more warps for fewer tokens, as long as each has a vector.
  int lw = 0;
  while (lw < 3 && (T << lw) < 148 * 64 && nvec > (32 << lw)) ++lw;
  const int64_t grid = std::min<int64_t>(ceil_div(T, 8 >> lw), 148 * 8);
  unpermute_rows_backward_kernel<TY, TD><<<(unsigned)grid, RTHREADS, 0, s>>>(
      static_cast<const TD*>(dout), static_cast<const TY*>(ys), pair_pos, offsets, w, static_cast<TY*>(dys), dw, T,
      (int)H, (int)k, (int)E, lw);
  return cudaGetLastError();
}

}  // namespace
}  // namespace stm

using namespace stm;

MOE_API moe_status moe_permute_rows(const moe_problem* p, const void* x, const int32_t* pair_pos,
                                    const int32_t* offsets, void* x_perm, moe_stream_t stream) {
  const moe_status st = check_problem(p);
  if (st != MOE_OK) return st;
  if (p->T == 0) return MOE_OK;
  if (!ok_ptr(x) || !ok_ptr(pair_pos) || !ok_ptr(offsets) || !ok_ptr(x_perm)) return MOE_ERR_INVALID_ARGUMENT;
  const int64_t nvec = p->H * (p->dtype == MOE_DTYPE_F32 ? 4 : 2) / 16;
  const int lg = lane_log2(nvec);
  permute_rows_kernel<<<lane_grid(p->T, nvec, lg), RTHREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint4*>(x), pair_pos, offsets, static_cast<uint4*>(x_perm), p->T, (int)nvec, (int)p->k,
      (int)p->E, lg);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

MOE_API moe_status moe_unpermute_rows(const moe_problem* p, int32_t y_dtype, const void* y_perm,
                                      const int32_t* pair_pos, const float* routing_weights, const float* shared_out,
                                      void* out, moe_stream_t stream) {
  const moe_status st = check_problem(p);
  if (st != MOE_OK) return st;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != p->dtype) return MOE_ERR_INVALID_ARGUMENT;
  if (p->T == 0) return MOE_OK;
  if (!ok_ptr(y_perm) || !ok_ptr(pair_pos) || !ok_opt(routing_weights) || !ok_opt(shared_out) || !ok_ptr(out))
    return MOE_ERR_INVALID_ARGUMENT;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->dtype == MOE_DTYPE_F32)
    e = launch_unpermute<float, float>(y_perm, pair_pos, routing_weights, shared_out, out, p->T, p->H, p->k, s);
  else if (y_dtype == MOE_DTYPE_F32)
    e = launch_unpermute<float, __nv_bfloat16>(y_perm, pair_pos, routing_weights, shared_out, out, p->T, p->H, p->k, s);
  else
    e = launch_unpermute<__nv_bfloat16, __nv_bfloat16>(y_perm, pair_pos, routing_weights, shared_out, out, p->T, p->H,
                                                       p->k, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

MOE_API moe_status moe_permute_rows_backward(const moe_problem* p, const void* dx_perm, const int32_t* pair_pos,
                                             void* dx, moe_stream_t stream) {
  if (p == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  return moe_unpermute_rows(p, p->dtype, dx_perm, pair_pos, nullptr, nullptr, dx, stream);
}

MOE_API moe_status moe_unpermute_rows_backward(const moe_problem* p, int32_t y_dtype, const void* dout,
                                               const void* y_perm, const int32_t* pair_pos, const int32_t* offsets,
                                               const float* routing_weights, void* dy_perm, float* d_routing_weights,
                                               moe_stream_t stream) {
  const moe_status st = check_problem(p);
  if (st != MOE_OK) return st;
  if (y_dtype != MOE_DTYPE_F32 && y_dtype != p->dtype) return MOE_ERR_INVALID_ARGUMENT;
  if (p->T == 0) return MOE_OK;
  if (!ok_ptr(dout) || !ok_ptr(pair_pos) || !ok_opt(routing_weights) || !ok_opt(dy_perm) ||
      !ok_opt(d_routing_weights))
    return MOE_ERR_INVALID_ARGUMENT;
  if (dy_perm == nullptr && d_routing_weights == nullptr) return MOE_ERR_INVALID_ARGUMENT;
  if (dy_perm != nullptr && !ok_ptr(offsets)) return MOE_ERR_INVALID_ARGUMENT;
  if (d_routing_weights != nullptr && !ok_ptr(y_perm)) return MOE_ERR_INVALID_ARGUMENT;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (p->dtype == MOE_DTYPE_F32)
    e = launch_unpermute_backward<float, float>(dout, y_perm, pair_pos, offsets, routing_weights, dy_perm,
                                                d_routing_weights, p->T, p->H, p->k, p->E, s);
  else if (y_dtype == MOE_DTYPE_F32)
    e = launch_unpermute_backward<float, __nv_bfloat16>(dout, y_perm, pair_pos, offsets, routing_weights, dy_perm,
                                                        d_routing_weights, p->T, p->H, p->k, p->E, s);
  else
    e = launch_unpermute_backward<__nv_bfloat16, __nv_bfloat16>(dout, y_perm, pair_pos, offsets, routing_weights,
                                                                dy_perm, d_routing_weights, p->T, p->H, p->k, p->E, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
