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
// 16-byte accesses that cover whole lines. What reaches the memory's rate is
// the loads in flight, so the kernels are compiled for each k up to 8 (more
// slots go eight at a time), and a thread takes several vectors of its token at
// once: 8 for k 1, 4 for k 2 and 3 (fp32 rows: to 5), else 2. The compiler issues
// their loads ahead as far as its registers go.
// (8192 x 8192 bf16, k 2: unpermute 130 us with one vector a thread, 64 with
// four.)
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "moe.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace stm {
namespace {

constexpr int RTHREADS = 256;
constexpr int kSlots = 8;  // sorted rows of a token in flight at once

// N values as they lie in memory: 16 bytes, or 8 (four bf16 beside four fp32).
template <int N, typename T>
using Raw = std::conditional_t<N * sizeof(T) == 16, uint4, uint2>;

template <int N, typename T>
__device__ __forceinline__ void unpackn(const Raw<N, T>& v, float* f) {
  if constexpr (N * sizeof(T) == 8) {
    static_assert(N == 4 && sizeof(T) == 2, "four bf16");
    f[0] = __uint_as_float(v.x << 16);
    f[1] = __uint_as_float(v.x & 0xffff0000u);
    f[2] = __uint_as_float(v.y << 16);
    f[3] = __uint_as_float(v.y & 0xffff0000u);
  } else if constexpr (sizeof(T) == 4) {
    unpack16(v, f, static_cast<float*>(nullptr));
  } else {
    unpack16_bf16(v, f);
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

// Sorted positions of a token's slots j0 .. j0 + SL - 1; -1 for a slot past k,
// one without a row, or (a plan that is not the dispatch's) one outside [0, P).
template <int SL>
__device__ __forceinline__ void load_slots(const int32_t* __restrict__ pp, int j0, int k, int64_t P, int (&p)[SL]) {
#pragma unroll
  for (int j = 0; j < SL; ++j) {
    p[j] = j0 + j < k ? __ldg(pp + j0 + j) : -1;
    if (p[j] >= P) p[j] = -1;
  }
}

// Their weights: 1 without a weight table, 0 for a slot without a row, which
// adds nothing whatever its weight.
template <int SL>
__device__ __forceinline__ void load_weights(const float* __restrict__ w, int j0, const int (&p)[SL], float (&ww)[SL]) {
#pragma unroll
  for (int j = 0; j < SL; ++j) ww[j] = p[j] < 0 ? 0.f : w == nullptr ? 1.f : __ldg(w + j0 + j);
}

// A vector of a sorted row; zeros where there is none (selected, not branched
// round, so that the loads of a thread go out together: branches around them
// made 8192 x 2048 bf16, k 8, 87 us instead of 53).
__device__ __forceinline__ uint4 load_row(const void* row, int v, bool has) {
  return has ? __ldcs(static_cast<const uint4*>(row) + v) : make_uint4(0u, 0u, 0u, 0u);
}

// Zeroes the rows [offsets[E], P) of `rows` (nvec 16-byte vectors each).
__device__ __forceinline__ void zero_unused_rows(uint4* __restrict__ rows, const int32_t* __restrict__ offsets, int E,
                                                 int64_t P, int nvec) {
  const int64_t b = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t nb = (int64_t)gridDim.x * gridDim.y;
  for (int64_t r = max(0, __ldg(offsets + E)) + b; r < P; r += nb)
    for (int v = threadIdx.x; v < nvec; v += RTHREADS) rows[r * nvec + v] = make_uint4(0u, 0u, 0u, 0u);
}

// A block is 256 >> lg teams of 1 << lg threads: a team handles one token at a
// time, a thread V of its vectors a pass, so no index needs a division.
template <int V>
__global__ void __launch_bounds__(RTHREADS) permute_rows_kernel(const uint4* __restrict__ x,
                                                                const int32_t* __restrict__ pair_pos,
                                                                const int32_t* __restrict__ offsets,
                                                                uint4* __restrict__ xs, int64_t Tn, int nvec, int k,
                                                                int E, int lg) {
  const int64_t P = Tn * k;
  const int tpb = RTHREADS >> lg, team = 1 << lg, col = threadIdx.x & (team - 1);
  for (int64_t t = (int64_t)blockIdx.x * tpb + (threadIdx.x >> lg); t < Tn; t += (int64_t)gridDim.x * tpb) {
    const int32_t* pp = pair_pos + t * k;
    int p[kSlots];
    load_slots(pp, 0, k, P, p);
    for (int v0 = blockIdx.y * team * V + col; v0 < nvec; v0 += gridDim.y * team * V) {
      uint4 val[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (v0 + i * team < nvec) val[i] = x[t * nvec + v0 + i * team];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        if (p[j] < 0) continue;
        uint4* o = xs + (int64_t)p[j] * nvec + v0;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (v0 + i * team < nvec) o[i * team] = val[i];
      }
      for (int j = kSlots; j < k; ++j) {
        const int q = __ldg(pp + j);
        if (q < 0 || q >= P) continue;
        uint4* o = xs + (int64_t)q * nvec + v0;
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (v0 + i * team < nvec) o[i * team] = val[i];
      }
    }
  }
  zero_unused_rows(xs, offsets, E, P, nvec);
}

// SL: the token's slots, or 8 of them at a time.
template <typename TY, typename TO, int SL, int V>
__global__ void __launch_bounds__(RTHREADS) unpermute_rows_kernel(const TY* __restrict__ ys,
                                                                  const int32_t* __restrict__ pair_pos,
                                                                  const float* __restrict__ w,
                                                                  const float* __restrict__ shared_out,
                                                                  TO* __restrict__ out, int64_t Tn, int H, int k,
                                                                  int lg) {
  constexpr int N = 16 / sizeof(TY);
  const int64_t P = Tn * k;
  const int nvec = H / N;
  const int tpb = RTHREADS >> lg, team = 1 << lg, col = threadIdx.x & (team - 1);
  for (int64_t t = (int64_t)blockIdx.x * tpb + (threadIdx.x >> lg); t < Tn; t += (int64_t)gridDim.x * tpb) {
    const int32_t* pp = pair_pos + t * k;
    const float* wt = w == nullptr ? nullptr : w + t * k;
    int p0[SL];
    float w0[SL];
    load_slots(pp, 0, k, P, p0);
    load_weights(wt, 0, p0, w0);
    for (int v0 = blockIdx.y * team * V + col; v0 < nvec; v0 += gridDim.y * team * V) {
      float acc[V][N];
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int n = 0; n < N; ++n) acc[i][n] = 0.f;
      auto add = [&](const int (&p)[SL], const float (&ww)[SL]) {
        uint4 raw[V][SL];
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < SL; ++j)
            raw[i][j] = load_row(ys + (int64_t)p[j] * H, v0 + i * team, p[j] >= 0 && v0 + i * team < nvec);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < SL; ++j) {
            float f[N];
            unpackn<N, TY>(raw[i][j], f);
#pragma unroll
            for (int n = 0; n < N; ++n) acc[i][n] = fmaf(ww[j], f[n], acc[i][n]);
          }
      };
      add(p0, w0);
      if constexpr (SL == kSlots) {
        for (int j0 = kSlots; j0 < k; j0 += kSlots) {
          int p[SL];
          float ww[SL];
          load_slots(pp, j0, k, P, p);
          load_weights(wt, j0, p, ww);
          add(p, ww);
        }
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = v0 + i * team;
        if (v >= nvec) break;
        if (shared_out != nullptr) {
#pragma unroll
          for (int n = 0; n < N; n += 4) {
            const float4 s = __ldcs(reinterpret_cast<const float4*>(shared_out + t * H + (int64_t)v * N + n));
            acc[i][n] += s.x;
            acc[i][n + 1] += s.y;
            acc[i][n + 2] += s.z;
            acc[i][n + 3] += s.w;
          }
        }
        storen<N>(out + t * H + (int64_t)v * N, acc[i]);
      }
    }
  }
}

// The sums of SL values over a team of 1 << lt lanes of a warp, the whole sum
// of value j in the team's lane j.
template <int SL>
__device__ __forceinline__ float team_sums(float (&a)[SL], int lt, int col) {
  if constexpr (SL == kSlots) {
    if (lt == 5) {
      // Each step halves what a lane keeps: eight sums in 9 shuffles instead
      // of 40, value (lane >> 2) in the lanes with (lane & 3) == 0, and one
      // more to lane j.
#pragma unroll
      for (int n = 4, o = 16; n >= 1; n >>= 1, o >>= 1) {
        const bool upper = col & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const float send = upper ? a[i] : a[i + n];
          const float keep = upper ? a[i + n] : a[i];
          a[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
      }
      a[0] += __shfl_xor_sync(0xffffffffu, a[0], 2);
      a[0] += __shfl_xor_sync(0xffffffffu, a[0], 1);
      return __shfl_sync(0xffffffffu, a[0], (col & 7) << 2);
    }
  }
  float mine = 0.f;
#pragma unroll
  for (int j = 0; j < SL; ++j) {
    for (int o = 1 << lt >> 1; o >= 1; o >>= 1) a[j] += __shfl_xor_sync(0xffffffffu, a[j], o);
    if (col == j) mine = a[j];
  }
  return mine;
}

// 1 << lt threads (8 to 256) share one token's columns, and its slots are taken
// SL at a time. dys and dw may each be absent.
template <typename TY, typename TD, int SL, int V>
__global__ void __launch_bounds__(RTHREADS) unpermute_rows_backward_kernel(
    const TD* __restrict__ dout, const TY* __restrict__ ys, const int32_t* __restrict__ pair_pos,
    const int32_t* __restrict__ offsets, const float* __restrict__ w, TY* __restrict__ dys, float* __restrict__ dw,
    int64_t Tn, int H, int k, int E, int lt) {
  constexpr int N = 16 / sizeof(TY);
  __shared__ float part[RTHREADS / 32][kSlots];
  const int64_t P = Tn * k;
  const int nvec = H / N;
  const int warp = threadIdx.x >> 5;
  const int tpb = RTHREADS >> lt, team = 1 << lt, col = threadIdx.x & (team - 1);
  for (int64_t tb = (int64_t)blockIdx.x * tpb; tb < Tn; tb += (int64_t)gridDim.x * tpb) {
    const int64_t t = tb + (threadIdx.x >> lt);
    const bool live = t < Tn;
    for (int j0 = 0; j0 < k; j0 += SL) {
      int p[SL];
      float ww[SL], acc[SL];
#pragma unroll
      for (int j = 0; j < SL; ++j) {
        p[j] = -1;
        ww[j] = 1.f;
        acc[j] = 0.f;
      }
      if (live) {
        load_slots(pair_pos + t * k, j0, k, P, p);
        load_weights(w == nullptr ? nullptr : w + t * k, j0, p, ww);
        for (int v0 = col; v0 < nvec; v0 += team * V) {
          Raw<N, TD> draw[V];
          uint4 raw[V][SL];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int v = v0 + i * team;
            draw[i] = v < nvec ? *reinterpret_cast<const Raw<N, TD>*>(dout + t * H + (int64_t)v * N) : Raw<N, TD>{};
            if (dw != nullptr) {
#pragma unroll
              for (int j = 0; j < SL; ++j)
                raw[i][j] = load_row(ys + (int64_t)p[j] * H, v, p[j] >= 0 && v < nvec);
            }
          }
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const int v = v0 + i * team;
            if (v >= nvec) break;
            float d[N];
            unpackn<N, TD>(draw[i], d);
            if (dys != nullptr) {
#pragma unroll
              for (int j = 0; j < SL; ++j) {
                float g[N];
#pragma unroll
                for (int n = 0; n < N; ++n) g[n] = ww[j] * d[n];
                if (p[j] >= 0) storen<N>(dys + (int64_t)p[j] * H + (int64_t)v * N, g);
              }
            }
            if (dw != nullptr) {
#pragma unroll
              for (int j = 0; j < SL; ++j) {
                float f[N];
                unpackn<N, TY>(raw[i][j], f);
#pragma unroll
                for (int n = 0; n < N; ++n) acc[j] = fmaf(d[n], f[n], acc[j]);
              }
            }
          }
        }
#pragma unroll
        for (int j = 0; j < SL; ++j)
          if (p[j] < 0) acc[j] = 0.f;  // dout may hold an infinity
      }
      if (dw != nullptr) {  // the same for the whole block
        if (lt <= 5) {
          const float s = team_sums(acc, lt, col);
          if (live && col < SL && j0 + col < k) dw[t * k + j0 + col] = s;
        } else {
          const int lane = threadIdx.x & 31;
          const float s = team_sums(acc, 5, lane);
          if (lane < SL) part[warp][lane] = s;
          __syncthreads();
          if (live && col < SL && j0 + col < k) {
            float sum = 0.f;
            for (int i = 0; i < team >> 5; ++i) sum += part[warp + i][col];
            dw[t * k + j0 + col] = sum;
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

// Vectors of a token that a thread takes at once for SL slots of rows with
// `bytes` an element. Of fp32 rows, whose vectors have half the values to sum,
// four up to five slots (unpermute of 8192 x 4096 into bf16, us with four and two:
// k 4 96 / 110; 8192 x 2048, k 5 in fp32 69 / 80, into bf16 57 / 54) and two from
// six on (8192 x 4096, k 6, with shared_out, four and two: 171 / 160; 8192 x 2048,
// k 7: 90 / 81); two or three slots with eight: 94 and 115, with four 84 and 111
// (8192 x 4096, shared_out).
constexpr int vectors_for(int SL, int bytes) { return SL == 1 ? 8 : SL <= (bytes == 4 ? 5 : 3) ? 4 : 2; }

// Several vectors a thread once that leaves 512 threads for each of 148 SMs:
// few tokens need the threads more (300 tokens of 2048 bf16, k 6: 4.6 us with
// two vectors, 4.1 with one; 1024 tokens, k 8: 9.3 and 10.1).
bool many(int64_t T, int64_t nvec, int V) { return T * nvec >= (int64_t)V * 148 * 512; }

// log2 of a team's threads for `passes` vectors (or groups of them): the most
// (up to 256) that leave at most a quarter of them idle on the last pass, and
// never fewer than 4.
int lane_log2(int64_t passes) {
  int lg = 8;
  while (lg > 2 && round_up(passes, int64_t(1) << lg) * 4 > passes * 5) --lg;
  return lg;
}

// Blocks for T tokens in teams of 1 << lg threads: at most `most`, and split
// over the columns too when the tokens alone give less than full residency
// (eight blocks of 256 threads on each of 148 SMs).
constexpr int64_t kResident = 148 * 8;
dim3 lane_grid(int64_t T, int64_t passes, int lg, int64_t most) {
  const int64_t bx = ceil_div(T, RTHREADS >> lg);
  const int64_t by =
      std::max<int64_t>(1, std::min<int64_t>(ceil_div(passes, int64_t(1) << lg), kResident / std::max<int64_t>(1, bx)));
  return dim3((unsigned)std::min(bx, most), (unsigned)by);
}

// f(slots) for the smallest compiled number of slots that takes k at once.
template <int SL = 1, typename F>
void with_slots(int64_t k, F&& f) {
  if constexpr (SL == kSlots) f(std::integral_constant<int, SL>{});
  else if (k <= SL) f(std::integral_constant<int, SL>{});
  else with_slots<SL + 1>(k, f);
}

template <typename TY, typename TO>
cudaError_t launch_unpermute(const void* ys, const int32_t* pair_pos, const float* w, const float* shared_out,
                             void* out, int64_t T, int64_t H, int64_t k, cudaStream_t s) {
  const int64_t nvec = H * sizeof(TY) / 16;
  with_slots(k, [&](auto slots) {
    constexpr int SL = decltype(slots)::value, V = vectors_for(SL, sizeof(TY));
    auto launch = [&](auto kernel, int per_thread) {
      const int64_t passes = ceil_div(nvec, per_thread);
      const int lg = lane_log2(passes);
      kernel<<<lane_grid(T, passes, lg, kResident), RTHREADS, 0, s>>>(
          static_cast<const TY*>(ys), pair_pos, w, shared_out, static_cast<TO*>(out), T, (int)H, (int)k, lg);
    };
    if (many(T, nvec, V)) launch(unpermute_rows_kernel<TY, TO, SL, V>, V);
    else launch(unpermute_rows_kernel<TY, TO, SL, 1>, 1);
  });
  return cudaGetLastError();
}

template <typename TY, typename TD>
cudaError_t launch_unpermute_backward(const void* dout, const void* ys, const int32_t* pair_pos,
                                      const int32_t* offsets, const float* w, void* dys, float* dw, int64_t T,
                                      int64_t H, int64_t k, int64_t E, cudaStream_t s) {
  const int64_t nvec = H * sizeof(TY) / 16;
  with_slots(k, [&](auto slots) {
    // half as many where each load is answered by a store
    constexpr int SL = decltype(slots)::value, V = std::max(2, vectors_for(SL, 2) / 2);
    auto launch = [&](auto kernel, int per_thread) {
      // A warp per token, or for short rows less (8 lanes at least: a lane
      // writes each slot's weight gradient); more for few tokens, as long as
      // each thread has a vector.
      const int64_t passes = ceil_div(nvec, per_thread);
      int lt = 5;
      while (lt > 3 && (int64_t(1) << lt) >= 2 * passes) --lt;
      while (lt >= 5 && lt < 8 && (T << lt) < 148 * 2048 && passes > (int64_t(1) << lt)) ++lt;
      const int64_t grid = std::min<int64_t>(ceil_div(T, RTHREADS >> lt), 148 * 8);
      kernel<<<(unsigned)grid, RTHREADS, 0, s>>>(static_cast<const TD*>(dout), static_cast<const TY*>(ys), pair_pos,
                                                 offsets, w, static_cast<TY*>(dys), dw, T, (int)H, (int)k, (int)E, lt);
    };
    if (many(T, nvec, V)) launch(unpermute_rows_backward_kernel<TY, TD, SL, V>, V);
    else launch(unpermute_rows_backward_kernel<TY, TD, SL, 1>, 1);
  });
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
  auto launch = [&](auto kernel, int per_thread) {
    const int64_t passes = ceil_div(nvec, per_thread);
    const int lg = lane_log2(passes);
    // Blocks that end early are replaced as they end, which evens out the stores
    // (8192 x 2048 bf16, k 8: 54 us with resident blocks, 49 so); with k 1 there
    // is nothing to even out (20.7 and 22.7 us of 8192 x 4096).
    const dim3 grid = lane_grid(p->T, passes, lg, p->k == 1 ? kResident : kResident * 64);
    kernel<<<grid, RTHREADS, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
        static_cast<const uint4*>(x), pair_pos, offsets, static_cast<uint4*>(x_perm), p->T, (int)nvec, (int)p->k,
        (int)p->E, lg);
  };
  // each load is followed by k stores: few of those leave the loads' time bare
  if (p->k <= 4 && many(p->T, nvec, 4)) launch(permute_rows_kernel<4>, 4);
  else launch(permute_rows_kernel<1>, 1);
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
