// Gradients of the two ends of the MoE expert-parallel local path: of the
// weighted unpermute and of the permute (mc2_moe.hip), for gfx950.
//
// Both move bytes: they are written for coalesced 16-byte accesses and for
// reading and writing each routed row once.
#include <type_traits>

#include "../../include/mc2_train.h"
#include "mc2_common.hpp"
#include "mc2_host.hpp"

namespace mc2 {

constexpr int kBwdThreads = 256;

template <bool F16>
__device__ __forceinline__ float in16(uint32_t bits) {
  if constexpr (F16) return f16_bits_to_f32(bits);
  else return bf16_bits_to_f32(bits);
}
template <bool F16>
__device__ __forceinline__ uint32_t out16x2(float a, float b) {
  if constexpr (F16) return f32_to_f16_bits(a) | (static_cast<uint32_t>(f32_to_f16_bits(b)) << 16);
  else return f32_to_bf16_bits(a) | (static_cast<uint32_t>(f32_to_bf16_bits(b)) << 16);
}

// Value of `v` in lane `kk` of each group of LPR lanes; a scalar where the
// group is the whole wave, so that row addresses are wave-uniform.
template <int LPR>
__device__ __forceinline__ int group_lane(int v, int kk) {
  if constexpr (LPR == 64) return __builtin_amdgcn_readlane(v, kk);
  else return __shfl(v, kk, LPR);
}

// A group of LPR lanes owns one token: its lanes own 16-byte column chunks, C
// per lane in a pass of LPR * C chunks. Rows of up to 512 elements use the
// smallest group that covers them, so that no lane idles; wider ones use the
// whole wave with C = 4 (one pass for H <= 2048).
//
// Sum over the H products of a slot: the lanes' partial sums of a group's 8
// slots are exchanged so that lane l ends with slot l & 7 (4 + 2 + 1 values
// instead of 8 each in the first three steps), then added over the rest of
// the group.
template <int LPR>
__device__ __forceinline__ float reduce_slots(float (&s)[8], int lane) {
  float q[4], r[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float mine = (lane & 4) ? s[4 + i] : s[i];
    const float other = (lane & 4) ? s[i] : s[4 + i];
    q[i] = mine + __shfl_xor(other, 4);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float mine = (lane & 2) ? q[2 + i] : q[i];
    const float other = (lane & 2) ? q[i] : q[2 + i];
    r[i] = mine + __shfl_xor(other, 2);
  }
  float v = ((lane & 1) ? r[1] : r[0]) + __shfl_xor((lane & 1) ? r[0] : r[1], 1);
#pragma unroll
  for (int off = 8; off < LPR; off <<= 1) v += __shfl_xor(v, off);
  return v;
}

// The index of slot s, or -1 where it is to be skipped; ok: its row is its own.
__device__ __forceinline__ int slot_row(const int32_t* __restrict__ idx,
                                        const int32_t* __restrict__ sorted, int64_t s,
                                        int64_t p_end, bool& ok, bool& bad) {
  int p = idx[s];
  ok = false;
  if (p < -1 || p >= p_end) {
    bad = true;
    p = -1;
  }
  if (p >= 0) {
    ok = sorted[p] == static_cast<int32_t>(s);
    bad |= !ok;
  }
  return p;
}

// dprobs[s] = <dout[t], y[idx[s]]>. The indices of 8 slots are loaded by the
// group's first 8 lanes and broadcast; the 8 rows' loads of a pass are all
// issued before any is used, and do not wait for the check against sorted_idx
// (the row lies inside y whatever that says; the check decides what is stored).
template <bool F16, int LPR, int C>
__device__ __forceinline__ bool probs_grad(const uint16_t* __restrict__ dout,
                                           const uint16_t* __restrict__ y, int64_t p_end,
                                           const int32_t* __restrict__ idx,
                                           const int32_t* __restrict__ sorted, int64_t t, int K,
                                           int64_t H, float* __restrict__ dprobs) {
  const int gl = threadIdx.x & (LPR - 1);
  const int64_t CR = H / 8;
  const u32x4_t* drow = reinterpret_cast<const u32x4_t*>(dout + t * H);
  bool bad = false;
  for (int k0 = 0; k0 < K; k0 += 8) {
    const int64_t s_l = t * K + k0 + gl;
    const bool mine = gl < 8 && k0 + gl < K;
    bool ok = false;
    const int p_l = mine ? slot_row(idx, sorted, s_l, p_end, ok, bad) : -1;
    float sum[8];
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) sum[kk] = 0.f;
    for (int64_t base = 0; base < CR; base += LPR * C) {
      u32x4_t d[C], v[8][C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t j = base + c * LPR + gl;
        d[c] = j < CR ? drow[j] : zero_v4();
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int p = group_lane<LPR>(p_l, kk);
        const u32x4_t* row = reinterpret_cast<const u32x4_t*>(y + (int64_t)(p < 0 ? 0 : p) * H);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int64_t j = base + c * LPR + gl;
          v[kk][c] = (p >= 0 && j < CR) ? __builtin_nontemporal_load(row + j) : zero_v4();
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float d0 = in16<F16>(d[c][q] & 0xFFFFu), d1 = in16<F16>(d[c][q] >> 16);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            sum[kk] = __builtin_fmaf(d0, in16<F16>(v[kk][c][q] & 0xFFFFu), sum[kk]);
            sum[kk] = __builtin_fmaf(d1, in16<F16>(v[kk][c][q] >> 16), sum[kk]);
          }
        }
    }
    const float r = reduce_slots<LPR>(sum, threadIdx.x & 63);
    if (mine) dprobs[s_l] = ok ? r : 0.f;
  }
  return bad;
}

// dy[idx[s]] = probs[s] * dout[t]: each row written once, non-temporal.
template <bool F16, int LPR, int C>
__device__ __forceinline__ bool rows_grad(const uint16_t* __restrict__ dout, int64_t p_end,
                                          const int32_t* __restrict__ idx,
                                          const int32_t* __restrict__ sorted,
                                          const float* __restrict__ probs, int64_t t, int K,
                                          int64_t H, uint16_t* __restrict__ dy) {
  const int gl = threadIdx.x & (LPR - 1);
  const int64_t CR = H / 8;
  const u32x4_t* drow = reinterpret_cast<const u32x4_t*>(dout + t * H);
  bool bad = false;
  for (int k0 = 0; k0 < K; k0 += 8) {
    const int64_t s_l = t * K + k0 + gl;
    bool ok = false;
    int p_l = -1;
    float w_l = 0.f;
    if (gl < 8 && k0 + gl < K) {
      w_l = probs[s_l];
      p_l = slot_row(idx, sorted, s_l, p_end, ok, bad);
      if (!ok) p_l = -1;
    }
    for (int64_t base = 0; base < CR; base += LPR * C) {
      float df[C][8];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t j = base + c * LPR + gl;
        const u32x4_t d = j < CR ? drow[j] : zero_v4();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          df[c][2 * q] = in16<F16>(d[q] & 0xFFFFu);
          df[c][2 * q + 1] = in16<F16>(d[q] >> 16);
        }
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int p = group_lane<LPR>(p_l, kk);
        const float w =
            __builtin_bit_cast(float, group_lane<LPR>(__builtin_bit_cast(int, w_l), kk));
        u32x4_t* row = reinterpret_cast<u32x4_t*>(dy + (int64_t)(p < 0 ? 0 : p) * H);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int64_t j = base + c * LPR + gl;
          if (p >= 0 && j < CR) {
            u32x4_t o;
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = out16x2<F16>(w * df[c][2 * q], w * df[c][2 * q + 1]);
            __builtin_nontemporal_store(o, row + j);
          }
        }
      }
    }
  }
  return bad;
}

// The first `readers` workgroups compute dprobs, the others dy: memory then
// sees mostly reads and, behind them, mostly writes, which is faster than both
// at once although dout is read twice (32768 tokens, top-8, 2048 wide: 371
// against 429 us, where dprobs alone takes 171 and dy alone 207; from 900 tokens
// of 256 up it never lost). Bound by HBM: 2.42 GB in 371 us, 6.5 TB/s counting dout twice.
template <bool F16, int LPR, int C>
__global__ __launch_bounds__(kBwdThreads) void unpermute_bwd_kernel(
    const uint16_t* __restrict__ dout, const uint16_t* __restrict__ y, int64_t p_end,
    const int32_t* __restrict__ idx, const int32_t* __restrict__ sorted,
    const float* __restrict__ probs, int64_t t0, int64_t T, int K, int64_t H,
    uint16_t* __restrict__ dy, float* __restrict__ dprobs, uint32_t readers, int32_t* dev_err) {
  const bool reads = blockIdx.x < readers;
  const int64_t blk = reads ? blockIdx.x : blockIdx.x - readers;
  const int64_t t = t0 + blk * (kBwdThreads / LPR) + threadIdx.x / LPR;
  if (t >= T) return;
  const bool bad = reads ? probs_grad<F16, LPR, C>(dout, y, p_end, idx, sorted, t, K, H, dprobs)
                         : rows_grad<F16, LPR, C>(dout, p_end, idx, sorted, probs, t, K, H, dy);
  if (bad) atomic_or_err(dev_err, MC2_DEVERR_INDEX);
}

// dx[t] = sum_k g[idx[t*K + k]], in fp32 with k ascending: the unpermute's
// gather without weights.
template <bool F16, int LPR, int C>
__global__ __launch_bounds__(kBwdThreads) void permute_bwd_kernel(
    const uint16_t* __restrict__ g, int64_t rows, const int32_t* __restrict__ idx, int64_t t0,
    int64_t T, int K, int64_t H, uint16_t* __restrict__ dx, int32_t* dev_err) {
  const int gl = threadIdx.x & (LPR - 1);
  const int64_t t = t0 + (int64_t)blockIdx.x * (kBwdThreads / LPR) + threadIdx.x / LPR;
  if (t >= T) return;
  const int64_t CR = H / 8;
  bool bad = false;
  for (int64_t base = 0; base < CR; base += LPR * C) {
    float acc[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[c][i] = 0.f;
    for (int k0 = 0; k0 < K; k0 += 8) {
      int p_l = -1;
      if (gl < 8 && k0 + gl < K) {
        p_l = idx[t * K + k0 + gl];
        if (p_l < -1 || p_l >= rows) {
          bad = true;
          p_l = -1;
        }
      }
      u32x4_t v[8][C];
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int p = group_lane<LPR>(p_l, kk);
        const u32x4_t* row = reinterpret_cast<const u32x4_t*>(g + (int64_t)(p < 0 ? 0 : p) * H);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int64_t j = base + c * LPR + gl;
          v[kk][c] = (p >= 0 && j < CR) ? __builtin_nontemporal_load(row + j) : zero_v4();
        }
      }
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[c][2 * q] += in16<F16>(v[kk][c][q] & 0xFFFFu);
            acc[c][2 * q + 1] += in16<F16>(v[kk][c][q] >> 16);
          }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t j = base + c * LPR + gl;
      if (j < CR) {
        u32x4_t o;
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = out16x2<F16>(acc[c][2 * q], acc[c][2 * q + 1]);
        __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>(dx + t * H) + j);
      }
    }
  }
  if (bad) atomic_or_err(dev_err, MC2_DEVERR_INDEX);
}

// Calls f(F16, LPR, C) as compile-time constants for a dtype and row width.
template <class F>
static void for_rows(int dtype, int64_t H, F&& f) {
  auto with = [&](auto half) {
    const int64_t chunks = H / 8;
    using I8 = std::integral_constant<int, 8>;
    using I16 = std::integral_constant<int, 16>;
    using I32 = std::integral_constant<int, 32>;
    using I64 = std::integral_constant<int, 64>;
    using C1 = std::integral_constant<int, 1>;
    using C4 = std::integral_constant<int, 4>;
    if (chunks <= 8) f(half, I8{}, C1{});
    else if (chunks <= 16) f(half, I16{}, C1{});
    else if (chunks <= 32) f(half, I32{}, C1{});
    else if (chunks <= 64) f(half, I64{}, C1{});
    else f(half, I64{}, C4{});
  };
  if (dtype == MC2_F16) with(std::true_type{});
  else with(std::false_type{});
}

// Calls f(t0, workgroups) for token ranges that cover T tokens, `per` of them a
// workgroup: a launch holds fewer than 2^32 threads, 2^31 are taken with up to
// two workgroups for the same tokens.
constexpr int64_t kMaxRangeBlocks = (int64_t{1} << 30) / kBwdThreads;
template <class F>
static void for_ranges(int64_t T, int per, F&& f) {
  for (int64_t t0 = 0; t0 < T; t0 += kMaxRangeBlocks * per) {
    const int64_t blocks = (T - t0 + per - 1) / per;
    f(t0, static_cast<unsigned>(blocks < kMaxRangeBlocks ? blocks : kMaxRangeBlocks));
  }
}

static int check_rows(int64_t T, int K, int64_t H, int64_t rows, int dtype) {
  if (dtype != MC2_BF16 && dtype != MC2_F16) return MC2_ERR_DTYPE;
  if (T < 1 || K < 1 || K > 64 || H < 8 || rows < 0) return MC2_ERR_SHAPE;
  if (T >= (int64_t)0x7fffffff || T * K >= (int64_t)0x7fffffff) return MC2_ERR_SHAPE;
  return H % 8 ? MC2_ERR_ALIGN : MC2_OK;
}

}  // namespace mc2

using namespace mc2;

extern "C" int mc2_moe_unpermute_backward(const void* dout, const void* y_full, int64_t y_rows,
                                          const int32_t* unpermute_idx, const int32_t* sorted_idx,
                                          const float* probs, int64_t T, int K, int64_t H,
                                          int dtype, void* dy, float* dprobs, int32_t* dev_err,
                                          hipStream_t stream) {
  if (!dout || !unpermute_idx || !sorted_idx || (!dy && !dprobs)) return MC2_ERR_NULL;
  if ((dy && !probs) || (dprobs && !y_full)) return MC2_ERR_NULL;
  const int st = check_rows(T, K, H, y_rows, dtype);
  if (st) return st;
  if (!aligned16(dout) || (dprobs && !aligned16(y_full)) || !aligned16(dy)) return MC2_ERR_ALIGN;
  const int64_t p_end = y_rows < T * K ? y_rows : T * K;
  for_rows(dtype, H, [&](auto half, auto lpr, auto c) {
    constexpr int LPR = decltype(lpr)::value;
    for_ranges(T, kBwdThreads / LPR, [&](int64_t t0, unsigned grid) {
      const unsigned readers = dprobs ? grid : 0u;
      hipLaunchKernelGGL((unpermute_bwd_kernel<decltype(half)::value, LPR, decltype(c)::value>),
                         dim3(readers + (dy ? grid : 0u)), dim3(kBwdThreads), 0, stream,
                         static_cast<const uint16_t*>(dout),
                         static_cast<const uint16_t*>(y_full), p_end, unpermute_idx, sorted_idx,
                         probs, t0, T, K, H, static_cast<uint16_t*>(dy), dprobs, readers, dev_err);
    });
  });
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}

extern "C" int mc2_moe_permute_backward(const void* dpermuted, int64_t rows,
                                        const int32_t* unpermute_idx, int64_t T, int K, int64_t H,
                                        int dtype, void* dx, int32_t* dev_err,
                                        hipStream_t stream) {
  if ((!dpermuted && rows != 0) || !unpermute_idx || !dx) return MC2_ERR_NULL;
  const int st = check_rows(T, K, H, rows, dtype);
  if (st) return st;
  if (!aligned16(dpermuted) || !aligned16(dx)) return MC2_ERR_ALIGN;
  for_rows(dtype, H, [&](auto half, auto lpr, auto c) {
    constexpr int LPR = decltype(lpr)::value;
    for_ranges(T, kBwdThreads / LPR, [&](int64_t t0, unsigned grid) {
      hipLaunchKernelGGL((permute_bwd_kernel<decltype(half)::value, LPR, decltype(c)::value>),
                         dim3(grid), dim3(kBwdThreads), 0, stream,
                         static_cast<const uint16_t*>(dpermuted), rows, unpermute_idx, t0, T, K, H,
                         static_cast<uint16_t*>(dx), dev_err);
    });
  });
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}
