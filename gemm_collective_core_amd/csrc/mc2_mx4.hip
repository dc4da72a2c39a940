// Quantisation to MX4 (blocks of 32 E2M1 values with a shared power of two) and
// back, for gfx950.
//
// All four kernels move bytes and are bound by memory: a value is read once and
// written once, in 8- and 16-byte accesses, and rounded by the conversion
// instructions, which divide by the power of two, round to nearest even and
// clamp at 6 by themselves. A block's largest magnitude is found on the bit
// patterns (they order as the magnitudes do), so that NaN and infinities need
// no case of their own until the exponent is known. Measured: 16384 x 8192 bf16
// 59 us (340 MB, 5.8 TB/s) and back 51 us; 16 matrices of 2048 x 1536 bf16 along
// the other axis 22 us (127 MB, 5.7 TB/s) and back 23 us.
#include "mc2_mx4.hpp"

namespace mc2 {

enum class In { BF16, F16, F32 };
template <In I> constexpr int kSize = I == In::F32 ? 4 : 2;

constexpr int kMxThreads = 256;
constexpr int64_t kMxMaxBlocks = 1 << 20;  // a launch holds fewer than 2^32 threads; more work loops

// Vectors of rows that start at any element.
typedef u32x4_t __attribute__((aligned(2))) u32x4_any_t;
typedef u32x2_t __attribute__((aligned(2))) u32x2_any_t;

// Scale byte of a block from the largest bit pattern (sign cleared) of its values.
template <In I>
__device__ __forceinline__ uint32_t scale_byte(uint32_t top) {
  uint32_t e;  // floor(log2) + 127; 255: NaN or infinity
  if constexpr (I == In::BF16) e = top >> 7;
  else if constexpr (I == In::F16)
    e = top >= 0x7c00u ? 255u : __float_as_uint(f16_bits_to_f32(top)) >> 23;
  else e = top >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// Byte B of a dword of codes from two values (16-bit: one dword of `v`).
template <In I, int B>
__device__ __forceinline__ uint32_t put_pair(uint32_t codes, uint32_t a, uint32_t b, float s) {
  if constexpr (I == In::BF16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, bit_cast<bf16x2_t>(a), s, B);
  else if constexpr (I == In::F16)
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(codes, bit_cast<f16x2_t>(a), s, B);
  else
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, __uint_as_float(a), __uint_as_float(b),
                                                    s, B);
}

__device__ __forceinline__ uint32_t umax32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The larger of `v` over each group of four lanes, in all of them.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = umax32(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 15, 15, true)));
  return umax32(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 15, 15, true)));
}

// Row t / nb for t * nb < 2^31 by a multiplication: mul = ceil(2^31 / nb).
__device__ __forceinline__ uint32_t div_nb(uint32_t t, uint32_t mul) {
  return static_cast<uint32_t>((static_cast<uint64_t>(t) * mul) >> 31);
}
static uint32_t div_mul(int64_t nb) {
  return static_cast<uint32_t>(((int64_t{1} << 31) + nb - 1) / nb);
}

// ------------------------------------------------------------ along the rows
//
// Four lanes share a block, eight values each: a wave reads 1 KiB (2 KiB of
// fp32) and writes 256 bytes of codes, both contiguous, and each thread keeps
// kUnits such pieces in flight. Piece q of the operand is codes dword q.
constexpr int kUnits = 4;

template <In I>
__global__ __launch_bounds__(kMxThreads) void quantize_rows_kernel(
    const char* __restrict__ x, int64_t pieces, int64_t k, uint32_t nb, uint32_t pitch,
    uint32_t mul, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int S = kSize<I>;
  constexpr int ND = 2 * S;  // dwords of eight values
  for (int64_t q0 = static_cast<int64_t>(blockIdx.x) * (kMxThreads * kUnits); q0 < pieces;
       q0 += static_cast<int64_t>(gridDim.x) * (kMxThreads * kUnits)) {
    const int64_t u0 = q0 >> 2, r0 = u0 / nb;
    const uint32_t rem0 = static_cast<uint32_t>(u0 - r0 * nb);
    uint32_t v[kUnits][ND], blk[kUnits];
    int64_t row[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t lq = threadIdx.x + i * kMxThreads;
      const uint32_t t = rem0 + (lq >> 2), rr = div_nb(t, mul);
      blk[i] = t - rr * nb;
      row[i] = r0 + rr;
      const int64_t k0 = blk[i] * 32 + (lq & 3) * 8;
#pragma unroll
      for (int d = 0; d < ND; ++d) v[i][d] = 0;
      if (q0 + lq < pieces) {
        const char* p = x + (row[i] * k + k0) * S;
        if (k0 + 8 <= k) {
#pragma unroll
          for (int d = 0; d < ND; d += 4) {
            const u32x4_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x4_any_t*>(p + 4 * d));
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][d + j] = w[j];
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (k0 + j < k) {
              if constexpr (S == 4) v[i][j] = reinterpret_cast<const uint32_t*>(p)[j];
              else v[i][j / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[j]) << (16 * (j & 1));
            }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t lq = threadIdx.x + i * kMxThreads;
      uint32_t top = 0;
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        if constexpr (S == 4) top = umax32(top, v[i][d] & 0x7fffffffu);
        else top = umax32(top, umax32(v[i][d] & 0x7fffu, (v[i][d] >> 16) & 0x7fffu));
      }
      const uint32_t e = scale_byte<I>(quad_max(top));
      const float s = mx4_scale(e);
      uint32_t c = 0;
      if constexpr (S == 4) {
        c = put_pair<I, 0>(c, v[i][0], v[i][1], s);
        c = put_pair<I, 1>(c, v[i][2], v[i][3], s);
        c = put_pair<I, 2>(c, v[i][4], v[i][5], s);
        c = put_pair<I, 3>(c, v[i][6], v[i][7], s);
      } else {
        c = put_pair<I, 0>(c, v[i][0], 0, s);
        c = put_pair<I, 1>(c, v[i][1], 0, s);
        c = put_pair<I, 2>(c, v[i][2], 0, s);
        c = put_pair<I, 3>(c, v[i][3], 0, s);
      }
      if (q0 + lq < pieces) {
        codes[q0 + lq] = e == 255u ? 0u : c;
        uint8_t* sr = scales + row[i] * pitch + blk[i];
        if ((lq & 3) == 0) *sr = static_cast<uint8_t>(e);
        if (blk[i] == nb - 1)  // the row's scales behind the last block
          for (uint32_t j = nb + (lq & 3); j < pitch; j += 4) sr[j - blk[i]] = 0;
      }
    }
  }
}

template <In O>
__global__ __launch_bounds__(kMxThreads) void dequantize_rows_kernel(
    const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t pieces,
    int64_t k, uint32_t nb, uint32_t pitch, uint32_t mul, char* __restrict__ out) {
  constexpr int S = kSize<O>;
  constexpr int ND = 2 * S;
  for (int64_t q0 = static_cast<int64_t>(blockIdx.x) * (kMxThreads * kUnits); q0 < pieces;
       q0 += static_cast<int64_t>(gridDim.x) * (kMxThreads * kUnits)) {
    const int64_t u0 = q0 >> 2, r0 = u0 / nb;
    const uint32_t rem0 = static_cast<uint32_t>(u0 - r0 * nb);
    uint32_t c[kUnits], e[kUnits], blk[kUnits];
    int64_t row[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t lq = threadIdx.x + i * kMxThreads;
      const uint32_t t = rem0 + (lq >> 2), rr = div_nb(t, mul);
      blk[i] = t - rr * nb;
      row[i] = r0 + rr;
      const bool in = q0 + lq < pieces;
      c[i] = in ? __builtin_nontemporal_load(codes + q0 + lq) : 0u;
      e[i] = in ? scales[row[i] * pitch + blk[i]] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t lq = threadIdx.x + i * kMxThreads;
      const int64_t k0 = blk[i] * 32 + (lq & 3) * 8;
      if (q0 + lq >= pieces || k0 >= k) continue;
      const float s = mx4_scale(e[i]);
      uint32_t v[ND];
      if constexpr (O == In::F32) {
        const f32x2_t p0 = mx4_pair_f32<0>(c[i], s), p1 = mx4_pair_f32<1>(c[i], s);
        const f32x2_t p2 = mx4_pair_f32<2>(c[i], s), p3 = mx4_pair_f32<3>(c[i], s);
        const float f[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __float_as_uint(f[j]);
      } else if constexpr (O == In::BF16) {
        const u32x4_t w = mx4_bf16x8(c[i], s);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = w[j];
      } else {
        v[0] = mx4_pair_f16<0>(c[i], s);
        v[1] = mx4_pair_f16<1>(c[i], s);
        v[2] = mx4_pair_f16<2>(c[i], s);
        v[3] = mx4_pair_f16<3>(c[i], s);
      }
      char* p = out + (row[i] * k + k0) * S;
      if (k0 + 8 <= k) {
#pragma unroll
        for (int d = 0; d < ND; d += 4)
          __builtin_nontemporal_store(u32x4_t{v[d], v[d + 1], v[d + 2], v[d + 3]},
                                      reinterpret_cast<u32x4_any_t*>(p + 4 * d));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (k0 + j < k) {
            if constexpr (S == 4) reinterpret_cast<uint32_t*>(p)[j] = v[j];
            else reinterpret_cast<uint16_t*>(p)[j] = static_cast<uint16_t>(v[j / 2] >> (16 * (j & 1)));
          }
      }
    }
  }
}

// ------------------------------------------------- along the other axis (trans)
//
// A workgroup takes 8 blocks (256 k rows) by 32 * CPL columns, a thread one
// block of CPL neighbouring columns: every access to x is 8 bytes a lane and
// 256 contiguous bytes a row. The blocks change places in LDS, so that the
// codes of a column leave as 128 contiguous bytes. 16-byte unit b of column c
// sits at b ^ (c / CPL & 7): the 32 lanes that write one column each, CPL
// columns apart, spread over all banks.
constexpr int kTB = 8;  // blocks a tile
template <In I> constexpr int kCpl = 8 / kSize<I>;
template <In I> constexpr int kTC = 32 * kCpl<I>;  // columns a tile

template <In I>
__device__ __forceinline__ int tile_unit(int c, int b) {
  return c * kTB + (b ^ ((c / kCpl<I>) & 7));
}

struct TileAt {
  int64_t mat, j0;  // matrix, first column
  int64_t b0;       // first block
};
__device__ __forceinline__ TileAt tile_at(int64_t t, int64_t tn, int64_t tk, int tc) {
  TileAt a;
  const int64_t u = t / tn;
  a.j0 = (t - u * tn) * tc;
  a.mat = u / tk;
  a.b0 = (u - a.mat * tk) * kTB;
  return a;
}

template <In I>
__global__ __launch_bounds__(kMxThreads) void quantize_cols_kernel(
    const char* __restrict__ x, int64_t tiles, int64_t tn, int64_t tk, int64_t n, int64_t k,
    int64_t nb, int64_t pitch, u32x4_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  constexpr int S = kSize<I>, CPL = kCpl<I>, TC = kTC<I>;
  __shared__ u32x4_t s_codes[TC * kTB];
  __shared__ __attribute__((aligned(8))) uint8_t s_sc[TC * kTB];
  const int lane = threadIdx.x & 63;
  const int b = (threadIdx.x >> 6) * 2 + (lane >> 5), cl = (lane & 31) * CPL;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const TileAt a = tile_at(t, tn, tk, TC);
    const int64_t k0 = (a.b0 + b) * 32, j0 = a.j0 + cl;
    u32x2_t v[32];
    const char* p = x + ((a.mat * k + k0) * n + j0) * S;
    const int64_t cols = n - j0;
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      v[r] = u32x2_t{0u, 0u};
      if (k0 + r < k) {
        const char* pr = p + r * n * S;
        if (cols >= CPL) {
          v[r] = __builtin_nontemporal_load(reinterpret_cast<const u32x2_any_t*>(pr));
        } else {
#pragma unroll
          for (int c = 0; c < CPL - 1; ++c)
            if (c < cols) {
              if constexpr (S == 4) v[r][c] = reinterpret_cast<const uint32_t*>(pr)[c];
              else v[r][c / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(pr)[c]) << (16 * (c & 1));
            }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      auto val = [&](int r) -> uint32_t {
        if constexpr (S == 4) return v[r][c];
        else return (v[r][c / 2] >> (16 * (c & 1))) & 0xffffu;
      };
      uint32_t top = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) top = umax32(top, val(r) & (S == 4 ? 0x7fffffffu : 0x7fffu));
      const uint32_t e = scale_byte<I>(top);
      const float s = mx4_scale(e);
      u32x4_t w;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        uint32_t cd = 0;
        auto pair = [&](int i) -> uint32_t {  // rows 8 d + 2 i and the next
          if constexpr (S == 4) return val(8 * d + 2 * i);
          else return __builtin_amdgcn_perm(v[8 * d + 2 * i + 1][c / 2], v[8 * d + 2 * i][c / 2],
                                            (c & 1) ? 0x07060302u : 0x05040100u);
        };
        cd = put_pair<I, 0>(cd, pair(0), val(8 * d + 1), s);
        cd = put_pair<I, 1>(cd, pair(1), val(8 * d + 3), s);
        cd = put_pair<I, 2>(cd, pair(2), val(8 * d + 5), s);
        cd = put_pair<I, 3>(cd, pair(3), val(8 * d + 7), s);
        w[d] = e == 255u ? 0u : cd;
      }
      s_codes[tile_unit<I>(cl + c, b)] = w;
      s_sc[(cl + c) * kTB + b] = a.b0 + b < nb ? static_cast<uint8_t>(e) : 0;
    }
    __syncthreads();
    const int64_t orow0 = a.mat * n + a.j0;
#pragma unroll
    for (int i = threadIdx.x; i < TC * kTB; i += kMxThreads) {
      const int c = i / kTB, bb = i % kTB;
      if (a.j0 + c < n && a.b0 + bb < nb)
        codes[(orow0 + c) * nb + a.b0 + bb] = s_codes[tile_unit<I>(c, bb)];
    }
    if (threadIdx.x < TC && a.j0 + threadIdx.x < n) {
      const int c = threadIdx.x;
      uint8_t* sr = scales + (orow0 + c) * pitch + a.b0;
      *reinterpret_cast<u32x2_t*>(sr) = *reinterpret_cast<const u32x2_t*>(s_sc + c * kTB);
      // the scales behind the last tile's blocks
      if (a.b0 + kTB >= nb && a.b0 + kTB < pitch) *reinterpret_cast<u32x2_t*>(sr + kTB) = u32x2_t{0u, 0u};
    }
    __syncthreads();
  }
}

template <In O>
__global__ __launch_bounds__(kMxThreads) void dequantize_cols_kernel(
    const u32x4_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t tiles,
    int64_t tn, int64_t tk, int64_t n, int64_t k, int64_t nb, int64_t pitch,
    char* __restrict__ out) {
  constexpr int S = kSize<O>, CPL = kCpl<O>, TC = kTC<O>;
  __shared__ u32x4_t s_codes[TC * kTB];
  __shared__ __attribute__((aligned(8))) uint8_t s_sc[TC * kTB];
  const int lane = threadIdx.x & 63;
  const int b = (threadIdx.x >> 6) * 2 + (lane >> 5), cl = (lane & 31) * CPL;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x) {
    const TileAt a = tile_at(t, tn, tk, TC);
    const int64_t orow0 = a.mat * n + a.j0;
#pragma unroll
    for (int i = threadIdx.x; i < TC * kTB; i += kMxThreads) {
      const int c = i / kTB, bb = i % kTB;
      if (a.j0 + c < n && a.b0 + bb < nb)
        s_codes[tile_unit<O>(c, bb)] =
            __builtin_nontemporal_load(codes + (orow0 + c) * nb + a.b0 + bb);
    }
    if (threadIdx.x < TC && a.j0 + threadIdx.x < n) {
      const int c = threadIdx.x;
      *reinterpret_cast<u32x2_t*>(s_sc + c * kTB) =
          *reinterpret_cast<const u32x2_t*>(scales + (orow0 + c) * pitch + a.b0);
    }
    __syncthreads();
    const int64_t k0 = (a.b0 + b) * 32, j0 = a.j0 + cl, cols = n - j0;
    if (k0 < k && cols > 0) {
      u32x4_t w[CPL];
      float s[CPL];
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        w[c] = s_codes[tile_unit<O>(cl + c, b)];
        s[c] = mx4_scale(s_sc[(cl + c) * kTB + b]);
      }
      char* p = out + ((a.mat * k + k0) * n + j0) * S;
      auto put = [&](int r, u32x2_t d) {
        if (k0 + r >= k) return;
        char* pr = p + r * n * S;
        if (cols >= CPL) {
          __builtin_nontemporal_store(d, reinterpret_cast<u32x2_any_t*>(pr));
        } else {
#pragma unroll
          for (int c = 0; c < CPL - 1; ++c)
            if (c < cols) {
              if constexpr (S == 4) reinterpret_cast<uint32_t*>(pr)[c] = d[c];
              else reinterpret_cast<uint16_t*>(pr)[c] = static_cast<uint16_t>(d[c / 2] >> (16 * (c & 1)));
            }
        }
      };
      // byte B of dword d of every column: rows 8 d + 2 B and the next
      auto two_rows = [&](int d, auto Bc) {
        constexpr int B = decltype(Bc)::value;
        const int r = 8 * d + 2 * B;
        if constexpr (O == In::F32) {
          const f32x2_t x0 = mx4_pair_f32<B>(w[0][d], s[0]), x1 = mx4_pair_f32<B>(w[1][d], s[1]);
          put(r, u32x2_t{__float_as_uint(x0.x), __float_as_uint(x1.x)});
          put(r + 1, u32x2_t{__float_as_uint(x0.y), __float_as_uint(x1.y)});
        } else {
          uint32_t y[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            y[c] = O == In::BF16 ? mx4_pair_bf16<B>(w[c][d], s[c]) : mx4_pair_f16<B>(w[c][d], s[c]);
          put(r, u32x2_t{__builtin_amdgcn_perm(y[1], y[0], 0x05040100u),
                         __builtin_amdgcn_perm(y[3], y[2], 0x05040100u)});
          put(r + 1, u32x2_t{__builtin_amdgcn_perm(y[1], y[0], 0x07060302u),
                             __builtin_amdgcn_perm(y[3], y[2], 0x07060302u)});
        }
      };
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        two_rows(d, std::integral_constant<int, 0>{});
        two_rows(d, std::integral_constant<int, 1>{});
        two_rows(d, std::integral_constant<int, 2>{});
        two_rows(d, std::integral_constant<int, 3>{});
      }
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side

static int check_operand(int64_t batch, int64_t rows, int64_t k, int dtype) {
  if (dtype != MC2_BF16 && dtype != MC2_F16 && dtype != MC2_F32) return MC2_ERR_DTYPE;
  constexpr int64_t kMost = int64_t{1} << 36;
  if (batch < 1 || rows < 1 || k < 1 || k > MC2_MX4_MAX_K) return MC2_ERR_SHAPE;
  if (batch > kMost || rows > kMost / batch) return MC2_ERR_SHAPE;
  return MC2_OK;
}

template <class F>
static void for_type(int dtype, F&& f) {
  if (dtype == MC2_BF16) f(std::integral_constant<In, In::BF16>{});
  else if (dtype == MC2_F16) f(std::integral_constant<In, In::F16>{});
  else f(std::integral_constant<In, In::F32>{});
}

static unsigned grid_of(int64_t work, int64_t per) {
  const int64_t g = (work + per - 1) / per;
  return static_cast<unsigned>(g < kMxMaxBlocks ? g : kMxMaxBlocks);
}

}  // namespace mc2

using namespace mc2;

extern "C" size_t mc2_mx4_row_bytes(int64_t k) {
  return k < 1 || k > MC2_MX4_MAX_K ? 0 : static_cast<size_t>(16 * mx4_blocks(k));
}

extern "C" size_t mc2_mx4_scale_bytes(int64_t k) {
  return k < 1 || k > MC2_MX4_MAX_K ? 0 : static_cast<size_t>(mx4_pitch(k));
}

extern "C" int mc2_mx4_quantize(const void* x, int64_t batch, int64_t rows, int64_t k, int trans,
                                int in_dtype, void* codes, void* scales, hipStream_t stream) {
  if (!x || !codes || !scales) return MC2_ERR_NULL;
  const int st = check_operand(batch, rows, k, in_dtype);
  if (st) return st;
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales)) return MC2_ERR_ALIGN;
  const int64_t nb = mx4_blocks(k), pitch = mx4_pitch(k);
  for_type(in_dtype, [&](auto type) {
    constexpr In I = decltype(type)::value;
    if (trans) {
      const int64_t tn = (rows + kTC<I> - 1) / kTC<I>, tk = (nb + kTB - 1) / kTB;
      hipLaunchKernelGGL((quantize_cols_kernel<I>), dim3(grid_of(batch * tn * tk, 1)),
                         dim3(kMxThreads), 0, stream, static_cast<const char*>(x), batch * tn * tk,
                         tn, tk, rows, k, nb, pitch, static_cast<u32x4_t*>(codes),
                         static_cast<uint8_t*>(scales));
    } else {
      const int64_t pieces = batch * rows * nb * 4;
      hipLaunchKernelGGL((quantize_rows_kernel<I>), dim3(grid_of(pieces, kMxThreads * kUnits)),
                         dim3(kMxThreads), 0, stream, static_cast<const char*>(x), pieces, k,
                         static_cast<uint32_t>(nb), static_cast<uint32_t>(pitch), div_mul(nb),
                         static_cast<uint32_t*>(codes), static_cast<uint8_t*>(scales));
    }
  });
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}

extern "C" int mc2_mx4_dequantize(const void* codes, const void* scales, int64_t batch,
                                  int64_t rows, int64_t k, int trans, int out_dtype, void* out,
                                  hipStream_t stream) {
  if (!codes || !scales || !out) return MC2_ERR_NULL;
  const int st = check_operand(batch, rows, k, out_dtype);
  if (st) return st;
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out)) return MC2_ERR_ALIGN;
  const int64_t nb = mx4_blocks(k), pitch = mx4_pitch(k);
  for_type(out_dtype, [&](auto type) {
    constexpr In O = decltype(type)::value;
    if (trans) {
      const int64_t tn = (rows + kTC<O> - 1) / kTC<O>, tk = (nb + kTB - 1) / kTB;
      hipLaunchKernelGGL((dequantize_cols_kernel<O>), dim3(grid_of(batch * tn * tk, 1)),
                         dim3(kMxThreads), 0, stream, static_cast<const u32x4_t*>(codes),
                         static_cast<const uint8_t*>(scales), batch * tn * tk, tn, tk, rows, k, nb,
                         pitch, static_cast<char*>(out));
    } else {
      const int64_t pieces = batch * rows * nb * 4;
      hipLaunchKernelGGL((dequantize_rows_kernel<O>), dim3(grid_of(pieces, kMxThreads * kUnits)),
                         dim3(kMxThreads), 0, stream, static_cast<const uint32_t*>(codes),
                         static_cast<const uint8_t*>(scales), pieces, k, static_cast<uint32_t>(nb),
                         static_cast<uint32_t>(pitch), div_mul(nb), static_cast<char*>(out));
    }
  });
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}
