// Orthogonalisation of a stack of matrices by Newton-Schulz products, gfx950.
//
//   X_0 = G / (|G|_F + eps);   X <- a X + (b A + c A^2) X,  A = X X^T
//
// on the smaller side (r = min(m, n), c = max(m, n)). The iterate is kept
// tall, Y = X^T for a wide G: (cp, rp), rows of rp values, both padded with
// zeros to multiples of 64. Then
//   A  = Y^T Y                 contraction over the rows of Y (k-major reads)
//   Q~ = a I + b A + c A A     A is symmetric: both operands are its rows
//   Y' = Y Q~                  Q~ is symmetric: Y's rows by its rows
// and the last step writes out = scale * Y Q~ (G tall) or scale * Q~ Y^T (G
// wide: the same two operands the other way round).
//
// Number formats. The products run on the fp16 matrix instructions with fp32
// accumulation: fp16 and bf16 run at the same rate and fp16 has three bits
// more (errors of the result 1e-3 instead of 1e-2). Powers of two keep the
// values in its range: Y is stored times 2^12 (entries up to 16), A and Q~
// times 2^9 (entries up to 128). Rounding Y to fp16 alone would not do: noise
// in a direction whose singular value is near zero (a gradient of fewer rows
// than the matrix has) grows by the factor a in every step, 484 times in five
// steps, and reached 1.5e-1 of the result. So Y is held as hi + lo, two fp16 (lo
// times 2^11 more): the products use hi,
//   Y' = hi Q~ + a lo,  Q~ = a I + b A + c A A,
// and errors are 4e-4 to 2.7e-3 whatever the rank, where roundings average out;
// few or equal singular values make them systematic (9e-3 for I, up to 3.5e-2).
// The last step leaves lo out, since what it loses is not multiplied again.
#include "../../include/mc2_train.h"
#include "mc2_tiles.hpp"

namespace mc2 {

constexpr int kNsThreads = 256;
constexpr int kNsPad = 64;        // rp and cp are multiples of one K stage
constexpr int kNsMaxPart = 256;   // partial sums of squares per matrix
constexpr float kXScale = 4096.f;             // stored Y = value * 2^12
constexpr float kLoScale = 2048.f;            // stored lo = rest * 2^11
constexpr float kGramScale = 0x1p-15f;        // 2^24 (Y * Y) -> 2^9
constexpr float kSqScale = 0x1p-9f;           // 2^18 (A * A) -> 2^9
constexpr float kUpdScale = 0x1p-9f;          // 2^21 (Y * Q) -> 2^12
constexpr float kOutScale = 0x1p-21f;         // 2^21 (Y * Q) -> 1
constexpr float kDiag = 512.f;                // 1 in Q's scale

template <int D>
__device__ __forceinline__ float ns_load(const void* p, int64_t i) {
  if constexpr (D == MC2_F32) return static_cast<const float*>(p)[i];
  else if constexpr (D == MC2_BF16) return bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
  else return f16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// 16 bytes at any element's address (rows of odd length start anywhere; such an
// access is one load or store here, not split)
typedef f32x4_t __attribute__((aligned(4))) f32x4_any_t;
typedef u32x4_t __attribute__((aligned(2))) u32x4_any_t;

// Eight consecutive values.
template <int D>
__device__ __forceinline__ void ns_load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (D == MC2_F32) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const f32x4_t a = *reinterpret_cast<const f32x4_any_t*>(static_cast<const float*>(p) + i + 4 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * h + j] = a[j];
    }
  } else {
    const u32x4_t q = *reinterpret_cast<const u32x4_any_t*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = D == MC2_BF16 ? bf16_bits_to_f32(q[j] & 0xFFFFu) : f16_bits_to_f32(q[j] & 0xFFFFu);
      v[2 * j + 1] = D == MC2_BF16 ? bf16_bits_to_f32(q[j] >> 16) : f16_bits_to_f32(q[j] >> 16);
    }
  }
}
// The same from row `row`, column `col` of a matrix of m rows of n values:
// zeros outside.
template <int D>
__device__ __forceinline__ void ns_load_in(const void* g, int64_t base, int64_t m, int64_t n,
                                           int64_t row, int64_t col, float (&v)[8]) {
  if (row < m && col + 8 <= n) {
    ns_load8<D>(g, base + row * n + col, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = row < m && col + j < n ? ns_load<D>(g, base + row * n + col + j) : 0.f;
  }
}

// Sum over the workgroup, the same in every thread; the order is fixed.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s_w[kNsThreads / 64];
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) v += __shfl_xor(v, off);
  if ((threadIdx.x & 63) == 0) s_w[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = 0;
#pragma unroll
  for (int w = 0; w < kNsThreads / 64; ++w) t += s_w[w];
  return t;
}

// part[b][i]: sums of squares, in double (gradients of 1e-30 or 1e30 neither
// vanish nor overflow). 16 values per thread in flight.
template <int D>
__global__ __launch_bounds__(kNsThreads) void ns_norm_kernel(const void* __restrict__ g, int64_t mn,
                                                             double* __restrict__ part) {
  const int nb = gridDim.x, b = blockIdx.y;
  const int64_t base = (int64_t)b * mn;
  const int64_t t = (int64_t)blockIdx.x * kNsThreads + threadIdx.x, step = (int64_t)nb * kNsThreads * 8;
  double s = 0;
  for (int64_t i = t * 8; i < mn; i += 2 * step) {
    float v[2][8];
    const bool two = i + step < mn;
    ns_load_in<D>(g, base, 1, mn, 0, i, v[0]);
    if (two) ns_load_in<D>(g, base, 1, mn, 0, i + step, v[1]);
#pragma unroll
    for (int j = 0; j < 8; ++j) s = __builtin_fma((double)v[0][j], (double)v[0][j], s);
    if (two)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fma((double)v[1][j], (double)v[1][j], s);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[(int64_t)b * nb + blockIdx.x] = s;
}

// x (in Y's scale) -> its two fp16 halves
__device__ __forceinline__ void ns_split(float x, uint32_t& hi, uint32_t& lo) {
  hi = f32_to_f16_bits(x);
  lo = f32_to_f16_bits((x - f16_bits_to_f32(hi)) * kLoScale);
}

// lo is kept in the order in which the update's lanes hold it, so that it moves
// in whole 512-byte pieces straight between registers and memory: by W x W tile,
// wave (2 x 2), 16 x 16 block, lane, each lane's 8 bytes holding four consecutive
// columns of one row. Index of the 8 bytes of (row, col), col a multiple of 4.
__device__ __forceinline__ int64_t ns_lo_place(int row, int col, int w, int tiles_n) {
  const int h = w / 2, f = w / 32;
  const int tile = (row / w) * tiles_n + col / w;
  const int in_r = row % w, in_c = col % w;
  const int wave = (in_r / h) * 2 + in_c / h;
  const int blk = (in_r % h) / 16 * f + (in_c % h) / 16;
  return ((int64_t)(tile * 4 + wave) * (f * f) + blk) * 64 + (row & 15) + ((col >> 2) & 3) * 16;
}

// One 64 x 64 tile of Y = G / (|G| + eps), transposed for a wide G, with zeros
// beyond G: read in whole pieces of G's rows into LDS, then hi written in whole
// 128-byte lines and lo in the update's lane order. Bound by HBM (16 x 2048 x
// 1536: 403 MB).
template <int D, bool TALL>
__global__ __launch_bounds__(kNsThreads) void ns_init_kernel(
    const void* __restrict__ g, int64_t m, int64_t n, const double* __restrict__ part, int nb,
    float eps, int64_t cp, int64_t rp, uint16_t* __restrict__ yhi, u32x2_t* __restrict__ ylo,
    int64_t lo_size, int w, int tiles_n) {
  __shared__ float s_t[64][65];
  const int b = blockIdx.y, tid = threadIdx.x;
  const int tc = static_cast<int>(rp / 64);
  const int64_t y0 = (int64_t)(blockIdx.x / tc) * 64, x0 = (int64_t)(blockIdx.x % tc) * 64;
  const int64_t gr0 = TALL ? y0 : x0, gc0 = TALL ? x0 : y0;  // the tile in G
  float u[2][8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = tid + h * kNsThreads;
    ns_load_in<D>(g, (int64_t)b * m * n, m, n, gr0 + (i >> 3), gc0 + (i & 7) * 8, u[h]);
  }
  const double norm2 = block_sum(tid < nb ? part[(int64_t)b * nb + tid] : 0.0);
  // a matrix of zeros stays one, also with eps = 0; in fp64 where fp32 does not
  // hold 1 / norm
  const double inv = norm2 == 0.0 ? 0.0 : kXScale / (sqrt(norm2) + static_cast<double>(eps));
  const float invf = static_cast<float>(inv);
  const bool fits = invf > 1e-30f && invf < 1e30f;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = tid + h * kNsThreads, r = i >> 3, c = (i & 7) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = fits ? u[h][j] * invf : static_cast<float>(static_cast<double>(u[h][j]) * inv);
      // (inv may be NaN: what lies beyond G stays zero)
      s_t[r][c + j] = gr0 + r < m && gc0 + c + j < n ? x : 0.f;
    }
  }
  __syncthreads();
  auto at = [&](int r, int c) { return TALL ? s_t[r][c] : s_t[c][r]; };
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = tid + h * kNsThreads, r = i >> 3, c = (i & 7) * 8;
    u32x4_t v;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = f32_to_f16_bits(at(r, c + 2 * j)) |
             (static_cast<uint32_t>(f32_to_f16_bits(at(r, c + 2 * j + 1))) << 16);
    *reinterpret_cast<u32x4_t*>(yhi + (int64_t)b * cp * rp + (y0 + r) * rp + x0 + c) = v;
  }
  // a wave takes one 16 x 16 block at a time, its lanes as the update's
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int blk = (tid >> 6) * 4 + k, l = tid & 63;
    const int r = (blk >> 2) * 16 + (l & 15), c = (blk & 3) * 16 + (l >> 4) * 4;
    uint32_t h, q[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) ns_split(at(r, c + j), h, q[j]);
    ylo[b * lo_size + ns_lo_place(static_cast<int>(y0) + r, static_cast<int>(x0) + c, w, tiles_n)] =
        u32x2_t{q[0] | (q[1] << 16), q[2] | (q[3] << 16)};
  }
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

typedef short s16x4_t __attribute__((ext_vector_type(4)));

enum NsMode : int { kGram = 0, kSquare = 1, kUpdate = 2, kOutTall = 3, kOutWide = 4 };

struct NsArgs {
  const uint16_t* y;   // (B, cp, rp) hi
  u32x2_t* ylo;        // lo of each matrix in the order of ns_lo_place, updated in place
  int64_t lo_size;     // places of it per matrix
  uint16_t* ynext;     // (B, cp, rp) hi of the next step
  uint16_t* gram;      // (B, rp, rp) A
  uint16_t* q;         // (B, rp, rp) Q~
  uint16_t* out;       // (B, m, n)
  int cp, rp;
  int om, on;          // m, n: rows and columns of the output
  int tiles_m, tiles_n, tiles;  // tiles per matrix (symmetric products: the upper triangle)
  int row_tiles;                // tiles per row in ns_tile's order
  float inv_tiles, inv_row_tiles;
  int keep_lo;                  // the update writes lo (a later update reads it)
  float a, b, c;       // this step's coefficients
  float scale;
  int out_bf16;
};

// Tile of workgroup b of n: workgroups go to the 8 XCDs in turn, so XCD x takes
// the x-th eighth of the tiles, whose rows and columns its L2 then shares (with
// 8 or 16 matrices, whole matrices, and what one launch wrote the next one finds
// there: 8 x 264 x 272 takes 73 us, with every other launch in reverse order 85).
__device__ __forceinline__ int ns_xcd_tile(int b, int n) {
  const int x = b & 7, q = n >> 3, rest = n & 7;
  return x * q + (x < rest ? x : rest) + (b >> 3);
}

// This workgroup's tile: matrix b, tile t of it, at row tm and column tn of tiles.
struct NsTile {
  int b, t, tm, tn;
};
// n / d for n < 2^24, with 1 / d at hand: a handful of instructions. (The time
// from a workgroup's start to its first load is mostly that of fetching its
// instructions: an integer division and a loop over the triangle's rows took
// 1500 cycles of it.)
__device__ __forceinline__ int ns_div(int n, int d, float inv) {
  int q = static_cast<int>(static_cast<float>(n) * inv);
  const int r = n - q * d;
  q += r >= d ? 1 : 0;
  q -= r < 0 ? 1 : 0;
  return uni(q);
}
template <bool SYM>
__device__ __forceinline__ NsTile ns_tile(const NsArgs& p) {
  const int lt = ns_xcd_tile(blockIdx.x, gridDim.x);
  const int b = ns_div(lt, p.tiles, p.inv_tiles);
  const int t = lt - b * p.tiles;
  const int tm = ns_div(t, p.row_tiles, p.inv_row_tiles), c = t - tm * p.row_tiles;
  if constexpr (SYM) {
    // the upper triangle of n x n tiles folded to rows of n + 1: row i of the
    // triangle, n - i tiles, and behind it row n - 1 - i, of i + 1 tiles
    const int n = p.tiles_n, i = n - 1 - tm;
    return c < n - tm ? NsTile{b, t, tm, tm + c} : NsTile{b, t, i, i + c - (n - tm)};
  } else {
    return {b, t, tm, c};
  }
}

// Swizzle of the 32-byte pairs (16 columns) of k row kr in a k-major stage W
// columns wide: the 16 k rows that one transposing read touches then fall on
// different banks. It depends on bits 0, 1 and 3 of kr only.
template <int W>
__device__ __forceinline__ int ns_kswz(int kr) {
  return W == 128 ? (kr & 3) | (((kr >> 3) & 1) << 2) : ((kr >> 1) & 1) | (((kr >> 3) & 1) << 1);
}

// This lane's place in lo of its tile (ns_lo_place)
__device__ __forceinline__ u32x2_t* ns_lo(const NsArgs& p, const NsTile& tl, int f) {
  return p.ylo + tl.b * p.lo_size + (int64_t)(tl.t * 4 + (threadIdx.x >> 6)) * (f * f * 64) +
         (threadIdx.x & 63);
}

// Eight 16-bit values to columns c .. of a row of n.
__device__ __forceinline__ void ns_put8(uint16_t* row, int c, int n, u32x4_t v) {
  if (c + 8 <= n) {
    *reinterpret_cast<u32x4_any_t*>(row + c) = v;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < n) row[c + e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
  }
}

// Place of 16-byte chunk c of row r of a W x W tile of 16-bit values staged in
// LDS: chunks swizzled in pairs by the row, so that 16 rows of 32 bytes each
// (what the blocks' lanes write, and what a transposing read takes) spread over
// the banks.
template <int W>
__device__ __forceinline__ int ns_spos(int r, int c) {
  constexpr int kPairs = W / 16;  // 32-byte pairs per row
  return r * (W * 2) + ((c ^ ((r & (kPairs - 1)) << 1)) << 4);
}

// Everything after the products of a W x W tile, held as F x F blocks of
// accumulators per wave (2 x 2 waves; a lane has four consecutive columns of
// one row), staged through `smem` for whole-row stores. ext(i, j): the block's
// four values of lo (update) or of A (square), asked for in order.
template <int W, int MODE, int F, class Ext>
__device__ __forceinline__ void ns_epilogue(const NsArgs& p, const NsTile& tl, lds_t* smem,
                                            const f32x4_t (&acc)[F][F], Ext&& ext) {
  constexpr bool SYM = MODE == kGram || MODE == kSquare;
  // The thread index through an assembly move: what is derived from it is then
  // computed here and not kept live through the main loop.
  int tid;
  asm volatile("v_mov_b32 %0, %1" : "=v"(tid) : "v"(static_cast<int>(threadIdx.x)));
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int b = tl.b, tm = tl.tm, tn = tl.tn, row0 = tm * W, col0 = tn * W;
  const int wr = (wave >> 1) * (W / 2), wc = (wave & 1) * (W / 2);
  const int64_t ysz = (int64_t)p.cp * p.rp, asz = (int64_t)p.rp * p.rp;
  // this lane's four values of block (i, j) in the staged tile
  auto place = [&](int i, int j) {
    const int r = wr + i * 16 + (lane & 15), c = wc + j * 16 + 4 * (lane >> 4);
    return reinterpret_cast<MC2_LDS u32x2_t*>(smem + ns_spos<W>(r, c >> 3) + ((c & 4) << 1));
  };
  auto pack = [](float x, float y) {
    return f32_to_f16_bits(x) | (static_cast<uint32_t>(f32_to_f16_bits(y)) << 16);
  };
  // the staged tile -> rows row0 .., columns col0 .. of a matrix of `rows`
  // rows of `ld` values, 16 bytes at a time (rows are whole pieces), eight LDS
  // reads in flight per thread
  auto store = [&](uint16_t* out, int ld, int rows, int cols) {
    constexpr int N = W * (W / 8) / kNsThreads, U = N < 8 ? N : 8;
    const int r0 = tid / (W / 8), c8 = tid % (W / 8);
    constexpr int RS = kNsThreads / (W / 8);  // rows per pass
    uint16_t* o = out + (int64_t)(row0 + r0) * ld + col0 + c8 * 8;
    const bool col_in = col0 + c8 * 8 < cols;
#pragma unroll 1
    for (int k0 = 0; k0 < N; k0 += U) {
      u32x4_t v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = *reinterpret_cast<const MC2_LDS u32x4_t*>(smem + ns_spos<W>(r0 + (k0 + u) * RS, c8));
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (col_in && row0 + r0 + (k0 + u) * RS < rows)
          *reinterpret_cast<u32x4_t*>(o + (int64_t)(k0 + u) * RS * ld) = v[u];
    }
  };

  if constexpr (SYM) {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        float v[4];
        if constexpr (MODE == kGram) {
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][e] * kGramScale;
        } else {
          const int r = row0 + wr + i * 16 + (lane & 15);
          const int c = col0 + wc + j * 16 + 4 * (lane >> 4);
          const u32x2_t x = ext(i, j);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float g = f16_bits_to_f32((x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
            v[e] = p.b * g + p.c * kSqScale * acc[i][j][e];
            if (tm == tn) v[e] += r == c + e ? p.a * kDiag : 0.f;
          }
        }
        *place(i, j) = u32x2_t{pack(v[0], v[1]), pack(v[2], v[3])};
      }
    __syncthreads();
    uint16_t* out = (MODE == kGram ? p.gram : p.q) + b * asz;
    store(out, p.rp, p.rp, p.rp);
    if (tm != tn) {
      // the mirrored tile: transposing reads of the staged one, each lane 8 rows
      // of one column, stored as 16 bytes of a row of the mirrored tile
      const int j = lane & 15, g = lane >> 4;
      constexpr int U = 4;  // passes with their reads in flight together
#pragma unroll 1
      for (int q0 = 0; q0 < W * W / 2048; q0 += W == 64 ? 2 : U) {
        constexpr int UU = W == 64 ? 2 : U;  // 16 columns by 32 rows per wave and pass
        u32x2_t h[UU][2];
#pragma unroll
        for (int u = 0; u < UU; ++u) {
          const int id = (q0 + u) * 4 + wave;
          const int c0 = (id % (W / 16)) * 16, kr = (id / (W / 16)) * 32 + g * 8 + (j >> 2);
          const int c = (c0 >> 3) + ((j & 3) >> 1), in = (j & 1) << 3;
#pragma unroll
          for (int k = 0; k < 2; ++k)
            h[u][k] = bit_cast<u32x2_t>(__builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<MC2_LDS s16x4_t*>(smem + ns_spos<W>(kr + 4 * k, c) + in)));
        }
#pragma unroll
        for (int u = 0; u < UU; ++u) {
          const int id = (q0 + u) * 4 + wave;
          const int c = col0 + (id % (W / 16)) * 16 + j, r8 = row0 + (id / (W / 16)) * 32 + g * 8;
          if (c < p.rp && r8 < p.rp)
            *reinterpret_cast<u32x4_t*>(out + (int64_t)c * p.rp + r8) =
                u32x4_t{h[u][0][0], h[u][0][1], h[u][1][0], h[u][1][1]};
        }
      }
    }
  } else if constexpr (MODE == kUpdate) {
    u32x2_t* lo = ns_lo(p, tl, F);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        uint32_t h[4], l[4];
        const u32x2_t x = ext(i, j);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float rest = f16_bits_to_f32((x[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
          ns_split(acc[i][j][e] * kUpdScale + p.a * (1.f / kLoScale) * rest, h[e], l[e]);
        }
        *place(i, j) = u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
        if (p.keep_lo) lo[(i * F + j) * 64] = u32x2_t{l[0] | (l[1] << 16), l[2] | (l[3] << 16)};
      }
    __syncthreads();
    store(p.ynext + b * ysz, p.rp, p.cp, p.rp);
  } else {
    // (the power of two first, which is exact: the factor of both is not for a
    // scale near the smallest numbers)
    auto scaled = [&](float v) { return v * kOutScale * p.scale; };
    auto stage = [&](auto cvt) {
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
          *place(i, j) = u32x2_t{cvt(scaled(acc[i][j][0]), scaled(acc[i][j][1])),
                                 cvt(scaled(acc[i][j][2]), scaled(acc[i][j][3]))};
    };
    if (p.out_bf16)
      stage([](float x, float y) {
        return f32_to_bf16_bits(x) | (static_cast<uint32_t>(f32_to_bf16_bits(y)) << 16);
      });
    else
      stage(pack);
    __syncthreads();
    uint16_t* out = p.out + (int64_t)b * p.om * p.on;
    if (p.on % 8 == 0) {
      store(out, p.on, p.om, p.on);
    } else {  // rows that are not whole 16-byte pieces
      for (int q = tid; q < W * (W / 8); q += kNsThreads) {
        const int r = q / (W / 8), c8 = (q % (W / 8)) * 8;
        const u32x4_t v = *reinterpret_cast<const MC2_LDS u32x4_t*>(smem + ns_spos<W>(r, c8 >> 3));
        if (row0 + r < p.om) ns_put8(out + (int64_t)(row0 + r) * p.on, col0 + c8, p.on, v);
      }
    }
  }
}

// One W x W tile of a product. 4 waves as 2 x 2; K in stages of 64 (two k-steps)
// through a ring of NS LDS buffers, filled by loads straight to LDS. A stage's
// second k-step is multiplied while the next stage's first fragments are read
// and the loads of stage s + NS are issued into the buffer just released.
// W = 64, NS = 4 and W = 128, NS = 2 take 64 KiB of LDS, two workgroups per CU;
// W = 128, NS = 4 is for launches of at most one workgroup per CU, which has
// nobody to hide its loads' latency. The 128 x 128 tiles move 96 KiB through LDS
// per stage, 768 cycles at 128 bytes each against 512 of MFMA (the square of
// 16 x 1536: MFMA pipes busy 34% of the launch, CUs with work 81%); the 64 x 64
// ones are bound by the CU's load path (16 KiB per stage, about 450 cycles against
// 128 of MFMA) and, in short contractions, by their start and end (4500 cycles).
// Each MFMA takes the second operand's fragment first, so a lane ends with
// four consecutive columns of one row.
template <int W, int NS, int MODE>
__global__ __launch_bounds__(kNsThreads, W == 128 && NS > 2 ? 1 : 2) void ns_gemm_kernel(NsArgs p) {
  constexpr bool KMAJ = MODE == kGram;
  constexpr bool SYM = MODE == kGram || MODE == kSquare;
  constexpr int OB = W * 128;      // bytes of one operand's stage
  constexpr int NL = OB / 4096;    // 1 KiB loads per wave, operand and stage
  constexpr int F = W / 32;        // 16-row fragments per wave and operand
  constexpr int NR = KMAJ ? 4 * F : 2 * F;  // LDS reads per wave and k-step
  __shared__ __attribute__((aligned(16))) char smem_raw[NS * 2 * OB];
  static_assert(W * W * 2 <= NS * 2 * OB, "the output tile is staged in the operands' place");
  lds_t* smem = (lds_t*)smem_raw;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const NsTile tl = ns_tile<SYM>(p);
  const int b = tl.b, t = tl.t, tm = tl.tm, tn = tl.tn;
  const int row0 = tm * W, col0 = tn * W;
  const int64_t ysz = (int64_t)p.cp * p.rp, asz = (int64_t)p.rp * p.rp;
  const uint16_t* Y = p.y + b * ysz;
  const uint16_t* A = p.gram + b * asz;
  const uint16_t* Q = p.q + b * asz;
  const uint16_t* opa = MODE == kGram ? Y : MODE == kSquare ? A : MODE == kOutWide ? Q : Y;
  const uint16_t* opb = MODE == kGram ? Y : MODE == kSquare ? A : MODE == kOutWide ? Y : Q;
  // rows (K-contiguous) or columns (k-major) of the two operands
  const int na = MODE == kUpdate || MODE == kOutTall ? p.cp : p.rp;
  const int nbn = MODE == kOutWide ? p.cp : p.rp;
  const int stages = (KMAJ ? p.cp : p.rp) / 64;

  // Byte offsets of this wave's loads: a load fills 1 KiB of LDS linearly, so
  // the lane's place there says which piece of the operand it takes. Rows or
  // columns beyond the matrix read its last ones; they are not stored.
  uint32_t off[2][NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int o = (wave * NL + i) * 1024 + lane * 16;
    if constexpr (KMAJ) {
      const int kr = o / (W * 2), in = o - kr * (W * 2);
      const int col = (((in >> 5) ^ ns_kswz<W>(kr)) << 4) + ((in & 16) >> 1);
      const int ca = row0 + col < na ? row0 + col : na - 8;
      const int cb = col0 + col < nbn ? col0 + col : nbn - 8;
      off[0][i] = static_cast<uint32_t>((kr * p.rp + ca) * 2);
      off[1][i] = static_cast<uint32_t>((kr * p.rp + cb) * 2);
    } else {
      const int r = o >> 7, ch = ((o >> 4) & 7) ^ ((r >> 1) & 7);
      const int ra = row0 + r < na ? r : na - 1 - row0;
      const int rb = col0 + r < nbn ? r : nbn - 1 - col0;
      off[0][i] = static_cast<uint32_t>(ra * p.rp * 2 + ch * 16);
      off[1][i] = static_cast<uint32_t>(rb * p.rp * 2 + ch * 16);
    }
  }
  const char* base_a = reinterpret_cast<const char*>(KMAJ ? opa : opa + (int64_t)row0 * p.rp);
  const char* base_b = reinterpret_cast<const char*>(KMAJ ? opb : opb + (int64_t)col0 * p.rp);
  const int64_t step = KMAJ ? (int64_t)128 * p.rp : 128;  // bytes per stage
  struct Stage {
    __amdgpu_buffer_rsrc_t ra, rb;
    lds_t* d;
  };
  auto stage_of = [&](int s) {
    // a stage past the last one gets resources of no records: its loads touch
    // no memory, and the count of loads in flight stays the same
    const int nrec = s < stages ? 0x7ffffff0 : 0;
    return Stage{__builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base_a + s * step), 0, nrec,
                                                   kBufFlags),
                 __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base_b + s * step), 0, nrec,
                                                   kBufFlags),
                 smem + (s % NS) * 2 * OB + wave * NL * 1024};
  };
  auto issue = [&](const Stage& s, int i) {
    if (i < NL) dma16(s.ra, s.d + i * 1024, off[0][i]);
    else dma16(s.rb, s.d + OB + (i - NL) * 1024, off[1][i - NL]);
  };

  f32x4_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int wr = (wave >> 1) * (W / 2), wc = (wave & 1) * (W / 2);

  // Operand fragments of one k-step: a lane supplies row lane & 15 of each 16
  // rows, K values 8 (lane >> 4) .. + 7 of the step's 32; from a k-major stage
  // as two transposing 8-byte reads of 4 k rows each.
  struct Frags {
    u32x4_t q[KMAJ ? 1 : F];
    u32x2_t h[KMAJ ? F : 1][2];
  };
  const uint32_t s0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
  // read q (of NR) of k-step ks from the stage at s: B's fragments, then A's
  auto read = [&](Frags& fa, Frags& fb, uint32_t s, int ks, int q) {
    constexpr int N = NR / 2;
    Frags& f = q < N ? fb : fa;
    const uint32_t base = q < N ? s + OB : s;
    const int x0 = q < N ? wc : wr, k = q < N ? q : q - N;
    if constexpr (KMAJ) {
      const int i = k >> 1, j = lane & 15, g = lane >> 4;
      const int kr = ks * 32 + g * 8 + (j >> 2);
      const uint32_t at =
          base + kr * (W * 2) + ((((x0 >> 4) + i) ^ ns_kswz<W>(kr)) << 5) + ((j & 3) << 3);
      if (k & 1)
        asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2"
                     : "=v"(f.h[i][1]) : "v"(at), "i"(4 * W * 2) : "memory");
      else
        asm volatile("ds_read_b64_tr_b16 %0, %1" : "=v"(f.h[i][0]) : "v"(at) : "memory");
    } else {
      const uint32_t at = base + row_off(x0 + k * 16 + (lane & 15), ks * 4 + (lane >> 4));
      asm volatile("ds_read_b128 %0, %1" : "=v"(f.q[k]) : "v"(at) : "memory");
    }
  };
  // ties the fragments to the wait before it: no use of them moves above
  auto tie = [&](Frags& f) {
#pragma unroll
    for (int i = 0; i < F; ++i) {
      if constexpr (KMAJ) {
        asm volatile("" : "+v"(f.h[i][0]));
        asm volatile("" : "+v"(f.h[i][1]));
      } else {
        asm volatile("" : "+v"(f.q[i]));
      }
    }
  };
  auto get = [&](const Frags& f, int i) {
    if constexpr (KMAJ)
      return bit_cast<f16x8_t>(u32x4_t{f.h[i][0][0], f.h[i][0][1], f.h[i][1][0], f.h[i][1][1]});
    else
      return bit_cast<f16x8_t>(f.q[i]);
  };
  auto multiply = [&](const Frags& fa, const Frags& fb, auto&& after) {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(get(fb, j), get(fa, i), acc[i][j], 0, 0, 0);
        after(i * F + j);
        __builtin_amdgcn_sched_barrier(0);
      }
  };

  // What the epilogue reads besides the products, loaded ahead of the main loop
  // (after it, each of these would cost a memory latency with nothing to hide it):
  // the update's lo, the square's tile of A
  constexpr int NE = MODE == kUpdate || MODE == kSquare ? F : 0;
  u32x2_t ext[NE ? NE : 1][NE ? NE : 1];
  auto fill = [&](int s) {
    const Stage st = stage_of(s);
#pragma unroll
    for (int i = 0; i < 2 * NL; ++i) issue(st, i);
  };
  fill(0);
  if constexpr (MODE == kUpdate) {
    const u32x2_t* lo = ns_lo(p, tl, F);
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) ext[i][j] = lo[(i * F + j) * 64];
  } else if constexpr (MODE == kSquare) {
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const int r = row0 + wr + i * 16 + (lane & 15);
        const int c = col0 + wc + j * 16 + 4 * (lane >> 4);
        ext[i][j] = u32x2_t{0u, 0u};
        if (r < p.rp && c < p.rp)
          ext[i][j] = *reinterpret_cast<const u32x2_t*>(A + (int64_t)r * p.rp + c);
      }
  }
#pragma unroll
  for (int s = 1; s < NS; ++s) fill(s);
  Frags a0, b0, a1, b1;
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * 2 * NL) : "memory");
  bar_sync();
#pragma unroll
  for (int q = 0; q < NR; ++q) read(a0, b0, s0, 0, q);
  // One MFMA, then up to two LDS reads and one load: a memory instruction that
  // waits to be taken then costs no more than the MFMAs in flight, and with one
  // workgroup per CU nobody else would fill that time.
  for (int s = 0; s < stages; ++s) {
    const uint32_t sa = s0 + (s % NS) * 2 * OB, sn = s0 + ((s + 1) % NS) * 2 * OB;
    lgkm_wait(0);
    tie(b0);
    tie(a0);
    multiply(a0, b0, [&](int q) {
#pragma unroll
      for (int r = 2 * q; r < 2 * q + 2; ++r)
        if (r < NR) read(a1, b1, sa, 1, r);
    });
    // every read of this stage is done, by every wave: its buffer may be
    // filled again; and the next stage has landed (this wave's loads of it,
    // those of later stages may be in flight: loads complete in order; then
    // every wave's)
    lgkm_wait(0);
    tie(b1);
    tie(a1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * 2 * NL) : "memory");
    bar_sync();
    // under the second k-step's products: the next stage's first fragments
    // (after the last stage: of a buffer nobody fills any more, never used),
    // and the loads of stage s + NS
    const Stage st = stage_of(s + NS);
    multiply(a1, b1, [&](int q) {
#pragma unroll
      for (int r = 2 * q; r < 2 * q + 2; ++r)
        if (r < NR) read(a0, b0, sn, 0, r);
      constexpr int kEvery = F * F / (2 * NL);
      if (q % kEvery == kEvery - 1) issue(st, q / kEvery);
    });
  }
  lgkm_wait(0);  // the last reads land in registers that stay theirs until then
  tie(b0);
  tie(a0);
  wait_vmcnt0();
  __syncthreads();  // every read of the operands is done: their place takes the output

  ns_epilogue<W, MODE, F>(p, tl, smem, acc, [&](int i, int j) { return ext[NE ? i : 0][NE ? j : 0]; });
}

// One 256 x 256 tile on the four-wave main loop (gemm_core_w4.hpp), whose waves
// of 128 x 128 read half as much LDS per product as the 128 x 128 tiles' waves:
// those are bound by LDS bandwidth. One workgroup per CU.
template <int MODE>
__global__ __launch_bounds__(TileW::NT, 1) void ns_gemm256_kernel(NsArgs p) {
  static_assert(MODE != kSquare, "the square takes narrower tiles");
  constexpr int F = TileW::FM;
  static_assert(TileW::BM == 256 && TileW::BN == 256 && TileW::FN == F && TileW::NT == kNsThreads,
                "2 x 2 waves of 128 x 128");
  static_assert(TileW::kStages * TileW::kStageBytes == 256 * 256 * 2,
                "the output tile is staged in the operands' place");
  __shared__ __attribute__((aligned(16))) char smem_raw[256 * 256 * 2];
  lds_t* smem = (lds_t*)smem_raw;
  const NsTile tl = ns_tile<MODE == kGram>(p);
  const int row0 = tl.tm * 256, col0 = tl.tn * 256;
  const int64_t ysz = (int64_t)p.cp * p.rp, asz = (int64_t)p.rp * p.rp;
  const char* Y = reinterpret_cast<const char*>(p.y + tl.b * ysz);
  const char* Q = reinterpret_cast<const char*>(p.q + tl.b * asz);
  const int64_t ld = (int64_t)p.rp * 2;
  const int na = MODE == kUpdate || MODE == kOutTall ? p.cp : p.rp;
  const int nb = MODE == kOutWide ? p.cp : p.rp;
  const int k = MODE == kGram ? p.cp : p.rp;
  const KSpan ks{k, 0, 0, k / 64, k / 64};
  f32x4_t acc[F][F];
  if constexpr (MODE == kGram) {
    mainloop_w4<Elem::F16, false, TileW, false, true>(smem, Y, ld, row0, na - 1, BDesc{Y, ld, nb},
                                                      col0, PlainCols{col0, nb - 8}, ks, acc);
  } else {
    const char* a = MODE == kOutWide ? Q : Y;
    const char* b = MODE == kOutWide ? Y : Q;
    mainloop_w4<Elem::F16, true, TileW, false>(smem, a, ld, row0, na - 1, BDesc{b, ld, nb}, col0,
                                               PlainCols{col0, nb - 8}, ks, acc);
  }
  // lo, two rows of blocks ahead of its use (the accumulators leave no room to
  // hold it through the main loop)
  u32x2_t ext[3][F];
  auto load = [&](int i) {
    if constexpr (MODE == kUpdate) {
      const u32x2_t* lo = ns_lo(p, tl, F);
#pragma unroll
      for (int j = 0; j < F; ++j) ext[i % 3][j] = lo[(i * F + j) * 64];
    }
  };
  load(0);
  load(1);
  ns_epilogue<256, MODE, F>(p, tl, smem, acc, [&](int i, int j) {
    if (j == 0 && i + 2 < F) load(i + 2);
    return ext[i % 3][j];
  });
}

// ---------------------------------------------------------------- one workgroup per matrix

// A small matrix (rp <= 128 and at most 64 Ki padded elements) is iterated by
// one workgroup in one launch: launches, not work, are what the general path
// costs there (17 of them, 56 us for 64 x 256).
//
// 8 waves. Y's high half lives in LDS (up to 128 KiB) as rows of rp values;
// wave w owns 16-row blocks w * RB .. + RB - 1 and holds their values in fp32 in
// registers, in the accumulator layout: the product Y Q is added onto a Y held
// there, so no low half is needed, and a wave's update touches its own rows
// only. A (less mu I) and Q take turns in one (rp, rp) LDS array. 64 x 256 takes
// 16 us: 35 k cycles, of them 8 k until the first product,
// 2100 a step for the Gram product (LDS bandwidth) and 2100 for the update;
// 64 x 1000 takes 54 us and 128 x 512 67 us.
constexpr int kTinyThreads = 512;
constexpr int64_t kTinyElems = 65536;
constexpr float kTinyScale = kXScale / kUpdScale;  // x's scale, that of hi Q: 2^21

struct TinyArgs {
  const void* g;
  uint16_t* out;
  int m, n, in_dtype, out_bf16, steps;
  float eps, scale;
  float co[3 * 32];
};

// Byte place of 16-byte chunk c of row r: RP values per row. Both the 16 rows
// that one row-wise fragment read touches and the 16 k rows of a transposing
// read (rows 8g + 0..3 or 8g + 4..7) spread over the banks.
template <int RP>
__device__ __forceinline__ uint32_t tiny_pos(int r, int c) {
  const int f = RP == 64 ? (r >> 1) & 7 : ((r & 3) << 1) | (((r >> 3) & 1) << 3) | ((r >> 2) & 1);
  return static_cast<uint32_t>(r * (RP * 2) + ((c ^ f) << 4));
}

template <int RP>
__device__ __forceinline__ f16x8_t tiny_row(const char* s, int r0, int ks) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const f16x8_t*>(s + tiny_pos<RP>(r0 + (lane & 15), ks * 4 + (lane >> 4)));
}

// 16 columns at c0 as a fragment over k rows ks * 32 .. + 31
template <int RP>
__device__ __forceinline__ f16x8_t tiny_col(const char* s, int c0, int ks) {
  const int lane = threadIdx.x & 63, j = lane & 15;
  const int kr = ks * 32 + (lane >> 4) * 8 + (j >> 2);
  const int c = (c0 >> 3) + ((j & 3) >> 1);
  s16x4_t h[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    h[i] = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (MC2_LDS s16x4_t*)(s + tiny_pos<RP>(kr + 4 * i, c) + ((j & 1) << 3)));
  const u32x2_t l = bit_cast<u32x2_t>(h[0]), u = bit_cast<u32x2_t>(h[1]);
  return bit_cast<f16x8_t>(u32x4_t{l[0], l[1], u[0], u[1]});
}

// four consecutive columns c .. c + 3 of row r
template <int RP>
__device__ __forceinline__ void tiny_put(char* s, int r, int c, float a, float b, float x, float y) {
  const uint32_t lo = f32_to_f16_bits(a) | (static_cast<uint32_t>(f32_to_f16_bits(b)) << 16);
  const uint32_t hi = f32_to_f16_bits(x) | (static_cast<uint32_t>(f32_to_f16_bits(y)) << 16);
  *reinterpret_cast<u32x2_t*>(s + tiny_pos<RP>(r, c >> 3) + ((c & 4) << 1)) = u32x2_t{lo, hi};
}

template <int RP, int RB>
__global__ __launch_bounds__(kTinyThreads) void ns_tiny_kernel(TinyArgs p) {
  constexpr int CB = RP / 16, KS = RB * 4;  // 32-row k steps of Y
  constexpr int kGramUnroll = RP == 64 && RB <= 4 ? 4 : 2;  // (registers)
  constexpr int kUpdUnroll = RP == 64 && RB <= 4 ? 2 : 1;
  constexpr int FA = RP / 64, FB = RP / 32;  // a wave's 16-row / 16-column blocks of A and Q
  __shared__ __attribute__((aligned(16))) char s_y[RB * 128 * RP * 2];
  __shared__ __attribute__((aligned(16))) char s_a[RP * RP * 2];
  double* s_n = reinterpret_cast<double*>(s_a);  // before A: its first write follows a barrier
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lc = 4 * (lane >> 4);
  const int m = p.m, n = p.n;
  const bool tall = m >= n;
  const int r = tall ? n : m, c = tall ? m : n;
  const int64_t gb = (int64_t)blockIdx.x * m * n;

  // element strides of Y's rows and columns in G
  const int sr = tall ? n : 1, sc = tall ? 1 : n;
  f32x4_t x[RB][CB];
  double sq = 0;
  // places outside G read its first element, all loads of a row of blocks being
  // in flight together, and become zeros
  auto load = [&](auto dtype) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int row = (wave * RB + i) * 16 + lr;
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = j * 16 + lc + e;
          const bool in = row < c && col < r;
          const float v = ns_load<decltype(dtype)::value>(p.g, gb + (in ? row * sr + col * sc : 0));
          x[i][j][e] = in ? v : 0.f;
        }
#pragma unroll
      for (int j = 0; j < CB; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sq = __builtin_fma((double)x[i][j][e], (double)x[i][j][e], sq);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (p.in_dtype == MC2_F32) load(std::integral_constant<int, MC2_F32>{});
  else if (p.in_dtype == MC2_BF16) load(std::integral_constant<int, MC2_BF16>{});
  else load(std::integral_constant<int, MC2_F16>{});
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) sq += __shfl_xor(sq, off);
  if (lane == 0) s_n[wave] = sq;
  __syncthreads();
  double norm2 = 0;
#pragma unroll
  for (int w = 0; w < kTinyThreads / 64; ++w) norm2 += s_n[w];
  const double inv = norm2 == 0.0 ? 0.0 : kTinyScale / (sqrt(norm2) + static_cast<double>(p.eps));
  const float invf = static_cast<float>(inv);
  // in fp64 only where fp32 does not hold 1 / norm (what lies outside G stays
  // zero: inv may be NaN)
  auto normalise = [&](auto mul) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const int row = (wave * RB + i) * 16 + lr;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          x[i][j][e] = row < c && j * 16 + lc + e < r ? mul(x[i][j][e]) : 0.f;
      }
  };
  if (invf > 1e-30f && invf < 1e30f) normalise([&](float v) { return v * invf; });
  else normalise([&](float v) { return static_cast<float>(static_cast<double>(v) * inv); });

  const int wm = (wave >> 1) * (RP / 4), wn = (wave & 1) * (RP / 2);  // this wave's part of A, Q
  for (int s = 0; s < p.steps; ++s) {
    // A is held as D = A - mu I, whose diagonal is smaller than A's once the
    // singular values are near 1 (there most of the rounding of A A comes from):
    // a I + b A + c A A = (a + b mu + c mu^2) I + (b + 2 c mu) D + c D D
    const float mu = s < 2 ? 0.f : 0.5f;
    const float cc = p.co[3 * s + 2], b = p.co[3 * s + 1] + 2.f * cc * mu;
    const float a = p.co[3 * s], am = (p.co[3 * s + 1] + cc * mu) * mu;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j)
        tiny_put<RP>(s_y, (wave * RB + i) * 16 + lr, j * 16 + lc, x[i][j][0] * kUpdScale,
                     x[i][j][1] * kUpdScale, x[i][j][2] * kUpdScale, x[i][j][3] * kUpdScale);
    __syncthreads();
    f32x4_t g[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) g[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll kGramUnroll
    for (int ks = 0; ks < KS; ++ks) {
      f16x8_t fa[FA], fb[FB];
#pragma unroll
      for (int i = 0; i < FA; ++i) fa[i] = tiny_col<RP>(s_y, wm + i * 16, ks);
#pragma unroll
      for (int j = 0; j < FB; ++j) fb[j] = tiny_col<RP>(s_y, wn + j * 16, ks);
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j)
          g[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], g[i][j], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          g[i][j][e] = g[i][j][e] * kGramScale -
                       (wm + i * 16 + lr == wn + j * 16 + lc + e ? mu * kDiag : 0.f);
        tiny_put<RP>(s_a, wm + i * 16 + lr, wn + j * 16 + lc, g[i][j][0], g[i][j][1], g[i][j][2],
                     g[i][j][3]);
      }
    __syncthreads();
    f32x4_t q[FA][FB];
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) q[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int ks = 0; ks < RP / 32; ++ks) {
      f16x8_t fa[FA], fb[FB];
#pragma unroll
      for (int i = 0; i < FA; ++i) fa[i] = tiny_row<RP>(s_a, wm + i * 16, ks);
#pragma unroll
      for (int j = 0; j < FB; ++j) fb[j] = tiny_row<RP>(s_a, wn + j * 16, ks);
#pragma unroll
      for (int i = 0; i < FA; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j)
          q[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], q[i][j], 0, 0, 0);
    }
    __syncthreads();  // every read of A is done: Q takes its place
#pragma unroll
    for (int i = 0; i < FA; ++i)
#pragma unroll
      for (int j = 0; j < FB; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) q[i][j][e] = b * g[i][j][e] + cc * (q[i][j][e] * kSqScale);
        tiny_put<RP>(s_a, wm + i * 16 + lr, wn + j * 16 + lc, q[i][j][0], q[i][j][1], q[i][j][2],
                     q[i][j][3]);
      }
    __syncthreads();
    // x = a x + (b mu + c mu^2) hi + hi Q: the part of the identity that the
    // product takes away again is added to what the product multiplies, hi (its
    // rounding would else stay in the directions of singular value zero)
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        // (opaque where registers are short: hi is formed anew here, not kept in
        // them from the step's start)
        if constexpr (RB * CB > 8) asm volatile("" : "+v"(x[i][j]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float hi = f16_bits_to_f32(f32_to_f16_bits(x[i][j][e] * kUpdScale));
          x[i][j][e] = __builtin_fmaf(hi, am * (1.f / kUpdScale), a * x[i][j][e]);
        }
      }
#pragma unroll kUpdUnroll
    for (int ks = 0; ks < RP / 32; ++ks) {
      f16x8_t fa[RB];
#pragma unroll
      for (int i = 0; i < RB; ++i) fa[i] = tiny_row<RP>(s_y, (wave * RB + i) * 16, ks);
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const f16x8_t fb = tiny_row<RP>(s_a, j * 16, ks);
#pragma unroll
        for (int i = 0; i < RB; ++i)
          x[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb, fa[i], x[i][j], 0, 0, 0);
      }
    }
    // (a wave reads only its own rows of Y above and writes only them in the
    // next step; the reads of Q end before that step's first barrier)
  }
  // The result takes Y's place (a wave's rows are read by that wave alone once Q
  // is formed) and leaves in 16-byte pieces of G's rows (2-byte stores from the registers took 18 us for 128 x 512).
  auto stage = [&](auto cvt) {
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int j = 0; j < CB; ++j) {
        const int row = (wave * RB + i) * 16 + lr, col = j * 16 + lc;
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) h[e] = cvt(x[i][j][e] * (1.f / kTinyScale) * p.scale);
        *reinterpret_cast<u32x2_t*>(s_y + tiny_pos<RP>(row, col >> 3) + ((col & 4) << 1)) =
            u32x2_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16)};
      }
  };
  if (p.out_bf16) stage([](float v) { return f32_to_bf16_bits(v); });
  else stage([](float v) { return f32_to_f16_bits(v); });
  __syncthreads();
  uint16_t* out = p.out + gb;
  if (tall) {
    for (int q = tid; q < c * (RP / 8); q += kTinyThreads) {
      const int row = q / (RP / 8), ch = q % (RP / 8);
      if (ch * 8 < r)
        ns_put8(out + row * n, ch * 8, n,
                *reinterpret_cast<const u32x4_t*>(s_y + tiny_pos<RP>(row, ch)));
    }
  } else {
    for (int q = wave; q < KS * CB; q += kTinyThreads / 64) {
      const int c0 = (q / KS) * 16, ks = q % KS;
      const u32x4_t v = bit_cast<u32x4_t>(tiny_col<RP>(s_y, c0, ks));
      const int col = c0 + lr, row = ks * 32 + (lane >> 4) * 8;
      if (col < r && row < c) ns_put8(out + col * n, row, n, v);
    }
  }
}

// ---------------------------------------------------------------- host

// The widest tiles that a matrix takes: none of twice its padded smaller side,
// of which half would be padding (five steps of 256 x 64 x 2048: 426 us, with
// 256 wide ones 922; 64 x 72 x 1300: 163 and 223; lo is as much smaller).
static int ns_widest(int64_t rp) { return rp <= 64 ? 64 : rp <= 128 ? 128 : 256; }

// Width of a product's tiles, and p's tile counts for it: 256 where those give
// every CU a tile (five steps of 16 x 2048 x 1536: 1774 us, with 128 at most
// 2025), else 128 where those give every second CU one (one 2048 x 3584: 440 us,
// asking for one on every CU 512; asking for one on every third, 16 x 300 x 2000
// goes from 198 to 263 us), else 64. The square stays at 128: its K is the short
// side, and two workgroups per CU hide more of its epilogue (16 x 2048 x 1536:
// 1845 us with 256, 300 x 130 x 190: 454 against 385).
template <int MODE>
static int ns_plan(NsArgs& p, int64_t batch) {
  constexpr bool SYM = MODE == kGram || MODE == kSquare;
  const int rows = MODE == kUpdate || MODE == kOutTall ? p.cp : p.rp;
  const int cols = MODE == kOutWide ? p.cp : p.rp;
  const int widest = ns_widest(p.rp);
  for (int w = MODE == kSquare && widest > 128 ? 128 : widest;; w /= 2) {
    p.tiles_m = (rows + w - 1) / w;
    p.tiles_n = (cols + w - 1) / w;
    p.tiles = SYM ? p.tiles_n * (p.tiles_n + 1) / 2 : p.tiles_m * p.tiles_n;
    p.row_tiles = SYM ? p.tiles_n + 1 : p.tiles_n;
    p.inv_tiles = 1.f / static_cast<float>(p.tiles);
    p.inv_row_tiles = 1.f / static_cast<float>(p.row_tiles);
    const int64_t n = batch * p.tiles;
    if (w == 64 || n >= (w == 256 ? num_cus() : num_cus() / 2)) return w;
  }
}

struct NsLayout {
  int64_t r, c, rp, cp;
  size_t part, y0, y1, lo, gram, q, total;
};

static bool ns_sizes_ok(int64_t batch, int64_t m, int64_t n) {
  return batch >= 1 && batch <= 65535 && m >= 1 && n >= 1 && m <= 65536 && n <= 65536;
}

// Rows per wave (in blocks of 16, a power of two) of ns_tiny_kernel for a matrix
// that one workgroup can hold, else 0.
static int ns_tiny_rows(int64_t rp, int64_t cp) {
  int rb = 1;
  while (rb * 128 < cp) rb *= 2;
  return rp <= 128 && rb * 128 * rp <= kTinyElems ? rb : 0;
}

// The workspace, from the sizes alone. Matrices that one workgroup holds use
// none of it: theirs is that of one matrix, whatever the batch.
static NsLayout ns_layout(int64_t batch, int64_t m, int64_t n) {
  NsLayout L{};
  L.r = m < n ? m : n;
  L.c = m < n ? n : m;
  L.rp = (L.r + kNsPad - 1) / kNsPad * kNsPad;
  L.cp = (L.c + kNsPad - 1) / kNsPad * kNsPad;
  if (ns_tiny_rows(L.rp, L.cp)) batch = 1;
  const size_t y = static_cast<size_t>(batch * L.cp * L.rp) * 2;  // multiples of 8 KiB
  const size_t a = static_cast<size_t>(batch * L.rp * L.rp) * 2;
  // lo in whole tiles of the update, of any width that it may take
  int64_t most = 0;
  for (int64_t w = 64; w <= ns_widest(L.rp); w *= 2) {
    const int64_t places = (L.cp + w - 1) / w * w * ((L.rp + w - 1) / w * w);
    most = most > places ? most : places;
  }
  const size_t l = static_cast<size_t>(batch * most) * 2;
  L.part = 0;
  L.y0 = (static_cast<size_t>(batch) * kNsMaxPart * sizeof(double) + 255) / 256 * 256;
  L.y1 = L.y0 + y;
  L.lo = L.y1 + y;
  L.gram = L.lo + l;
  L.q = L.gram + a;
  L.total = L.q + a;
  return L;
}

template <int D>
static void ns_start(const void* g, int64_t batch, int64_t m, int64_t n, const NsLayout& L,
                     float eps, double* part, uint16_t* y, const NsArgs& p, int w,
                     hipStream_t stream) {
  const int64_t mn = m * n;
  int64_t nb = (mn + kNsThreads * 16 - 1) / (kNsThreads * 16);
  nb = nb < kNsMaxPart ? nb : kNsMaxPart;
  const dim3 blk(kNsThreads);
  hipLaunchKernelGGL(ns_norm_kernel<D>, dim3(static_cast<unsigned>(nb), static_cast<unsigned>(batch)),
                     blk, 0, stream, g, mn, part);
  auto init = [&](auto kernel) {
    hipLaunchKernelGGL(kernel,
                       dim3(static_cast<unsigned>(L.cp / 64 * (L.rp / 64)), static_cast<unsigned>(batch)),
                       blk, 0, stream, g, m, n, part, static_cast<int>(nb), eps, L.cp, L.rp, y, p.ylo,
                       p.lo_size, w, static_cast<int>((L.rp + w - 1) / w));
  };
  if (m >= n) init(ns_init_kernel<D, true>);
  else init(ns_init_kernel<D, false>);
}

template <int MODE>
static void ns_product(NsArgs p, int64_t batch, hipStream_t stream) {
  const int w = ns_plan<MODE>(p, batch);
  const int64_t n = batch * p.tiles;
  const dim3 grid(static_cast<unsigned>(n)), blk(kNsThreads);
  if constexpr (MODE != kSquare) {
    if (w == 256) {
      hipLaunchKernelGGL(ns_gemm256_kernel<MODE>, grid, blk, 0, stream, p);
      return;
    }
  }
  if (w == 128 && n <= num_cus())
    hipLaunchKernelGGL((ns_gemm_kernel<128, 4, MODE>), grid, blk, 0, stream, p);
  else if (w == 128)
    hipLaunchKernelGGL((ns_gemm_kernel<128, 2, MODE>), grid, blk, 0, stream, p);
  else
    hipLaunchKernelGGL((ns_gemm_kernel<64, 4, MODE>), grid, blk, 0, stream, p);
}

// The whole call as one launch, for matrices that one workgroup can hold.
// Returns false for others.
static bool ns_tiny(const TinyArgs& p, int64_t batch, const NsLayout& L, hipStream_t stream) {
  const int rb = ns_tiny_rows(L.rp, L.cp);
  if (rb == 0) return false;
  const dim3 grid(static_cast<unsigned>(batch)), blk(kTinyThreads);
  auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, blk, 0, stream, p); };
  if (L.rp == 64) {
    if (rb == 1) go(ns_tiny_kernel<64, 1>);
    else if (rb == 2) go(ns_tiny_kernel<64, 2>);
    else if (rb == 4) go(ns_tiny_kernel<64, 4>);
    else go(ns_tiny_kernel<64, 8>);
  } else {
    if (rb == 1) go(ns_tiny_kernel<128, 1>);
    else if (rb == 2) go(ns_tiny_kernel<128, 2>);
    else go(ns_tiny_kernel<128, 4>);
  }
  return true;
}

}  // namespace mc2

using namespace mc2;

extern "C" size_t mc2_ns_workspace_size(int64_t batch, int64_t m, int64_t n) {
  return ns_sizes_ok(batch, m, n) ? ns_layout(batch, m, n).total : 0;
}

extern "C" int mc2_ns_orthogonalize(const void* g, int64_t batch, int64_t m, int64_t n,
                                    int in_dtype, int steps, const float* coeffs, float eps,
                                    float scale, int out_dtype, void* out, void* workspace,
                                    size_t ws_bytes, hipStream_t stream) {
  if (!g || !coeffs || !out || !workspace) return MC2_ERR_NULL;
  if (in_dtype != MC2_F32 && in_dtype != MC2_BF16 && in_dtype != MC2_F16) return MC2_ERR_DTYPE;
  if (out_dtype != MC2_BF16 && out_dtype != MC2_F16) return MC2_ERR_DTYPE;
  if (!ns_sizes_ok(batch, m, n) || steps < 1 || steps > 32) return MC2_ERR_SHAPE;
  if (!(eps >= 0.f) || eps > 3.0e38f || !(scale >= -3.0e38f && scale <= 3.0e38f))
    return MC2_ERR_SHAPE;
  for (int i = 0; i < 3 * steps; ++i)
    if (!(coeffs[i] >= -16.f && coeffs[i] <= 16.f)) return MC2_ERR_SHAPE;
  if (!aligned16(g) || !aligned16(out) || !aligned16(workspace)) return MC2_ERR_ALIGN;
  const NsLayout L = ns_layout(batch, m, n);
  // tiles of 64 x 64 of the largest product (ns_div; 128 GiB of iterate)
  if (batch * (L.cp / 64) * (L.rp / 64) >= 1 << 24) return MC2_ERR_SHAPE;
  if (ws_bytes < L.total) return MC2_ERR_WORKSPACE;
  TinyArgs ta{};
  ta.g = g;
  ta.out = static_cast<uint16_t*>(out);
  ta.m = static_cast<int>(m);
  ta.n = static_cast<int>(n);
  ta.in_dtype = in_dtype;
  ta.out_bf16 = out_dtype == MC2_BF16;
  ta.steps = steps;
  ta.eps = eps;
  ta.scale = scale;
  for (int i = 0; i < 3 * steps; ++i) ta.co[i] = coeffs[i];
  if (ns_tiny(ta, batch, L, stream)) return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
  char* ws = static_cast<char*>(workspace);
  double* part = reinterpret_cast<double*>(ws + L.part);
  uint16_t* y[2] = {reinterpret_cast<uint16_t*>(ws + L.y0), reinterpret_cast<uint16_t*>(ws + L.y1)};
  NsArgs p{};
  p.cp = static_cast<int>(L.cp);
  p.rp = static_cast<int>(L.rp);
  p.ylo = reinterpret_cast<u32x2_t*>(ws + L.lo);
  const int w = ns_plan<kUpdate>(p, batch);  // lo's order is that of the update's tiles
  p.lo_size = static_cast<int64_t>(p.tiles) * w * w / 4;
  if (in_dtype == MC2_F32) ns_start<MC2_F32>(g, batch, m, n, L, eps, part, y[0], p, w, stream);
  else if (in_dtype == MC2_BF16) ns_start<MC2_BF16>(g, batch, m, n, L, eps, part, y[0], p, w, stream);
  else ns_start<MC2_F16>(g, batch, m, n, L, eps, part, y[0], p, w, stream);
  p.gram = reinterpret_cast<uint16_t*>(ws + L.gram);
  p.q = reinterpret_cast<uint16_t*>(ws + L.q);
  p.out = static_cast<uint16_t*>(out);
  p.om = static_cast<int>(m);
  p.on = static_cast<int>(n);
  p.scale = scale;
  p.out_bf16 = out_dtype == MC2_BF16;
  for (int s = 0; s < steps; ++s) {
    const bool last = s + 1 == steps;
    p.y = y[s & 1];
    p.ynext = y[1 - (s & 1)];
    p.a = coeffs[3 * s];
    p.b = coeffs[3 * s + 1];
    p.c = coeffs[3 * s + 2];
    p.keep_lo = s + 2 < steps;  // the last step reads hi only
    ns_product<kGram>(p, batch, stream);
    ns_product<kSquare>(p, batch, stream);
    if (!last) ns_product<kUpdate>(p, batch, stream);
    else if (m >= n) ns_product<kOutTall>(p, batch, stream);
    else ns_product<kOutWide>(p, batch, stream);
  }
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}
