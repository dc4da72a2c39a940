// Orthogonalisation of a stack of matrices by Newton-Schulz products, gfx950.
//
//   X_0 = G / (|G|_F + eps);   X <- a X + (b A + c A^2) X,  A = X X^T
//
// on the smaller side (r = min(m, n), c = max(m, n)). The iterate is kept
// tall, Y = X^T for a wide G: (cp, rp), rows of rp values, both padded with
// zeros to multiples of 64. Then
//   A  = Y^T Y                 contraction over the rows of Y (k-major reads)
//   Q  = b A + c A A           A is symmetric: both operands are its rows
//   Y' = a Y + Y Q             Q is symmetric: Y's rows by Q's rows
// and the last step writes out = scale * Y Q~ (G tall) or scale * Q~ Y^T (G
// wide: the same two operands the other way round), Q~ = a I + Q.
//
// Number formats. The products run on the fp16 matrix instructions with fp32
// accumulation: fp16 and bf16 run at the same rate and fp16 has three bits
// more (errors of the result 1e-3 instead of 1e-2). Powers of two keep the
// values in its range: Y is stored times 2^12 (entries up to 16), A and Q
// times 2^9 (entries up to 128). Rounding Y to fp16 alone would not do: noise
// in a direction whose singular value is near zero (a gradient of fewer rows
// than the matrix has) grows by the factor a in every step, 484 times in five
// steps, and reached 1.5e-1 of the result. So Y is held as hi + lo, two fp16
// (lo 2^11 times finer): the products use hi, the term a Y both. Errors are
// then 1e-3 whatever the rank. The last step reads hi only, since what it
// loses is not multiplied again.
#include "../../include/mc2_train.h"
#include "mc2_common.hpp"
#include "mc2_host.hpp"

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

// Eight consecutive values from a 16-byte aligned place.
template <int D>
__device__ __forceinline__ void ns_load8(const void* p, int64_t i, float (&v)[8]) {
  if constexpr (D == MC2_F32) {
    const f32x4_t* q = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i);
    const f32x4_t a = q[0], b = q[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = a[j];
      v[4 + j] = b[j];
    }
  } else {
    const u32x4_t q = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = D == MC2_BF16 ? bf16_bits_to_f32(q[j] & 0xFFFFu) : f16_bits_to_f32(q[j] & 0xFFFFu);
      v[2 * j + 1] = D == MC2_BF16 ? bf16_bits_to_f32(q[j] >> 16) : f16_bits_to_f32(q[j] >> 16);
    }
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
// vanish nor overflow).
template <int D, bool VEC>
__global__ __launch_bounds__(kNsThreads) void ns_norm_kernel(const void* __restrict__ g, int64_t mn,
                                                             double* __restrict__ part) {
  const int nb = gridDim.x, b = blockIdx.y;
  const int64_t base = (int64_t)b * mn;
  double s = 0;
  if constexpr (VEC) {
    for (int64_t i = ((int64_t)blockIdx.x * kNsThreads + threadIdx.x) * 8; i < mn;
         i += (int64_t)nb * kNsThreads * 8) {
      float v[8];
      ns_load8<D>(g, base + i, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = __builtin_fma((double)v[j], (double)v[j], s);
    }
  } else {
    for (int64_t i = (int64_t)blockIdx.x * kNsThreads + threadIdx.x; i < mn;
         i += (int64_t)nb * kNsThreads) {
      const double v = ns_load<D>(g, base + i);
      s = __builtin_fma(v, v, s);
    }
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[(int64_t)b * nb + blockIdx.x] = s;
}

// x (in Y's scale) -> its two fp16 halves
__device__ __forceinline__ void ns_split(float x, uint16_t& hi, uint16_t& lo) {
  hi = f32_to_f16_bits(x);
  lo = f32_to_f16_bits((x - f16_bits_to_f32(hi)) * kLoScale);
}

// One 64 x 64 tile of Y = G / (|G| + eps), transposed for a wide G, with zeros
// beyond G. VEC: G's rows are whole 16-byte pieces.
template <int D, bool TALL, bool VEC>
__global__ __launch_bounds__(kNsThreads) void ns_init_kernel(
    const void* __restrict__ g, int64_t m, int64_t n, const double* __restrict__ part, int nb,
    float eps, int64_t cp, int64_t rp, uint16_t* __restrict__ yhi, uint16_t* __restrict__ ylo) {
  __shared__ float s_t[64][65];
  const int b = blockIdx.y, tid = threadIdx.x;
  const double norm2 = block_sum(tid < nb ? part[(int64_t)b * nb + tid] : 0.0);
  // a matrix of zeros stays one, also with eps = 0
  const double inv = norm2 == 0.0 ? 0.0 : kXScale / (sqrt(norm2) + static_cast<double>(eps));
  const int tc = static_cast<int>(rp / 64);
  const int64_t y0 = (int64_t)(blockIdx.x / tc) * 64, x0 = (int64_t)(blockIdx.x % tc) * 64;
  const int64_t gb = (int64_t)b * m * n;
  // G's tile: rows gr0 .., columns gc0 ..
  const int64_t gr0 = TALL ? y0 : x0, gc0 = TALL ? x0 : y0;
  for (int i = tid; i < 64 * 8; i += kNsThreads) {
    const int r = i >> 3, c8 = (i & 7) * 8;
    float v[8];
    const bool row_in = gr0 + r < m;
    if (VEC && row_in && gc0 + c8 < n) {
      ns_load8<D>(g, gb + (gr0 + r) * n + gc0 + c8, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = row_in && gc0 + c8 + j < n ? ns_load<D>(g, gb + (gr0 + r) * n + gc0 + c8 + j) : 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool in = row_in && gc0 + c8 + j < n;
      s_t[r][c8 + j] = in ? static_cast<float>(static_cast<double>(v[j]) * inv) : 0.f;
    }
  }
  __syncthreads();
  for (int i = tid; i < 64 * 8; i += kNsThreads) {
    const int r = i >> 3, c8 = (i & 7) * 8;
    u32x4_t h, l;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint16_t h0, h1, l0, l1;
      ns_split(TALL ? s_t[r][c8 + 2 * j] : s_t[c8 + 2 * j][r], h0, l0);
      ns_split(TALL ? s_t[r][c8 + 2 * j + 1] : s_t[c8 + 2 * j + 1][r], h1, l1);
      h[j] = h0 | (static_cast<uint32_t>(h1) << 16);
      l[j] = l0 | (static_cast<uint32_t>(l1) << 16);
    }
    const int64_t at = (int64_t)b * cp * rp + (y0 + r) * rp + x0 + c8;
    *reinterpret_cast<u32x4_t*>(yhi + at) = h;
    *reinterpret_cast<u32x4_t*>(ylo + at) = l;
  }
}

// ---------------------------------------------------------------- products

enum NsMode : int { kGram = 0, kSquare = 1, kUpdate = 2, kOutTall = 3, kOutWide = 4 };

struct NsArgs {
  const uint16_t* y;   // (B, cp, rp) hi
  uint16_t* ylo;       // (B, cp, rp) lo, updated in place
  uint16_t* ynext;     // (B, cp, rp) hi of the next step
  uint16_t* gram;      // (B, rp, rp) A
  uint16_t* q;         // (B, rp, rp) Q
  uint16_t* out;       // (B, m, n)
  int cp, rp;
  int om, on;          // m, n: rows and columns of the output
  int tiles_m, tiles_n, tiles;  // tiles per matrix (symmetric products: the upper triangle)
  float a, b, c;       // this step's coefficients
  float diag;          // added to Q's diagonal (a in the last step)
  float scale;
  int out_bf16;
};

typedef short s16x4_t __attribute__((ext_vector_type(4)));

// Swizzled place of 16-byte chunk ch (8 columns) of k row kr in a k-major
// stage W columns wide: 32-byte pairs move so that the 16 k rows that one
// transposing read touches fall on different banks.
template <int W>
__device__ __forceinline__ int ns_kpos(int kr, int ch) {
  const int swz = W == 128 ? (kr & 3) | (((kr >> 3) & 1) << 2) : ((kr >> 1) & 1) | (((kr >> 3) & 1) << 1);
  return kr * (W * 2) + (((ch >> 1) ^ swz) << 5) + ((ch & 1) << 4);
}
// Place of 16-byte chunk c of row r in a K-contiguous stage (128-byte rows).
__device__ __forceinline__ int ns_rpos(int r, int c) { return r * 128 + ((c ^ ((r >> 1) & 7)) << 4); }

// One W x W tile of a product. 4 waves as 2 x 2, K in stages of 64 through a
// two-buffer LDS ring: the next stage is loaded into registers while this one
// is multiplied. Each MFMA takes the second operand's fragment first, so a
// lane ends with four consecutive columns of one row.
template <int W, int MODE>
__global__ __launch_bounds__(kNsThreads) void ns_gemm_kernel(NsArgs p) {
  constexpr bool KMAJ = MODE == kGram;
  constexpr bool SYM = MODE == kGram || MODE == kSquare;
  constexpr int OB = W * 128;      // bytes of one operand's stage
  constexpr int NL = W / 32;       // 16-byte loads per thread, operand and stage
  constexpr int F = W / 32;        // 16-row fragments per wave and operand
  constexpr int PITCH = W * 2 + 16;
  __shared__ __attribute__((aligned(16))) char smem[4 * OB];
  static_assert(W * PITCH <= 4 * OB, "the output tile is staged in the operands' place");

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int b = blockIdx.x / p.tiles;
  int t = blockIdx.x - b * p.tiles;
  int tm, tn;
  if constexpr (SYM) {
    tm = 0;
    while (t >= p.tiles_n - tm) {
      t -= p.tiles_n - tm;
      ++tm;
    }
    tn = tm + t;
  } else {
    tm = t / p.tiles_n;
    tn = t - tm * p.tiles_n;
  }
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

  // this thread's loads: source of stage 0, LDS place
  const u32x4_t* src[2][NL];
  int dst[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int q = tid + i * kNsThreads;
    if constexpr (KMAJ) {
      const int kr = q / (W / 8), ch = q - kr * (W / 8);
      // columns beyond the matrix read its last ones; they are not stored
      const int ca = row0 + ch * 8 < na ? row0 + ch * 8 : na - 8;
      const int cb = col0 + ch * 8 < nbn ? col0 + ch * 8 : nbn - 8;
      src[0][i] = reinterpret_cast<const u32x4_t*>(opa + (int64_t)kr * p.rp + ca);
      src[1][i] = reinterpret_cast<const u32x4_t*>(opb + (int64_t)kr * p.rp + cb);
      dst[i] = ns_kpos<W>(kr, ch);
    } else {
      const int r = q >> 3, ch = q & 7;
      const int ra = row0 + r < na ? row0 + r : na - 1;
      const int rb = col0 + r < nbn ? col0 + r : nbn - 1;
      src[0][i] = reinterpret_cast<const u32x4_t*>(opa + (int64_t)ra * p.rp + ch * 8);
      src[1][i] = reinterpret_cast<const u32x4_t*>(opb + (int64_t)rb * p.rp + ch * 8);
      dst[i] = ns_rpos(r, ch);
    }
  }
  const int64_t step = KMAJ ? (int64_t)8 * p.rp : 8;  // 16-byte pieces per stage

  f32x4_t acc[F][F];
#pragma unroll
  for (int i = 0; i < F; ++i)
#pragma unroll
    for (int j = 0; j < F; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int wr = (wave >> 1) * (W / 2), wc = (wave & 1) * (W / 2);

  auto frag = [&](const char* s, int x0, int ks) {
    if constexpr (KMAJ) {
      const int j = lane & 15, g = lane >> 4;
      const int kr = ks * 32 + g * 8 + (j >> 2);
      // the half h = 1 lies 4 k rows on, where the swizzle is the same for
      // W = 128 and for W = 64 (bits 0, 1 and 3 of the k row)
      const char* q = s + ns_kpos<W>(kr, x0 >> 3) + ((j & 3) << 3);
      const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4_t*)(q));
      const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (__attribute__((address_space(3))) s16x4_t*)(q + 4 * W * 2));
      const u32x2_t l2 = bit_cast<u32x2_t>(lo), h2 = bit_cast<u32x2_t>(hi);
      return bit_cast<f16x8_t>(u32x4_t{l2[0], l2[1], h2[0], h2[1]});
    } else {
      return *reinterpret_cast<const f16x8_t*>(s + ns_rpos(x0 + (lane & 15), ks * 4 + (lane >> 4)));
    }
  };

  u32x4_t va[NL], vb[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    va[i] = src[0][i][0];
    vb[i] = src[1][i][0];
  }
  for (int s = 0; s < stages; ++s) {
    char* sa = smem + (s & 1) * 2 * OB;
    char* sb = sa + OB;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      *reinterpret_cast<u32x4_t*>(sa + dst[i]) = va[i];
      *reinterpret_cast<u32x4_t*>(sb + dst[i]) = vb[i];
    }
    __syncthreads();
    if (s + 1 < stages) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        va[i] = src[0][i][(s + 1) * step];
        vb[i] = src[1][i][(s + 1) * step];
      }
    }
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      f16x8_t fa[F], fb[F];
#pragma unroll
      for (int i = 0; i < F; ++i) fa[i] = frag(sa, wr + i * 16, ks);
#pragma unroll
      for (int i = 0; i < F; ++i) fb[i] = frag(sb, wc + i * 16, ks);
#pragma unroll
      for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(fb[j], fa[i], acc[i][j], 0, 0, 0);
    }
  }
  __syncthreads();  // every read of the operands is done: their place takes the output

  auto stage4 = [&](int i, int j, uint32_t x, uint32_t y) {
    *reinterpret_cast<u32x2_t*>(smem + (wr + i * 16 + (lane & 15)) * PITCH +
                                (wc + j * 16 + 4 * (lane >> 4)) * 2) = u32x2_t{x, y};
  };
  auto pack = [](float x, float y) {
    return f32_to_f16_bits(x) | (static_cast<uint32_t>(f32_to_f16_bits(y)) << 16);
  };
  // the staged tile -> rows row0 .., columns col0 .. of a matrix of `rows`
  // rows of `ld` values, 16 bytes at a time (rows are whole pieces)
  auto store = [&](uint16_t* out, int ld, int rows, int cols) {
    for (int q = tid; q < W * (W / 8); q += kNsThreads) {
      const int r = q / (W / 8), c8 = (q - r * (W / 8)) * 8;
      if (row0 + r < rows && col0 + c8 < cols)
        *reinterpret_cast<u32x4_t*>(out + (int64_t)(row0 + r) * ld + col0 + c8) =
            *reinterpret_cast<const u32x4_t*>(smem + r * PITCH + c8 * 2);
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
          u32x2_t av{0u, 0u};
          if (r < p.rp && c < p.rp)
            av = *reinterpret_cast<const u32x2_t*>(A + (int64_t)r * p.rp + c);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float g = f16_bits_to_f32((av[e >> 1] >> (16 * (e & 1))) & 0xFFFFu);
            v[e] = p.b * g + p.c * (acc[i][j][e] * kSqScale) + (r == c + e ? p.diag * kDiag : 0.f);
          }
        }
        stage4(i, j, pack(v[0], v[1]), pack(v[2], v[3]));
      }
    __syncthreads();
    uint16_t* out = (MODE == kGram ? p.gram : p.q) + b * asz;
    store(out, p.rp, p.rp, p.rp);
    if (tm != tn) {  // the mirrored tile: columns of the staged one as rows
      for (int q = tid; q < W * (W / 8); q += kNsThreads) {
        const int r8 = (q / W) * 8, c = q - (q / W) * W;
        if (col0 + c < p.rp && row0 + r8 < p.rp) {
          u32x4_t o;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint16_t x = *reinterpret_cast<const uint16_t*>(smem + (r8 + 2 * e) * PITCH + c * 2);
            const uint16_t y =
                *reinterpret_cast<const uint16_t*>(smem + (r8 + 2 * e + 1) * PITCH + c * 2);
            o[e] = x | (static_cast<uint32_t>(y) << 16);
          }
          *reinterpret_cast<u32x4_t*>(out + (int64_t)(col0 + c) * p.rp + row0 + r8) = o;
        }
      }
    }
  } else if constexpr (MODE == kUpdate) {
    uint16_t* lo = p.ylo + b * ysz;
    u32x2_t keep[F][F];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const int r = row0 + wr + i * 16 + (lane & 15);
        const int c = col0 + wc + j * 16 + 4 * (lane >> 4);
        u32x2_t hv{0u, 0u}, lv{0u, 0u};
        if (r < p.cp && c < p.rp) {
          hv = *reinterpret_cast<const u32x2_t*>(Y + (int64_t)r * p.rp + c);
          lv = *reinterpret_cast<const u32x2_t*>(lo + (int64_t)r * p.rp + c);
        }
        uint16_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = f16_bits_to_f32((hv[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) +
                          f16_bits_to_f32((lv[e >> 1] >> (16 * (e & 1))) & 0xFFFFu) * (1.f / kLoScale);
          ns_split(p.a * x + acc[i][j][e] * kUpdScale, h[e], l[e]);
        }
        stage4(i, j, h[0] | ((uint32_t)h[1] << 16), h[2] | ((uint32_t)h[3] << 16));
        keep[i][j] = u32x2_t{l[0] | ((uint32_t)l[1] << 16), l[2] | ((uint32_t)l[3] << 16)};
      }
    __syncthreads();
    store(p.ynext + b * ysz, p.rp, p.cp, p.rp);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) stage4(i, j, keep[i][j][0], keep[i][j][1]);
    __syncthreads();
    store(lo, p.rp, p.cp, p.rp);
  } else {
    const float sc = p.scale * kOutScale;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
      for (int j = 0; j < F; ++j) {
        uint32_t w[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = acc[i][j][2 * e] * sc, y = acc[i][j][2 * e + 1] * sc;
          w[e] = p.out_bf16 ? f32_to_bf16_bits(x) | (static_cast<uint32_t>(f32_to_bf16_bits(y)) << 16)
                            : pack(x, y);
        }
        stage4(i, j, w[0], w[1]);
      }
    __syncthreads();
    uint16_t* out = p.out + (int64_t)b * p.om * p.on;
    if (p.on % 8 == 0) {
      store(out, p.on, p.om, p.on);
    } else {  // rows that are not whole 16-byte pieces
      for (int q = tid; q < W * W; q += kNsThreads) {
        const int r = q / W, c = q - r * W;
        if (row0 + r < p.om && col0 + c < p.on)
          out[(int64_t)(row0 + r) * p.on + col0 + c] =
              *reinterpret_cast<const uint16_t*>(smem + r * PITCH + c * 2);
      }
    }
  }
}

// ---------------------------------------------------------------- host

struct NsLayout {
  int64_t r, c, rp, cp;
  size_t part, y0, y1, lo, gram, q, total;
};

static bool ns_sizes_ok(int64_t batch, int64_t m, int64_t n) {
  return batch >= 1 && batch <= 65535 && m >= 1 && n >= 1 && m <= 65536 && n <= 65536;
}

static NsLayout ns_layout(int64_t batch, int64_t m, int64_t n) {
  NsLayout L{};
  L.r = m < n ? m : n;
  L.c = m < n ? n : m;
  L.rp = (L.r + kNsPad - 1) / kNsPad * kNsPad;
  L.cp = (L.c + kNsPad - 1) / kNsPad * kNsPad;
  const size_t y = static_cast<size_t>(batch * L.cp * L.rp) * 2;  // multiples of 8 KiB
  const size_t a = static_cast<size_t>(batch * L.rp * L.rp) * 2;
  L.part = 0;
  L.y0 = (static_cast<size_t>(batch) * kNsMaxPart * sizeof(double) + 255) / 256 * 256;
  L.y1 = L.y0 + y;
  L.lo = L.y1 + y;
  L.gram = L.lo + y;
  L.q = L.gram + a;
  L.total = L.q + a;
  return L;
}

template <int D>
static void ns_start(const void* g, int64_t batch, int64_t m, int64_t n, const NsLayout& L,
                     float eps, double* part, uint16_t* y, uint16_t* lo, hipStream_t stream) {
  const int64_t mn = m * n;
  constexpr int per16 = D == MC2_F32 ? 4 : 8;
  int64_t nb = (mn + kNsThreads * 32 - 1) / (kNsThreads * 32);
  nb = nb < kNsMaxPart ? nb : kNsMaxPart;
  const dim3 gn(static_cast<unsigned>(nb), static_cast<unsigned>(batch)), blk(kNsThreads);
  const bool flat = mn % 8 == 0;  // every matrix starts on 16 bytes and is whole pieces
  if (flat) hipLaunchKernelGGL((ns_norm_kernel<D, true>), gn, blk, 0, stream, g, mn, part);
  else hipLaunchKernelGGL((ns_norm_kernel<D, false>), gn, blk, 0, stream, g, mn, part);
  const dim3 gi(static_cast<unsigned>(L.cp / 64 * (L.rp / 64)), static_cast<unsigned>(batch));
  const bool rows16 = n % 8 == 0;
  static_assert(per16 == 4 || per16 == 8, "16-byte pieces");
  auto init = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, gi, blk, 0, stream, g, m, n, part, static_cast<int>(nb), eps, L.cp,
                       L.rp, y, lo);
  };
  if (m >= n) rows16 ? init(ns_init_kernel<D, true, true>) : init(ns_init_kernel<D, true, false>);
  else rows16 ? init(ns_init_kernel<D, false, true>) : init(ns_init_kernel<D, false, false>);
}

template <int MODE>
static void ns_product(NsArgs p, int64_t batch, hipStream_t stream) {
  constexpr bool SYM = MODE == kGram || MODE == kSquare;
  const int rows = MODE == kUpdate || MODE == kOutTall ? p.cp : p.rp;
  const int cols = MODE == kOutWide ? p.cp : p.rp;
  auto plan = [&](int w) {
    p.tiles_m = (rows + w - 1) / w;
    p.tiles_n = (cols + w - 1) / w;
    p.tiles = SYM ? p.tiles_n * (p.tiles_n + 1) / 2 : p.tiles_m * p.tiles_n;
    return batch * p.tiles;
  };
  // 128 x 128 tiles where they fill the chip, else 64 x 64
  int64_t grid = plan(128);
  if (grid >= num_cus()) {
    hipLaunchKernelGGL((ns_gemm_kernel<128, MODE>), dim3(static_cast<unsigned>(grid)),
                       dim3(kNsThreads), 0, stream, p);
  } else {
    grid = plan(64);
    hipLaunchKernelGGL((ns_gemm_kernel<64, MODE>), dim3(static_cast<unsigned>(grid)),
                       dim3(kNsThreads), 0, stream, p);
  }
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
  // grids are 32-bit: tiles of 64 x 64 of the largest product
  if (batch * (L.cp / 64) * (L.cp / 64) > 0x7fffffff) return MC2_ERR_SHAPE;
  if (ws_bytes < L.total) return MC2_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  double* part = reinterpret_cast<double*>(ws + L.part);
  uint16_t* y[2] = {reinterpret_cast<uint16_t*>(ws + L.y0), reinterpret_cast<uint16_t*>(ws + L.y1)};
  uint16_t* lo = reinterpret_cast<uint16_t*>(ws + L.lo);
  if (in_dtype == MC2_F32) ns_start<MC2_F32>(g, batch, m, n, L, eps, part, y[0], lo, stream);
  else if (in_dtype == MC2_BF16) ns_start<MC2_BF16>(g, batch, m, n, L, eps, part, y[0], lo, stream);
  else ns_start<MC2_F16>(g, batch, m, n, L, eps, part, y[0], lo, stream);
  NsArgs p{};
  p.ylo = lo;
  p.gram = reinterpret_cast<uint16_t*>(ws + L.gram);
  p.q = reinterpret_cast<uint16_t*>(ws + L.q);
  p.out = static_cast<uint16_t*>(out);
  p.cp = static_cast<int>(L.cp);
  p.rp = static_cast<int>(L.rp);
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
    p.diag = last ? p.a : 0.f;
    ns_product<kGram>(p, batch, stream);
    ns_product<kSquare>(p, batch, stream);
    if (!last) ns_product<kUpdate>(p, batch, stream);
    else if (m >= n) ns_product<kOutTall>(p, batch, stream);
    else ns_product<kOutWide>(p, batch, stream);
  }
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}
