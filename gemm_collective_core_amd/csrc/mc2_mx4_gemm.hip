// Product of two MX4 operands in the chunk schedule of the rank-chunked GEMM
// (MatmulReduceScatter / AllGatherMatmul compute share), for gfx950.
//
// Two kernels. Where there are tiles enough, mx4_tile_kernel computes 256 x 256
// or 128 x 128 of the output in a workgroup (mx4_core.hpp), bound by the matrix
// instructions. With few rows the weights' bytes bound the call, and
// mx4_rows_kernel reads them straight into registers, each wave a part of K.
#include "mc2_tiles.hpp"
#include "mx4_core.hpp"

namespace mc2 {

struct Mx4Args {
  const char* A;
  const char* As;
  const char* B;
  const char* Bs;
  char* out;
  const uint16_t* bias;
  int64_t m, n, nb, pitch, ldo;
  // chunk schedule, as the rank-chunked GEMM's: W chunks of mc rows from
  // first_chunk on, each in `sub` pieces of sq rows, one more for the first sr
  int64_t mc, sq;
  int world, first_chunk, sub, sr;
  int tiles_n, tiles_m1, tiles_m0;  // tile columns, tile rows of a long and a short piece
  int tiles_per_chunk;
  int round;
  int n_full;  // work units below are whole tiles, the rest half tiles (two a tile)
  uint32_t* flags;
  uint32_t* counters;
  uint32_t epoch;
  int store_wt;
};

// Tile t: its first row and column, the end of its piece, the piece and how
// many tiles that has. Row blocks are fastest inside a piece.
struct Mx4Pos {
  int64_t row0, row_end, col0;
  int seg, seg_tiles;
};

__device__ __forceinline__ Mx4Pos mx4_pos(const Mx4Args& p, int tile, int bm, int bn) {
  Mx4Pos q;
  const int seq = tile / p.tiles_per_chunk;
  int t = tile - seq * p.tiles_per_chunk;
  int c = p.first_chunk + seq;
  c = c >= p.world ? c - p.world : c;
  const int per_long = p.tiles_m1 * p.tiles_n, per_short = p.tiles_m0 * p.tiles_n;
  int j = 0;
  const bool in_long = t < p.sr * per_long;
  if (in_long) {
    j = t / per_long;
    t -= j * per_long;
  } else {
    t -= p.sr * per_long;
    j = t / per_short;
    t -= j * per_short;
    j += p.sr;
  }
  const int rows = in_long ? p.tiles_m1 : p.tiles_m0;
  q.seg = c * p.sub + j;
  q.seg_tiles = in_long ? per_long : per_short;
  const int64_t seg0 = c * p.mc + j * p.sq + (j < p.sr ? j : p.sr);
  q.row_end = seg0 + p.sq + (j < p.sr ? 1 : 0);
  const int tn = t / rows;
  q.row0 = seg0 + static_cast<int64_t>(t - tn * rows) * bm;
  q.col0 = static_cast<int64_t>(tn) * bn;
  return q;
}

// Counts `weight` half tiles as done; the last of a segment raises its flag (the
// protocol of the rank-chunked GEMM: a release per tile, one acquire per
// segment).
__device__ __forceinline__ void mx4_count(const Mx4Args& p, int seg, int seg_tiles,
                                          uint32_t weight) {
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (threadIdx.x == 0) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "agent");
    const uint32_t prev = __hip_atomic_fetch_add(&p.counters[seg], weight, __ATOMIC_RELAXED,
                                                 __HIP_MEMORY_SCOPE_AGENT);
    if (prev + weight == 2u * static_cast<uint32_t>(seg_tiles)) {
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
      __hip_atomic_store(&p.counters[seg], 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      __hip_atomic_store(&p.flags[seg], p.epoch, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_SYSTEM);
    }
  }
}

template <class TS>
constexpr int mx4_smem() {
  constexpr int staged = TS::BM * (TS::BN * 2 + 16);
  return TS::kLoopBytes > staged ? TS::kLoopBytes : staged;
}

// The tile at t, which has rows.
template <class TS, Out O, bool KTAIL>
__device__ __forceinline__ void mx4_tile(const Mx4Args& p, lds_t* smem, const Mx4Pos& t) {
  constexpr int OS = OutInfo<O>::bytes;
  constexpr int pitch = TS::BN * 2 + 16;  // staged 16-bit rows
  const int64_t ld = p.nb * 16;
  const MxSide a{p.A + t.row0 * ld, p.As + t.row0 * p.pitch, t.row_end - 1 - t.row0};
  const MxSide b{p.B + t.col0 * ld, p.Bs + t.col0 * p.pitch, p.n - 1 - t.col0};
  f32x16_t acc[TS::FM][TS::FN];
  mainloop_mx4<TS, KTAIL>(smem, a, b, p.nb, p.pitch, acc);

  // A lane holds, of each 32 x 32 block, row (lane & 31) and the four columns
  // 8 g + 4 (lane >> 5) .. + 3 for g = 0 .. 3.
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wrow0 = (wave >> 1) * TS::WTM, wcol0 = (wave & 1) * TS::WTN;
  char* base = p.out + t.row0 * p.ldo + t.col0 * OS;
  const int64_t nrows = t.row_end - t.row0, ncols = p.n - t.col0;
  const __amdgpu_buffer_rsrc_t r = make_rsrc(base);
#pragma unroll
  for (int fn = 0; fn < TS::FN; ++fn)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int cc = wcol0 + fn * 32 + 8 * g + 4 * (lane >> 5);
      float bv[4] = {0.f, 0.f, 0.f, 0.f};
      if (p.bias && cc < ncols) {
#pragma unroll
        for (int i = 0; i < 4; ++i) bv[i] = bf16_bits_to_f32(p.bias[t.col0 + cc + i]);
      }
#pragma unroll
      for (int fm = 0; fm < TS::FM; ++fm) {
        const int rr = wrow0 + fm * 32 + (lane & 31);
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = acc[fm][fn][4 * g + i] + bv[i];
        if constexpr (OS == 2)
          *reinterpret_cast<MC2_LDS u32x2_t*>(smem + rr * pitch + cc * 2) = pack4<O>(v);
        else if (rr < nrows && cc < ncols)
          store4<O>(base, r, rr * p.ldo + cc * OS, v, p.store_wt != 0);
      }
    }
  if constexpr (OS == 2) {
    __syncthreads();
    store_staged<TS::NT>(smem, pitch, TS::BN * 2, TS::BM, p.out + t.row0 * p.ldo, p.ldo, nrows,
                         t.col0 * 2, p.n * 2, p.store_wt != 0);
  }
}

using MxL = MxTile<256, 256, 1>;
using MxH = MxTile<128, 256, 2>;  // half a large tile
using MxS = MxTile<128, 128, 2>;

// One workgroup per work unit: a tile, or of a last round of 256 x 256 tiles
// that would leave half of the CUs idle, the upper or lower half of one.
template <class TS, Out O, bool KTAIL>
__global__ __launch_bounds__(TS::NT, TS::BM == 256 ? 1 : 2) void mx4_tile_kernel(Mx4Args p) {
  __shared__ __attribute__((aligned(16))) char smem_raw[mx4_smem<TS>()];
  lds_t* smem = (lds_t*)smem_raw;
  const int u = xcd_tile(blockIdx.x, p.round, gridDim.x);
  Mx4Pos t;
  if (TS::BM == 256 && u >= p.n_full) {
    if constexpr (TS::BM == 256) {
      const int v = u - p.n_full;
      t = mx4_pos(p, p.n_full + (v >> 1), TS::BM, TS::BN);
      t.row0 += (v & 1) * MxH::BM;
      if (t.row0 < t.row_end) mx4_tile<MxH, O, KTAIL>(p, smem, t);
      if (p.flags) mx4_count(p, t.seg, t.seg_tiles, 1u);
    }
    return;
  }
  t = mx4_pos(p, u, TS::BM, TS::BN);
  mx4_tile<TS, O, KTAIL>(p, smem, t);
  if (p.flags) mx4_count(p, t.seg, t.seg_tiles, 2u);
}

// ------------------------------------------------------------------- few rows
//
// A workgroup of NW waves computes MT x 16 rows by NT x 16 columns: wave w sums the
// 512-value chunks w, w + NW, ... of K, and the waves' sums are added in order
// through LDS. A lane takes row (lane & 15) of A and of B and, of a chunk, the
// blocks 4 j + g, g = lane >> 4: a load is 64 contiguous bytes of 16 rows. The 16
// scale bytes of a row's chunk are one load, from which a lane picks its own.
// The weights are read once, straight into registers. Bound by latency: 1 x 8192
// x 3584 (15.6 MB) 5.8 us, 64 x 8192 x 3584 11.6 us.
typedef int i32x8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ i32x8_t mx4_op(u32x4_t v) {
  return i32x8_t{static_cast<int>(v[0]), static_cast<int>(v[1]), static_cast<int>(v[2]),
                 static_cast<int>(v[3]), 0, 0, 0, 0};
}

template <int MT, int NT, int NW, Out O>
__global__ __launch_bounds__(NW * 64) void mx4_rows_kernel(Mx4Args p) {
  constexpr int OS = OutInfo<O>::bytes;
  __shared__ f32x4_t red[NW][NT][MT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, g = lane >> 4;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * (MT * 16);
  const int64_t col0 = static_cast<int64_t>(blockIdx.x) * (NT * 16);
  const int64_t ld = p.nb * 16;
  const char* bc[NT];
  const char* bs[NT];
#pragma unroll
  for (int f = 0; f < NT; ++f) {
    const int64_t col = col0 + f * 16 + r < p.n ? col0 + f * 16 + r : p.n - 1;
    bc[f] = p.B + col * ld + g * 16;
    bs[f] = p.Bs + col * p.pitch;
  }
  const char* ac[MT];
  const char* as[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int64_t row = row0 + i * 16 + r < p.m ? row0 + i * 16 + r : p.m - 1;
    ac[i] = p.A + row * ld + g * 16;
    as[i] = p.As + row * p.pitch;
  }
  f32x4_t acc[NT][MT];
#pragma unroll
  for (int f = 0; f < NT; ++f)
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[f][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int64_t chunks = p.pitch / 16;
  for (int64_t c = wave; c < chunks; c += NW) {
    const int64_t left = p.nb - c * 16 - g;  // block 4 j of the lane's exists where 4 j < left
    u32x4_t vb[NT][4], sb[NT], va[MT][4], sa[MT];
#pragma unroll
    for (int f = 0; f < NT; ++f) {
      sb[f] = *reinterpret_cast<const u32x4_t*>(bs[f] + c * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        vb[f][j] = 4 * j < left ? *reinterpret_cast<const u32x4_t*>(bc[f] + c * 256 + j * 64) : zero_v4();
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
      sa[i] = *reinterpret_cast<const u32x4_t*>(as[i] + c * 16);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        va[i][j] = 4 * j < left ? *reinterpret_cast<const u32x4_t*>(ac[i] + c * 256 + j * 64) : zero_v4();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int f = 0; f < NT; ++f)
#pragma unroll
        for (int i = 0; i < MT; ++i)
          acc[f][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              mx4_op(vb[f][j]), mx4_op(va[i][j]), acc[f][i], 4, 4, 0,
              static_cast<int>(sb[f][j] >> (8 * g)), 0, static_cast<int>(sa[i][j] >> (8 * g)));
  }
#pragma unroll
  for (int f = 0; f < NT; ++f)
#pragma unroll
    for (int i = 0; i < MT; ++i) red[wave][f][i][lane] = acc[f][i];
  __syncthreads();
  // B was the first operand: a lane holds row (lane & 15), columns 4 g .. + 3
  for (int q = threadIdx.x; q < NT * MT * 64; q += NW * 64) {
    const int f = q / (MT * 64), i = (q >> 6) % MT, l = q & 63;
    f32x4_t s = red[0][f][i][l];
#pragma unroll
    for (int w = 1; w < NW; ++w) s += red[w][f][i][l];
    const int64_t row = row0 + i * 16 + (l & 15), cc = col0 + f * 16 + 4 * (l >> 4);
    if (row < p.m && cc < p.n) {
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = s[j] + (p.bias ? bf16_bits_to_f32(p.bias[cc + j]) : 0.f);
      char* o = p.out + row * p.ldo + cc * OS;
      const auto d = pack4<O>(v);
      if constexpr (OS == 2) *reinterpret_cast<u32x2_t*>(o) = d;
      else *reinterpret_cast<u32x4_t*>(o) = d;
    }
  }
}

// ------------------------------------------------------------------ host side

template <int MT, int NT, Out O>
static void launch_rows_of(const Mx4Args& a, hipStream_t s) {
  constexpr int NW = 8;
  const dim3 grid(static_cast<unsigned>((a.n + 16 * NT - 1) / (16 * NT)),
                  static_cast<unsigned>((a.m + 16 * MT - 1) / (16 * MT)));
  hipLaunchKernelGGL((mx4_rows_kernel<MT, NT, NW, O>), grid, dim3(NW * 64), 0, s, a);
}
// Workgroups of 32 rows by 16 * nt columns.
static int64_t rows_groups(const Mx4Args& a, int64_t nt) {
  return (a.m + 31) / 32 * ((a.n + 16 * nt - 1) / (16 * nt));
}

// The narrowest tile whose workgroups find a CU each, else the widest (us on the
// GPU at 32 x 8192 x 8192, 16 / 32 / 64 columns, 512 / 256 / 128 workgroups: 17.2
// / 13.9 / 17.3; at 64 x 8192 x 3584, 448 / 224 / 112: 16.9 / 12.6 / 17.4; for up
// to 16 rows, which 16-row tiles serve, at 16 x 8192 x 8192: 12.4 / 11.4 / 14.7).
template <Out O>
static hipError_t launch_rows(const Mx4Args& a, hipStream_t s) {
  const int64_t cus = num_cus();
  if (a.m <= 16) {
    if (rows_groups(a, 1) <= cus) launch_rows_of<1, 1, O>(a, s);
    else launch_rows_of<1, 2, O>(a, s);
  } else {
    if (rows_groups(a, 1) <= cus) launch_rows_of<2, 1, O>(a, s);
    else if (rows_groups(a, 2) <= cus) launch_rows_of<2, 2, O>(a, s);
    else launch_rows_of<2, 4, O>(a, s);
  }
  return hipGetLastError();
}

template <class TS, Out O>
static hipError_t launch_tiles(const Mx4Args& a, unsigned blocks, hipStream_t s) {
  if (a.nb % 8 == 0)
    hipLaunchKernelGGL((mx4_tile_kernel<TS, O, false>), dim3(blocks), dim3(TS::NT), 0, s, a);
  else
    hipLaunchKernelGGL((mx4_tile_kernel<TS, O, true>), dim3(blocks), dim3(TS::NT), 0, s, a);
  return hipGetLastError();
}

// Tiles of one chunk for tiles of bm rows and tn tile columns.
static int64_t mx4_chunk_tiles(const Mx4Args& a, int bm, int64_t tn) {
  return (a.sr * ((a.sq + bm) / bm) + (a.sub - a.sr) * ((a.sq + bm - 1) / bm)) * tn;
}

// A call without flags takes mx4_rows_kernel for up to 64 rows, and for more
// where its widest tiles find a CU each (128 x 8192 x 3584: 17.4 us against 21.0
// with 128 x 128 tiles; 256 x 2048 x 1024: 5.2 against 7.6; past one round the
// tiles win: 256 x 8192 x 3584 32 against 21).
static bool few_rows(const Mx4Args& a) {
  return !a.flags && (a.m <= 64 || rows_groups(a, 4) <= num_cus());
}

template <Out O>
static int run_mx4(Mx4Args a, hipStream_t s) {
  if (few_rows(a)) return launch_rows<O>(a, s) == hipSuccess ? MC2_OK : MC2_ERR_HIP;
  const int64_t cus = num_cus();
  const int64_t tl = mx4_chunk_tiles(a, 256, (a.n + 255) / 256) * a.world;
  // 128 x 128 tiles while they find a CU each, then 256 x 256 (us, small against
  // large: 1024 x 4096 x 4096, 64 large tiles, 15.2 / 18.4; 1280 x 4096 x 4096, 80,
  // 22.0 / 18.8; 1024 x 8192 x 5120, 80, 38.6 / 33.6)
  const bool large = 4 * tl > cus;
  const int bm = large ? 256 : 128;
  a.tiles_n = static_cast<int>((a.n + bm - 1) / bm);
  const int64_t m1 = (a.sq + bm) / bm, m0 = (a.sq + bm - 1) / bm;
  const int64_t per = mx4_chunk_tiles(a, bm, a.tiles_n);
  if (m1 * a.tiles_n > 0x3fffff || per > 0x7fffff || per * a.world > 0x7fffff) return MC2_ERR_SHAPE;
  a.tiles_m1 = static_cast<int>(m1);
  a.tiles_m0 = static_cast<int>(m0);
  a.tiles_per_chunk = static_cast<int>(per);
  a.round = static_cast<int>(cus / 8 * 8) * (large ? 1 : 2);
  // A last (or only) round of 256 x 256 tiles that is at most half full runs as
  // half tiles (us, whole against halves: 16384 x 8192 x 3584 in 8 chunks 242 /
  // 234; 8192 x 4096 x 2560 67 / 58.5; 2048 x 4096 x 4096 29.7 / 22.4).
  const int64_t tiles = per * a.world, rem = large ? tiles % cus : 0;
  const int64_t halves = 2 * rem <= cus ? rem : 0;
  a.n_full = static_cast<int>(tiles - halves);
  const unsigned blocks = static_cast<unsigned>(tiles + halves);
  const hipError_t e = large ? launch_tiles<MxL, O>(a, blocks, s) : launch_tiles<MxS, O>(a, blocks, s);
  return e == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}

static int mx4_mm(const void* x1, const void* s1, const void* x2, const void* s2, int64_t m,
                  int64_t k, int64_t n, int W, int rank, bool gather, const void* bias,
                  int out_dtype, void* out, uint32_t* flags, uint32_t* counters, uint32_t epoch,
                  int comm_turn, hipStream_t stream) {
  if (!x1 || !s1 || !x2 || !s2 || !out) return MC2_ERR_NULL;
  if (!valid_world(W) || rank < 0 || rank >= W) return MC2_ERR_SHAPE;
  if (m < 1 || m > (int64_t{1} << 40) || m % W || k < 1 || k > MC2_MX4_MAX_K || n < 1 ||
      n > (int64_t{1} << 20))
    return MC2_ERR_SHAPE;
  if (out_dtype != MC2_BF16 && out_dtype != MC2_F16 && out_dtype != MC2_F32) return MC2_ERR_DTYPE;
  if (n % 8) return MC2_ERR_ALIGN;
  if (!aligned16(x1) || !aligned16(s1) || !aligned16(x2) || !aligned16(s2) || !aligned16(out))
    return MC2_ERR_ALIGN;
  if ((flags == nullptr) != (counters == nullptr)) return MC2_ERR_NULL;
  if (flags && epoch == 0) return MC2_ERR_SHAPE;
  if (comm_turn < 0 || comm_turn > m / W) return MC2_ERR_SHAPE;
  Mx4Args a{};
  a.A = static_cast<const char*>(x1);
  a.As = static_cast<const char*>(s1);
  a.B = static_cast<const char*>(x2);
  a.Bs = static_cast<const char*>(s2);
  a.out = static_cast<char*>(out);
  a.bias = static_cast<const uint16_t*>(bias);
  a.m = m;
  a.n = n;
  a.nb = mx4_blocks(k);
  a.pitch = mx4_pitch(k);
  a.ldo = n * (out_dtype == MC2_F32 ? 4 : 2);
  a.mc = m / W;
  a.world = W;
  a.first_chunk = gather ? rank : (rank + 1) % W;
  a.sub = comm_turn > 1 ? comm_turn : 1;
  a.sq = a.mc / a.sub;
  a.sr = static_cast<int>(a.mc % a.sub);
  a.flags = flags;
  a.counters = counters;
  a.epoch = epoch;
  a.store_wt = flags != nullptr;
  if (out_dtype == MC2_BF16) return run_mx4<Out::BF16>(a, stream);
  if (out_dtype == MC2_F16) return run_mx4<Out::F16>(a, stream);
  return run_mx4<Out::F32>(a, stream);
}

}  // namespace mc2

using namespace mc2;

extern "C" int mc2_mx4_mm_rs_local(const void* x1, const void* x1_scale, const void* x2,
                                   const void* x2_scale, int64_t m, int64_t k, int64_t n,
                                   int world_size, int rank, const void* bias, int out_dtype,
                                   void* out, uint32_t* ready_flags, uint32_t* flag_counters,
                                   uint32_t epoch, int comm_turn, hipStream_t stream) {
  return mx4_mm(x1, x1_scale, x2, x2_scale, m, k, n, world_size, rank, false, bias, out_dtype, out,
                ready_flags, flag_counters, epoch, comm_turn, stream);
}

extern "C" int mc2_mx4_ag_mm_local(const void* x_gathered, const void* x_scale, const void* x2,
                                   const void* x2_scale, int64_t m_c, int64_t k, int64_t n,
                                   int world_size, int rank, const void* bias, int out_dtype,
                                   void* out, uint32_t* ready_flags, uint32_t* flag_counters,
                                   uint32_t epoch, int comm_turn, hipStream_t stream) {
  if (m_c < 1 || m_c > (int64_t{1} << 32)) {
    if (!x_gathered || !x_scale || !x2 || !x2_scale || !out) return MC2_ERR_NULL;
    return MC2_ERR_SHAPE;
  }
  if (!valid_world(world_size)) {
    if (!x_gathered || !x_scale || !x2 || !x2_scale || !out) return MC2_ERR_NULL;
    return MC2_ERR_SHAPE;
  }
  return mx4_mm(x_gathered, x_scale, x2, x2_scale, m_c * world_size, k, n, world_size, rank, true,
                bias, out_dtype, out, ready_flags, flag_counters, epoch, comm_turn, stream);
}
