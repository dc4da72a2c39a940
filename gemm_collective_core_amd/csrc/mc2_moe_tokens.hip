// A whole MoE layer for few tokens (mc2_moe_tokens), for gfx950: two launches.
//
// Decoding reads every named expert's weights for a handful of rows, so the
// weights' bytes bound it: 75 MB for one token, top-8, of the layer with 2048 x
// 1536 and 768 x 2048 bf16 experts. Both kernels stream them once, straight from
// memory into the registers that the matrix instructions take them from:
//
//   tokens_fc1_kernel: a workgroup computes a strip of gate columns and the same
//     strip of up columns for all the rows of one expert, each wave over a part
//     of H; the waves' sums meet in LDS, SwiGLU follows, and h leaves as the sum
//     of three bf16 numbers, all the 24 bits of fp32 (see split_h).
//   tokens_fc2_kernel: the same with h and w2 for a strip of output columns. The
//     results y of a slot stay fp32 in the workspace; the workgroup that brings
//     the last one of a token adds the token's strip up, in slot order, with the
//     routing weights.
//
// A workgroup of fc1 finds its expert by itself, the a-th that a slot names, and
// that expert's slots (no sorting launch, no count on the host); a row of
// workgroups more writes what fc2 needs: the same as a plan, and each token's
// count of local slots. Rows of the 16-row operand that no slot fills are zeros,
// which load nothing, and are dropped: rows of a product do not mix, so neither
// do their NaN.
//
// Measured, fc1 and fc2: one token of the layer above 14.6 + 10.9 us (75 MB, 2.9
// TB/s); 64 tokens, all 128 experts in MX4, 52 + 52 us (316 MB). Bound by chains
// of latencies (ids, rows, products, LDS, y, counter, sum) with two workgroups a
// CU: without any read of w1 the 64 tokens still take 90 of 112 us, without one of
// w2 105, without both 80.
#include "mc2_mx4.hpp"
#include "mc2_tiles.hpp"

namespace mc2 {

constexpr int kTokMaxSlots = 4096;   // T * K
constexpr int kTokMaxExperts = 1024;
constexpr int kCpolAgent = 0x10;     // sc1: coherent over the XCDs' L2s
constexpr int kTokMaxPer = 2;        // strips a workgroup
constexpr int kHParts = 3;           // bf16 numbers that hold an h
constexpr int kTokMany = 2;          // 16-row operands at a time where an expert has more slots
                                     // (four would leave one workgroup a CU its registers)

// Strips of fc2 at most: 16 columns each.
__host__ __device__ constexpr int64_t tok_strips(int64_t H) { return (H + 15) / 16; }

struct TokArgs {
  const uint16_t* x;
  const int32_t* sel;
  const float* probs;
  const char* w1;
  const char* w1s;
  const char* w2;
  const char* w2s;
  uint16_t* out;
  int32_t* left;      // (strip of fc2, token): local slots whose y is still to come
  i32x4_t* plan;      // expert, slots, place of the first in list, experts named
  uint16_t* list;     // local slots, expert after expert
  uint16_t* h[kHParts];
  float* y;
  int32_t* dev_err;
  int64_t H, I;
  int T, K, TK, E, e0, El;
  int strips1, strips2, per1, per2;  // strips of a matrix, and of a workgroup
};

// Which expert (of this rank's) a workgroup works for, and how many slots of it.
struct Expert {
  int e, count;
};

struct PickMem {
  int count;
  uint16_t list[kTokMaxSlots];
};

__device__ __forceinline__ int local_id(const TokArgs& p, int s) {
  const int e = p.sel[s] - p.e0;
  return s < p.TK && e >= 0 && e < p.El ? e : -1;
}

// The expert of row `a` of workgroups (e = -1: none) and its slots in mem.list,
// in any order: rows of a product do not mix.
//   Up to 64 slots: the a-th expert that they name, in the order of their first
// slots; a lane each and no barrier, every wave finds the same and writes the
// same list.
//   More: expert a, of which the row may find no slot.
template <int NT>
__device__ __forceinline__ Expert pick_expert(const TokArgs& p, int a, PickMem& mem) {
  const int lane = threadIdx.x & 63;
  Expert r{-1, 0};
  if (p.TK <= 64) {
    const int id = local_id(p, lane < p.TK ? lane : p.TK - 1);
    const uint64_t valid = __ballot(id >= 0 && lane < p.TK);
    uint64_t left = valid;
    for (;; --a) {
      if (left == 0) return r;
      const int e = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
      const uint64_t same = __ballot(id == e) & valid;
      left &= ~same;
      if (a == 0) {
        if ((same >> lane) & 1)
          mem.list[__popcll(same & ((uint64_t{1} << lane) - 1))] = static_cast<uint16_t>(lane);
        r.e = e;
        r.count = __popcll(same);
        return r;
      }
    }
  }
  if (threadIdx.x == 0) mem.count = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < p.TK; b += 4 * NT) {  // four loads in flight
    int id[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) id[i] = p.sel[b + i * NT < p.TK ? b + i * NT : p.TK - 1] - p.e0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (id[i] == a && b + i * NT < p.TK)
        mem.list[atomicAdd(&mem.count, 1)] = static_cast<uint16_t>(b + i * NT);
  }
  __syncthreads();
  r.count = __builtin_amdgcn_readfirstlane(mem.count);
  if (r.count > 0) r.e = a;
  return r;
}

// The plan of fc2, by one workgroup: every expert named, in order of id, with its
// slots; ids out of range reported.
template <int NT>
__device__ __forceinline__ void write_plan(const TokArgs& p, int slots) {
  __shared__ int cnt[kTokMaxExperts];  // slots of an expert, then the next place of its list
  const int lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kTokMaxExperts; i += NT) cnt[i] = 0;
  __syncthreads();
  for (int s = threadIdx.x; s < p.TK; s += NT) {
    const int e = local_id(p, s);
    if (e >= 0) atomicAdd(&cnt[e], 1);
    if (p.sel[s] < 0 || p.sel[s] >= p.E) atomic_or_err(p.dev_err, MC2_DEVERR_EXPERT_ID);
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    constexpr int PER = kTokMaxExperts / 64;  // neighbours a lane
    int named = 0, rows = 0;
    for (int i = 0; i < PER; ++i) {
      const int c = cnt[lane * PER + i];
      named += c > 0;
      rows += c;
    }
    int n = named, r = rows;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int on = __shfl_up(n, d), orr = __shfl_up(r, d);
      if (lane >= d) {
        n += on;
        r += orr;
      }
    }
    const int total = __builtin_amdgcn_readlane(n, 63);
    n -= named;
    r -= rows;
    for (int i = 0; i < PER; ++i) {
      const int c = cnt[lane * PER + i];
      if (c > 0) p.plan[n++] = i32x4_t{lane * PER + i, c, r, total};
      cnt[lane * PER + i] = r;
      r += c;
    }
    for (int i = total + lane; i < slots; i += 64) p.plan[i] = i32x4_t{-1, 0, 0, total};
  }
  __syncthreads();
  for (int s = threadIdx.x; s < p.TK; s += NT) {
    const int e = local_id(p, s);
    if (e >= 0) p.list[atomicAdd(&cnt[e], 1)] = static_cast<uint16_t>(s);
  }
}

// Token t's counters of every strip of fc2, or its row of zeros where no slot of
// it is local.
template <int NT>
__device__ __forceinline__ void count_slots(const TokArgs& p, int t) {
  const int lane = threadIdx.x & 63;  // K is 64 at most
  const int n = __popcll(__ballot(lane < p.K && local_id(p, t * p.K + (lane < p.K ? lane : 0)) >= 0));
  for (int s = threadIdx.x; s < p.strips2; s += NT) p.left[s * p.T + t] = n;
  if (n == 0)
    for (int64_t c = threadIdx.x * 8; c < p.H; c += NT * 8)
      *reinterpret_cast<u32x4_t*>(p.out + t * p.H + c) = zero_v4();
}

// ------------------------------------------------------------------- weights
//
// The weights of a strip of 16 * NF columns of one matrix, KS of K a step, taken
// in groups of U neighbouring steps a wave: Group holds this lane's part of one.
// load(st, step, u) brings step u of a group into registers and scales(st, step)
// what its U steps share, which take() puts in force; frag<T>(u, f) is the
// operand of fragment f (16 columns) for sub-step T of KT, 32 K values each. The
// rows of x are loaded with row_k(s, T, g) the first of the eight K values that
// lane group g loads, and order(a) then gives every lane the values that frag<T>
// goes with. h is written in the lanes' order instead: frag<T> goes with the eight
// values from lane_k(s, T, g) on, and value k of a row of K stands at h_at(k, K).
// Column c of the strip is lane lane_of(c) & 15 of fragment frag_of(c).
// (Addresses are 32-bit offsets from scalar bases: 64-bit ones would take two
// registers for each load in flight.)

// Exchange the upper 32 lanes of a with the lower 32 of b; the odd rows of 16
// lanes of a with the even ones of b.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// bf16 weights (rows of K, columns contiguous): a lane loads LC neighbouring
// columns of eight K rows; the eight values of a column then lie in one lane
// and a byte permute pairs them up, so that the strip's columns go to fragments
// by their place among the LC: fragment f holds columns LC * n + f.
template <int LC_>
struct WBf16 {
  static constexpr int NF = LC_, LC = LC_, KS = 32, KT = 1, NW = 8;
  static constexpr int U1 = LC_ == 2 ? 4 : 2, U2 = 4;  // steps a group, fc1 and fc2
  static constexpr int U1m = U1, U2m = U2;             // ... of kTokMany operands

  struct Strip {
    const char* base;  // column 0 of the strip in K row 0
    uint32_t off;      // this lane's columns in K row 8 g
    uint32_t ld;       // bytes between K rows
    int64_t k;
  };
  static __device__ __forceinline__ Strip strip(const char* w, const char*, int64_t e, int64_t K,
                                                int64_t cols, int64_t first, int64_t c0,
                                                int64_t limit) {
    const int lane = threadIdx.x & 63;
    const int64_t mine = LC * (lane & 15), most = limit - LC - c0;
    return {w + (e * K * cols + first + c0) * 2,
            static_cast<uint32_t>((8 * (lane >> 4) * cols + (mine < most ? mine : most)) * 2),
            static_cast<uint32_t>(cols * 2), K};
  }
  template <int U>
  struct Group {
    uint32_t r[U][8][LC_ / 2];
    __device__ __forceinline__ void load(const Strip& st, int64_t s, int u) {
      const int64_t row = s * 32 + 8 * ((threadIdx.x & 63) >> 4);
      // k is a multiple of 8: all eight rows or none
      const uint32_t off = row < st.k ? st.off : kOffNone;
      const __amdgpu_buffer_rsrc_t q = make_rsrc(st.base + s * 32 * st.ld);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (LC == 4) {
          const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(q, off, i * st.ld, 0);
          r[u][i][0] = v[0];
          r[u][i][1] = v[1];
        } else {
          r[u][i][0] = __builtin_amdgcn_raw_buffer_load_b32(q, off, i * st.ld, 0);
        }
      }
    }
    __device__ __forceinline__ void scales(const Strip&, int64_t) {}
    __device__ __forceinline__ void take() {}
    template <int T>
    __device__ __forceinline__ bf16x8_t frag(int u, int f) const {
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = __builtin_amdgcn_perm(r[u][2 * i + 1][f >> 1], r[u][2 * i][f >> 1],
                                     (f & 1) ? 0x07060302u : 0x05040100u);
      return bit_cast<bf16x8_t>(v);
    }
  };
  static __device__ __forceinline__ int64_t row_k(int64_t s, int, int g) { return s * 32 + 8 * g; }
  static __device__ __forceinline__ void order(u32x4_t (&)[1]) {}
  static __device__ __forceinline__ int64_t lane_k(int64_t s, int, int g) { return s * 32 + 8 * g; }
  static __device__ __forceinline__ int64_t h_at(int64_t k, int64_t) { return k; }
  // w[e][k .. k + 7][c]
  static __device__ __forceinline__ void eight(const char* w, const char*, int64_t e, int64_t K,
                                               int64_t cols, int64_t k, int64_t c, float (&v)[8]) {
    const uint16_t* q = reinterpret_cast<const uint16_t*>(w) + (e * K + k) * cols + c;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_bits_to_f32(q[i * cols]);
  }
  static __device__ __forceinline__ int frag_of(int c) { return c % LC; }
  static __device__ __forceinline__ int lane_of(int c) { return c / LC; }
};

// MX4 weights (a row per column, K contiguous): a lane holds a block of 32 K
// values of each of its NF columns, 16 n + the fragment's first, and turns eight
// of them at a time into exact bf16 numbers. The four scale bytes of a step's
// blocks are one dword of the row, and those of a group's steps one load (a
// byte load for each step and fragment took 30 of 171 us at 64 tokens).
template <int NF_>
struct WMx4 {
  static constexpr int NF = NF_, KS = 128, KT = 4, NW = 4;
  static constexpr int U1 = 4, U2 = 2, U1m = 2, U2m = 1;

  struct Strip {
    const char* base;
    const char* sbase;
    uint32_t off[NF_], soff[NF_];  // this lane's column: block g, scales
    int64_t nb;
  };
  static __device__ __forceinline__ Strip strip(const char* w, const char* ws, int64_t e, int64_t K,
                                                int64_t cols, int64_t first, int64_t c0,
                                                int64_t limit) {
    const int lane = threadIdx.x & 63;
    Strip st;
    st.nb = (K + 31) / 32;
    const int64_t pitch = (st.nb + 15) / 16 * 16, row0 = e * cols + first + c0;
    st.base = w + row0 * st.nb * 16;
    st.sbase = ws + row0 * pitch;
#pragma unroll
    for (int f = 0; f < NF; ++f) {
      const int64_t mine = 16 * f + (lane & 15), most = limit - 1 - c0;
      const int64_t c = mine < most ? mine : most;
      st.off[f] = static_cast<uint32_t>((c * st.nb + (lane >> 4)) * 16);
      st.soff[f] = static_cast<uint32_t>(c * pitch);
    }
    return st;
  }
  template <int U>
  struct Group {
    static_assert(U == 1 || U == 2 || U == 4, "scales of a group in one load");
    u32x4_t c[U][NF_];
    uint32_t sc[NF_][U], nx[NF_][U];
    __device__ __forceinline__ void load(const Strip& st, int64_t s, int u) {
      const bool in = s * 4 + ((threadIdx.x & 63) >> 4) < st.nb;
      const __amdgpu_buffer_rsrc_t q = make_rsrc(st.base + s * 64);
#pragma unroll
      for (int f = 0; f < NF; ++f)
        c[u][f] = __builtin_amdgcn_raw_buffer_load_b128(q, in ? st.off[f] : kOffNone, 0, 0);
    }
    // s: the group's first step, a multiple of U
    __device__ __forceinline__ void scales(const Strip& st, int64_t s) {
      const __amdgpu_buffer_rsrc_t q = make_rsrc(st.sbase + s * 4);
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        const uint32_t off = s * 4 < st.nb ? st.soff[f] : kOffNone;
        if constexpr (U == 4) {
          const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(q, off, 0, 0);
#pragma unroll
          for (int u = 0; u < U; ++u) nx[f][u] = v[u];
        } else if constexpr (U == 2) {
          const u32x2_t v = __builtin_amdgcn_raw_buffer_load_b64(q, off, 0, 0);
          nx[f][0] = v[0];
          nx[f][U - 1] = v[1];
        } else {
          nx[f][0] = __builtin_amdgcn_raw_buffer_load_b32(q, off, 0, 0);
        }
      }
    }
    __device__ __forceinline__ void take() {
#pragma unroll
      for (int f = 0; f < NF; ++f)
#pragma unroll
        for (int u = 0; u < U; ++u) sc[f][u] = nx[f][u];
    }
    template <int T>
    __device__ __forceinline__ bf16x8_t frag(int u, int f) const {
      const uint32_t byte = (sc[f][u] >> (((threadIdx.x & 63) >> 4) * 8)) & 255u;
      return bit_cast<bf16x8_t>(mx4_bf16x8(c[u][f][T], mx4_scale(byte)));
    }
  };
  // Sub-step T goes with K values 32 g + 8 T + .. of lane group g. A load of those
  // would touch 16 bytes in every 64 of a row; instead the four groups load 64
  // contiguous bytes, 32 T + 8 g + .., and the 4 x 4 pieces (T, g) change places.
  static __device__ __forceinline__ int64_t row_k(int64_t s, int t, int g) {
    return s * 128 + 32 * t + 8 * g;
  }
  static __device__ __forceinline__ void order(u32x4_t (&a)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t r[4] = {a[0][i], a[1][i], a[2][i], a[3][i]};
      swap32(r[0], r[2]);
      swap32(r[1], r[3]);
      swap16(r[0], r[1]);
      swap16(r[2], r[3]);
#pragma unroll
      for (int t = 0; t < 4; ++t) a[t][i] = r[t];
    }
  }
  static __device__ __forceinline__ int64_t lane_k(int64_t s, int t, int g) {
    return s * 128 + 32 * g + 8 * t;
  }
  // Piece (T, g) of 128 values, T first; the last values of a row, K % 128 of them,
  // are `full` groups of four pieces and `more` pieces of one further group.
  static __device__ __forceinline__ int64_t h_at(int64_t k, int64_t K) {
    const int64_t first = k & ~int64_t{127};
    const int left = static_cast<int>(K - first < 128 ? K - first : 128) >> 3;
    const int full = left >> 2, more = left & 3;
    const int r = static_cast<int>(k - first), t = (r >> 3) & 3, g = r >> 5;
    return first + 8 * (t * full + (t < more ? t : more) + g) + (r & 7);
  }
  // w[e][k .. k + 7][c]
  static __device__ __forceinline__ void eight(const char* w, const char* ws, int64_t e, int64_t K,
                                               int64_t cols, int64_t k, int64_t c, float (&v)[8]) {
    const int64_t nb = (K + 31) / 32, pitch = (nb + 15) / 16 * 16, row = e * cols + c;
    const uint32_t codes = *reinterpret_cast<const uint32_t*>(w + row * nb * 16 + k / 2);
    const u32x4_t q = mx4_bf16x8(codes, mx4_scale(static_cast<uint8_t>(ws[row * pitch + k / 32])));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = bf16_bits_to_f32((q[i / 2] >> (16 * (i & 1))) & 0xffffu);
  }
  static __device__ __forceinline__ int frag_of(int c) { return c / 16; }
  static __device__ __forceinline__ int lane_of(int c) { return c % 16; }
};

__device__ __forceinline__ f32x4_t mfma_bf16(bf16x8_t a, bf16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Workgroup barrier for LDS alone: loads from memory stay in flight across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// The waves' sums of NV values a lane (one 16-row tile), through LDS: element
// (m, v, c) of the tile is red[w][v][(m >> 2) * 16 + n][m & 3] of every wave.
template <int NW, int NV>
__device__ __forceinline__ float tile_sum(const f32x4_t (&red)[NW][NV][64], int v, int m, int n) {
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) s += red[w][v][(m >> 2) * 16 + n][m & 3];
  return s;
}

// ----------------------------------------------------------------------- fc1

// Both kernels walk the strips [s0, s1) of one expert with the loads a group of
// U K steps ahead: a step's registers are loaded again for the next group, of
// this strip or the next, as soon as its products are done, so that memory is
// read on while the waves' sums meet in LDS. Where one group covers K, the rows'
// operands are loaded once for all strips. A wave takes V neighbouring steps of K
// in every V * NW, in this order whatever U is: the sums of a slot are then the
// same bits however many slots share its operand (which varies, see pick_expert).

// h as three bf16 numbers: the upper half of h, of what that leaves, and of what is
// left then, eight bits each. They sum to h exactly (from 2^-110 on; below, the last
// one leaves bf16's range), and none is larger, so that a finite h has finite parts.
// (Two of them, 16 bits, took 10 us of 250 less at 256 tokens with 4-bit weights, 6
// of 110 at 64; 25 in 10000 outputs were then not the nearest bf16 number to the
// result in 64 bits, with three 2.)
__device__ __forceinline__ void split_h(float h, uint32_t (&part)[kHParts]) {
  // (an infinite h has no rest)
  const bool finite = __builtin_fabsf(h) < __builtin_inff();
#pragma unroll
  for (int i = 0; i < kHParts; ++i) {
    part[i] = __float_as_uint(h) >> 16;
    h = finite ? h - bf16_bits_to_f32(part[i]) : 0.f;
  }
}

// h of up to 16 * MT slots, list[0 .. count).
template <class W, int MT>
__device__ __forceinline__ void fc1_rows(const TokArgs& p, int64_t e, const uint16_t* list,
                                         int count, int s0, int s1,
                                         f32x4_t (&red)[W::NW][2 * W::NF][64]) {
  constexpr int NF = W::NF, NW = W::NW, V = W::U1, U = MT == 1 ? V : W::U1m, CW = 16 * NF;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = static_cast<int>((p.H + W::KS * NW * V - 1) / (W::KS * NW * V)) * (V / U);
  typename W::Strip sg, su;
  auto at_strip = [&](int s) {
    sg = W::strip(p.w1, p.w1s, e, p.H, 2 * p.I, 0, static_cast<int64_t>(s) * CW, p.I);
    su = W::strip(p.w1, p.w1s, e, p.H, 2 * p.I, p.I, static_cast<int64_t>(s) * CW, p.I);
  };
  static_assert(V % U == 0, "groups are parts of V steps");
  auto step = [&](int grp, int u) {
    const int q = grp * U + u;
    return static_cast<int64_t>((q / V * NW + wave) * V + q % V);
  };
  typename W::template Group<U> wg, wu;
  at_strip(s0);
  wg.scales(sg, step(0, 0));
  wu.scales(su, step(0, 0));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    wg.load(sg, step(0, u), u);
    wu.load(su, step(0, u), u);
  }
  const __amdgpu_buffer_rsrc_t rx = make_rsrc(reinterpret_cast<const char*>(p.x));
  uint32_t xr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 16 * i + (lane & 15);
    xr[i] = r < count ? static_cast<uint32_t>(list[r] / p.K * p.H * 2) : kOffNone;
  }
  u32x4_t a[U][MT][W::KT];
  auto load_rows = [&](int grp) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < W::KT; ++t) {
        const int64_t k = W::row_k(step(grp, u), t, g);
#pragma unroll
        for (int i = 0; i < MT; ++i)
          a[u][i][t] = __builtin_amdgcn_raw_buffer_load_b128(
              rx, k < p.H ? xr[i] + static_cast<uint32_t>(2 * k) : kOffNone, 0, 0);
      }
  };
  load_rows(0);
  for (int s = s0; s < s1; ++s) {
    f32x4_t ag[NF][MT], au[NF][MT];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < MT; ++i) ag[f][i] = au[f][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int grp = 0; grp < groups; ++grp) {
      const bool turn = grp + 1 == groups;
      const int ng = turn ? 0 : grp + 1;
      const bool more = !turn || s + 1 < s1;
      if (turn && more) at_strip(s + 1);
      if (s == s0 || groups > 1) {  // rows newly loaded
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int i = 0; i < MT; ++i) W::order(a[u][i]);
      }
      wg.take();
      wu.take();
      if (more) {
        wg.scales(sg, step(ng, 0));
        wu.scales(su, step(ng, 0));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        sfor<W::KT>([&](auto Tc) {
          constexpr int t = decltype(Tc)::value;
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const bf16x8_t bg = wg.template frag<t>(u, f), bu = wu.template frag<t>(u, f);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              ag[f][i] = mfma_bf16(bit_cast<bf16x8_t>(a[u][i][t]), bg, ag[f][i]);
              au[f][i] = mfma_bf16(bit_cast<bf16x8_t>(a[u][i][t]), bu, au[f][i]);
            }
          }
        });
        if (more) {
          wg.load(sg, step(ng, u), u);
          wu.load(su, step(ng, u), u);
        }
      }
      if (more && groups > 1) load_rows(ng);
    }
    const int64_t c0 = static_cast<int64_t>(s) * CW;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int f = 0; f < NF; ++f) {
        red[wave][f][lane] = ag[f][i];
        red[wave][NF + f][lane] = au[f][i];
      }
      lds_barrier();
      const int rows = count - 16 * i < 16 ? count - 16 * i : 16;
      for (int q = threadIdx.x; q < rows * CW; q += NW * 64) {
        const int m = q / CW, c = q - m * CW;
        const int f = W::frag_of(c), n = W::lane_of(c);
        if (c0 + c >= p.I) continue;
        const float gate = tile_sum<NW>(red, f, m, n), up = tile_sum<NW>(red, NF + f, m, n);
        const float h = gate / (1.f + __expf(-gate)) * up;
        uint32_t part[kHParts];
        split_h(h, part);
        const int64_t at = static_cast<int64_t>(list[16 * i + m]) * p.I + W::h_at(c0 + c, p.I);
#pragma unroll
        for (int j = 0; j < kHParts; ++j) p.h[j][at] = static_cast<uint16_t>(part[j]);
      }
      lds_barrier();
    }
  }
}

// Strips of a kernel's workgroup: `per` neighbouring ones.
struct Strips {
  int s0, s1;
};
__device__ __forceinline__ Strips my_strips(int strips, int per) {
  const int s0 = blockIdx.x * per;
  return {s0, s0 + per < strips ? s0 + per : strips};
}

// MANY: more than 16 tokens, so that an expert may have more than 16 slots of
// different tokens; they are then taken 32 at a time.
template <class W, bool MANY>
__global__ __launch_bounds__(W::NW * 64, 2) void tokens_fc1_kernel(TokArgs p) {
  constexpr int NT = W::NW * 64;
  __shared__ PickMem mem;
  __shared__ f32x4_t red[W::NW][2 * W::NF][64];
  if (blockIdx.y == 0) {  // a row of workgroups ahead of the experts': what fc2 needs
    if (blockIdx.x == 0) write_plan<NT>(p, p.TK < p.El ? p.TK : p.El);
    for (int t = blockIdx.x; t < p.T; t += gridDim.x) count_slots<NT>(p, t);
    return;
  }
  const Expert ex = pick_expert<NT>(p, blockIdx.y - 1, mem);
  if (ex.e < 0) return;
  const Strips st = my_strips(p.strips1, p.per1);
  for (int b = 0; b < ex.count;) {
    const int left = ex.count - b;
    if (MANY && left > 16) {
      fc1_rows<W, kTokMany>(p, ex.e, mem.list + b, left < 16 * kTokMany ? left : 16 * kTokMany,
                            st.s0, st.s1, red);
      b += 16 * kTokMany;
    } else {
      fc1_rows<W, 1>(p, ex.e, mem.list + b, left < 16 ? left : 16, st.s0, st.s1, red);
      b += 16;
    }
  }
}

// ----------------------------------------------------------------------- fc2

// y of one slot and column, from the numbers that its parts of h stand for. The
// products of the parts give NaN where an infinite weight meets a part that is zero,
// though h times the weight is infinite. (The call costs about 1% where no y is NaN,
// 110.2 -> 111.5 us for 64 tokens in MX4; sums of their own for the first parts, which
// would be infinite, cost 1 to 3% and 16 to 32 registers more.)
template <class W>
__device__ __forceinline__ float whole_dot(const TokArgs& p, int64_t e, int64_t slot, int64_t c) {
  float y = 0.f;
  for (int64_t k = 0; k < p.I && y == y; k += 8) {
    const int64_t at = slot * p.I + W::h_at(k, p.I);
    float w[8];
    W::eight(p.w2, p.w2s, e, p.I, p.H, k, c, w);
    u32x4_t h[kHParts];
#pragma unroll
    for (int j = 0; j < kHParts; ++j) h[j] = *reinterpret_cast<const u32x4_t*>(p.h[j] + at);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = 0.f;
#pragma unroll
      for (int j = kHParts - 1; j >= 0; --j)
        v += bf16_bits_to_f32((h[j][i / 2] >> (16 * (i & 1))) & 0xffffu);
      y = __builtin_fmaf(v, w[i], y);
    }
  }
  return y;
}

template <class W, int MT>
__device__ __forceinline__ void fc2_rows(const TokArgs& p, int64_t e, const uint16_t* list,
                                         int count, int s0, int s1,
                                         f32x4_t (&red)[W::NW][W::NF][64],
                                         uint16_t (&slots)[16 * kTokMany]) {
  constexpr int NF = W::NF, NW = W::NW, V = W::U2, U = MT == 1 ? V : W::U2m, CW = 16 * NF;
  const int lane = threadIdx.x & 63, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int groups = static_cast<int>((p.I + W::KS * NW * V - 1) / (W::KS * NW * V)) * (V / U);
  typename W::Strip sw;
  auto at_strip = [&](int s) {
    sw = W::strip(p.w2, p.w2s, e, p.I, p.H, 0, static_cast<int64_t>(s) * CW, p.H);
  };
  static_assert(V % U == 0, "groups are parts of V steps");
  auto step = [&](int grp, int u) {
    const int q = grp * U + u;
    return static_cast<int64_t>((q / V * NW + wave) * V + q % V);
  };
  typename W::template Group<U> w;
  at_strip(s0);
  w.scales(sw, step(0, 0));
#pragma unroll
  for (int u = 0; u < U; ++u) w.load(sw, step(0, u), u);
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(reinterpret_cast<const char*>(p.y));
  uint32_t hr[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = 16 * i + (lane & 15);
    hr[i] = r < count ? static_cast<uint32_t>(list[r] * p.I * 2) : kOffNone;
  }
  u32x4_t h[U][MT][W::KT][kHParts];
  auto load_rows = [&](int grp) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < W::KT; ++t) {
        const int64_t k = W::lane_k(step(grp, u), t, g);
        const uint32_t at = static_cast<uint32_t>(2 * W::h_at(k, p.I));
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < kHParts; ++j)
            h[u][i][t][j] = __builtin_amdgcn_raw_buffer_load_b128(
                make_rsrc(reinterpret_cast<const char*>(p.h[j])), k < p.I ? hr[i] + at : kOffNone, 0, 0);
      }
  };
  load_rows(0);
  // the slots again, in LDS: a load of them after the products would wait for
  // every load that is under way by then (there before the sums' barrier)
  if (threadIdx.x < count) slots[threadIdx.x] = list[threadIdx.x];
  for (int s = s0; s < s1; ++s) {
    f32x4_t acc[NF][MT];
#pragma unroll
    for (int f = 0; f < NF; ++f)
#pragma unroll
      for (int i = 0; i < MT; ++i) acc[f][i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int grp = 0; grp < groups; ++grp) {
      const bool turn = grp + 1 == groups;
      const int ng = turn ? 0 : grp + 1;
      const bool more = !turn || s + 1 < s1;
      if (turn && more) at_strip(s + 1);
      w.take();
      if (more) w.scales(sw, step(ng, 0));
#pragma unroll
      for (int u = 0; u < U; ++u) {
        sfor<W::KT>([&](auto Tc) {
          constexpr int t = decltype(Tc)::value;
#pragma unroll
          for (int f = 0; f < NF; ++f) {
            const bf16x8_t b = w.template frag<t>(u, f);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int j = 0; j < kHParts; ++j)
                acc[f][i] = mfma_bf16(bit_cast<bf16x8_t>(h[u][i][t][j]), b, acc[f][i]);
          }
        });
        if (more) w.load(sw, step(ng, u), u);
      }
      if (more && groups > 1) load_rows(ng);
    }
    const int64_t c0 = static_cast<int64_t>(s) * CW;
#pragma unroll
    for (int i = 0; i < MT; ++i) {
#pragma unroll
      for (int f = 0; f < NF; ++f) red[wave][f][lane] = acc[f][i];
      lds_barrier();
      const int rows = count - 16 * i < 16 ? count - 16 * i : 16;
      for (int q = threadIdx.x; q < rows * CW; q += NW * 64) {
        const int m = q / CW, c = q - m * CW;
        if (c0 + c >= p.H) continue;
        float v = tile_sum<NW>(red, W::frag_of(c), m, W::lane_of(c));
        if (__builtin_expect(v != v, 0)) v = whole_dot<W>(p, e, slots[16 * i + m], c0 + c);
        const int64_t at = static_cast<int64_t>(slots[16 * i + m]) * p.H + c0 + c;
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), ry, static_cast<int>(at * 4), 0,
                                              kCpolAgent);
      }
      lds_barrier();
    }
  }
}

// out[t] = sum over the local slots of t, in slot order, of probs * y: four
// columns from c on.
__device__ __forceinline__ void sum_slots(const TokArgs& p, int t, int64_t c) {
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(reinterpret_cast<const char*>(p.y));
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  for (int k0 = 0; k0 < p.K; k0 += 8) {  // eight slots' loads in flight
    u32x4_t y[8];
    float w[8];
    bool in[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = t * p.K + (k0 + j < p.K ? k0 + j : p.K - 1);
      // (rows of slots that are not local are read too, and dropped: the loads do
      // not wait for the ids)
      in[j] = k0 + j < p.K && local_id(p, s) >= 0;
      w[j] = p.probs[s];
      y[j] = __builtin_amdgcn_raw_buffer_load_b128(
          ry, static_cast<uint32_t>((static_cast<int64_t>(s) * p.H + c) * 4), 0, kCpolAgent);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (in[j]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(w[j], __uint_as_float(y[j][i]), v[i]);
      }
  }
  *reinterpret_cast<u32x2_t*>(p.out + static_cast<int64_t>(t) * p.H + c) = pack4<Out::BF16>(v);
}

constexpr int kTokDone = 2048;  // finished (strip, token) pairs held at a time

template <class W, bool MANY>
__global__ __launch_bounds__(W::NW * 64, 2) void tokens_fc2_kernel(TokArgs p) {
  constexpr int NT = W::NW * 64, CW = 16 * W::NF;
  __shared__ f32x4_t red[W::NW][W::NF][64];
  __shared__ uint16_t slots[16 * kTokMany];
  __shared__ uint16_t done[kTokDone];  // strip (from the workgroup's first) * 256 + token
  __shared__ int ndone;
  const i32x4_t plan = p.plan[blockIdx.y];
  const int count = plan[1];
  const Strips st = my_strips(p.strips2, p.per2);
  if (plan[0] < 0) return;
  const uint16_t* list = p.list + plan[2];
  for (int b = 0; b < count;) {
    const int left = count - b;
    if (MANY && left > 16) {
      fc2_rows<W, kTokMany>(p, plan[0], list + b, left < 16 * kTokMany ? left : 16 * kTokMany,
                            st.s0, st.s1, red, slots);
      b += 16 * kTokMany;
    } else {
      fc2_rows<W, 1>(p, plan[0], list + b, left < 16 ? left : 16, st.s0, st.s1, red, slots);
      b += 16;
    }
  }
  // The workgroup that brings the last y of a token's strip adds the token up.
  // y was written through to memory and is read from there: once the stores
  // are done (the wait), no cache needs a write-back or an invalidation, which
  // would cost the other workgroups their weights.
  if (threadIdx.x == 0) ndone = 0;
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  const int most = count < p.T ? count : p.T;  // tokens that a strip can finish here
  const int batch = kTokDone / most;
  for (int s0 = st.s0; s0 < st.s1; s0 += batch) {
    const int ns = s0 + batch < st.s1 ? batch : st.s1 - s0;
    for (int q = threadIdx.x; q < ns * count; q += NT) {
      const int s = q / count, t = list[q - s * count] / p.K;
      if (__hip_atomic_fetch_add(&p.left[(s0 + s) * p.T + t], -1, __ATOMIC_RELAXED,
                                 __HIP_MEMORY_SCOPE_AGENT) == 1)
        done[atomicAdd(&ndone, 1)] = static_cast<uint16_t>((s0 - st.s0 + s) * 256 + t);
    }
    __syncthreads();
    const int items = ndone * (CW / 4);
    for (int q = threadIdx.x; q < items; q += NT) {
      const int d = done[q / (CW / 4)];
      const int64_t c = static_cast<int64_t>(st.s0 + (d >> 8)) * CW + 4 * (q % (CW / 4));
      if (c < p.H) sum_slots(p, d & 255, c);
    }
    __syncthreads();
    if (threadIdx.x == 0) ndone = 0;
    __syncthreads();
  }
}

// ------------------------------------------------------------------ host side

struct TokWorkspace {
  size_t left, plan, list, h, y, bytes;
};

static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

static bool tok_workspace(int64_t T, int K, int64_t H, int64_t I, TokWorkspace& w) {
  if (T < 1 || T > 256 || K < 1 || K > 64 || T * K > kTokMaxSlots) return false;
  if (H < 8 || H > 65536 || I < 8 || I > 65536) return false;
  const int64_t TK = T * K;
  if (TK * H >= int64_t{1} << 28 || TK * I >= int64_t{1} << 28) return false;
  w.left = 0;
  w.plan = up256(static_cast<size_t>(tok_strips(H) * T) * 4);
  w.list = w.plan + up256(static_cast<size_t>(TK < kTokMaxExperts ? TK : kTokMaxExperts) * 16);
  w.h = w.list + up256(static_cast<size_t>(TK) * 2);
  w.y = w.h + up256(static_cast<size_t>(TK * I) * 2) * kHParts;
  w.bytes = w.y + up256(static_cast<size_t>(TK * H) * 4);
  return true;
}

// Strips a workgroup: two where twelve workgroups a CU would each have one (us at
// 1 / 2 / 3 / as many as leave six workgroups a CU: 64 tokens above, MX4, 122 / 111
// / 119 / 112; 256 tokens of 1024 / 256, 8 of 1024 experts, MX4 219 / 181 / 188 /
// 315, of 512 experts, bf16 274 / 251 / 280 / 262): the second strip's weights are
// on their way while the first one's sums are made.
static int strips_per(int64_t strips, int64_t rows, int64_t cus) {
  return strips * rows >= 12 * cus ? kTokMaxPer : 1;
}

template <class W1, class W2, bool MANY>
static void launch_both(TokArgs a, int rows1, int rows2, int64_t cus, hipStream_t s) {
  a.strips1 = static_cast<int>((a.I + 16 * W1::NF - 1) / (16 * W1::NF));
  a.strips2 = static_cast<int>((a.H + 16 * W2::NF - 1) / (16 * W2::NF));
  a.per1 = strips_per(a.strips1, rows1, cus);
  a.per2 = strips_per(a.strips2, rows2, cus);
  const dim3 grid1((a.strips1 + a.per1 - 1) / a.per1, rows1 + 1);
  const dim3 grid2((a.strips2 + a.per2 - 1) / a.per2, rows2);
  hipLaunchKernelGGL((tokens_fc1_kernel<W1, MANY>), grid1, dim3(W1::NW * 64), 0, s, a);
  hipLaunchKernelGGL((tokens_fc2_kernel<W2, MANY>), grid2, dim3(W2::NW * 64), 0, s, a);
}

// Wide strips where 64-column ones make workgroups for a quarter of the CUs. fc1, us
// wide / narrow for bf16 and for MX4 (whose wide strips are of 32 columns), by that
// number: 96 (one token above) 28.9 / 30.4, 19.3 / 19.1; 72 (six experts) 25.0 / 25.3,
// 17.9 / 17.7; 64 (40 tokens of 1024 / 512, 8 experts) 23.5 / 23.8, 21.5 / 19.9; 48 (one
// token, I = 384) 24.5 / 22.9, 17.7 / 16.4; 32 (37 tokens of 1416 / 200, 8 experts)
// 25.2 / 23.2, 18.8 / 17.3. fc2: 256 (one token, I = 256) 22.4 / 25.1, 15.9 / 19.2; 184
// (the 37 tokens) 23.2 / 27.2, 17.3 / 21.4; 128 (two experts of 4096 / 1536) 35.5 /
// 37.5, 19.4 / 18.7; 64 (two of 2048 / 768) 20.2 / 19.9, 13.8 / 12.6.
template <bool MANY>
static void launch_tokens(const TokArgs& a, bool mx4, hipStream_t s) {
  const int slots = a.TK < a.El ? a.TK : a.El;
  const int rows1 = a.TK <= 64 ? slots : a.El;  // see pick_expert
  const int64_t cus = num_cus();
  const bool wide1 = slots * ((a.I + 63) / 64) >= cus / 4, wide2 = slots * ((a.H + 63) / 64) >= cus / 4;
  auto both = [&](auto w1, auto w2) {
    launch_both<decltype(w1), decltype(w2), MANY>(a, rows1, slots, cus, s);
  };
  if (mx4) {
    if (wide1) wide2 ? both(WMx4<2>{}, WMx4<4>{}) : both(WMx4<2>{}, WMx4<1>{});
    else wide2 ? both(WMx4<1>{}, WMx4<4>{}) : both(WMx4<1>{}, WMx4<1>{});
  } else {
    if (wide1) wide2 ? both(WBf16<4>{}, WBf16<4>{}) : both(WBf16<4>{}, WBf16<2>{});
    else wide2 ? both(WBf16<2>{}, WBf16<4>{}) : both(WBf16<2>{}, WBf16<2>{});
  }
}

}  // namespace mc2

using namespace mc2;

extern "C" size_t mc2_moe_tokens_workspace_size(int64_t T, int K, int64_t H, int64_t I) {
  TokWorkspace w;
  return tok_workspace(T, K, H, I, w) ? w.bytes : 0;
}

extern "C" int mc2_moe_tokens(const void* x, const int32_t* sel, const float* probs, int64_t T,
                              int K, int64_t H, int num_experts, int ep_rank, int local_experts,
                              int w_dtype, const void* w1, const void* w1_scale, const void* w2,
                              const void* w2_scale, int64_t I, void* out, void* workspace,
                              size_t ws_bytes, int32_t* dev_err, hipStream_t stream) {
  if (!x || !sel || !probs || !w1 || !w2 || !out || !workspace) return MC2_ERR_NULL;
  if (w_dtype != MC2_BF16 && w_dtype != MC2_MX4) return MC2_ERR_DTYPE;
  const bool mx4 = w_dtype == MC2_MX4;
  if (mx4 && (!w1_scale || !w2_scale)) return MC2_ERR_NULL;
  if (!mx4 && (w1_scale || w2_scale)) return MC2_ERR_DTYPE;
  TokWorkspace w;
  if (!tok_workspace(T, K, H, I, w)) return MC2_ERR_SHAPE;
  if (num_experts < 1 || local_experts < 1 || local_experts > kTokMaxExperts || ep_rank < 0 ||
      (static_cast<int64_t>(ep_rank) + 1) * local_experts > num_experts)
    return MC2_ERR_SHAPE;
  if (H % 8 || I % 8) return MC2_ERR_ALIGN;
  if (!aligned16(x) || !aligned16(w1) || !aligned16(w2) || !aligned16(w1_scale) ||
      !aligned16(w2_scale) || !aligned16(out) || !aligned16(workspace))
    return MC2_ERR_ALIGN;
  if (ws_bytes < w.bytes) return MC2_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  TokArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.sel = sel;
  a.probs = probs;
  a.w1 = static_cast<const char*>(w1);
  a.w1s = static_cast<const char*>(w1_scale);
  a.w2 = static_cast<const char*>(w2);
  a.w2s = static_cast<const char*>(w2_scale);
  a.out = static_cast<uint16_t*>(out);
  a.left = reinterpret_cast<int32_t*>(ws + w.left);
  a.plan = reinterpret_cast<i32x4_t*>(ws + w.plan);
  a.list = reinterpret_cast<uint16_t*>(ws + w.list);
  for (int j = 0; j < kHParts; ++j)
    a.h[j] = reinterpret_cast<uint16_t*>(ws + w.h + (w.y - w.h) / kHParts * j);
  a.y = reinterpret_cast<float*>(ws + w.y);
  a.dev_err = dev_err;
  a.H = H;
  a.I = I;
  a.T = static_cast<int>(T);
  a.K = K;
  a.TK = static_cast<int>(T) * K;
  a.E = num_experts;
  a.e0 = ep_rank * local_experts;
  a.El = local_experts;
  if (T > 16) launch_tokens<true>(a, mx4, stream);
  else launch_tokens<false>(a, mx4, stream);
  return hipGetLastError() == hipSuccess ? MC2_OK : MC2_ERR_HIP;
}
