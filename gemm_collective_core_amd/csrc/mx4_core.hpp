// Main loop of the product of two MX4 operands, both held K-contiguous (A as
// (m, k), B as (n, k)), gfx950: four waves, a 256 x 256 or 128 x 128 tile.
//
// An MX4 row is the same to the loads and to LDS as a 16-bit row of a quarter
// of the values: K advances in stages of 128 bytes per row (256 values), held
// in the two-buffer LDS ring, the swizzled rows and the loads straight into LDS
// of the 16-bit loops. What differs:
//  * v_mfma_scale_f32_32x32x64_f8f6f4, four k-steps a stage. Lane l supplies 32
//    values (16 bytes) of row l & 31; in k-step j the lanes of group g = l >> 5
//    take the stage's block 4 g + j. (The loop in the 16 x 16 x 128 shape, with
//    the 16-bit loop's order of a stage, takes the same time at long K, 484 us
//    at 16384 x 8192 x 8192, and 127.5 against 119 us at k = 1024.)
//  * The powers of two go to the instruction as one byte a lane, picked from a
//    register by the instruction itself: the four blocks that a lane takes in a
//    stage are neighbours, so one 4-byte LDS read per 32 rows and stage brings
//    all four. Scales are loaded 16 bytes a row, for two stages at a time, into
//    a ring of their own.
//  * One stage is 64 (4 x 4 blocks of 32 x 32 a wave, four k-steps) instructions
//    of 32 cycles. The operands of k-steps 1 to 3 are all read in its first
//    slots (the accumulators live in the accumulation registers, which leaves
//    128 vector registers for a stage's operands), which frees the buffer for
//    the loads of the stage after next for the rest of the stage.
// 16384 x 8192 x 3584 takes 220 us (4.4 PFLOP/s). The matrix cores' power leaves a
// clock of 1.8 GHz, at which the pipes are busy 60% of the time that a workgroup is
// resident. The rest are waits of the loop: without any loads it takes 207 of 235 us
// (whole tiles, 16 x 16 x 128 shape), without the operand reads 217, without the
// scales 228; and the first loads and the stores of a tile, which nothing overlaps
// with one workgroup a CU.
#pragma once

#include <utility>

#include "gemm_core_w4.hpp"
#include "mc2_mx4.hpp"

namespace mc2 {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

// acc = or += B A^T of one k-step with the scale bytes J of sb and sa, the
// accumulators in the accumulation registers. The compiler sees no matrix
// instruction here: the loop's end waits before anything reads a result.
template <int J>
__device__ __forceinline__ void mfma_mx4_init(f32x16_t& c, u32x4_t b, u32x4_t a, uint32_t sb,
                                              uint32_t sa) {
  asm volatile(
      "v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, 0, %3, %4 "
      "op_sel:[%5,%5,0] op_sel_hi:[%6,%6,0] cbsz:4 blgp:4"
      : "=a"(c)
      : "v"(b), "v"(a), "v"(sb), "v"(sa), "i"(J & 1), "i"(J >> 1));
}
template <int J>
__device__ __forceinline__ void mfma_mx4(f32x16_t& c, u32x4_t b, u32x4_t a, uint32_t sb,
                                         uint32_t sa) {
  asm volatile(
      "v_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 "
      "op_sel:[%5,%5,0] op_sel_hi:[%6,%6,0] cbsz:4 blgp:4"
      : "+a"(c)
      : "v"(b), "v"(a), "v"(sb), "v"(sa), "i"(J & 1), "i"(J >> 1));
}

// 4-byte LDS read at addr + OFF; valid only after a matching lgkm_wait.
template <int OFF>
__device__ __forceinline__ uint32_t lds_rd32_at(uint32_t addr) {
  static_assert(OFF >= 0 && OFF < 65536, "ds_read offset field");
  uint32_t v;
  asm volatile("ds_read_b32 %0, %1 offset:%2" : "=v"(v) : "v"(addr), "i"(OFF) : "memory");
  return v;
}

// Operands of a k-step and scales of a stage; tie(): the values are used, and
// in their registers, from here on.
template <int FM, int FN>
struct MxOps {
  u32x4_t a[FM], b[FN];
  __device__ __forceinline__ void tie() {
#pragma unroll
    for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(a[i]));
#pragma unroll
    for (int i = 0; i < FN; ++i) asm volatile("" : "+v"(b[i]));
  }
};
template <int FM, int FN>
struct MxScales {
  uint32_t a[FM], b[FN];
  __device__ __forceinline__ void tie() {
#pragma unroll
    for (int i = 0; i < FM; ++i) asm volatile("" : "+v"(a[i]));
#pragma unroll
    for (int i = 0; i < FN; ++i) asm volatile("" : "+v"(b[i]));
  }
};

// RS: operand reads a slot in the first slots of a stage.
template <int BM_, int BN_, int RS_>
struct MxTile {
  static constexpr int BM = BM_, BN = BN_, RS = RS_;
  static constexpr int WTM = BM / 2, WTN = BN / 2;  // 2 x 2 waves
  static constexpr int FM = WTM / 32, FN = WTN / 32;
  static constexpr int NT = 256;
  static constexpr int kABytes = BM * kKBytes, kBBytes = BN * kKBytes;
  // scales of a pair of stages: loads of 64 rows, the same number for every wave
  static constexpr int NS = (BM + BN + 255) / 256;
  static constexpr int kScBytes = 4 * NS * 1024;
  static constexpr int kSc0 = 2 * (kABytes + kBBytes);
  static constexpr int kLoopBytes = kSc0 + 2 * kScBytes;
};

// The operand of one side: codes and scales at their first row, bytes a row,
// last row of the matrix relative to the tile's first.
struct MxSide {
  const char* codes;
  const char* scales;
  int64_t last;
};

// Sums the whole K extent (nb blocks) of the tile whose first rows `a` and `b`
// point to. KTAIL: nb is not a multiple of 8, so the last stage's loads check
// the blocks left (lanes past the end load zeros).
template <class TS, bool KTAIL>
__device__ __forceinline__ void mainloop_mx4(lds_t* smem, const MxSide& a, const MxSide& b,
                                             int64_t nb, int64_t pitch,
                                             f32x16_t (&acc)[TS::FM][TS::FN]) {
  constexpr int FM = TS::FM, FN = TS::FN, MM = FM * FN, Q = 4 * MM;
  constexpr int NA = TS::BM / 32, NB = TS::BN / 32, NL = NA + NB;  // loads a wave, 8 rows each
  constexpr int NS = TS::NS;  // scale loads a wave, 64 rows each, per two stages
  constexpr int NF = FM + FN;                  // operand reads per k-step
  static_assert(TS::BM % 64 == 0 && TS::BN % 64 == 0, "a scale load is of one side");
  // slots of a stage, one MFMA each: the reads of k-steps 1 to 3 (RS a slot),
  // kBarA (wait for them; the buffer is free), the loads of the stage after
  // next spread over the rest, kBarB (this wave's loads of the next stage have
  // landed), the next stage's reads of k-step 0 and of its scales
  constexpr int kReadSlots = (3 * NF + TS::RS - 1) / TS::RS;
  constexpr int kBarA = kReadSlots + 1;
  constexpr int kNextReads = 2 * NF;  // operands and scales
  constexpr int kNextSlots = (kNextReads + TS::RS - 1) / TS::RS;
  constexpr int kBarB = Q - kNextSlots - 1;
  constexpr int kLSpan = Q - kBarA - 1;
  static_assert(kBarB > kBarA, "slots for the reads");
  // (load j is issued after slot kBarA + 1 + j * kLSpan / NL)
  constexpr int kLoadsBeforeB = [] {
    int c = 0;
    for (int j = 0; j < NL; ++j) c += kBarA + 1 + j * kLSpan / NL < kBarB;
    return c;
  }();
  static_assert(NL + NS <= 63, "vmcnt range");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wrow0 = (wave >> 1) * TS::WTM, wcol0 = (wave & 1) * TS::WTN;
  const int64_t ld = nb * 16;

  uint32_t l_off[NL];
  int l_chunk[NL];
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    const bool isa = j < NA;
    const int r = 8 * ((isa ? NA : NB) * wave + (isa ? j : j - NA)) + (lane >> 3);
    const int c = (row_off(r, lane & 7) - r * kKBytes) >> 4;
    const int64_t last = isa ? a.last : b.last;
    l_off[j] = static_cast<uint32_t>((r < last ? r : last) * ld + c * 16);
    l_chunk[j] = c;
  }
  // scale loads: 64 rows each, A's rows first
  uint32_t s_off[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    const int r = 64 * (NS * wave + j) + lane;
    const bool isa = 64 * (NS * wave + j) < TS::BM;
    const int rr = isa ? r : r - TS::BM;
    const int64_t last = isa ? a.last : b.last;
    // (past the last row of both sides: nothing is loaded)
    s_off[j] = r < TS::BM + TS::BN ? static_cast<uint32_t>((rr < last ? rr : last) * pitch) : kOffNone;
  }

  const int n = static_cast<int>((nb + 7) / 8);
  int ld_it = 0;
  struct StageLd {
    __amdgpu_buffer_rsrc_t ra, rb;
    int left;  // blocks left
    lds_t* st;
  };
  auto prep = [&]() {
    StageLd s;
    s.left = static_cast<int>(nb) - ld_it * 8;
    s.st = smem + (ld_it & 1) * (TS::kABytes + TS::kBBytes);
    const int nrec = ld_it < n ? 0x7ffffff0 : 0;
    const int64_t k0 = static_cast<int64_t>(ld_it) * kKBytes;
    s.ra = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(a.codes + k0), 0, nrec, kBufFlags);
    s.rb = __builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(b.codes + k0), 0, nrec, kBufFlags);
    ++ld_it;
    return s;
  };
  auto issue_j = [&](const StageLd& s, int j) {
    uint32_t off = l_off[j];
    if constexpr (KTAIL) off = l_chunk[j] < s.left ? off : kOffNone;
    if (j < NA) dma16(s.ra, s.st + 8 * (NA * wave + j) * kKBytes, off);
    else dma16(s.rb, s.st + TS::kABytes + 8 * (NB * wave + (j - NA)) * kKBytes, off);
  };
  // scales of the stages 2 pair and 2 pair + 1
  auto issue_scales = [&](int pair) {
    const int nrec = 2 * pair < n ? 0x7ffffff0 : 0;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const bool isa = 64 * (NS * wave + j) < TS::BM;
      const char* base = (isa ? a.scales : b.scales) + static_cast<int64_t>(pair) * 16;
      dma16(__builtin_amdgcn_make_buffer_rsrc(const_cast<char*>(base), 0, nrec, kBufFlags),
            smem + TS::kSc0 + (pair & 1) * TS::kScBytes + 1024 * (NS * wave + j), s_off[j]);
    }
  };

  // LDS read addresses of the wave's first fragment for k-step j of buffer p;
  // fragment f sits 32 rows (4096 bytes) further on
  const uint32_t s0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(smem));
  constexpr uint32_t kStage = TS::kABytes + TS::kBBytes;
  uint32_t adA[4], adB[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ch = 4 * (lane >> 5) + j;
    adA[j] = s0 + row_off(wrow0 + (lane & 31), ch);
    adB[j] = s0 + TS::kABytes + row_off(wcol0 + (lane & 31), ch);
  }
  const uint32_t adSA = s0 + TS::kSc0 + (wrow0 + (lane & 31)) * 16 + (lane >> 5) * 4;
  const uint32_t adSB = s0 + TS::kSc0 + (TS::BM + wcol0 + (lane & 31)) * 16 + (lane >> 5) * 4;

  MxOps<FM, FN> x[4];     // operands of the four k-steps
  MxScales<FM, FN> sc[2];  // scales of a stage of either parity
  // operand read i of k-step J of buffer P
  auto read_op = [&](auto I, auto Jc, auto Pc) {
    constexpr int i = decltype(I)::value, J = decltype(Jc)::value, P = decltype(Pc)::value;
    constexpr int kFrag = 32 * kKBytes;
    // (the second buffer's offset does not fit the read's offset field)
    if constexpr (i < FN) x[J].b[i] = lds_rd128_at<i * kFrag>(adB[J] + P * kStage);
    else x[J].a[i - FN] = lds_rd128_at<(i - FN) * kFrag>(adA[J] + P * kStage);
  };
  auto read_scale = [&](auto I, auto Pc, uint32_t ring) {
    constexpr int i = decltype(I)::value, P = decltype(Pc)::value;
    if constexpr (i < FN) sc[P].b[i] = lds_rd32_at<i * 512 + 8 * P>(adSB + ring);
    else sc[P].a[i - FN] = lds_rd32_at<(i - FN) * 512 + 8 * P>(adSA + ring);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  StageLd nx;
  issue_scales(0);
  nx = prep();
#pragma unroll
  for (int j = 0; j < NL; ++j) issue_j(nx, j);
  nx = prep();
#pragma unroll
  for (int j = 0; j < NL; ++j) issue_j(nx, j);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NL) : "memory");  // stage 0 and its scales have landed
  bar_sync();
  sfor<NF>([&](auto I) { read_op(I, I0{}, I0{}); });
  sfor<NF>([&](auto I) { read_scale(I, I0{}, 0u); });

  auto stage = [&](auto Pc, auto First, int it) {
    constexpr int P = decltype(Pc)::value;
    constexpr bool FIRST = decltype(First)::value;
    using NP = std::integral_constant<int, 1 - P>;
    lgkm_wait(0);  // this stage's k-step 0 and scales (read during the previous stage)
    x[0].tie();
    sc[P].tie();
    // scale ring of the next stage
    const uint32_t ring = static_cast<uint32_t>(((it + 1) >> 1) & 1) * TS::kScBytes;
    sfor<Q>([&](auto Qc) {
      constexpr int q = decltype(Qc)::value;
      constexpr int J = q / MM, s = q % MM, fm = s / FN, fn = s % FN;
      if constexpr (s == 0 && J > 0) {
        // operands of k-step J: reads issued after them may be in flight
        constexpr int issued = q * TS::RS < 3 * NF ? q * TS::RS : 3 * NF;
        constexpr int need = J * NF;
        static_assert(issued >= need, "operands read ahead of their k-step");
        if constexpr (q <= kBarA) lgkm_wait(issued - need);
        x[J].tie();
      }
      if constexpr (FIRST && J == 0)
        mfma_mx4_init<J>(acc[fm][fn], x[J].b[fn], x[J].a[fm], sc[P].b[fn], sc[P].a[fm]);
      else
        mfma_mx4<J>(acc[fm][fn], x[J].b[fn], x[J].a[fm], sc[P].b[fn], sc[P].a[fm]);
      if constexpr (q < kReadSlots) {
        sfor<TS::RS>([&](auto R) {
          constexpr int i = q * TS::RS + decltype(R)::value;
          if constexpr (i < 3 * NF)
            read_op(std::integral_constant<int, i % NF>{},
                    std::integral_constant<int, 1 + i / NF>{}, Pc);
        });
      } else if constexpr (q == kBarA) {
        lgkm_wait(0);  // every read of this stage's buffer is done
        bar_sync();    // ... by every wave: the buffer may be refilled
        nx = prep();
        if constexpr (P == 0) issue_scales((it + 2) >> 1);
      } else if constexpr (q == kBarB) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoadsBeforeB + (P == 0 ? NS : 0)) : "memory");
        bar_sync();
      } else if constexpr (q > kBarB) {
        sfor<TS::RS>([&](auto R) {
          constexpr int i = (q - kBarB - 1) * TS::RS + decltype(R)::value;
          if constexpr (i < NF)
            read_op(std::integral_constant<int, i>{}, I0{}, NP{});
          else if constexpr (i < kNextReads)
            read_scale(std::integral_constant<int, i - NF>{}, NP{}, ring);
        });
      }
      sfor<NL>([&](auto Jl) {
        constexpr int j = decltype(Jl)::value;
        if constexpr (kBarA + 1 + j * kLSpan / NL == q) issue_j(nx, j);
      });
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using T = std::true_type;
  using F = std::false_type;
  stage(I0{}, T{}, 0);
  for (int it = 1; it < n; it += 2) {
    stage(I1{}, F{}, it);
    if (it + 1 < n) stage(I0{}, F{}, it + 1);
  }
  // the last stage's reads of the next one (never used) stay in their registers
  // until they have landed
  lgkm_wait(0);
  x[0].tie();
  sc[0].tie();
  sc[1].tie();
  wait_vmcnt0();
  bar_sync();
  // the last MFMAs' results are complete before anything reads them
  asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int fm = 0; fm < FM; ++fm)
#pragma unroll
    for (int fn = 0; fn < FN; ++fn) asm volatile("" : "+a"(acc[fm][fn]));
}

}  // namespace mc2
