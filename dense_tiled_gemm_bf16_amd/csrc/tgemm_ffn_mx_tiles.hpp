// Tiled products of MXFP4 operands with a fused epilogue for gfx950, dense and
// grouped.  256 x 256 tiles take the MXFP4 K loop of tgemm_kernel.hpp; MxTile
// here is the kernel of smaller tiles, and of scale rows that do not start on
// a dword.  The epilogues are those of the 16-bit products
// (tgemm_ffn_tiles.hpp): sums, bias, activation and residual are binary32, C is
// rounded once.
#pragma once

#include "tgemm_ffn_tiles.hpp"

namespace tgemm {
namespace ffn {
namespace {

// The MXFP4 operands of the 256 x 256 kernel, C in bf16 or fp16.
template <bool F16>
struct MxTraits : Traits<kFp4, true, true, true> {
  static constexpr bool kOutF16 = F16;
};

typedef __attribute__((ext_vector_type(8))) int v8i;

// Bytes of a slice row.  TWO: two workgroups share a CU.
template <int TM, bool TWO>
constexpr int kMxSlice = TM == 64 && !TWO ? 256 : 128;

struct MxSlots {
  LDS_AS uint8_t *a[4], *b[4];  // kNS slots of TM, TN rows
  LDS_AS uint8_t *s[4];         // scales, 16 bytes of a row: of B's rows, then A's; then the same from 4 bytes on
};

// MxTile: TM x TN of C by 4 waves (2 x 2), K in slices of SL bytes (2 SL
// elements) of a row through a ring of kNS slots, rows and scales loaded into
// LDS directly.
//
// Lane l of the scaled v_mfma 16x16x128 takes row l % 16 and one block of 32
// elements.  Over the kP = SL / 64 products of a slice lane group g = l / 16
// takes blocks kP g .. kP g + kP - 1 of the slice, one a product, of both
// operands alike: its scales of a slice are then kP bytes side by side, byte s
// for product s, and no scale moves between lanes.  A slot row keeps block c at
// 16-byte chunk c ^ perm(row % 16): the rows of a fragment read fall on
// different LDS banks (no conflict in 21 million reads), and four lanes side by
// side load 64 bytes side by side.  (With the chunks of one product side by
// side instead, four lanes loaded from four places: 24 bytes a clock and CU at
// most.)  A row's scales come 16 bytes at a time, those of 512 elements: a load
// of 4 bytes a lane and slice cost the texture path as much as the rows.
//
// Few 64 x 64 tiles, one a CU: slices of 256 bytes and four slots (128 KiB), 96 KiB
// on their way.  TWO, for more tiles than CUs: slices of 128 bytes, four slots
// of 64 x 64 or two of 128 x 128 (64 KiB), so that two workgroups share a CU and
// the one multiplies while the other waits or stores.
//
// ALIGNED: every row's scales start on a dword.  If not, a lane loads from the
// dword that holds the first, and shifts.
template <int DT, int TM, int TN, bool TWO, bool ALIGNED, class EXT>
struct MxTile {
  static constexpr int kBlk = 16;
  static constexpr int kWM = TM / 2, kWN = TN / 2, kNBm = kWM / 16, kNBn = kWN / 16;
  static constexpr int SL = kMxSlice<TM, TWO>, kP = SL / 64;  // bytes of a slice row; products of a slice
  static constexpr int kNS = TM == 64 ? 4 : 2;
  static constexpr int kIR = 1024 / SL;                  // rows of a load instruction
  static constexpr int kLA = TM / 4 / kIR, kLB = TN / 4 / kIR;  // row load instructions of a wave and slice
  static constexpr int kPer16 = 16 / kIR;                // instructions after which the rows' permutation repeats
  static constexpr int kPairs = 256 / SL;                // slices that share a load of scales
  // Scale loads: 64 rows an instruction, 16 bytes (those of a slice) each, one
  // instruction a wave (the rows past TM + TN: nothing).
  static constexpr int kPlanes = ALIGNED ? 1 : 2, kPlane = 4 * 1024;
  static constexpr int kLoads = kLA + kLB + kPlanes;
  static constexpr int kScaleBytes = kPlane * kPlanes;
  static_assert(kLA % kPer16 == 0 && kLB % kPer16 == 0 && TN % 64 == 0 && TM + TN <= 256, "whole instructions");
  static_assert((kNS - 1) * kLoads < 64, "vmcnt is 6 bits");
  static_assert(kNS == 4 || (kP == 2 && kPairs == 2), "two slots: two products, scales of two slices");
  // Loads behind slice kt + 1 that may be on their way when it is waited for in
  // slice kt, S = kt % 4: of the two slices after it, or with two slots of the one.
  // (Of two slices one is even; if they share scales, those come with it.)
  static constexpr int ahead(int S) {
    return kNS == 2 ? kLA + kLB + (S % 2 == 0 ? kPlanes : 0) : 2 * (kLA + kLB) + 2 / kPairs * kPlanes;
  }

  const Args &a;
  MxSlots slots;
  EXT x;
  int kbv;  // scales of a row from the first slice on (rows are a.kb apart)
  int lane, wave, wave_m, wave_n, m0, n0;
  __amdgpu_buffer_rsrc_t ra, rb, rsa, rsb;
  uint32_t offa[kLA], offb[kLB];
  int at_a[kLA], at_s;     // gathered: the rows of offa and offs
  int kcol[kPer16];        // this lane's byte in a slice row, by instruction % kPer16
  uint32_t offs;           // aligned offset of this lane's row of scales in slice 0
  uint32_t sh_x[2], sh_y[EXT::kGather ? kNBm : 1];  // where this lane's scales start in their dword
  uint32_t frag;           // this lane's chunk of product 0
  f32x4 acc[kNBn][kNBm];

  __device__ __forceinline__ MxTile(const Args &args, const MxSlots &s, const EXT &ext) : a(args), slots(s), x(ext), kbv(args.kb) {}

  // Banks repeat every 256 bytes, one row or two.  LDS serves a read of 16
  // bytes a lane in groups of 16 lanes; whether those are 16 rows of one lane
  // group, or rows 0-3 and 12-15 of one and 4-11 of the next, their chunks differ.
  __device__ static __forceinline__ int perm(int r) {
    if constexpr (SL == 256) return r ^ ((r & 4) << 1);
    return ((r >> 1) & 3) | ((((r >> 2) ^ (r >> 3)) & 1) << 2);
  }

  // Row of B (from the tile's first on) that LDS row r holds, or -1.
  __device__ __forceinline__ int b_row(int r) const {
    if constexpr (EXT::kGated) {
      const int c = ((r >> 5) << 4) + (r & 15);
      return c < min(a.N - n0, TN / 2) ? c + ((r >> 4) & 1 ? x.half : 0) : -1;
    } else {
      return r < min(a.N - n0, TN) ? r : -1;
    }
  }
  // Row of A (of the array if gathered, else from the tile's first on) that
  // LDS row r holds, or -1.  at: what index(r) read.
  __device__ __forceinline__ int index(int r) const {
    if constexpr (EXT::kGather)
      if (x.rows) return x.rows[m0 + min(r, a.M - m0 - 1)];
    return 0;
  }
  __device__ __forceinline__ int a_row(int r, int at) const {
    if constexpr (EXT::kGather)
      if (x.rows) return r < min(a.M - m0, TM) && at >= 0 && at < x.src_rows ? at : -1;
    return r < min(a.M - m0, TM) ? r : -1;
  }

  // Up to B's rows.
  __device__ __forceinline__ void init_b() {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    wave_m = wave >> 1;
    wave_n = wave & 1;
    m0 = x.m0;
    n0 = x.n0;
    constexpr int kCh = SL / 16;
    const int lr = lane / kCh;
    // (Read ahead: B's loads do not wait for them.)
#pragma unroll
    for (int i = 0; i < kLA; ++i) at_a[i] = index(kIR * (wave * kLA + i) + lr);
    at_s = index(max(64 * wave - TN + lane, 0));
    const int brows = EXT::kGated ? ext_half() + min(a.N - n0, TN / 2) : min(a.N - n0, TN);
    rb = make_rsrc(a.B + (size_t)n0 * a.ldb, (uint32_t)(brows - 1) * (uint32_t)a.ldb + (uint32_t)a.K);
    // Rows: lane l of instruction i writes chunk l % kCh of row kIR i + l / kCh
    // of the wave's rows, whose number % 16 goes by i % kPer16.
#pragma unroll
    for (int p = 0; p < kPer16; ++p) kcol[p] = 16 * ((lane % kCh) ^ perm(kIR * p + lr));
#pragma unroll
    for (int i = 0; i < kLB; ++i) {
      const int row = b_row(kIR * (wave * kLB + i) + lr);
      offb[i] = row >= 0 ? (uint32_t)row * (uint32_t)a.ldb + (uint32_t)kcol[i % kPer16] : kOOB;
    }
  }
  // The rest.
  __device__ __forceinline__ void init_a() {
    bool gather = false;
    if constexpr (EXT::kGather) gather = x.rows != nullptr;
    int src = min(a.M - m0, TM);
    if constexpr (EXT::kGather) src = gather ? x.src_rows : src;
    ra = make_rsrc(a.A + (gather ? (size_t)0 : (size_t)m0 * a.lda),
                   src > 0 ? (uint32_t)(src - 1) * (uint32_t)a.lda + (uint32_t)a.K : 0u);
    const int brows = EXT::kGated ? ext_half() + min(a.N - n0, TN / 2) : min(a.N - n0, TN);
    // Scales: based at the dword that holds the first byte, up to the one that
    // holds the last.
    const uintptr_t pa = (uintptr_t)(a.SA + (gather ? (size_t)0 : (size_t)m0 * a.kb));
    const uintptr_t pb = (uintptr_t)(a.SB + (size_t)n0 * a.kb);
    const uint32_t mis_a = (uint32_t)(pa & 3), mis_b = (uint32_t)(pb & 3);
    rsa = make_rsrc((const void *)(pa - mis_a), src > 0 ? (mis_a + (uint32_t)(src - 1) * (uint32_t)a.kb + (uint32_t)kbv + 3u) & ~3u : 0u);
    rsb = make_rsrc((const void *)(pb - mis_b), (mis_b + (uint32_t)(brows - 1) * (uint32_t)a.kb + (uint32_t)kbv + 3u) & ~3u);

    const int r = lane & 15, g = lane >> 4;
    const int lr = lane / (SL / 16);
#pragma unroll
    for (int i = 0; i < kLA; ++i) {
      const int row = a_row(kIR * (wave * kLA + i) + lr, at_a[i]);
      offa[i] = row >= 0 ? (uint32_t)row * (uint32_t)a.lda + (uint32_t)kcol[i % kPer16] : kOOB;
    }
    // Scales: lane l of wave w takes row 64 w + l of B's and A's together.
    {
      const bool isb = wave < TN / 64;
      const int row = isb ? b_row(64 * wave + lane) : a_row(64 * wave - TN + lane, at_s);
      offs = row >= 0 ? ((isb ? mis_b : mis_a) + (uint32_t)row * (uint32_t)a.kb) & ~3u : kOOB;
    }
    if constexpr (!ALIGNED) {
      // (16 rows are 16 kb bytes: one shift for all blocks, of each half.)
      sh_x[0] = (mis_b + (uint32_t)r * (uint32_t)a.kb) & 3u;
      sh_x[1] = (mis_b + (uint32_t)(r + ext_half()) * (uint32_t)a.kb) & 3u;
      if constexpr (EXT::kGather) {
#pragma unroll
        for (int j = 0; j < kNBm; ++j)
        {
          const int row = wave_m * kWM + 16 * j + r;
          sh_y[j] = (mis_a + (uint32_t)max(a_row(row, index(row)), 0) * (uint32_t)a.kb) & 3u;
        }
      } else {
        sh_y[0] = (mis_a + (uint32_t)r * (uint32_t)a.kb) & 3u;
      }
    }
    frag = (uint32_t)(r * SL + (((kP * g) ^ perm(r)) << 4));
#pragma unroll
    for (int i = 0; i < kNBn; ++i)
#pragma unroll
      for (int j = 0; j < kNBm; ++j) acc[i][j] = f32x4{};
  }
  __device__ __forceinline__ int ext_half() const {
    if constexpr (EXT::kGated) return x.half;
    return 0;
  }

  // S below is kt % 4: rows in slot kt % kNS, scales in slot S / kPairs.
  // Load I of slice kt into its slot.  The last slices check columns: what lies
  // past K arrives as zeros, and a slice past the last is all zeros.
  template <int S, int I>
  __device__ __forceinline__ void load_one(int kt) const {
    const int left = a.K - kt * SL;  // bytes of a row from this slice on
    const bool whole = left >= SL;
    if constexpr (I < kLA + kLB) {
      constexpr bool isb = I >= kLA;
      constexpr int i = isb ? I - kLA : I;
      const uint32_t v = whole || kcol[i % kPer16] < left ? (isb ? offb[i % kLB] : offa[i % kLA]) : kOOB;
      LDS_AS uint8_t *dst = (isb ? slots.b[S % kNS] : slots.a[S % kNS]) + (wave * (isb ? kLB : kLA) + i) * 1024;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(isb ? rb : ra, (LDS_AS void *)dst, 16, v, (uint32_t)(kt * SL), 0, 0);
    } else if constexpr (S % kPairs == 0) {
      constexpr int p = I - kLA - kLB;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(wave < TN / 64 ? rsb : rsa,
                                               (LDS_AS void *)(slots.s[S / kPairs] + p * kPlane + wave * 1024), 16,
                                               left > 0 ? offs : kOOB, (uint32_t)(kt / kPairs) * 16u + 4u * (uint32_t)p, 0, 0);
    }
  }

  struct Frags {
    u32x4 x[kNBn], y[kNBm];
  };
  // Scales as read (block R: x blocks, then y blocks), and as the MFMAs take them.
  struct Raw {
    uint32_t w[kNBn + kNBm][kPairs == 2 ? 4 : ALIGNED ? 1 : 2];
  };
  uint32_t sc[kNBn + kNBm];
  static constexpr int kPer = kNBn * kNBm, kNR = kNBn + kNBm;  // MFMAs and fragment reads of a product
  // Fragment R (x blocks, then y blocks) of product P.
  template <int S, int P, int R>
  __device__ __forceinline__ void read_frag(Frags &f) const {
    const uint32_t at = frag ^ (uint32_t)(P << 4);
    if constexpr (R < kNBn)
      f.x[R] = *(const LDS_AS u32x4 *)(slots.b[S % kNS] + (wave_n * kWN + 16 * R) * SL + at);
    else
      f.y[R - kNBn] = *(const LDS_AS u32x4 *)(slots.a[S % kNS] + (wave_m * kWM + 16 * (R - kNBn)) * SL + at);
  }
  // This lane's scales of block R: of slice kt, or of slices kt and kt + 1 (kt
  // even, kPairs == 2; both at once, so that the slot is free for the pair after
  // the next when slice kt begins).  Read in front of slice kt, made up in it
  // (finish_scale): on the spot, each would wait for its read.
  template <int S, int R>
  __device__ __forceinline__ void read_scale(Raw &c) const {
    const int b = R < kNBn ? wave_n * kNBn + R : TN / 16 + wave_m * kNBm + R - kNBn;
    const int g = lane >> 4;
    const LDS_AS uint8_t *p = slots.s[S / kPairs] + b * 256 + 16 * (lane & 15);
    if constexpr (ALIGNED && kPairs == 2) {
      const u32x4 v = *(const LDS_AS u32x4 *)p;
#pragma unroll
      for (int i = 0; i < 4; ++i) c.w[R][i] = v[i];
      return;
    }
    p += (kP * g) & ~3;
#pragma unroll
    for (int h = 0; h < kPairs; ++h) {
      c.w[R][h] = *(const LDS_AS uint32_t *)(p + 8 * h);
      if constexpr (!ALIGNED) c.w[R][kPairs + h] = *(const LDS_AS uint32_t *)(p + 8 * h + kPlane);
    }
  }
  template <int R>
  __device__ __forceinline__ void finish_scale(const Raw &c, uint32_t keep) {
    if constexpr (ALIGNED) {
      if constexpr (kPairs == 1) {
        sc[R] = c.w[R][0] & keep;
      } else {
        const uint32_t pick = 0x0100u + 0x0202u * (uint32_t)(lane >> 4);  // bytes 2 g and 2 g + 1 of eight
        sc[R] = (__builtin_amdgcn_perm(c.w[R][1], c.w[R][0], 0x0c0c0000u | pick) |
                 __builtin_amdgcn_perm(c.w[R][3], c.w[R][2], pick << 16 | 0x0c0cu)) & keep;
      }
    } else {
      const uint32_t sh = R < kNBn ? sh_x[EXT::kGated ? R & 1 : 0] : sh_y[EXT::kGather ? (R < kNBn ? 0 : R - kNBn) : 0];
      if constexpr (kPairs == 1) {
        sc[R] = __builtin_amdgcn_alignbyte(c.w[R][1], c.w[R][0], sh) & keep;
      } else {
        const uint32_t by = 8 * sh + 16 * ((lane >> 4) & 1);  // (up to 5 bytes on)
        const uint32_t lo = (uint32_t)(((uint64_t)c.w[R][2] << 32 | c.w[R][0]) >> by);
        const uint32_t hi = (uint32_t)(((uint64_t)c.w[R][3] << 32 | c.w[R][1]) >> by);
        sc[R] = __builtin_amdgcn_perm(hi, lo, 0x05040100u) & keep;
      }
    }
  }
  // The bytes of a lane's scales that are the row's: those behind its last are
  // the next row's, and a NaN among them would meet the zeros past K.
  __device__ __forceinline__ uint32_t keep_of(int kt) const {
    const int left = kbv - kP * (4 * kt + (lane >> 4));
    auto low = [](int n, int most) { return n >= most ? ~0u >> (32 - 8 * most) : n <= 0 ? 0u : ~0u >> (32 - 8 * n); };
    if constexpr (kPairs == 1) return low(left, 4);
    return low(left, 2) | low(left - 8, 2) << 16;
  }
  template <int S, int... R>
  __device__ __forceinline__ void read_first(std::integer_sequence<int, R...>, Frags &f, Raw &c) const {
    (read_frag<S, 0, R>(f), ...);
    (read_scale<S, R>(c), ...);
  }

  template <int SEL>
  __device__ static __forceinline__ f32x4 mma(const u32x4 &p, const u32x4 &q, const f32x4 &c, uint32_t sp, uint32_t sq) {
    const v8i p8 = {(int)p[0], (int)p[1], (int)p[2], (int)p[3], 0, 0, 0, 0};
    const v8i q8 = {(int)q[0], (int)q[1], (int)q[2], (int)q[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p8, q8, c, 4, 4, SEL, (int)sp, SEL, (int)sq);
  }

  // MFMA Q of product P of slice kt in slot S, its fragments in f.  Between
  // the MFMAs the next product's fragments are read into fn, and the loads of
  // the slice kNS behind the one that just left its slot go out.  Four slots:
  //  * before the last product a wait and a barrier: slice kt + 1 has landed in
  //    every wave, and every wave holds the last fragments of slice kt, so that
  //    its slot may take slice kt + 4;
  //  * the last product reads the first fragments and the scales of slice kt + 1
  //    (of the pair that it begins);
  //  * the loads go out over kWindow MFMAs behind the barrier.
  // Two slots (and two products): a slot is read in as short a time as goes, so
  // that its next slice is loaded for one and a half slices, not one.
  //  * The first half of the first product reads the second's fragments; then a
  //    barrier, and the loads of slice kt + 2 go out over kWindow MFMAs.
  //  * In the middle of the second product slice kt + 1 is waited for (slice
  //    kt + 2 is on its way), a barrier, and its first fragments and scales are read.
  // (Freed and waited for at one place, as with four slots: 1024 x 4096 x 4096 16.4
  // -> 14.9 us, 32768 gathered rows of 32 experts, 4096 x 2048, 235 -> 227; 32768 x 4096 x
  // 8192 swiglu 634 -> 640.)  What is left is the loads themselves: without them 392
  // of 622 us there, without the reads of fragments 576.  Loads over half as many MFMAs: 626.
  // (Left to the compiler, the loads sank to the end of the slice, in front of
  // the wait for them, and the fragments' reads to their use: 1123 us.)
  static constexpr int kWindow = kNS == 2 ? kPer : (kP - 1) * kPer;
  static constexpr int kHalf = kPer / 2;
  // The MFMA of load i, from the barrier on.
  static constexpr int load_pos(int i) { return i * kWindow / kLoads; }
  template <int S, int P, int Q, int R>
  __device__ __forceinline__ void read_at(int kt, Frags &fn, Raw &cn) const {
    // (The compiler waits for loads into the scales' slots in front of these
    // reads, whichever slot they read: right behind the barrier, in front of the next loads,
    // it has none or few to wait for.)
    constexpr int kAt = kNS == 2 && P == kP - 1 ? kHalf : 0;  // the first MFMA with reads
    if constexpr (P == kP - 1 && Q == kAt && (S + 1) % kPairs == 0) read_scale<(S + 1) % 4, R>(cn);
    if constexpr (kAt + R * (kNS == 2 ? kHalf : kPer) / kNR == Q) {
      if constexpr (P < kP - 1)
        read_frag<S, P + 1, R>(fn);
      else
        read_frag<(S + 1) % 4, 0, R>(fn);
    }
  }
  template <int S, int P, int Q, int I>
  __device__ __forceinline__ void load_at(int kt) const {
    if constexpr (kNS == 2) {
      if constexpr (load_pos(I) + kHalf == P * kPer + Q) load_one<(S + 2) % 4, I>(kt + 2);
    } else if constexpr (load_pos(I) == (P + 1) % kP * kPer + Q) {
      if constexpr (P == kP - 1)
        load_one<(S + kNS) % 4, I>(kt + kNS);
      else
        load_one<(S + kNS - 1) % 4, I>(kt + kNS - 1);
    }
  }
  template <int S, int P, int Q, int... R>
  __device__ __forceinline__ void reads_at(std::integer_sequence<int, R...>, int kt, Frags &fn, Raw &cn) const {
    (read_at<S, P, Q, R>(kt, fn, cn), ...);
  }
  template <int S, int P, int Q, int... I>
  __device__ __forceinline__ void loads_at(std::integer_sequence<int, I...>, int kt) const {
    (load_at<S, P, Q, I>(kt), ...);
  }
  template <int S, int P, int Q>
  __device__ __forceinline__ void mfma_one(int kt, const Frags &f, Frags &fn, Raw &c) {
    if constexpr (kNS == 2 && P == 0 && Q == kHalf) {
      wait_vm_lgkm0<63>();  // (the reads alone)
      barrier();
    }
    if constexpr (P == kP - 1 && Q == (kNS == 2 ? kHalf : 0)) {
      wait_vm_lgkm0<ahead(S)>();
      barrier();
    }
    constexpr bool kNewScales = P == 0 && S % kPairs == 0;
    if constexpr (kNewScales) {
      // Blocks that this MFMA is the first to take.
      const uint32_t keep = keep_of(kt);
      if constexpr (Q < kNBm) finish_scale<kNBn + Q>(c, keep);
      if constexpr (Q % kNBm == 0) finish_scale<Q / kNBm>(c, keep);
    }
    reads_at<S, P, Q>(std::make_integer_sequence<int, kNR>(), kt, fn, c);
    loads_at<S, P, Q>(std::make_integer_sequence<int, kLoads>(), kt);
    // (The y blocks snake, so that MFMAs side by side share an operand.)
    constexpr int I = Q / kNBm, J0 = Q % kNBm, J = (I & 1) ? kNBm - 1 - J0 : J0;
    acc[I][J] = mma<P + kP * (S % kPairs)>(f.x[I], f.y[J], acc[I][J], sc[I], sc[kNBn + J]);
    __builtin_amdgcn_sched_barrier(0);
  }
  template <int S, int P, int... Q>
  __device__ __forceinline__ void product(std::integer_sequence<int, Q...>, int kt, const Frags &f, Frags &fn, Raw &c) {
    (mfma_one<S, P, Q>(kt, f, fn, c), ...);
  }
  // Slice kt (S = kt % 4); its first fragments are in f0, its scales, if they
  // are new, in c.
  template <int S>
  __device__ __forceinline__ void step(int kt, Frags &f0, Frags &f1, Raw &c) {
    constexpr auto all = std::make_integer_sequence<int, kPer>();
    product<S, 0>(all, kt, f0, f1, c);
    product<S, 1>(all, kt, f1, f0, c);
    if constexpr (kP == 4) {
      product<S, 2>(all, kt, f0, f1, c);
      product<S, 3>(all, kt, f1, f0, c);
    }
  }
  // Loads of slice kNS - 1 that go out in front of the first barrier (scales
  // come with every kPairs-th slice).  Two slots: all of them.
  static constexpr int early() {
    if (kNS == 2) return kLA + kLB;
    int n = 0;
    for (int i = 0; i < kLoads; ++i) n += load_pos(i) < kPer && (i < kLA + kLB || (kNS - 1) % kPairs == 0);
    return n;
  }

  // Loads I0 .. I0 + N - 1 of slice S, one of the first.
  template <int S, int I0, int... I>
  __device__ __forceinline__ void load_from(std::integer_sequence<int, I...>) const {
    (load_one<S, I0 + I>(S), ...);
  }
  template <int S, int I0, int N>
  __device__ __forceinline__ void load_part() const {
    load_from<S, I0>(std::make_integer_sequence<int, N>());
  }
  template <int S>
  __device__ __forceinline__ void load_a() const {
    load_part<S, 0, kLA>();
    load_part<S, kLA + kLB, kPlanes>();
  }

  __device__ __forceinline__ void run() {
    init_b();
    const int nk = (a.K + SL - 1) / SL;
    // Slices 0 .. kNS - 2, and of slice kNS - 1 what a slice before the first
    // would have loaded behind its barrier (two slots: all; an odd slice brings no scales).
    if constexpr (EXT::kGather) {
      // B's rows first, which wait for no index.  (With the groups read once, below:
      // 37 tokens of 64 experts 32.4 -> 31.1 us, 200 tokens 38.7 -> 37.2, 32768 rows of 32
      // experts 240 -> 232, 4000 rows of 16 experts on 64 x 64 tiles 17.9 -> 16.4.)  Loads
      // are waited for in their order: with slice 0 for slice 1's too if there are
      // four slots, as the first step's wait counts on B's loads of slice 2 behind those.
      load_part<0, kLA, kLB>();
      load_part<1, kLA, kLB>();
      if constexpr (kNS == 4) load_part<2, kLA, kLB>();
      init_a();
      load_a<0>();
      load_a<1>();
      if constexpr (kNS == 4) load_a<2>();
    } else {
      init_a();
      load_part<0, 0, kLoads>();
      load_part<1, 0, kNS == 2 ? early() : kLoads>();
      if constexpr (kNS == 4) load_part<2, 0, kLoads>();
    }
    if constexpr (kNS == 4) load_part<3, 0, early()>();  // (row loads come first)
    constexpr int kLate = EXT::kGather ? kLA + (kNS == 4 && 2 % kPairs == 0 ? kPlanes : 0) : kNS == 2 ? 0 : ahead(0);
    wait_vm_lgkm0<kLate + (EXT::kGather && kNS == 2 ? 0 : early())>();
    barrier();
    Frags f0, f1;
    Raw c;
    read_first<0>(std::make_integer_sequence<int, kNR>(), f0, c);
    int kt = 0;
    for (; kt + 3 < nk; kt += 4) {
      step<0>(kt, f0, f1, c);
      step<1>(kt + 1, f0, f1, c);
      step<2>(kt + 2, f0, f1, c);
      step<3>(kt + 3, f0, f1, c);
    }
    if (kt < nk) step<0>(kt, f0, f1, c);
    if (kt + 1 < nk) step<1>(kt + 1, f0, f1, c);
    if (kt + 2 < nk) step<2>(kt + 2, f0, f1, c);
    // The loads still in flight into the slots.
    wait_vm_lgkm0<0>();
    x.store(*this);
  }

  // The rounding alone (see the plain products' epilogue): lane swaps leave a
  // lane 8 columns of a row.
  __device__ __forceinline__ void epilogue() {
    static_assert(kNBn % 2 == 0, "blocks pair up along N");
    const int q = lane >> 4;
#pragma unroll
    for (int j = 0; j < kNBm; ++j) {
      const int m = m0 + wave_m * kWM + j * 16 + (lane & 15);
      uint8_t *crow = a.C + (size_t)m * a.ldc * 2;
#pragma unroll
      for (int i = 0; i < kNBn; i += 2) {
        const f32x4 &u = acc[i][j], &v = acc[i + 1][j];
        const uint32_t us[2] = {pack2<DT>(u[0], u[1]), pack2<DT>(u[2], u[3])};
        const uint32_t vs[2] = {pack2<DT>(v[0], v[1]), pack2<DT>(v[2], v[3])};
        uint32_t xo[2], yo[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const auto h = __builtin_amdgcn_permlane32_swap(us[d], vs[d], false, false);
          const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
          xo[d] = r[0];
          yo[d] = r[1];
        }
        const int n = n0 + wave_n * kWN + i * 16 + 8 * q;
        if (m < a.M && n < a.N) store_c(crow + (size_t)n * 2, u32x4{xo[0], xo[1], yo[0], yo[1]});
      }
    }
  }
};

// (Arrays, not one: the compiler then sees that a read of one slot needs no
// wait for loads into another. It tells at most eight apart.)
#define TGEMM_MX_SLOTS(TM, TN, SL, NS, SCALES)                              \
  __shared__ __attribute__((aligned(1024))) uint8_t sR0[(TM + TN) * SL];    \
  __shared__ __attribute__((aligned(1024))) uint8_t sR1[(TM + TN) * SL];    \
  __shared__ __attribute__((aligned(1024))) uint8_t sS0[SCALES];            \
  __shared__ __attribute__((aligned(1024))) uint8_t sS1[SCALES];            \
  MxSlots slots;                                                            \
  slots.a[0] = (LDS_AS uint8_t *)sR0;                                       \
  slots.a[1] = (LDS_AS uint8_t *)sR1;                                       \
  slots.b[0] = (LDS_AS uint8_t *)sR0 + TM * SL;                             \
  slots.b[1] = (LDS_AS uint8_t *)sR1 + TM * SL;                             \
  slots.s[0] = (LDS_AS uint8_t *)sS0;                                       \
  slots.s[1] = (LDS_AS uint8_t *)sS1;                                       \
  if constexpr (NS == 4) {                                                  \
    __shared__ __attribute__((aligned(1024))) uint8_t sR2[(TM + TN) * SL];  \
    __shared__ __attribute__((aligned(1024))) uint8_t sR3[(TM + TN) * SL];  \
    slots.a[2] = (LDS_AS uint8_t *)sR2;                                     \
    slots.a[3] = (LDS_AS uint8_t *)sR3;                                     \
    slots.b[2] = (LDS_AS uint8_t *)sR2 + TM * SL;                           \
    slots.b[3] = (LDS_AS uint8_t *)sR3 + TM * SL;                           \
  }                                                                         \
  if constexpr (SL == 256) {                                                \
    __shared__ __attribute__((aligned(1024))) uint8_t sS2[SCALES];          \
    __shared__ __attribute__((aligned(1024))) uint8_t sS3[SCALES];          \
    slots.s[2] = (LDS_AS uint8_t *)sS2;                                     \
    slots.s[3] = (LDS_AS uint8_t *)sS3;                                     \
  }

// A bias alone, straight from the accumulators (as the rounding alone): lane l
// holds row l % 16 and columns 4 (l / 16) .. + 3 of each block.  (4096 x 4096 x 2048
// through LDS 29 us, this way 21.)
template <int DT, bool GROUPED>
struct BiasExt {
  static constexpr bool kOn = true, kGated = false, kGather = GROUPED, kPrefetch = true;
  int m0, n0;
  int half;
  const int32_t *rows;
  int src_rows;
  Tail t;
  template <class K>
  __device__ __forceinline__ void store(K &k) const {
    const int q = k.lane >> 4;
    float b[K::kNBn][4];
#pragma unroll
    for (int i = 0; i < K::kNBn; ++i) {
      const int n = min(n0 + k.wave_n * K::kWN + 16 * i + 4 * q, k.a.N - 4);
      const v2u w = *(const v2u *)(t.bias + (size_t)n * 2);
      unpack2<DT>(w[0], b[i]);
      unpack2<DT>(w[1], b[i] + 2);
    }
#pragma unroll
    for (int j = 0; j < K::kNBm; ++j) {
      const int m = m0 + k.wave_m * K::kWM + j * 16 + (k.lane & 15);
      uint8_t *crow = k.a.C + (size_t)m * k.a.ldc * 2;
#pragma unroll
      for (int i = 0; i < K::kNBn; i += 2) {
        const f32x4 &u = k.acc[i][j], &v = k.acc[i + 1][j];
        const uint32_t us[2] = {pack2<DT>(u[0] + b[i][0], u[1] + b[i][1]), pack2<DT>(u[2] + b[i][2], u[3] + b[i][3])};
        const uint32_t vs[2] = {pack2<DT>(v[0] + b[i + 1][0], v[1] + b[i + 1][1]),
                                pack2<DT>(v[2] + b[i + 1][2], v[3] + b[i + 1][3])};
        uint32_t xo[2], yo[2];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const auto h = __builtin_amdgcn_permlane32_swap(us[d], vs[d], false, false);
          const auto r = __builtin_amdgcn_permlane16_swap(h[0], h[1], false, false);
          xo[d] = r[0];
          yo[d] = r[1];
        }
        const int n = n0 + k.wave_n * K::kWN + i * 16 + 8 * q;
        if (m < k.a.M && n < k.a.N) store_c(crow + (size_t)n * 2, u32x4{xo[0], xo[1], yo[0], yo[1]});
      }
    }
  }
};

// What the epilogue has to do: the rounding alone or a gated activation alone, a
// bias alone, or anything.
enum : int { kBare = 0, kBias = 1, kFull = 2 };
template <int DT, bool GATED, bool GROUPED, int EPI, int AREA>
using MxExt = typename std::conditional<
    EPI == kFull, FfnExt<DT, GATED, GROUPED, AREA>,
    typename std::conditional<EPI == kBias, BiasExt<DT, GROUPED>,
                              typename std::conditional<GATED, GatedExt<DT, GROUPED>, PlainExt>::type>::type>::type;

// One tile with its first row m0 and first column n0, by the kernel of its size.
template <int DT, int TM, int TN, bool TWO, bool ALIGNED, class X>
__device__ __forceinline__ void mx_tile(const Args &a, const X &x) {
  if constexpr (TM == 256) {
    using T = MxTraits<DT == 1>;
    __shared__ __attribute__((aligned(1024))) uint8_t sA0[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sA1[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sB0[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t sB1[256 * kRowBytes];
    __shared__ __attribute__((aligned(1024))) uint8_t st[Kernel<T, 256, 256, false, X>::kStageBytes];
    Slots slots;
    slots.a[0] = (LDS_AS uint8_t *)sA0;
    slots.a[1] = (LDS_AS uint8_t *)sA1;
    slots.b[0] = (LDS_AS uint8_t *)sB0;
    slots.b[1] = (LDS_AS uint8_t *)sB1;
    slots.junk = nullptr;
    slots.stage = (LDS_AS uint8_t *)st;
    Kernel<T, 256, 256, false, X> k(a, slots, x);
    k.run();
  } else {
    using K = MxTile<DT, TM, TN, TWO, ALIGNED, X>;
    TGEMM_MX_SLOTS(TM, TN, K::SL, K::kNS, K::kScaleBytes)
    K k(a, slots, x);
    k.run();
  }
}

template <int DT, int TM, int TN, bool TWO, bool ALIGNED, bool GATED, int EPI>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(TWO ? 2 : 1, TWO ? 2 : 1)))
void mx_epilogue_kernel(const Args a, const Tail t) {
#if defined(__HIP_DEVICE_COMPILE__)
  int tm, tn;
  tile_of((int)blockIdx.x, a.tiles_m * a.tiles_n, a.tiles_m, a.tiles_n, tm, tn);
  constexpr int kArea = (TM < TN ? TM : TN) * kMxSlice<TM, TWO>;
  const MxExt<DT, GATED, false, EPI, kArea> x{tm * TM, tn * (GATED ? TN / 2 : TN), t.half, nullptr, 0, t};
  mx_tile<DT, TM, TN, TWO, ALIGNED>(a, x);
#endif
}

// The K split: workgroup w computes tile w % tiles over its range of slices and
// leaves its sums in plane w / tiles of the workspace.
struct MxSplitExt {
  static constexpr bool kOn = true, kGated = false, kGather = false, kPrefetch = false;
  int m0, n0, split;
  template <class K>
  __device__ __forceinline__ void store(K &k) const {
    float *plane = k.a.ws + (size_t)split * (size_t)k.a.M * (size_t)k.a.N;
#pragma unroll
    for (int j = 0; j < K::kNBm; ++j) {
      const int m = m0 + k.wave_m * K::kWM + j * 16 + (k.lane & 15);
#pragma unroll
      for (int i = 0; i < K::kNBn; ++i) {
        const int n = n0 + k.wave_n * K::kWN + 16 * i + 4 * (k.lane >> 4);
        if (m < k.a.M && n < k.a.N) store_c((uint8_t *)(plane + (size_t)m * k.a.N + n), __builtin_bit_cast(u32x4, k.acc[i][j]));
      }
    }
  }
};

template <bool ALIGNED>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(1, 1)))
void mx_split_kernel(const Args a0) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int tiles = a0.tiles_m * a0.tiles_n, split = (int)blockIdx.x / tiles, t = (int)blockIdx.x - split * tiles;
  const int s0 = split * a0.kq;
  Args a = a0;
  a.A += (size_t)s0 * 256;
  a.B += (size_t)s0 * 256;
  a.SA += (size_t)s0 * 16;
  a.SB += (size_t)s0 * 16;
  a.K = min(a0.K - s0 * 256, a0.kq * 256);
  using K = MxTile<0, 64, 64, false, ALIGNED, MxSplitExt>;
  TGEMM_MX_SLOTS(64, 64, K::SL, K::kNS, K::kScaleBytes)
  K k(a, slots, MxSplitExt{t % a0.tiles_m * 64, t / a0.tiles_m * 64, split});
  k.kbv = a0.kb - s0 * 16;
  k.run();
#endif
}

struct MxGroups {
  const int32_t *offsets;
  const int32_t *rows;  // or nullptr
  int groups, R, src_rows;
  int64_t stride_b, stride_sb, stride_bias;  // bytes, bytes, elements
};

// Unit `order(total)` of all the groups' tiles (none if that is negative).  Up to
// 64 groups are read once for both, one a lane: every workgroup's loads wait for this.
template <class F>
__device__ __forceinline__ Found find_ordered(const MxGroups &g, int size, int times, int lane, F order) {
  if (g.groups > 64) {
    const int at = order(total_units(g.offsets, g.groups, g.R, size, times, lane));
    return at < 0 ? Found{-1, 0, 0, 0, 0} : find_unit(g.offsets, g.groups, g.R, at, size, times, lane);
  }
  const Range r = lane_rows(g.offsets, g.groups, g.R, lane);
  const int n = (r.hi - r.lo + size - 1) / size * times, upto = wave_scan(n);
  const int at = order(__builtin_amdgcn_readlane(upto, 63));
  const uint64_t past = at < 0 ? 0 : __ballot(at < upto);
  if (!past) return {-1, 0, 0, 0, 0};
  const int l = (int)__builtin_ctzll(past), before = __builtin_amdgcn_readlane(upto - n, l);
  // (Only offsets that are no offsets can leave the unit outside the group.)
  if (at < before || l >= g.groups) return {-1, 0, 0, 0, 0};
  return {l, __builtin_amdgcn_readlane(r.lo, l), __builtin_amdgcn_readlane(r.hi, l), at - before, before};
}

template <int DT, int TM, int TN, bool TWO, bool ALIGNED, bool GATED, int EPI>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(TWO ? 2 : 1, TWO ? 2 : 1)))
void mx_grouped_kernel(const Args a0, const Tail t0, const MxGroups g) {
#if defined(__HIP_DEVICE_COMPILE__)
  const int lane = threadIdx.x & 63;
  const int wg = (int)blockIdx.x;
  const Found f = find_ordered(g, TM, a0.tiles_n, lane, [&](int total) { return wg < total ? xcd_order(wg, total) : -1; });
  if (f.e < 0) return;
  int tm, tn;
  tile_in_group(f.unit, (f.hi - f.lo + TM - 1) / TM, a0.tiles_n, tm, tn);
  // The group's own product: its rows, its weight, its bias.
  Args a = a0;
  Tail t = t0;
  a.M = f.hi - f.lo;
  a.B += (size_t)f.e * (size_t)g.stride_b;
  a.SB += (size_t)f.e * (size_t)g.stride_sb;
  a.C += (size_t)f.lo * a.ldc * 2;
  if (!g.rows) {
    a.A += (size_t)f.lo * a.lda;
    a.SA += (size_t)f.lo * a.kb;
  }
  if (t.bias) t.bias += (size_t)f.e * (size_t)g.stride_bias * 2;
  if (t.pre) t.pre += (size_t)f.lo * t.ldp * 2;
  constexpr int kArea = (TM < TN ? TM : TN) * kMxSlice<TM, TWO>;
  const MxExt<DT, GATED, true, EPI, kArea> x{__builtin_amdgcn_readfirstlane(tm * TM),
                                               __builtin_amdgcn_readfirstlane(tn * (GATED ? TN / 2 : TN)), t.half,
                                               g.rows ? g.rows + f.lo : nullptr, g.src_rows, t};
  mx_tile<DT, TM, TN, TWO, ALIGNED>(a, x);
#endif
}

inline Args mx_args(const MxGemm &g) {
  Args a{};
  a.A = static_cast<const uint8_t *>(g.A);
  a.B = static_cast<const uint8_t *>(g.B);
  a.SA = static_cast<const uint8_t *>(g.SA);
  a.SB = static_cast<const uint8_t *>(g.SB);
  a.C = static_cast<uint8_t *>(g.C);
  a.M = (int)g.M;
  a.N = (int)(is_gated(g.act) ? g.N / 2 : g.N);  // output columns
  a.K = (int)(g.K / 2);                          // bytes
  a.lda = (int)g.lda;
  a.ldb = (int)g.ldb;
  a.ldc = (int)g.ldc;
  a.kb = (int)(g.K / 32);
  a.ksteps = (int)(g.K / 256);  // (256-row tiles)
  a.splits = 1;
  return a;
}

inline hipError_t launch_mx_split_tiles(const MxGemm &g) {
  Args a = mx_args(g);
  a.N = (int)g.N;  // the product's columns, gated or not
  a.tiles_m = (int)((g.M + 63) / 64);
  a.tiles_n = (int)((g.N + 63) / 64);
  a.ws = g.ws;
  const int slices = (a.K + 255) / 256;
  a.kq = (slices + g.splits - 1) / g.splits;  // (mx_splits leaves no split empty)
  a.splits = g.splits;
  const int64_t wgs = (int64_t)a.tiles_m * a.tiles_n * a.splits;
  if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
  void *args[] = {&a};
  const void *fn = mx_scales_aligned(g) ? reinterpret_cast<const void *>(&mx_split_kernel<true>)
                                        : reinterpret_cast<const void *>(&mx_split_kernel<false>);
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
}

template <int DT, int TM, int TN, bool TWO, bool ALIGNED, bool GATED>
hipError_t launch_mx_tile(const MxGemm &g) {
  Args a = mx_args(g);
  constexpr int kCols = GATED ? TN / 2 : TN;
  a.tiles_m = (int)((g.M + TM - 1) / TM);
  a.tiles_n = (a.N + kCols - 1) / kCols;
  Tail t{static_cast<const uint8_t *>(g.bias), static_cast<const uint8_t *>(g.residual), static_cast<uint8_t *>(g.preact),
         (int)g.ldr, (int)g.ldp, g.act, GATED ? a.N : 0};
  // (A gated 256 x 256 tile straight from the accumulators would spill.)
  const int epi = g.residual || g.preact || (GATED ? g.bias || TM == 256 : g.act != kNone) ? kFull : g.bias ? kBias : kBare;
  if (g.groups == 0) {
    const int64_t wgs = (int64_t)a.tiles_m * a.tiles_n;
    if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
    void *args[] = {&a, &t};
    const void *fn = reinterpret_cast<const void *>(&mx_epilogue_kernel<DT, TM, TN, TWO, ALIGNED, GATED, kFull>);
    if constexpr (!(GATED && TM == 256))
      if (epi == kBare) fn = reinterpret_cast<const void *>(&mx_epilogue_kernel<DT, TM, TN, TWO, ALIGNED, GATED, kBare>);
    if constexpr (!GATED)
      if (epi == kBias) fn = reinterpret_cast<const void *>(&mx_epilogue_kernel<DT, TM, TN, TWO, ALIGNED, GATED, kBias>);
    return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
  }
  // The most tiles the groups can have: each one's last may be partial.
  const int64_t wgs = (g.M / TM + (g.groups < g.M ? g.groups : g.M)) * (int64_t)a.tiles_n;
  if (!grid_ok(wgs)) return hipErrorInvalidConfiguration;
  MxGroups gr{g.offsets, g.rows, (int)g.groups, (int)g.M, (int)g.src_rows, g.stride_b, g.stride_sb, g.N};
  void *args[] = {&a, &t, &gr};
  const void *fn = reinterpret_cast<const void *>(&mx_grouped_kernel<DT, TM, TN, TWO, ALIGNED, GATED, kFull>);
  if constexpr (!(GATED && TM == 256))
    if (epi == kBare) fn = reinterpret_cast<const void *>(&mx_grouped_kernel<DT, TM, TN, TWO, ALIGNED, GATED, kBare>);
  if constexpr (!GATED)
    if (epi == kBias) fn = reinterpret_cast<const void *>(&mx_grouped_kernel<DT, TM, TN, TWO, ALIGNED, GATED, kBias>);
  return hipLaunchKernel(fn, dim3((unsigned)wgs), dim3(kThreads), args, 0, g.stream);
}

template <int DT, int TM, int TN, bool TWO, bool ALIGNED>
hipError_t launch_mx_gated(const MxGemm &g) {
  return is_gated(g.act) ? launch_mx_tile<DT, TM, TN, TWO, ALIGNED, true>(g)
                         : launch_mx_tile<DT, TM, TN, TWO, ALIGNED, false>(g);
}
template <int DT, int TM, int TN, bool TWO>
hipError_t launch_mx_aligned(const MxGemm &g) {
  return mx_scales_aligned(g) ? launch_mx_gated<DT, TM, TN, TWO, true>(g) : launch_mx_gated<DT, TM, TN, TWO, false>(g);
}

}  // namespace
}  // namespace ffn
}  // namespace tgemm
