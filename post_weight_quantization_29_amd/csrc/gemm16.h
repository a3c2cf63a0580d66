// C = A B^T for 16-bit A [m x K] and B [n x K], both k-contiguous, with a fused
// epilogue: the tile loop of the large products on the packed layer (B is the
// weight dequantized to the workspace; 2 m n K operations dwarf that pass).
//
// A workgroup of WM x WN waves takes 32 MB WM rows of A by 32 NB WN rows of B; a
// wave holds NB x MB accumulators of v_mfma_f32_32x32x16.  Stages of 32 k are
// copied HBM -> LDS by buffer_load ... lds (16 bytes per lane, no staging
// registers) into a ring of kRing slots, kRing - 2 stages ahead.  A stage row
// is 64 bytes; its 16-byte chunk c sits at c ^ ((row / 4) % 4), so the sixteen
// lanes that read sixteen consecutive rows of one chunk hit sixteen different
// 16-byte columns of the 64 banks (the copy applies the swizzle by permuting
// the lanes' source addresses).  The sync point of stage k sits before the last
// k-slice of stage k-1: there every wave has waited for its copies of stage k
// and has finished reading stage k-2, whose slot takes the next copies; the
// last slice's MFMAs overlap the first operand reads of stage k.
//
// What bounds it: the matrix pipe.  The 256 x 256 tile (MB = NB = 4) reads
// 8 KB of operands from LDS per wave and 16 MFMAs, half of what LDS delivers;
// the 128 x 128 tile (MB = NB = 2, two workgroups per CU) reads twice that per
// MFMA and serves products with too few large tiles for 256 CUs.
#pragma once
#include "w4.h"

namespace gptq {

typedef int i32x4g_t __attribute__((ext_vector_type(4)));

struct Gemm16Args {
  const uint16_t* A0;   // stages [0, k0_stages)
  const uint16_t* A1;   // stages after them (a second matrix of A's shape, its k from 0)
  int64_t lda;          // elements, a multiple of 8
  const uint16_t* B;
  int64_t ldb;
  int64_t m;
  int n;                // rows of B that exist
  int k0_stages, n_stages;
  int tiles_m, tiles_n;
};

constexpr int kGk = 32;          // k per stage
constexpr int kRing = 5;         // stage slots
constexpr int kEpPitch = 36;     // floats per token row of the epilogue's LDS tile

GPTQ_DEV void copy16_lds(uint32_t lds_dst, const i32x4g_t& rsrc, int voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds_dst)), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
GPTQ_DEV void copy4_lds(uint32_t lds_dst, const i32x4g_t& rsrc, int voff) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds_dst)), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
template <int N> GPTQ_DEV void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
GPTQ_DEV void ring_barrier() { asm volatile("s_barrier" ::: "memory"); }

// rows past the end carry an offset beyond every buffer range: they read zero
constexpr int kPastEnd = 0x7ffffff0;
constexpr int64_t kMaxRowBytes = 0x7fff0000 / 256;   // a tile's row offsets stay below kPastEnd

GPTQ_DEV i32x4g_t tile_rsrc(uint64_t base, bool live) {
  i32x4g_t r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));
  r[2] = live ? 0x7fffff00 : 0;
  r[3] = 0x00020000;
  return r;
}

// Workgroups are dealt round-robin to the 8 XCDs, each with its own L2: XCD x
// takes the x-th eighth of the tiles, in strips of four tile rows of A, so its
// co-resident workgroups share panels of both operands.
GPTQ_DEV bool tile_of(int wg, int tm, int tn, int& im, int& in) {
  const int T = tm * tn, per = (T + 7) / 8;
  const int idx = (wg & 7) * per + (wg >> 3);
  if ((wg >> 3) >= per || idx >= T) return false;
  const int strip = idx / (4 * tn), rest = idx - strip * 4 * tn;
  const int h = min(4, tm - 4 * strip);
  im = 4 * strip + rest % h;
  in = rest / h;
  return true;
}

template <typename T, int MB, int NB, int WM, int WN, typename Epi>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm16_kernel(Gemm16Args g, Epi epi) {
  typedef typename T16<T>::v8 v8;
  constexpr int W = WM * WN, TM = 32 * MB * WM, TN = 32 * NB * WN;
  constexpr uint32_t kSlot = (TM + TN) * 64;
  constexpr int CA = TM / (16 * W), CB = TN / (16 * W), kCopies = CA + CB;   // copies per wave and stage
  constexpr int kEpWave = 32 * kEpPitch * 4 * Epi::kPlanes;
  constexpr uint32_t kLds = kRing * kSlot;
  static_assert(W * kEpWave <= (int)kLds && TM % (16 * W) == 0 && TN % (16 * W) == 0, "tile");
  __shared__ __attribute__((aligned(1024))) char smem[kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  int im, in;
  if (!tile_of(blockIdx.x, g.tiles_m, g.tiles_n, im, in)) return;
  const int64_t m0 = (int64_t)im * TM;
  const int n0 = in * TN;
  const uint32_t lds = (uint32_t)(uintptr_t)(LDS_AS const char*)smem;

  // copy i of a stage: rows 16 (wave + W i) + lane / 4, chunk lane % 4
  int voffA[CA], voffB[CB];
  {
    const int R = 16 * wave + (lane >> 2);
    const int c = (lane & 3) ^ ((R >> 2) & 3);
#pragma unroll
    for (int i = 0; i < CA; ++i)
      voffA[i] = m0 + R + 16 * W * i < g.m ? (int)((R + 16 * W * i) * g.lda * 2) + 16 * c : kPastEnd;
#pragma unroll
    for (int i = 0; i < CB; ++i)
      voffB[i] = n0 + R + 16 * W * i < g.n ? (int)((R + 16 * W * i) * g.ldb * 2) + 16 * c : kPastEnd;
  }
  const uint64_t a0 = reinterpret_cast<uint64_t>(g.A0 + m0 * g.lda), a1 = reinterpret_cast<uint64_t>(g.A1 + m0 * g.lda);
  const uint64_t b0 = reinterpret_cast<uint64_t>(g.B + (int64_t)n0 * g.ldb);
  const int nk = g.n_stages;
  auto rsrc_of = [&](int k, i32x4g_t& ra, i32x4g_t& rb) {
    const bool live = k < nk;
    ra = tile_rsrc(k < g.k0_stages ? a0 + (uint64_t)k * (kGk * 2) : a1 + (uint64_t)(k - g.k0_stages) * (kGk * 2), live);
    rb = tile_rsrc(b0 + (uint64_t)k * (kGk * 2), live);
  };
  auto copy = [&](const i32x4g_t& ra, const i32x4g_t& rb, int slot, int q) {
    if (q < CA) copy16_lds(lds + slot * kSlot + 1024u * (W * q + wave), ra, voffA[q < CA ? q : 0]);
    else copy16_lds(lds + slot * kSlot + TM * 64 + 1024u * (W * (q - CA) + wave), rb, voffB[q >= CA ? q - CA : 0]);
  };
  // operand reads: row lane % 32 of a 32-row block, k chunk 2 slice + lane / 32
  const uint32_t sw = ((lane & 31) * 64) + (((lane >> 5) ^ ((lane >> 2) & 3)) << 4);
  const uint32_t rdA = lds + wm * (32 * MB * 64) + sw, rdB = lds + TM * 64 + wn * (32 * NB * 64) + sw;
  const uint32_t rdA1 = rdA ^ 32u, rdB1 = rdB ^ 32u;   // slice 1: chunk 2 + lane / 32
  auto rd = [&](uint32_t at) { return *(LDS_AS const v8*)(uintptr_t)at; };

  f32x16_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  constexpr int kInFlight = (kRing - 3) * kCopies;
#pragma unroll
  for (int a = 0; a <= kRing - 3; ++a) {
    i32x4g_t ra, rb;
    rsrc_of(a, ra, rb);
#pragma unroll
    for (int q = 0; q < kCopies; ++q) copy(ra, rb, a, q);
  }
  wait_copies<kInFlight>();
  ring_barrier();
  {
    i32x4g_t ra, rb;
    rsrc_of(kRing - 2, ra, rb);
#pragma unroll
    for (int q = 0; q < kCopies; ++q) copy(ra, rb, kRing - 2, q);
  }
  v8 opA[2][MB], opB[2][NB];
#pragma unroll
  for (int j = 0; j < MB; ++j) opA[0][j] = rd(rdA + 2048u * j);
#pragma unroll
  for (int i = 0; i < NB; ++i) opB[0][i] = rd(rdB + 2048u * i);

  auto stage = [&]<int SLOT>(int k) {
    constexpr int NS = (SLOT + 1) % kRing, DS = (SLOT + kRing - 1) % kRing;
    i32x4g_t ra, rb;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bool last = ks == 1;
      if (last) {
        wait_copies<kInFlight>();
        ring_barrier();
        rsrc_of(k + kRing - 1, ra, rb);
      }
      constexpr int P = MB * NB, F = MB + NB;
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int i = q / MB, j = q % MB;
        acc[i][j] = T16<T>::mfma32(opB[ks][i], opA[ks][j], acc[i][j]);
        // the next slice's operands and (last slice) the copies, spread over the MFMAs
#pragma unroll
        for (int f = q * F / P; f < (q + 1) * F / P; ++f) {
          if (!last) {
            if (f < MB) opA[1][f < MB ? f : 0] = rd(rdA1 + SLOT * kSlot + 2048u * f);
            else opB[1][f >= MB ? f - MB : 0] = rd(rdB1 + SLOT * kSlot + 2048u * (f - MB));
          } else {
            if (f < MB) opA[0][f < MB ? f : 0] = rd(rdA + NS * kSlot + 2048u * f);
            else opB[0][f >= MB ? f - MB : 0] = rd(rdB + NS * kSlot + 2048u * (f - MB));
          }
        }
        if (last) {
#pragma unroll
          for (int f = q * kCopies / P; f < (q + 1) * kCopies / P; ++f) copy(ra, rb, DS, f);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  static_assert(kRing == 5, "stages run in groups of five");
  int k = 0;
  for (; k + 5 <= nk; k += 5) {
    stage.template operator()<0>(k);
    stage.template operator()<1>(k + 1);
    stage.template operator()<2>(k + 2);
    stage.template operator()<3>(k + 3);
    stage.template operator()<4>(k + 4);
  }
  if (k < nk) stage.template operator()<0>(k++);
  if (k < nk) stage.template operator()<1>(k++);
  if (k < nk) stage.template operator()<2>(k++);
  if (k < nk) stage.template operator()<3>(k++);

  // the copies issued past the end (they write zeros) land before the ring is reused
  wait_copies<0>();
  __syncthreads();

  // Epilogue: blocks of 32 tokens x 32 values (x kPlanes) go through the wave's
  // own part of LDS, so that a lane finishes eight neighbouring values of one
  // token and stores 16 bytes.
  float* ep = reinterpret_cast<float*>(smem) + wave * (kEpWave / 4);
  constexpr int PL = Epi::kPlanes;
  const int64_t mw = m0 + wm * 32 * MB;
#pragma unroll
  for (int ib = 0; ib < NB; ib += PL)
#pragma unroll
    for (int j = 0; j < MB; ++j) {
#pragma unroll
      for (int p = 0; p < PL; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[ib + p][j][4 * q + e];
          *reinterpret_cast<f32x4_t*>(ep + (32 * p + (lane & 31)) * kEpPitch + 8 * q + 4 * (lane >> 5)) = v;
        }
      __builtin_amdgcn_wave_barrier();
      const int nb = (n0 + wn * 32 * NB + 32 * ib) / PL;   // first output column of the block
#pragma unroll 1
      for (int t = 0; t < 2; ++t) {
        const int tok = 16 * t + (lane >> 2), c = 8 * (lane & 3);
        if (mw + 32 * j + tok < g.m) {
          float v[PL][8];
#pragma unroll
          for (int p = 0; p < PL; ++p) {
            const f32x4_t lo = *reinterpret_cast<const f32x4_t*>(ep + (32 * p + tok) * kEpPitch + c);
            const f32x4_t hi = *reinterpret_cast<const f32x4_t*>(ep + (32 * p + tok) * kEpPitch + c + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              v[p][e] = lo[e];
              v[p][4 + e] = hi[e];
            }
          }
          epi.template finish<8>(v, mw + 32 * j + tok, nb + c);
        }
      }
      __builtin_amdgcn_wave_barrier();
    }
}

}  // namespace gptq
