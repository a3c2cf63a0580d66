// C = A B^T for 16-bit A [m x K] and B [n x K], both k-contiguous, with a fused
// epilogue: the tile loop of the large products on the packed layer (B is the
// weight dequantized to the workspace; 2 m n K operations dwarf that pass).
//
// A workgroup of WM x WN waves takes 32 MB WM rows of A by 32 NB WN rows of B; a
// wave holds NB x MB accumulators of v_mfma_f32_32x32x16.  Stages of 32 k are
// copied HBM -> LDS by buffer_load ... lds (16 bytes per lane, no staging
// registers) into a ring of five slots.  Two stages share each 128-byte cache
// line of A and B, so they are copied as a pair, the second half of a line
// right behind the first: copied a stage at a time, each line came through the
// CU's L1 twice, and that path was busier than the matrix pipe.  Pair (k+4,
// k+5) is issued when stage k (even) has been read, into its slot and the spare
// one, three stages before it is needed.  Measured with no tile split (8192 x
// 13824 x 5120, 4096 x 4096 x 22016, 4096 x 22016 x 4096): 1.11, 1.18, 1.26
// PFLOP/s, a stage at a time 1.04, 1.08, 1.18; stages of 64 k in two slots the
// same within 2 %.  The matrix pipe is busy in 59-60 % of the cycles (at the 1.87
// GHz that the chip's power leaves it) and the waves wait for a third of their
// time: the two waves of a SIMD meet the same barriers.
// A stage row is 64 bytes; its 16-byte chunk c sits at c ^ ((row / 4) % 4), so
// the sixteen lanes that read sixteen consecutive rows of one chunk hit sixteen
// different 16-byte columns of the 64 banks (the copy applies the swizzle by
// permuting the lanes' source addresses).  The sync point of a stage sits before
// the last 16-k slice of the stage before it, whose MFMAs overlap the copies
// and the next stage's first operand reads.
//
// The 256 x 256 tile (eight waves, two a SIMD) reads 6 KB of operands from LDS
// per wave and 8 MFMAs; the 128 x 128 tile (four waves, two workgroups per CU)
// serves products with too few large tiles for 256 CUs.  Tiles past the last full
// round may be split over k: their sums go to the workspace as they lie in
// registers, and gemm16_join_kernel adds them in order and finishes them.
#pragma once
#include "w4.h"

namespace gptq {

struct Gemm16Args {
  const uint16_t* A0;   // pairs of stages [0, k0_pairs)
  const uint16_t* A1;   // pairs after them (a second matrix of A's shape, its k from 0)
  int64_t lda;          // elements, a multiple of 8
  const uint16_t* B;
  int64_t ldb;
  int64_t m;
  int n;                // rows of B that exist
  int k0_pairs, n_pairs;
  int tiles_m, tiles_n;
  int whole;            // tiles that one workgroup takes whole; the others' k is split
  int slices, slice_pairs;
  float* part;          // [slice][split tile][wave][block][4][lane] of four sums
};

constexpr int kGk = 64;          // k per pair of stages
constexpr int kSlots = 5;        // stage slots
constexpr int kEpPitch = 36;     // floats per token row of the epilogue's LDS tile

template <int N> GPTQ_DEV void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
// before a slot is given back: the wave's own LDS reads of it are done
GPTQ_DEV void wait_lds_reads() { __builtin_amdgcn_s_waitcnt(0xC07F); }
GPTQ_DEV void ring_barrier() { asm volatile("s_barrier" ::: "memory"); }

// rows past the end carry an offset beyond every buffer range: they read zero
constexpr int kPastEnd = 0x7ffffff0;
constexpr int64_t kMaxRowBytes = 0x7fff0000 / 256;   // a tile's row offsets stay below kPastEnd

GPTQ_DEV i32x4_t tile_rsrc(uint64_t base, bool live) {
  i32x4_t r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)base);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(base >> 32));
  r[2] = live ? 0x7fffff00 : 0;
  r[3] = 0x00020000;
  return r;
}

// Workgroups are dealt round-robin to the 8 XCDs, each with its own L2: XCD x
// takes the x-th eighth of the items, so its co-resident workgroups share panels
// of both operands.  Tiles are counted in strips of four tile rows of A.
GPTQ_DEV int item_of(int wg, int n) {
  const int per = (n + 7) / 8, i = (wg & 7) * per + (wg >> 3);
  return (wg >> 3) < per && i < n ? i : -1;
}
GPTQ_DEV void tile_of(int idx, int tm, int tn, int& im, int& in) {
  const int strip = idx / (4 * tn), rest = idx - strip * 4 * tn;
  const int h = min(4, tm - 4 * strip);
  im = 4 * strip + rest % h;
  in = rest / h;
}

// 32 tokens x 32 values (x kPlanes) go through the wave's own part of LDS, so
// that a lane finishes eight neighbouring values of one token and stores 16
// bytes.  Token tok0 + lane % 32 has values 8 q + 4 (lane / 32) + e in x[p][4 q + e].
template <typename Epi>
GPTQ_DEV void finish_block(const Epi& epi, float* ep, const f32x16_t (&x)[Epi::kPlanes], int64_t tok0, int64_t m, int col) {
  constexpr int PL = Epi::kPlanes;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int p = 0; p < PL; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f32x4_t v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = x[p][4 * q + e];
      *reinterpret_cast<f32x4_t*>(ep + (32 * p + (lane & 31)) * kEpPitch + 8 * q + 4 * (lane >> 5)) = v;
    }
  __builtin_amdgcn_wave_barrier();
#pragma unroll 1
  for (int t = 0; t < 2; ++t) {
    const int tok = 16 * t + (lane >> 2), c = 8 * (lane & 3);
    if (tok0 + tok < m) {
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
      epi.template finish<8>(v, tok0 + tok, col + c);
    }
  }
  __builtin_amdgcn_wave_barrier();
}

template <typename T, int MB, int NB, int WM, int WN, typename Epi>
__global__ __launch_bounds__(64 * WM * WN, 2) void gemm16_kernel(Gemm16Args g, Epi epi) {
  typedef typename T16<T>::v8 v8;
  constexpr int W = WM * WN, TM = 32 * MB * WM, TN = 32 * NB * WN;
  constexpr uint32_t kRow = kGk, kSlot = (TM + TN) * kRow;       // bytes of a stage row, of a stage
  constexpr int CA = TM / (16 * W), CB = TN / (16 * W), kCopies = 2 * (CA + CB);   // copies per wave and pair
  constexpr int kEpWave = 32 * kEpPitch * 4 * Epi::kPlanes;
  constexpr uint32_t kLds = kSlots * kSlot;
  static_assert(W * kEpWave <= (int)kLds && TM % (16 * W) == 0 && TN % (16 * W) == 0, "tile");
  __shared__ __attribute__((aligned(1024))) char smem[kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // whole tiles first, then slice by slice the split ones
  const int n_whole = (g.whole + 7) / 8 * 8, n_split = g.tiles_m * g.tiles_n - g.whole;
  const bool split = (int)blockIdx.x >= n_whole;
  const int item = split ? item_of(blockIdx.x - n_whole, n_split * g.slices) : item_of(blockIdx.x, g.whole);
  if (item < 0) return;
  const int slice = split ? item / n_split : 0;
  int im, in;
  tile_of(split ? g.whole + item - slice * n_split : item, g.tiles_m, g.tiles_n, im, in);
  const int p0 = slice * g.slice_pairs, np = split ? min(p0 + g.slice_pairs, g.n_pairs) : g.n_pairs;
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
  // descriptors of a pair's first and second stages (an instruction offset
  // would move the LDS address as well)
  struct Pair {
    i32x4_t a[2], b[2];
  };
  auto rsrc_of = [&](int p) {
    const bool live = p < np;
    const uint64_t pa = p < g.k0_pairs ? a0 + (uint64_t)p * (kGk * 2) : a1 + (uint64_t)(p - g.k0_pairs) * (kGk * 2);
    const uint64_t pb = b0 + (uint64_t)p * (kGk * 2);
    return Pair{{tile_rsrc(pa, live), tile_rsrc(pa + 64, live)}, {tile_rsrc(pb, live), tile_rsrc(pb + 64, live)}};
  };
  // copy y of a pair, both halves of its lines, into slots s0, s1
  auto copy = [&](const Pair& r, int s0, int s1, int y) {
    const uint32_t at = lds + 1024u * wave + (y < CA ? 1024u * W * y : TM * kRow + 1024u * W * (y - CA));
    if (y < CA) copy16_lds_two(at + s0 * kSlot, r.a[0], at + s1 * kSlot, r.a[1], voffA[y < CA ? y : 0]);
    else copy16_lds_two(at + s0 * kSlot, r.b[0], at + s1 * kSlot, r.b[1], voffB[y >= CA ? y - CA : 0]);
  };
  // operand reads: row lane % 32 of a 32-row block, k chunk 2 slice + lane / 32
  const uint32_t sw = (lane & 31) * kRow + (((lane >> 5) ^ ((lane >> 2) & 3)) << 4);
  const uint32_t rdA = lds + wm * (32 * MB * kRow) + sw, rdB = lds + TM * kRow + wn * (32 * NB * kRow) + sw;
  auto rd = [&](uint32_t at) { return *(LDS_AS const v8*)(uintptr_t)at; };

  // Of the two workgroups that share a CU (workgroups 256 apart, as they are
  // dealt) one goes first at every pipe: the other's waits fall into its
  // products.  Measured, 577 x 5120 x 13824: 166 us the whole call without, 160.
  if constexpr (W == 4) {
    if ((blockIdx.x >> 8) & 1) __builtin_amdgcn_s_setprio(1);
  }
  f32x16_t acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  auto copy_pair = [&](int p, int s0, int s1) {
    const Pair r = rsrc_of(p);
#pragma unroll
    for (int y = 0; y < CA + CB; ++y) copy(r, s0, s1, y);
  };
  copy_pair(p0, 0, 1);
  copy_pair(p0 + 1, 2, 3);
  wait_copies<kCopies>();
  ring_barrier();
  v8 opA[2][MB], opB[2][NB];
#pragma unroll
  for (int j = 0; j < MB; ++j) opA[0][j] = rd(rdA + 32 * kRow * j);
#pragma unroll
  for (int i = 0; i < NB; ++i) opB[0][i] = rd(rdB + 32 * kRow * i);

  // Stage S of ten (the ring's period and the pairs'), in pair p
  auto stage = [&]<int S>(int p) {
    constexpr int SLOT = S % kSlots, NS = (S + 1) % kSlots, SPARE = (S + 4) % kSlots;
    constexpr bool even = S % 2 == 0;
    Pair r;
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      const bool last = ks == 1;
      if (last) {
        if constexpr (even) {
          // stage S's slot and the spare one are free once every wave has its last operands
          wait_lds_reads();
          ring_barrier();
          r = rsrc_of(p + 2);
        } else {
          wait_copies<kCopies>();            // the next pair has landed
          ring_barrier();
        }
      }
      constexpr int P = MB * NB, F = MB + NB;
#pragma unroll
      for (int q = 0; q < P; ++q) {
        const int i = q / MB, j = q % MB;
        acc[i][j] = T16<T>::mfma32(opB[ks][i], opA[ks][j], acc[i][j]);
        // The next slice's operands, one (or two) per MFMA from the first on, in
        // the order in which its MFMAs want them: B's first block, A's blocks,
        // B's others.
#pragma unroll
        for (int f = q * F / (P < F ? P : F); f < (q + 1) * F / (P < F ? P : F) && f < F; ++f) {
          const bool isA = f >= 1 && f <= MB;
          const int x = f == 0 ? 0 : isA ? f - 1 : f - MB;
          // slice 1 is chunk 2 + lane / 32: bit 5 flips
          const uint32_t at = ((isA ? rdA : rdB) ^ (last ? 0u : 32u)) + (last ? NS : SLOT) * kSlot + 32 * kRow * x;
          if (isA) opA[ks ^ 1][isA ? x : 0] = rd(at);
          else opB[ks ^ 1][isA ? 0 : x] = rd(at);
        }
        if (last && even) {
#pragma unroll
          for (int f = q * kCopies / P; f < (q + 1) * kCopies / P; ++f)
            if (f % 2 == 0) copy(r, SPARE, SLOT, f / 2);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  auto pair = [&]<int S>(int p) {
    stage.template operator()<S>(p);
    stage.template operator()<S + 1>(p);
  };
  static_assert(kSlots == 5, "ten stages to a turn");
  int p = p0;
  for (; p + 5 <= np; p += 5) {
    pair.template operator()<0>(p);
    pair.template operator()<2>(p + 1);
    pair.template operator()<4>(p + 2);
    pair.template operator()<6>(p + 3);
    pair.template operator()<8>(p + 4);
  }
  if (p < np) pair.template operator()<0>(p++);
  if (p < np) pair.template operator()<2>(p++);
  if (p < np) pair.template operator()<4>(p++);
  if (p < np) pair.template operator()<6>(p++);

  // the copies issued past the end (they write zeros) land before the ring is reused
  wait_copies<0>();
  __syncthreads();

  if (split) {
    f32x4_t* to = reinterpret_cast<f32x4_t*>(g.part) + ((int64_t)item * W + wave) * (NB * MB * 4 * 64) + lane;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * q + e];
          to[((i * MB + j) * 4 + q) * 64] = v;
        }
    return;
  }
  float* ep = reinterpret_cast<float*>(smem) + wave * (kEpWave / 4);
  constexpr int PL = Epi::kPlanes;
#pragma unroll
  for (int ib = 0; ib < NB; ib += PL)
#pragma unroll
    for (int j = 0; j < MB; ++j) {
      f32x16_t x[PL];
#pragma unroll
      for (int p = 0; p < PL; ++p) x[p] = acc[ib + p][j];
      finish_block(epi, ep, x, m0 + wm * 32 * MB + 32 * j, g.m, (n0 + wn * 32 * NB + 32 * ib) / PL);
    }
}

// The split tiles: their slices' sums in order, and the epilogue, 32 tokens x 32
// values (x kPlanes) per wave.
template <int MB, int NB, int WM, int WN, typename Epi>
__global__ __launch_bounds__(256) void gemm16_join_kernel(Gemm16Args g, Epi epi) {
  constexpr int PL = Epi::kPlanes, W = WM * WN, BLOCKS = NB * MB / PL;   // blocks of a wave's accumulators
  __shared__ __attribute__((aligned(16))) float smem[4 * 32 * kEpPitch * PL];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n_split = g.tiles_m * g.tiles_n - g.whole;
  const int64_t id = (int64_t)blockIdx.x * 4 + wave;
  const int b = (int)(id % BLOCKS), w = (int)(id / BLOCKS % W), tile = (int)(id / (BLOCKS * W));
  if (tile >= n_split) return;
  const int ib = b / MB * PL, j = b % MB;
  f32x16_t x[PL];
#pragma unroll
  for (int p = 0; p < PL; ++p)
#pragma unroll
    for (int e = 0; e < 16; ++e) x[p][e] = 0.0f;
#pragma unroll 2
  for (int s = 0; s < g.slices; ++s) {
    const f32x4_t* from = reinterpret_cast<const f32x4_t*>(g.part) + (((int64_t)s * n_split + tile) * W + w) * (NB * MB * 4 * 64) + lane;
#pragma unroll
    for (int p = 0; p < PL; ++p)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t v = from[(((ib + p) * MB + j) * 4 + q) * 64];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[p][4 * q + e] += v[e];
      }
  }
  int im, in;
  tile_of(g.whole + tile, g.tiles_m, g.tiles_n, im, in);
  finish_block(epi, smem + wave * (32 * kEpPitch * PL), x, (int64_t)im * (32 * MB * WM) + (w / WN) * 32 * MB + 32 * j, g.m,
               (in * (32 * NB * WN) + (w % WN) * 32 * NB + 32 * ib) / PL);
}

}  // namespace gptq
