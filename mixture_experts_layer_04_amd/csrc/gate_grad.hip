// moe_gate_grad: the router's gradient from the logits to the hidden states
// and the gate,
//
//   dx[t, h]     = sum_e d_logits[t, e] gate[e, h] (+ dx_in[t, h])
//   d_gate[e, h] = sum_t d_logits[t, e] x[t, h]
//
// on the matrix cores.  The fp32 operands are split into bf16 planes that add
// up to them (hi: the value rounded, mid: the remainder rounded, lo: the
// rest), every product of two planes is exact in fp32 and
// v_mfma_f32_16x16x32_bf16 accumulates in fp32:
//  * d_gate takes all three planes of d_logits against the bf16 x: the sums
//    are fp32 sums of exact products.
//  * dx is rounded to bf16 (a half step of 2^-8), so it takes two planes of
//    d_logits and of an fp32 gate, without the product of the two mid planes.
//    Left out are mid mid and the two lo parts, each below 2^-16 of the
//    product: under 2^-14 together.  A bf16 gate is its own hi plane.
//
// Bound by the matrix cores: three MFMA products for each fp32 one (two with
// a bf16 gate).  At 8192 tokens, 7168 columns and 256 experts each of the two
// products runs in 67 us (kernel alone), 1.35 PFLOP/s of bf16, the rate that
// a large library product sustains on the card (1.38); the planes take 11 us
// and the addition of d_gate's 4 splits 7.
//
// A first launch writes the planes in the order the MFMA operands read them:
// fragments of 16 rows x 32 K values, 1 KiB each, lane l of a wave holding
// row l % 16, K values 8 (l / 16) .. + 7 at byte 16 l.  A fragment is then
// one contiguous copy into LDS and one conflict-free 16-byte read per lane.

#include <type_traits>
#include <utility>

#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kFrag = 512;  // bf16 values of a fragment (1 KiB)
constexpr int kMaxMf = 4;   // 16-expert fragments per wave of the d_gate kernel

typedef __amdgpu_buffer_rsrc_t rsrc_t;
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

// Buffer range at `base`: loads at or past its end give zero, stores there
// are dropped, and either way the instruction is issued (the waits below
// count instructions).
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(hi << 32 | lo), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
// The same range as the four words of a descriptor, in scalar registers.
__device__ __forceinline__ i32x4_t make_desc(const void* base, uint32_t bytes) {
  const uint64_t b = (uint64_t)base;
  return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
                 __builtin_amdgcn_readfirstlane((int)((uint32_t)(b >> 32) & 0xFFFFu)),
                 __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000};
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
// Copy of 16 bytes per lane from byte voff + soff of the range to LDS address
// dst + 16 lane (copy_frag: 64 lanes x 16 contiguous bytes).  Written as
// assembly (it has no result register) because the compiler puts a wait for
// every copy that it knows of ahead of LDS reads it cannot tell from the
// copy's target, which here would be a wait for the whole pipeline in each
// step; the waits below are the ones that are needed.  s_mov and s_nop 4 give
// the wait states that the compiler does not see the need of: one between a
// write of m0 and its use, five between a vector instruction (readfirstlane)
// that writes a scalar register and a memory instruction that reads it.
__device__ __forceinline__ void copy16(const i32x4_t& r, uint32_t voff, uint32_t soff, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(
                   __builtin_amdgcn_readfirstlane(dst)),
               "v"(voff), "s"(r), "s"(__builtin_amdgcn_readfirstlane(soff))
               : "memory", "m0");
}
__device__ __forceinline__ void copy_frag(const i32x4_t& r, uint32_t soff, uint32_t dst, int lane) {
  copy16(r, lane * 16, soff, dst);
}
template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N < 63 ? N : 63) : "memory");
}
// Memory operations stay on their side of it.
__device__ __forceinline__ void keep_order() { asm volatile("" ::: "memory"); }
// Barrier that waits for this wave's LDS operations but leaves its vector
// memory operations in flight; what others need of those, the wave has
// waited for before it.
__device__ __forceinline__ void step_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// v = hi + mid + lo, each a bf16 (its 16 bits): hi is v rounded to nearest,
// mid what remains rounded again, and the rest fits a bf16 (24 bits of v, 8 a
// plane, and the signs).  A value that is not finite is its own hi plane; one
// that rounds to infinity keeps its upper bits.
__device__ __forceinline__ void split3(float v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t u = __float_as_uint(v);
  hi = cvt_bf16x2(v, 0.f) & 0xFFFFu;
  const bool special = (hi & 0x7F80u) == 0x7F80u;
  const bool finite = (u & 0x7F800000u) != 0x7F800000u;
  if (special && finite) hi = u >> 16;
  const float r = v - __uint_as_float(hi << 16);
  mid = cvt_bf16x2(r, 0.f) & 0xFFFFu;
  lo = cvt_bf16x2(r - __uint_as_float(mid << 16), 0.f) & 0xFFFFu;
  if (!finite) mid = lo = 0u;
}

struct GateGradP {
  const uint16_t* x;
  const void* gate;
  const float* dl;
  const uint16_t* dx_in;
  uint16_t* dx;
  float* d_gate;
  int T, H, E, gate_fp32;
  int Kf;       // K fragments of dx: E / 32 rounded up (to one of the kernel's counts)
  int mt;       // 16-token fragments per wave of dx: 2, 1, or 0 for the kernel of many experts
  int hsplits, hper;  // column splits of dx, 64-column blocks of each
  int tiles_t;  // 128-token tiles
  int nt32;     // K steps of d_gate: T / 32 rounded up
  int Ef;       // 16-expert fragments of d_gate, all M tiles
  int mtiles, mf;  // M tiles of d_gate, of 2 mf fragments each
  int splits, steps;  // K splits of d_gate, steps of each
  uint16_t* dxa;  // [tiles_t][Kf][2][8][kFrag]   d_logits, rows t
  uint16_t* dxb;  // [H / 64][Kf][1 or 2][4][kFrag]  gate, rows h
  uint16_t* dga;  // [nt32][3][Ef][kFrag]  d_logits, rows e
  float* part;    // [splits][E][H]
};

// 8 values from column c of a row of n, zeros past its end
__device__ __forceinline__ void load8(const float* row, int c, int n, float (&f)[8]) {
  if (c + 8 <= n) {
    f32x4_t a, b;
    __builtin_memcpy(&a, row + c, 16);
    __builtin_memcpy(&b, row + c + 4, 16);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = a[i];
      f[i + 4] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < n ? row[c + i] : 0.f;
  }
}
// 8 values' planes, one 16-byte piece each, `plane` values apart
template <int N>
__device__ __forceinline__ void store_planes(const float (&f)[8], uint16_t* at, size_t plane) {
  uint32_t v[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split3(f[i], v[0][i], v[1][i], v[2][i]);
#pragma unroll
  for (int q = 0; q < N; ++q)
    *reinterpret_cast<u32x4_t*>(at + q * plane) = u32x4_t{v[q][0] | (v[q][1] << 16), v[q][2] | (v[q][3] << 16),
                                                          v[q][4] | (v[q][5] << 16), v[q][6] | (v[q][7] << 16)};
}

// The planes of both products in one launch, a tile of 32 x 64 values
// through LDS per workgroup: the first `logit_tiles` workgroups take d_logits
// (32 tokens x 64 experts: rows t for dx as they are, rows e for d_gate
// across), the others the gate (32 experts x 64 columns, across).
__global__ __launch_bounds__(256) void split_kernel(GateGradP p, int logit_tiles, int e_tiles) {
  __shared__ float tile[32][65];
  const int r = threadIdx.x / 8, c8 = (threadIdx.x % 8) * 8;    // loads: row, 8 columns
  const int c = threadIdx.x % 64, g8 = (threadIdx.x / 64) * 8;  // across: column, 8 rows
  float f[8];
  if ((int)blockIdx.x < logit_tiles) {
    const int bt = blockIdx.x / e_tiles, t = bt * 32 + r, e0 = (blockIdx.x % e_tiles) * 64;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
    if (t < p.T) load8(p.dl + (size_t)t * p.E, e0 + c8, p.E, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[r][c8 + i] = f[i];
    const int e = e0 + c8;
    if (p.dxa && e / 32 < p.Kf)  // t < 128 tiles_t by the grid
      store_planes<2>(f,
                      p.dxa + (((size_t)(t / 128) * p.Kf + e / 32) * 2 * 8 + (t % 128) / 16) * kFrag +
                          (t % 16 + 16 * ((e % 32) / 8)) * 8,
                      8 * kFrag);
    __syncthreads();
    if (p.dga && (e0 + c) / 16 < p.Ef && bt < p.nt32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = tile[g8 + i][c];
      store_planes<3>(f, p.dga + ((size_t)bt * 3 * p.Ef + (e0 + c) / 16) * kFrag + (c % 16 + 16 * (g8 / 8)) * 8,
                      (size_t)p.Ef * kFrag);
    }
  } else {
    const int b = blockIdx.x - logit_tiles, be = b % p.Kf, e = be * 32 + r, h = b / p.Kf * 64 + c8;
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
    if (e < p.E) {
      if (p.gate_fp32) {
        load8(static_cast<const float*>(p.gate) + (size_t)e * p.H, h, p.H, f);
      } else {
        const u32x4_t u = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p.gate) + (size_t)e * p.H + h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f[2 * i] = bf16_lo(u[i]);
          f[2 * i + 1] = bf16_hi(u[i]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) tile[r][c8 + i] = f[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = tile[g8 + i][c];
    const int planes = p.gate_fp32 ? 2 : 1;
    uint16_t* at =
        p.dxb + ((size_t)(b / p.Kf) * p.Kf + be) * planes * 4 * kFrag + (c / 16) * kFrag + (c % 16 + 16 * (g8 / 8)) * 8;
    if (planes == 2)
      store_planes<2>(f, at, 4 * kFrag);
    else
      store_planes<1>(f, at, 0);
  }
}

__device__ __forceinline__ bf16x8_t frag(const uint16_t* lds, int lane) {
  return *reinterpret_cast<const bf16x8_t*>(lds + lane * 8);
}

// A division's result is in a vector register, also a uniform one's.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

// Item of a grid of 8 ceil(items / 8) workgroups such that each XCD
// (workgroups are dealt to the XCDs in turn) has a contiguous run of them;
// -1: none.
__device__ __forceinline__ int xcd_item(int items) {
  const int per = (items + 7) / 8, item = (blockIdx.x % 8) * per + blockIdx.x / 8;
  return (int)blockIdx.x / 8 < per && item < items ? item : -1;
}

// dx up to 512 experts: a wave keeps both planes of its 16 MT tokens in
// registers (all KF steps of them) and the workgroup, 8 waves of different
// tokens, streams the gate's planes through an LDS ring: per 64 columns, KF
// steps of 4 GP fragments, SK of them a stage, in memory order, asked for
// D - 1 stages ahead.
// The gate is the MFMA's row operand, so a lane holds 4 consecutive columns
// of a token.
//
// A wave's vector memory operations complete in issue order, so a wave that
// waits for the ring waits for everything it issued before: waves 0-3 copy
// the ring (from the L2) and do nothing else, waves 4-7 move the rows of
// dx_in and dx (HBM).  dx_in comes into LDS one block of 64 columns ahead;
// the sums, rounded, replace it there; the waves that brought it store them
// as whole 128-byte rows during the next block.  The 16-byte pieces of row r
// are XORed with r % 8, so that the 16 rows which an access touches lie in
// different banks.
// Items in (token group, column range) order per XCD: its L2 serves a token
// group's planes to all column ranges, and a gate stage to the few token
// groups that run beside each other.
template <int KF, int MT, int GP, bool ADD>
__global__ __launch_bounds__(512, 2) void dx_kernel(GateGradP p) {
  // K steps per ring stage and barrier (level with one at 8 KF, 8192 x 7168 x
  // 256: 80 / 78 us with 1 / 2, planes included)
  constexpr int SK = KF % 2 == 0 ? 2 : KF % 3 == 0 ? 3 : 1;
  constexpr int D = SK == 1 ? 8 : SK == 2 ? 4 : 3, SF = 4 * GP * SK, ROWS = 8 * MT * 16;
  constexpr int RC = ROWS / 4 / 8;  // 1 KiB copies (8 rows) of a row-moving wave and block
  __shared__ __align__(16) uint16_t ring[D][SF * kFrag];
  __shared__ __align__(16) uint16_t rowbuf[2][ROWS * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int item = xcd_item((p.T + ROWS - 1) / ROWS * p.hsplits);
  if (item < 0) return;
  const int tg = uniform(item / p.hsplits), hs = item - tg * p.hsplits;
  const int hb0 = hs * p.hper, hb1 = min(p.H / 64, hb0 + p.hper);
  const int total = (hb1 - hb0) * (KF / SK);  // stages, >= 1
  const i32x4_t gb = make_desc(p.dxb + (size_t)hb0 * KF * 4 * GP * kFrag, (uint32_t)total * SF * kFrag * 2);
  auto copy = [&](int s) {  // past the end: the last stage again, into a slot nobody reads
    if (wave < 4) {
#pragma unroll
      for (int i = 0; i < GP * SK; ++i)
        copy_frag(gb, (uint32_t)((min(s, total - 1) * SF + wave * GP * SK + i) * kFrag * 2),
                  lds_addr(ring[s % D] + (wave * GP * SK + i) * kFrag), lane);
    }
  };
  // the rows that waves 4-7 move: 8 per copy, lane l the 16-byte piece l % 8
  // (XORed) of row l / 8
  const int t0 = tg * ROWS, r0 = (wave & 3) * (ROWS / 4);
  const uint32_t bytes = (uint32_t)min(p.T - t0, ROWS) * p.H * 2;  // of the rows below T
  const size_t origin = (size_t)t0 * p.H;
  const i32x4_t in = make_desc(ADD ? p.dx_in + origin : nullptr, bytes);
  const rsrc_t out = make_rsrc(p.dx + origin, bytes);
  uint32_t row_at[RC];
#pragma unroll
  for (int c = 0; c < RC; ++c)
    row_at[c] = (r0 + c * 8 + lane / 8) * (uint32_t)p.H * 2 + ((lane % 8) ^ (lane / 8)) * 16;
  auto copy_rows = [&](int hb) {  // past the end: the last block again
    if (ADD && wave >= 4) {
#pragma unroll
      for (int c = 0; c < RC; ++c)
        copy16(in, row_at[c], (uint32_t)min(hb, hb1 - 1) * 128, lds_addr(rowbuf[hb & 1] + (r0 + c * 8) * 64));
    }
  };
  auto store_rows = [&](int hb) {
    if (wave >= 4) {
#pragma unroll
      for (int c = 0; c < RC; ++c) {
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(rowbuf[hb & 1] + (r0 + c * 8) * 64 + lane * 8);
        __builtin_amdgcn_raw_buffer_store_b128(v, out, row_at[c], (uint32_t)hb * 128, 0);
      }
    }
  };
  copy_rows(hb0);
#pragma unroll
  for (int s = 0; s < D - 1; ++s) copy(s);
  bf16x8_t th[MT][KF], tm[MT][KF];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int tf = min((tg * 8 + wave) * MT + m, p.tiles_t * 8 - 1);
    const uint16_t* at = p.dxa + ((size_t)(tf / 8) * KF * 16 + tf % 8) * kFrag + lane * 8;
#pragma unroll
    for (int k = 0; k < KF; ++k) {
      th[m][k] = *reinterpret_cast<const bf16x8_t*>(at + (size_t)k * 16 * kFrag);
      tm[m][k] = *reinterpret_cast<const bf16x8_t*>(at + (size_t)(k * 16 + 8) * kFrag);
    }
  }
  int done = 0;  // stages
  for (int hb = hb0; hb < hb1; ++hb) {
    f32x4_t acc[4][MT];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    auto step = [&](auto tag) {
      constexpr int k = decltype(tag)::value;
      // waves 0-3: the stage has landed when only the D - 2 behind it are in
      // flight.  Waves 4-7, ahead of the block's last barrier: this block's
      // dx_in has when only the stores and dx_in copies of this block's
      // first step are (with one step a block, those come after the wait).
      if (wave < 4)
        wait_vm<(D - 2) * GP * SK>();
      else if (ADD && k == KF / SK - 1)
        hb == hb0 ? wait_vm<KF == SK ? 0 : RC>() : wait_vm<KF == SK ? 0 : 2 * RC>();
      step_barrier();  // all of that is there for every wave; the step before is read
      copy(done + D - 1);
      if (k == 0) {
        if (hb > hb0) store_rows(hb - 1);
        // their reads of that buffer are done before dx_in comes into it
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy_rows(hb + 1);
      }
#pragma unroll
      for (int kk = 0; kk < SK; ++kk) {
        const uint16_t* B = ring[done % D] + kk * 4 * GP * kFrag;
        const int q = k * SK + kk;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8_t gh = frag(B + i * kFrag, lane);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            acc[i][m] = mfma_16x16x32_bf16(gh, th[m][q], acc[i][m]);
            acc[i][m] = mfma_16x16x32_bf16(gh, tm[m][q], acc[i][m]);
          }
          if (GP == 2) {
            const bf16x8_t gm = frag(B + (4 + i) * kFrag, lane);
#pragma unroll
            for (int m = 0; m < MT; ++m) acc[i][m] = mfma_16x16x32_bf16(gm, th[m][q], acc[i][m]);
          }
        }
      }
      ++done;
    };
    [&]<int... K>(std::integer_sequence<int, K...>) { (step(std::integral_constant<int, K>{}), ...); }
    (std::make_integer_sequence<int, KF / SK>{});
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f32x4_t v = acc[i][m];
        const int r = (wave * MT + m) * 16 + lane % 16, g = lane / 16;
        u32x2_t* at = reinterpret_cast<u32x2_t*>(rowbuf[hb & 1] + r * 64 + ((2 * i + g / 2) ^ (r % 8)) * 8 + (g & 1) * 4);
        if (ADD) {
          const u32x2_t u = *at;
          v += f32x4_t{bf16_lo(u[0]), bf16_hi(u[0]), bf16_lo(u[1]), bf16_hi(u[1])};
        }
        *at = u32x2_t{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
      }
  }
  step_barrier();
  store_rows(hb1 - 1);
  wait_vm<0>();  // no copy into LDS outlives the workgroup
}

// dx above 512 experts: 128 columns x 128 tokens per workgroup, 2 x 2 waves
// of 64 x 64, both operands through LDS.  GP planes of the gate.
template <int GP>
__global__ __launch_bounds__(256) void dx_wide_kernel(GateGradP p) {
  constexpr int AF = 2 * 8, BF = GP * 8;  // fragments per K step
  __shared__ __align__(16) uint16_t lds[2][(AF + BF) * kFrag];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wh = wave & 1, wt = wave >> 1;
  const uint32_t step_b = GP * 4 * kFrag * 2;  // bytes of a 64-column block's step
  const i32x4_t gb = make_desc(p.dxb + (size_t)blockIdx.x * 2 * p.Kf * GP * 4 * kFrag, 2u * p.Kf * step_b);
  for (int ty = blockIdx.y; ty < p.tiles_t; ty += gridDim.y) {
    const i32x4_t ga = make_desc(p.dxa + (size_t)ty * p.Kf * AF * kFrag, (uint32_t)p.Kf * AF * kFrag * 2);
    auto copy = [&](int s) {
      uint16_t* to = lds[s & 1];
      for (int f = wave; f < AF + BF; f += 4) {
        const int i = f - AF, blk = (i % 8) / 4;  // gate: plane i / 8, fragment i % 8 of two blocks
        if (f < AF)
          copy_frag(ga, (uint32_t)((s * AF + f) * kFrag * 2), lds_addr(to + f * kFrag), lane);
        else
          copy_frag(gb, (blk * p.Kf + s) * step_b + (uint32_t)(((i / 8) * 4 + i % 4) * kFrag * 2), lds_addr(to + f * kFrag),
                    lane);
      }
    };
    f32x4_t acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    copy(0);
    for (int s = 0; s < p.Kf; ++s) {
      wait_vm<0>();
      __syncthreads();  // step s has landed; step s - 1 is read
      if (s + 1 < p.Kf) copy(s + 1);
      const uint16_t* A = lds[s & 1];
      const uint16_t* B = A + AF * kFrag;
      bf16x8_t th[4], tm[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        th[j] = frag(A + (wt * 4 + j) * kFrag, lane);
        tm[j] = frag(A + (8 + wt * 4 + j) * kFrag, lane);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bf16x8_t gh = frag(B + (wh * 4 + i) * kFrag, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = mfma_16x16x32_bf16(gh, th[j], acc[i][j]);
          acc[i][j] = mfma_16x16x32_bf16(gh, tm[j], acc[i][j]);
        }
        if (GP == 2) {
          const bf16x8_t gm = frag(B + (8 + wh * 4 + i) * kFrag, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16x16x32_bf16(gm, th[j], acc[i][j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = ty * 128 + wt * 64 + j * 16 + lane % 16;
      if (t >= p.T) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = blockIdx.x * 128 + wh * 64 + i * 16 + 4 * (lane / 16);
        const size_t at = (size_t)t * p.H + h;
        f32x4_t v = acc[i][j];
        if (p.dx_in) {
          const uint2 u = *reinterpret_cast<const uint2*>(p.dx_in + at);
          v += f32x4_t{bf16_lo(u.x), bf16_hi(u.x), bf16_lo(u.y), bf16_hi(u.y)};
        }
        *reinterpret_cast<uint2*>(p.dx + at) = uint2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
      }
    }
    __syncthreads();  // the last step is read before the next tile's copies
  }
}

// d_gate: 32 MF experts x 256 columns per workgroup and K split, 2 x 4 waves
// of 16 MF x 64.
//  * The planes of d_logits (24 KiB a step at MF = 4) are copied into a ring
//    of three steps, two steps ahead.
//  * x has its rows along K: a thread loads 4 columns of 4 tokens R steps
//    ahead into registers, transposes them there and stores 8-byte pieces
//    (4 tokens of a column) into the step's fragments one step ahead.  The
//    operations of a wave complete in issue order and the compiler's waits
//    for the loads do not know of the copies, so they cover about half of
//    those R steps; a step's copies go out before its loads.  The
//    16-byte slot of a fragment is XORed with the fragment's number, so that
//    lanes which write the same slot of 8 fragments meet different banks.
//  * Workgroups of one K split that share columns or planes run on the same
//    XCD (contiguous runs of (split, column tile, expert tile) per XCD).
template <int MF>
__global__ __launch_bounds__(512, 2) void d_gate_kernel(GateGradP p) {
  constexpr int AF = 3 * 2 * MF, BF = 16;
  constexpr int R = 6, N_X = 4, N_A = AF / 8;  // loads of x, and copies (at least), of a wave and step
  __shared__ __align__(16) uint16_t alds[3][AF * kFrag];
  __shared__ __align__(16) uint16_t blds[2][BF * kFrag];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave & 1, wn = wave >> 1;
  const int ht = (p.H + 255) / 256;
  const int item = xcd_item(ht * p.mtiles * p.splits);
  if (item < 0) return;
  const int col = uniform(item / p.mtiles), mt = item - col * p.mtiles;
  const int z = uniform(col / ht), hx = col - z * ht;
  const int h0 = hx * 256;
  const int s0 = z * p.steps, n = min(p.nt32, s0 + p.steps) - s0;  // >= 1
  // Everything a step needs beside its operands is scalar or set up here: the
  // descriptors move along with the steps, the offsets inside a step stay.
  const uint32_t a_step = 3u * p.Ef * kFrag * 2;
  const uint16_t* const a_first = p.dga + (size_t)s0 * 3 * p.Ef * kFrag;
  uint32_t a_at[(AF + 7) / 8];
#pragma unroll
  for (int c = 0; c < (AF + 7) / 8; ++c) {
    const int f = c * 8 + wave;
    a_at[c] = (uint32_t)(((f / (2 * MF)) * p.Ef + mt * 2 * MF + f % (2 * MF)) * kFrag * 2);
  }
  auto copy_a = [&](int s, int slot) {  // past the end: the last step again
    const i32x4_t r = make_desc(reinterpret_cast<const char*>(a_first) + (size_t)min(s, n - 1) * a_step, a_step);
#pragma unroll
    for (int c = 0; c < (AF + 7) / 8; ++c)
      if (c * 8 + 8 <= AF || c * 8 + wave < AF) copy_frag(r, a_at[c], lds_addr(alds[slot] + (c * 8 + wave) * kFrag), lane);
  };
  // this thread's 4 tokens and 4 columns of a step; rows at or past T are
  // outside the range and read as zeros, columns past H (of the last tile)
  // are not stored
  const int quad = (wave & 3) * 2 + lane / 32, hq = (wave >> 2) * 32 + lane % 32;
  uint32_t x_at[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x_at[i] = (uint32_t)(quad * 4 + i) * p.H * 2 + min(h0 + hq * 4, p.H - 4) * 2;
  u32x2_t xr[R][4];
  auto load_x = [&](int s, u32x2_t(&to)[4]) {
    const int t = (s0 + s) * 32, rows = max(0, min(p.T - t, 32));
    const rsrc_t r = make_rsrc(p.x + (size_t)(rows > 0 ? t : 0) * p.H, (uint32_t)rows * p.H * 2);
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i] = __builtin_amdgcn_raw_buffer_load_b64(r, x_at[i], 0, 0);
  };
  uint32_t b_at[4];  // where this thread's piece of each of its columns goes, in 16-bit values
#pragma unroll
  for (int c = 0; c < 4; ++c)
    b_at[c] = (hq / 4) * kFrag + (((quad / 2) * 16 + (hq % 4) * 4 + c) ^ (hq / 4)) * 8 + (quad & 1) * 4;
  auto store_x = [&](int slot, const u32x2_t(&v)[4]) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t sel = c & 1 ? 0x07060302u : 0x05040100u;
      *reinterpret_cast<u32x2_t*>(blds[slot] + b_at[c]) =
          u32x2_t{__builtin_amdgcn_perm(v[1][c / 2], v[0][c / 2], sel),
                  __builtin_amdgcn_perm(v[3][c / 2], v[2][c / 2], sel)};
    }
  };
  f32x4_t acc[MF][4];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // x of step s sits in xr[s % R], its fragments in blds[s % 2], the planes
  // in alds[s % 3]: with R a multiple of 6 all fixed in the unrolled loop
  static_assert(R % 6 == 0, "slots by the place in the loop");
#pragma unroll
  for (int i = 0; i < R - 2; ++i) load_x(i, xr[i]);
  copy_a(0, 0);
  keep_order();
  load_x(R - 2, xr[R - 2]);
  copy_a(1, 1);
  keep_order();
  load_x(R - 1, xr[R - 1]);
  store_x(0, xr[0]);
  // BEHIND: vector memory operations behind step s's copies (issued at step
  // s - 2): that step's loads of x, then the copies and loads of step s - 1.
  // Steps past the unrolled loop load no x.
  auto step = [&](int s, auto place, auto behind, auto loads) {
    constexpr int I = decltype(place)::value;
    wait_vm<decltype(behind)::value>();
    step_barrier();
    const uint16_t* A = alds[I % 3] + wm * MF * kFrag + lane * 8;
    const uint16_t* B = blds[I % 2] + wn * 4 * kFrag;
    bf16x8_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = frag(B + j * kFrag, lane ^ (wn * 4 + j));
    bf16x8_t a[3];
#pragma unroll
    for (int q = 0; q < 3; ++q) a[q] = frag(A + q * 2 * MF * kFrag, 0);
    // the next steps' operands are asked for while these reads are under way
    copy_a(s + 2, (I + 2) % 3);
    keep_order();
    if (decltype(loads)::value) load_x(s + R, xr[I]);
    keep_order();
    store_x((I + 1) % 2, xr[(I + 1) % R]);
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const bf16x8_t now = a[q];
        if (i + 1 < MF) a[q] = frag(A + (q * 2 * MF + i + 1) * kFrag, 0);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16x16x32_bf16(now, b[j], acc[i][j]);
      }
  };
  int s = 0;
  for (; s + R <= n; s += R) {
    [&]<int... I>(std::integer_sequence<int, I...>) {
      (step(s + I, std::integral_constant<int, I>{}, std::integral_constant<int, 2 * N_X + N_A>{}, std::true_type{}), ...);
    }
    (std::make_integer_sequence<int, R>{});
  }
  [&]<int... I>(std::integer_sequence<int, I...>) {
    ((s + I < n ? step(s + I, std::integral_constant<int, I>{},
                       std::integral_constant<int, I == 0 ? 2 * N_X + N_A : I == 1 ? N_X + N_A : N_A>{},
                       std::false_type{})
                : void()),
     ...);
  }
  (std::make_integer_sequence<int, R - 1>{});
  wait_vm<0>();  // no copy into LDS outlives the workgroup
  float* out = p.splits > 1 ? p.part + (size_t)z * p.E * p.H : p.d_gate;
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = (mt * 2 * MF + wm * MF + i) * 16 + 4 * (lane / 16) + r;
      if (e >= p.E) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int h = h0 + wn * 64 + j * 16 + lane % 16;
        if (h < p.H) out[(size_t)e * p.H + h] = acc[i][j][r];
      }
    }
}

// out = sum of n arrays of 4 len4 values, in order
__global__ __launch_bounds__(256) void add_parts_kernel(const f32x4_t* part, int n, size_t len4, f32x4_t* out) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < len4; i += (size_t)gridDim.x * 256) {
    f32x4_t v = part[i];
    for (int s = 1; s < n; ++s) v += part[(size_t)s * len4 + i];
    out[i] = v;
  }
}
__global__ __launch_bounds__(256) void zero_kernel(f32x4_t* out, size_t len4) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < len4; i += (size_t)gridDim.x * 256)
    out[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
}

// d_gate's tile height (mf) and K splits: the least of an estimate of its time
// in us, per round of 256 workgroups a start and the steps, and for more than
// one split the launch that adds them up and the bytes they write and read.
// Fitted to a sweep of both over eleven shapes (1 to 8192 tokens, 64 to 288
// experts), where its choice was within 3 us of the best of each; splitting
// to fill the chip with the tallest tiles alone took 23 us instead of 14 at
// 512 tokens, 4096 columns and 288 experts.
void d_gate_split(GateGradP& p) {
  static const double kStep[kMaxMf] = {0.45, 0.58, 0.82, 1.03};  // us per step by mf
  static const int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  const int ht = ceil_div(p.H, 256), nt = p.nt32 > 0 ? p.nt32 : 1;
  const double write = (double)p.E * p.H * 4 / 5.5e6;  // us for one array of partial sums
  double best = 0;
  for (int mf = 1; mf <= kMaxMf; ++mf) {
    const int mtiles = ceil_div(p.E, 32 * mf);
    for (int splits : kSplits) {
      if (splits > nt) break;
      const int steps = ceil_div(nt, splits), n = ceil_div(nt, steps);
      const int64_t rounds = ceil_div64((int64_t)ht * mtiles * n, 256);
      const double us = rounds * (3.0 + steps * kStep[mf - 1]) +
                        (n > 1 ? 3.0 + 0.15 * n + (2 * n + 1) * write : write);
      if (best == 0 || us < best) {
        best = us;
        p.mf = mf;
        p.mtiles = mtiles;
        p.steps = steps;
        p.splits = n;
      }
    }
  }
  p.Ef = p.mtiles * 2 * p.mf;
}

// Shape-derived numbers and the workspace (offsets; 0-size parts included).
struct GateGradPlan {
  GateGradP p;
  size_t dxa, dxb, dga, part, total;
};
GateGradPlan gate_grad_plan(int T, int H, int E) {
  GateGradPlan L;
  GateGradP& p = L.p;
  p.T = T;
  p.H = H;
  p.E = E;
  p.Kf = ceil_div(E, 32);
  p.tiles_t = ceil_div(T, 128);
  p.nt32 = ceil_div(T, 32);
  // dx: 32 tokens per wave in registers up to 256 experts, 16 up to 512
  p.mt = p.Kf <= 8 ? 2 : p.Kf <= 16 ? 1 : 0;
  if (p.Kf == 7) p.Kf = 8;
  if (p.mt == 1) p.Kf = p.Kf <= 10 ? p.Kf : p.Kf <= 12 ? 12 : 16;
  const int blocks = H / 64, groups = ceil_div(T, p.mt == 1 ? 128 : 256);
  p.hsplits = groups >= 32 ? 8 : ceil_div(256, groups > 0 ? groups : 1);
  if (p.hsplits > blocks) p.hsplits = blocks;
  p.hper = ceil_div(blocks, p.hsplits);
  p.hsplits = ceil_div(blocks, p.hper);
  d_gate_split(p);
  size_t off = kCtrlBytes;  // the control block stays as it is
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  const size_t fb = (size_t)kFrag * 2;
  L.dxa = take((size_t)p.tiles_t * p.Kf * 16 * fb);
  L.dxb = take((size_t)(H / 64) * p.Kf * 8 * fb);
  L.dga = take((size_t)p.nt32 * 3 * p.Ef * fb);
  L.part = take(p.splits > 1 ? (size_t)p.splits * E * H * sizeof(float) : 0);
  L.total = off;
  return L;
}

template <int KF, int MT>
void launch_dx_kf(const GateGradP& p, hipStream_t s) {
  const int grid = ceil_div(ceil_div(p.T, 128 * MT) * p.hsplits, 8) * 8;
  if (p.gate_fp32) {
    if (p.dx_in)
      dx_kernel<KF, MT, 2, true><<<grid, 512, 0, s>>>(p);
    else
      dx_kernel<KF, MT, 2, false><<<grid, 512, 0, s>>>(p);
  } else {
    if (p.dx_in)
      dx_kernel<KF, MT, 1, true><<<grid, 512, 0, s>>>(p);
    else
      dx_kernel<KF, MT, 1, false><<<grid, 512, 0, s>>>(p);
  }
}
void launch_dx(const GateGradP& p, hipStream_t s) {
  switch (p.Kf) {
    case 1: launch_dx_kf<1, 2>(p, s); break;
    case 2: launch_dx_kf<2, 2>(p, s); break;
    case 3: launch_dx_kf<3, 2>(p, s); break;
    case 4: launch_dx_kf<4, 2>(p, s); break;
    case 5: launch_dx_kf<5, 2>(p, s); break;
    case 6: launch_dx_kf<6, 2>(p, s); break;
    case 8: launch_dx_kf<8, 2>(p, s); break;
    case 9: launch_dx_kf<9, 1>(p, s); break;
    case 10: launch_dx_kf<10, 1>(p, s); break;
    case 12: launch_dx_kf<12, 1>(p, s); break;
    default: launch_dx_kf<16, 1>(p, s); break;
  }
}

bool gate_grad_shape(int T, int H, int E) {
  return T >= 0 && T <= (1 << 24) && H >= 128 && H % 128 == 0 && H <= (1 << 20) && E >= 1 && E <= 1024;
}

}  // namespace

}  // namespace moe

extern "C" size_t moe_gate_grad_workspace_size(int T, int H, int E) {
  return moe::gate_grad_shape(T, H, E) ? moe::gate_grad_plan(T, H, E).total : 0;
}

extern "C" moe_status moe_gate_grad(const void* x, const void* gate, int gate_is_fp32, const float* d_logits,
                                    const void* dx_in, int T, int H, int E, void* dx, float* d_gate, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream) {
  using namespace moe;
  if (!gate_grad_shape(T, H, E) || gate_is_fp32 < 0 || gate_is_fp32 > 1) return MOE_E_INVAL;
  if (!dx && !d_gate) return MOE_E_INVAL;
  if (dx_in && !dx) return MOE_E_INVAL;
  for (const void* q : {x, gate, dx_in, (const void*)dx, (const void*)d_gate, (const void*)workspace})
    if (!aligned(q, 16)) return MOE_E_INVAL;
  const size_t len4 = (size_t)E * H / 4;
  if (T == 0) {
    if (!d_gate) return MOE_OK;
    zero_kernel<<<(int)(ceil_div64(len4, 256) < 2048 ? ceil_div64(len4, 256) : 2048), 256, 0, stream>>>(
        reinterpret_cast<f32x4_t*>(d_gate), len4);
    MOE_CHECK_LAUNCH();
    return MOE_OK;
  }
  if (!d_logits || (d_gate && !x) || (dx && !gate) || !workspace) return MOE_E_INVAL;
  GateGradPlan L = gate_grad_plan(T, H, E);
  if (workspace_bytes < L.total) return MOE_E_WORKSPACE;
  char* b = static_cast<char*>(workspace);
  GateGradP& p = L.p;
  p.x = static_cast<const uint16_t*>(x);
  p.gate = gate;
  p.gate_fp32 = gate_is_fp32;
  p.dl = d_logits;
  p.dx_in = static_cast<const uint16_t*>(dx_in);
  p.dx = static_cast<uint16_t*>(dx);
  p.d_gate = d_gate;
  p.dxa = dx ? reinterpret_cast<uint16_t*>(b + L.dxa) : nullptr;
  p.dxb = reinterpret_cast<uint16_t*>(b + L.dxb);
  p.dga = d_gate ? reinterpret_cast<uint16_t*>(b + L.dga) : nullptr;
  p.part = reinterpret_cast<float*>(b + L.part);
  const int cols = p.Kf * 32 > p.Ef * 16 ? p.Kf * 32 : p.Ef * 16;
  const int e_tiles = ceil_div(cols, 64), logit_tiles = p.tiles_t * 4 * e_tiles;
  const int gate_tiles = dx ? p.Kf * (H / 64) : 0;
  split_kernel<<<logit_tiles + gate_tiles, 256, 0, stream>>>(p, logit_tiles, e_tiles);
  MOE_CHECK_LAUNCH();
  if (dx) {
    if (p.mt == 0) {
      const dim3 grid((unsigned)(H / 128), (unsigned)(p.tiles_t < 65535 ? p.tiles_t : 65535));
      if (gate_is_fp32)
        dx_wide_kernel<2><<<grid, 256, 0, stream>>>(p);
      else
        dx_wide_kernel<1><<<grid, 256, 0, stream>>>(p);
    } else {
      launch_dx(p, stream);
    }
    MOE_CHECK_LAUNCH();
  }
  if (d_gate) {
    const int items = ceil_div(H, 256) * p.mtiles * p.splits, grid = ceil_div(items, 8) * 8;
    switch (p.mf) {
      case 1: d_gate_kernel<1><<<grid, 512, 0, stream>>>(p); break;
      case 2: d_gate_kernel<2><<<grid, 512, 0, stream>>>(p); break;
      case 3: d_gate_kernel<3><<<grid, 512, 0, stream>>>(p); break;
      default: d_gate_kernel<4><<<grid, 512, 0, stream>>>(p); break;
    }
    MOE_CHECK_LAUNCH();
    if (p.splits > 1) {
      add_parts_kernel<<<(int)(ceil_div64(len4, 256) < 2048 ? ceil_div64(len4, 256) : 2048), 256, 0, stream>>>(
          reinterpret_cast<const f32x4_t*>(p.part), p.splits, len4, reinterpret_cast<f32x4_t*>(d_gate));
      MOE_CHECK_LAUNCH();
    }
  }
  return MOE_OK;
}
