// moe_rms_norm and moe_rms_norm_grad: the root-mean-square norm in front of
// an MoE layer, with the residual's addition before it and the experts'
// activation quantisation behind it, and its gradient.
//
//   h = x + residual                       (fp32; stored in the residual's type)
//   y = h rsqrt(mean(h^2) + eps) w         (fp32 from the unrounded h; stored as bf16)
//   q = e4m3(y / s)                        (s from the group's largest |y|, in fp32)
//
// The 8-bit codes are rounded once, from the fp32 y: rounding to bf16 first
// would put many values exactly on an e4m3 tie and send half of those to the
// wrong side.
//
//   g = dy w,  r = rsqrt(mean(h^2) + eps)
//   dx = r g - h r^3 mean(g h) + dh        (gradient of x and of the residual)
//   dw = sum_t dy h r                      (fp32)
//
// Both are bound by memory: one pass, a row lives in registers between its
// loads and its stores.  All row vectors are 16-byte accesses at the
// alignment of an element (the hardware takes them at any address), so odd
// widths keep the wide accesses.  Measured: 8192 x 4096 with a residual and MX
// codes 59 us (5.1 TB/s; a large copy reaches 4.9 here), its gradient at
// 8192 x 7168 with an fp32 residual stream 155 us (5.3 TB/s); 1 x 7168 3.8
// us, an empty kernel 3.5.
//
// Rows of up to 256 values share a wave, 8, 16 or 32 lanes each: 100000 x 128
// 22.9 us with a wave per row, 9.6 so, its gradient 49.9 and 23.2.

#include <cmath>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "quant.h"

namespace moe {

namespace {

constexpr int kMaxNormH = 32768;  // 16 waves x 64 lanes x 4 vectors x 8 values
constexpr int kVec = 8;           // values per vector

// The 8 values of a row of n that a thread's vector i (its first element)
// stands for.  A vector that runs past the row's end is moved back to end
// with it: its first `skip` values are its neighbour's, which are left out of
// sums and scales and stored twice with the same value.  Rows of fewer than
// 8 values (SHORT: they may be) go element by element.
struct Span {
  uint32_t base;
  int skip;  // 8: no vector
};
template <bool SHORT>
__device__ __forceinline__ Span span_of(int i, int n) {
  if (i >= n) return Span{0, 8};
  if (i + kVec <= n || (SHORT && n < kVec)) return Span{(uint32_t)i, 0};
  return Span{(uint32_t)(n - kVec), i + kVec - n};
}

// Where it begins: a 32-bit offset in bytes, so that the row's address stays
// scalar where it is.
template <class T>
__device__ __forceinline__ T* vector_at(T* row, Span s) {
  typedef typename std::conditional<std::is_const<T>::value, const char, char>::type Byte;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(row) + s.base * (uint32_t)sizeof(T));
}

// A vector as it comes from memory (bf16: two values a word).  pin: values
// taken from it before are not kept in registers for what follows.
template <class T>
struct Raw;
template <>
struct Raw<uint16_t> {
  u32x4_t v;
  template <bool SHORT>
  __device__ __forceinline__ void load(const uint16_t* row, Span s, int n) {
    v = u32x4_t{0u, 0u, 0u, 0u};
    if (s.skip == 8) return;
    if (!SHORT || n >= kVec) {
      __builtin_memcpy(&v, vector_at(row, s), 16);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) v[j / 2] |= (uint32_t)row[j] << (16 * (j & 1));
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(v[j]);
      f[2 * j + 1] = bf16_hi(v[j]);
    }
  }
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(v)); }
};
template <>
struct Raw<float> {
  f32x4_t a, b;
  template <bool SHORT>
  __device__ __forceinline__ void load(const float* row, Span s, int n) {
    a = b = f32x4_t{0.f, 0.f, 0.f, 0.f};
    if (s.skip == 8) return;
    if (!SHORT || n >= kVec) {
      __builtin_memcpy(&a, vector_at(row, s), 16);
      __builtin_memcpy(&b, vector_at(row, s) + 4, 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (j < n) a[j] = row[j];
        if (j + 4 < n) b[j] = row[j + 4];
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[j + 4] = b[j];
    }
  }
  __device__ __forceinline__ void pin() { asm volatile("" : "+v"(a), "+v"(b)); }
};
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
// once: nobody reads the values soon (a hint to the caches)
template <bool SHORT>
__device__ __forceinline__ void store8(uint16_t* row, Span s, int n, const float (&f)[8], bool once = false) {
  if (s.skip == 8) return;
  u32x4_t v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = cvt_bf16x2(f[2 * j], f[2 * j + 1]);
  if (!SHORT || n >= kVec) {
    u32x4_any_t* at = reinterpret_cast<u32x4_any_t*>(vector_at(row, s));
    if (once)
      __builtin_nontemporal_store(v, at);
    else
      *at = v;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) row[j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
  }
}
template <bool SHORT>
__device__ __forceinline__ void store8(float* row, Span s, int n, const float (&f)[8], bool once = false) {
  if (s.skip == 8) return;
  if (!SHORT || n >= kVec) {
    const f32x4_t a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
    f32x4_any_t* at = reinterpret_cast<f32x4_any_t*>(vector_at(row, s));
    if (once) {
      __builtin_nontemporal_store(a, at);
      __builtin_nontemporal_store(b, at + 1);
    } else {
      at[0] = a;
      at[1] = b;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) row[j] = f[j];
  }
}
template <bool SHORT>
__device__ __forceinline__ void load_weight8(const void* w, int w_fp32, Span s, int n, float (&f)[8]) {
  if (w_fp32) {
    Raw<float> r;
    r.load<SHORT>(static_cast<const float*>(w), s, n);
    r.get(f);
  } else {
    Raw<uint16_t> r;
    r.load<SHORT>(static_cast<const uint16_t*>(w), s, n);
    r.get(f);
  }
}
// a thread's sum over a moved vector starts behind its neighbour's values
__device__ __forceinline__ float sum8(const float (&f)[8], int skip) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s += j >= skip ? f[j] : 0.f;
  return s;
}

struct NormP {
  const uint16_t* x;
  const void* res;
  const void* w;
  void* h;      // optional, the residual's type
  uint16_t* y;  // optional
  uint8_t* q;   // QF != 0
  void* s;
  int first;  // row of the launch's first workgroup
  int T, H;
  float eps, inv_h;
  int w_fp32;
  int waves;  // waves per row
  bool once;  // outputs past the caches: store them with the hint
};

// e4m3 codes and scales of 8 values of a row; a scale group is 16 (FP8: 128
// values) or 4 (MX: 32 values) neighbouring lanes, all of them in range or
// all past the row's end.  No clamp: |v| <= 448 (1 + 2^-23) rounds to at
// most 448, and a NaN stays one (code 0x7F).
template <int QF>
__device__ __forceinline__ void quant8(const NormP& p, size_t row, int i, const float (&v)[8]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
  float g[8];
  if (QF == 1) {
    m = row_max16(m);
    const float s = fp8_group_scale(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = v[j] / s;
    if (i < p.H && (threadIdx.x & 15) == 0) static_cast<float*>(p.s)[row * (p.H / 128) + i / 128] = s;
  } else {
    m = fmaxf(m, dpp_f32<0xB1>(m));
    m = fmaxf(m, dpp_f32<0x4E>(m));
    const uint32_t c = mx_group_code(m);
    const float inv = e8m0_inv(c);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = v[j] * inv;
    if (i < p.H && (threadIdx.x & 3) == 0) static_cast<uint8_t*>(p.s)[row * (p.H / 32) + i / 32] = (uint8_t)c;
  }
  if (i < p.H) {
    uint2 u;
    u.x = pack4_e4m3(g[0], g[1], g[2], g[3]);
    u.y = pack4_e4m3(g[4], g[5], g[6], g[7]);
    *reinterpret_cast<uint2*>(p.q + row * p.H + i) = u;
  }
}

// Threads per row: ROW lanes of a wave, or (ROW 64) whole waves.
template <int ROW>
__device__ __forceinline__ int row_threads(int waves) {
  return ROW < kWave ? ROW : waves * kWave;
}

// The thread's row in the workgroup (uniform, and known to be, for whole waves).
template <int ROW>
__device__ __forceinline__ int row_of_thread(int waves) {
  if (ROW < kWave) return threadIdx.x / ROW;
  return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave / waves);
}

// RT: residual type, 0 none, 1 bf16, 2 fp32.  NV vectors per thread, as many
// rows per workgroup as its size holds.
template <int NV, int ROW, int QF, int RT>
__global__ __launch_bounds__(1024) void norm_kernel(NormP p) {
  typedef typename std::conditional<RT == 2, float, uint16_t>::type ResT;
  constexpr bool SHORT = ROW == 8;
  const int lanes = row_threads<ROW>(p.waves);
  const int sub = row_of_thread<ROW>(p.waves), tid = threadIdx.x - sub * lanes;
  const int rows = blockDim.x / lanes;
  const size_t row = (size_t)p.first + (size_t)blockIdx.x * rows + sub;
  const bool live = row < (size_t)p.T;
  const bool moved = p.H % kVec != 0;
  Span sp[NV];
#pragma unroll
  for (int v = 0; v < NV; ++v) sp[v] = span_of<SHORT>((v * lanes + tid) * kVec, p.H);
  float h[NV][8], w[NV][8];
  float ss = 0.f;
  if (live) {
    Raw<uint16_t> x[NV];
    Raw<ResT> res[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) x[v].template load<SHORT>(p.x + row * p.H, sp[v], p.H);
    if (RT != 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) res[v].template load<SHORT>(static_cast<const ResT*>(p.res) + row * p.H, sp[v], p.H);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) load_weight8<SHORT>(p.w, p.w_fp32, sp[v], p.H, w[v]);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      x[v].get(h[v]);
      if (RT != 0) {
        float r[8];
        res[v].get(r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] += r[j];
      }
      float sq[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) sq[j] = h[v][j] * h[v][j];
      ss += moved ? sum8(sq, sp[v].skip) : sum8(sq, 0);
    }
  }
  ss = group_sum<ROW>(ss);
  if (ROW == kWave && p.waves > 1) {
    __shared__ float part[16];
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = ss;
    __syncthreads();
    ss = 0.f;
    for (int i = 0; i < p.waves; ++i) ss += part[sub * p.waves + i];
  }
  if (!live) return;
  const float r = rsqrtf(ss * p.inv_h + p.eps);
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (RT != 0 && p.h) store8<SHORT>(static_cast<ResT*>(p.h) + row * p.H, sp[v], p.H, h[v], p.once);
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[v][j] * r * w[v][j];
    if (p.y) store8<SHORT>(p.y + row * p.H, sp[v], p.H, y, p.once);
    if (QF != 0) quant8<QF>(p, row, (v * lanes + tid) * kVec, y);
  }
}

template <int NV, int ROW, int QF>
void launch_norm_rt(const NormP& p, int rt, dim3 grid, int threads, hipStream_t s) {
  switch (rt) {
    case 0: norm_kernel<NV, ROW, QF, 0><<<grid, threads, 0, s>>>(p); break;
    case 1: norm_kernel<NV, ROW, QF, 1><<<grid, threads, 0, s>>>(p); break;
    default: norm_kernel<NV, ROW, QF, 2><<<grid, threads, 0, s>>>(p); break;
  }
}
template <int NV, int ROW>
void launch_norm_q(const NormP& p, int qf, int rt, dim3 grid, int threads, hipStream_t s) {
  switch (qf) {
    case 0: launch_norm_rt<NV, ROW, 0>(p, rt, grid, threads, s); break;
    case 1:
      if constexpr (ROW != 8) launch_norm_rt<NV, ROW, 1>(p, rt, grid, threads, s);  // H >= 128
      break;
    default: launch_norm_rt<NV, ROW, 2>(p, rt, grid, threads, s); break;
  }
}

// A value of the loop's turn alone: keeps the compiler from carrying a 64-bit
// address per lane and vector from turn to turn instead of a scalar one.
template <int ROW, class T>
__device__ __forceinline__ T this_turn(T v) {
  if (ROW == kWave) asm volatile("" : "+s"(v));
  return v;
}

struct NormGradP {
  const uint16_t* dy;
  const void* dh;  // optional, h's type
  const void* h;
  const void* w;
  void* dx;     // h's type
  float* part;  // [gridDim.x][H] sums of dy h r over this workgroup's rows; null: no weight gradient
  int T, H;
  float eps, inv_h;
  int w_fp32;
  int waves;  // waves per row
};

// A workgroup holds blockDim / row_threads rows at a time, and takes the next
// ones gridDim further on; a thread keeps the same columns for every row, so
// the weight and the weight gradient's sums stay in its registers (the rows'
// sums are added across lanes and in LDS at the end, in order).  The next rows
// are on their way while a row is reduced and stored.  Above 16384 columns
// (NV 4) the sums lie in LDS and scalar row addresses leave the registers to
// the row: 2048 x 20000 198 us with all of it in registers (spilled), 102 so.
template <int NV, int ROW, bool HF32>
__global__ __launch_bounds__(1024) void norm_grad_kernel(NormGradP p) {
  typedef typename std::conditional<HF32, float, uint16_t>::type HT;
  constexpr bool SHORT = ROW == 8;
  const int lanes = row_threads<ROW>(p.waves);
  const int sub = row_of_thread<ROW>(p.waves), tid = threadIdx.x - sub * lanes;
  const int rows = blockDim.x / lanes;
  const bool moved = p.H % kVec != 0;
  __shared__ float part[2][2][16];
  // at NV 4 the 128 registers hold neither the weight (read per row, from the
  // L1) nor the weight gradient's sums (in LDS) beside the row.  The row stays
  // in registers: dx may take the place of h or dh
  constexpr bool AHEAD = NV == 1, WIDE = NV > 2;
  __shared__ float wide[WIDE ? NV * kVec * 1024 : 1];
  Span sp[NV];
  float w[WIDE ? 1 : NV][8], dw[WIDE ? 1 : NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    sp[v] = span_of<SHORT>((v * lanes + tid) * kVec, p.H);
    if (!WIDE) load_weight8<SHORT>(p.w, p.w_fp32, sp[v], p.H, w[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (WIDE)
        wide[(v * kVec + j) * 1024 + threadIdx.x] = 0.f;
      else
        dw[v][j] = 0.f;
    }
  }
  Raw<HT> hr[NV], dhr[NV], hn[NV], dhn[NV];
  Raw<uint16_t> dyr[NV], dyn[NV];
  auto load = [&](int64_t row, Raw<HT>(&h)[NV], Raw<uint16_t>(&dy)[NV], Raw<HT>(&dh)[NV]) {
    if (row >= p.T) return;
    const size_t at = (size_t)row * p.H;
    const HT* h_row = this_turn<ROW>(static_cast<const HT*>(p.h) + at);
    const uint16_t* dy_row = this_turn<ROW>(p.dy + at);
    const HT* dh_row = this_turn<ROW>(static_cast<const HT*>(p.dh) + at);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v].template load<SHORT>(h_row, sp[v], p.H);
      dy[v].template load<SHORT>(dy_row, sp[v], p.H);
      if (p.dh) dh[v].template load<SHORT>(dh_row, sp[v], p.H);
    }
  };
  int flip = 0;
  int64_t row = (int64_t)blockIdx.x * rows + sub;
  const int64_t stride = (int64_t)gridDim.x * rows;
  if (AHEAD) load(row, hr, dyr, dhr);
  // every wave of the workgroup takes the same number of turns
  for (int64_t first = (int64_t)blockIdx.x * rows; first < p.T; first += stride, row += stride, flip ^= 1) {
    if (AHEAD)
      load(row + stride, hn, dyn, dhn);
    else
      load(row, hr, dyr, dhr);
    const bool live = row < p.T;
    HT* dx_row = this_turn<ROW>(static_cast<HT*>(p.dx) + (size_t)row * p.H);
    float ss = 0.f, gh = 0.f;
    if (live) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float h[8], g[8], a[8], b[8];
        hr[v].get(h);
        dyr[v].get(g);
        if (WIDE) load_weight8<SHORT>(this_turn<ROW>(p.w), p.w_fp32, sp[v], p.H, w[0]);
        const float(&wv)[8] = w[WIDE ? 0 : v];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          a[j] = h[j] * h[j];
          b[j] = g[j] * wv[j] * h[j];
        }
        ss += moved ? sum8(a, sp[v].skip) : sum8(a, 0);
        gh += moved ? sum8(b, sp[v].skip) : sum8(b, 0);
      }
    }
    ss = group_sum<ROW>(ss);
    gh = group_sum<ROW>(gh);
    if (ROW == kWave && p.waves > 1) {
      if ((threadIdx.x & 63) == 0) {
        part[flip][0][threadIdx.x >> 6] = ss;
        part[flip][1][threadIdx.x >> 6] = gh;
      }
      // one barrier a turn: a wave writes the other half next time, and this
      // half again only after the next turn's barrier
      __syncthreads();
      ss = gh = 0.f;
      for (int i = 0; i < p.waves; ++i) {
        ss += part[flip][0][sub * p.waves + i];
        gh += part[flip][1][sub * p.waves + i];
      }
    }
    if (live) {
      const float r = rsqrtf(ss * p.inv_h + p.eps);
      const float c = r * r * r * (gh * p.inv_h);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        float h[8], g[8], d[8], dh[8];
        if (WIDE) {
          hr[v].pin();
          dyr[v].pin();
        }
        hr[v].get(h);
        dyr[v].get(g);
        if (p.dh) dhr[v].get(dh);
        if (WIDE) load_weight8<SHORT>(this_turn<ROW>(p.w), p.w_fp32, sp[v], p.H, w[0]);
        const float(&wv)[8] = w[WIDE ? 0 : v];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = r * (g[j] * wv[j]) - h[j] * c;
          d[j] = p.dh ? n + dh[j] : n;
          if (WIDE)
            wide[(v * kVec + j) * 1024 + threadIdx.x] += g[j] * (h[j] * r);
          else
            dw[v][j] += g[j] * (h[j] * r);
        }
        store8<SHORT>(dx_row, sp[v], p.H, d);
      }
    }
    if (AHEAD) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        hr[v] = hn[v];
        dyr[v] = dyn[v];
        dhr[v] = dhn[v];
      }
    }
  }
  if (!p.part) return;
  if constexpr (WIDE) {  // one row at a time: the sums are whole
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[0][j] = wide[(v * kVec + j) * 1024 + threadIdx.x];
      store8<SHORT>(p.part + (size_t)blockIdx.x * p.H, sp[v], p.H, dw[0]);
    }
    return;
  } else {
#pragma unroll
    for (int off = ROW; off < kWave; off *= 2)  // the rows of a wave
#pragma unroll
      for (int j = 0; j < 8; ++j) dw[0][j] += __shfl_xor(dw[0][j], off, kWave);
    // then the waves, or the groups of waves, that hold the same columns
    const int group = ROW < kWave ? threadIdx.x / kWave : sub, groups = ROW < kWave ? blockDim.x / kWave : rows;
    if (ROW < kWave && (threadIdx.x & 63) >= ROW) sp[0].skip = 8;
    if (groups > 1) {
      extern __shared__ float sums[];  // [groups][8][NV][lanes]
      const int width = NV * lanes * kVec;
      __syncthreads();
      if (sp[0].skip < 8)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) sums[group * width + (j * NV + v) * lanes + tid] = dw[v][j];
      __syncthreads();
      if (group > 0 || sp[0].skip == 8) return;
      for (int i = 1; i < groups; ++i)
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int j = 0; j < 8; ++j) dw[v][j] += sums[i * width + (j * NV + v) * lanes + tid];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) store8<SHORT>(p.part + (size_t)blockIdx.x * p.H, sp[v], p.H, dw[v]);
  }
}

// out[c] = sum of n rows of part[., c], in a fixed order: 32 slices of the
// rows per workgroup of 32 columns, then the slices.  n = 0: zeros.
__global__ __launch_bounds__(256) void column_sum_kernel(const float* part, int n, int H, float* out) {
  __shared__ float s[32][33];
  const int q = threadIdx.x & 7, c = blockIdx.x * 32 + q * 4, slice = threadIdx.x >> 3;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  if (c + 4 <= H) {
#pragma unroll 4
    for (int r = slice; r < n; r += 32) {
      f32x4_t v;
      __builtin_memcpy(&v, part + (size_t)r * H + c, 16);
      acc += v;
    }
  } else {
    for (int r = slice; r < n; r += 32)
      for (int j = 0; j < 4; ++j)
        if (c + j < H) acc[j] += part[(size_t)r * H + c + j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[slice][q * 4 + j] = acc[j];
  __syncthreads();
  const int col = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x < 32 && col < H) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][threadIdx.x];
    out[col] = t;
  }
}

int norm_waves(int H, int nv) { return ceil_div(H, kWave * kVec * nv); }
// lanes per row: 8, 16 or 32 where one vector each holds it, else whole waves
int norm_row(int H) { return H <= 8 * kVec ? 8 : H <= 16 * kVec ? 16 : H <= 32 * kVec ? 32 : kWave; }

// The backward pass: vectors per thread, rows per workgroup (about 8 waves
// where rows are short) and workgroups: 16 waves per CU, as the registers
// allow; each workgroup leaves one fp32 row of weight gradient sums, and more
// workgroups than stay resident cost more in those than they hide (8192 x
// 7168 fp32: 157 / 165 / 170 us with 256 / 512 / 768; 8192 x 4096 bf16 54 /
// 61 with 512 / 768 of 8 waves).
struct GradShape {
  int nv, row, waves, rows, grid;
};
GradShape grad_shape(int T, int H) {
  GradShape g;
  g.nv = norm_waves(H, 1) <= 16 ? 1 : norm_waves(H, 2) <= 16 ? 2 : 4;
  g.waves = norm_waves(H, g.nv);
  g.row = norm_row(H);
  g.rows = (g.waves >= 8 ? 1 : 8 / g.waves) * (kWave / g.row);
  const int turns = ceil_div(T, g.rows), fit = 256 * (g.waves > 8 ? 1 : 2);
  g.grid = turns < fit ? turns : fit;
  return g;
}

template <int NV, int ROW>
void launch_grad_nv(const NormGradP& p, int h_fp32, const GradShape& g, hipStream_t s) {
  const int threads = g.rows * (ROW < kWave ? ROW : g.waves * kWave);
  const size_t lds = g.rows > 1 ? (size_t)threads * NV * kVec * sizeof(float) : 0;
  if (h_fp32)
    norm_grad_kernel<NV, ROW, true><<<g.grid, threads, lds, s>>>(p);
  else
    norm_grad_kernel<NV, ROW, false><<<g.grid, threads, lds, s>>>(p);
}

moe_status norm_shape(int T, int H, float eps) {
  if (T < 0 || T > (1 << 24) || H < 1 || !(eps >= 0.f) || std::isinf(eps)) return MOE_E_INVAL;
  return H > kMaxNormH ? MOE_E_UNSUPPORTED : MOE_OK;
}

}  // namespace

moe_status norm_validate(const void* x, const void* residual, int residual_is_fp32, const void* weight,
                         int weight_is_fp32, int T, int H, float eps, int qformat, const void* h, const void* y,
                         const void* q, const void* s) {
  const moe_status st = norm_shape(T, H, eps);
  if (st != MOE_OK) return st;
  if (residual_is_fp32 < 0 || residual_is_fp32 > 1 || weight_is_fp32 < 0 || weight_is_fp32 > 1) return MOE_E_INVAL;
  if (qformat != MOE_W_BF16 && qformat != MOE_W_FP8_BLOCK128 && qformat != MOE_W_MXFP4) return MOE_E_INVAL;
  if (h && !residual) return MOE_E_INVAL;
  if (qformat != MOE_W_BF16 && !aligned(q, 8)) return MOE_E_INVAL;
  if ((qformat == MOE_W_FP8_BLOCK128 && H % 128) || (qformat == MOE_W_MXFP4 && H % 32)) return MOE_E_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !weight) return MOE_E_INVAL;
  if (qformat == MOE_W_BF16 ? !y : (!q || !s)) return MOE_E_INVAL;
  return MOE_OK;
}

moe_status launch_norm(const void* x, const void* residual, int residual_is_fp32, const void* weight,
                       int weight_is_fp32, int T, int H, float eps, int qformat, void* h, void* y, void* q, void* s,
                       hipStream_t stream) {
  NormP p;
  p.x = static_cast<const uint16_t*>(x);
  p.res = residual;
  p.w = weight;
  p.h = h;
  p.y = static_cast<uint16_t*>(y);
  p.q = static_cast<uint8_t*>(q);
  p.s = s;
  p.T = T;
  p.H = H;
  p.eps = eps;
  p.inv_h = 1.f / (float)H;
  p.w_fp32 = weight_is_fp32;
  // One vector per thread up to 8192 columns, two where rows are short and
  // many; about 8 waves per workgroup.  Measured (bf16, us): 8192 x 4096 with
  // MX codes 59.8 / 62.9 / 68.1 with 1 / 2 / 4 vectors, 8192 x 1024 12.9 /
  // 11.9 / 14.5, 1 x 7168 with fp8 codes 4.7 / 4.9 / 5.8.
  int nv = norm_waves(H, 1) <= 16 ? 1 : norm_waves(H, 2) <= 16 ? 2 : 4;
  if (H <= 2048 && H > 512 && T >= 4096) nv = 2;
  p.waves = norm_waves(H, nv);
  const int row = norm_row(H);
  const int rows = (p.waves >= 8 ? 1 : 8 / p.waves) * (kWave / row);
  // h and y of more than 64 MiB do not stay in the caches until the next
  // kernel reads them: stored with the non-temporal hint (8192 x 4096 with MX
  // codes 58.8 -> 54.9 us, 8192 x 7168 with an fp32 residual 142 -> 139)
  p.once = (uint64_t)T * H * (2 + (!residual ? 0 : residual_is_fp32 ? 4 : 2)) > (64ull << 20);
  const int threads = rows * (row < kWave ? row : p.waves * kWave), rt = !residual ? 0 : residual_is_fp32 ? 2 : 1;
  // a grid holds fewer than 2^32 threads: more rows go by several launches
  const int most = (int)((1u << 31) / threads) * rows;
  for (int64_t first = 0; first < T; first += most) {
    p.first = (int)first;
    const dim3 grid((unsigned)ceil_div(T - first < most ? T - p.first : most, rows));
    switch (row < kWave ? row : nv) {
      case 8: launch_norm_q<1, 8>(p, qformat, rt, grid, threads, stream); break;
      case 16: launch_norm_q<1, 16>(p, qformat, rt, grid, threads, stream); break;
      case 32: launch_norm_q<1, 32>(p, qformat, rt, grid, threads, stream); break;
      case 1: launch_norm_q<1, kWave>(p, qformat, rt, grid, threads, stream); break;
      case 2: launch_norm_q<2, kWave>(p, qformat, rt, grid, threads, stream); break;
      default: launch_norm_q<4, kWave>(p, qformat, rt, grid, threads, stream); break;
    }
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}

}  // namespace moe

extern "C" moe_status moe_rms_norm(const void* x, const void* residual, int residual_is_fp32, const void* weight,
                                   int weight_is_fp32, int T, int H, float eps, int qformat, void* h, void* y,
                                   void* q, void* s, hipStream_t stream) {
  const moe_status st = moe::norm_validate(x, residual, residual_is_fp32, weight, weight_is_fp32, T, H, eps, qformat,
                                           h, y, q, s);
  if (st != MOE_OK || T == 0) return st;
  return moe::launch_norm(x, residual, residual_is_fp32, weight, weight_is_fp32, T, H, eps, qformat, h, y, q, s,
                          stream);
}

extern "C" size_t moe_rms_norm_grad_workspace_size(int T, int H) {
  if (T < 0 || H < 1 || H > moe::kMaxNormH) return 0;
  return moe::kCtrlBytes + moe::align_up((size_t)moe::grad_shape(T, H).grid * H * sizeof(float), 256);
}

extern "C" moe_status moe_rms_norm_grad(const void* dy, const void* dh, const void* h, int h_is_fp32,
                                        const void* weight, int weight_is_fp32, int T, int H, float eps, void* dx,
                                        float* d_weight, void* workspace, size_t workspace_bytes,
                                        hipStream_t stream) {
  using namespace moe;
  const moe_status st = norm_shape(T, H, eps);
  if (st != MOE_OK) return st;
  if (h_is_fp32 < 0 || h_is_fp32 > 1 || weight_is_fp32 < 0 || weight_is_fp32 > 1) return MOE_E_INVAL;
  if (T > 0 && (!dy || !h || !weight || !dx)) return MOE_E_INVAL;
  if (d_weight) {
    if (!workspace) return MOE_E_INVAL;
    if (workspace_bytes < moe_rms_norm_grad_workspace_size(T, H)) return MOE_E_WORKSPACE;
  }
  const GradShape g = grad_shape(T, H);
  NormGradP p;
  p.dy = static_cast<const uint16_t*>(dy);
  p.dh = dh;
  p.h = h;
  p.w = weight;
  p.dx = dx;
  p.part = d_weight ? reinterpret_cast<float*>(static_cast<char*>(workspace) + kCtrlBytes) : nullptr;
  p.T = T;
  p.H = H;
  p.eps = eps;
  p.inv_h = 1.f / (float)H;
  p.w_fp32 = weight_is_fp32;
  p.waves = g.waves;
  if (T > 0) {
    switch (g.row < kWave ? g.row : g.nv) {
      case 8: launch_grad_nv<1, 8>(p, h_is_fp32, g, stream); break;
      case 16: launch_grad_nv<1, 16>(p, h_is_fp32, g, stream); break;
      case 32: launch_grad_nv<1, 32>(p, h_is_fp32, g, stream); break;
      case 1: launch_grad_nv<1, kWave>(p, h_is_fp32, g, stream); break;
      case 2: launch_grad_nv<2, kWave>(p, h_is_fp32, g, stream); break;
      default: launch_grad_nv<4, kWave>(p, h_is_fp32, g, stream); break;
    }
    MOE_CHECK_LAUNCH();
  }
  if (d_weight) {
    column_sum_kernel<<<ceil_div(H, 32), 256, 0, stream>>>(p.part, T > 0 ? g.grid : 0, H, d_weight);
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}
