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
// widths keep the wide accesses; only the last vector of a row that 8 does
// not divide goes element by element.

#include <cmath>
#include <type_traits>

#include "common.h"
#include "launch.h"
#include "quant.h"

namespace moe {

namespace {

constexpr int kMaxNormH = 32768;  // 16 waves x 4 vectors x 8 values
constexpr int kVec = 8;           // values per vector

// 8 values from element i of a row of n (zeros past its end)
__device__ __forceinline__ void load8(const uint16_t* row, int i, int n, float (&f)[8]) {
  if (i + kVec <= n) {
    u32x4_t v;
    __builtin_memcpy(&v, row + i, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = bf16_lo(v[j]);
      f[2 * j + 1] = bf16_hi(v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = i + j < n ? bf16_to_f32(row[i + j]) : 0.f;
  }
}
__device__ __forceinline__ void load8(const float* row, int i, int n, float (&f)[8]) {
  if (i + kVec <= n) {
    f32x4_t a, b;
    __builtin_memcpy(&a, row + i, 16);
    __builtin_memcpy(&b, row + i + 4, 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[j] = a[j];
      f[j + 4] = b[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = i + j < n ? row[i + j] : 0.f;
  }
}
__device__ __forceinline__ void store8(uint16_t* row, int i, int n, const float (&f)[8]) {
  u32x4_t v;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = cvt_bf16x2(f[2 * j], f[2 * j + 1]);
  if (i + kVec <= n) {
    __builtin_memcpy(row + i, &v, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) row[i + j] = (uint16_t)(v[j / 2] >> (16 * (j & 1)));
  }
}
__device__ __forceinline__ void store8(float* row, int i, int n, const float (&f)[8]) {
  if (i + kVec <= n) {
    const f32x4_t a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
    __builtin_memcpy(row + i, &a, 16);
    __builtin_memcpy(row + i + 4, &b, 16);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i + j < n) row[i + j] = f[j];
  }
}
__device__ __forceinline__ void load_weight8(const void* w, int w_fp32, int i, int n, float (&f)[8]) {
  if (w_fp32)
    load8(static_cast<const float*>(w), i, n, f);
  else
    load8(static_cast<const uint16_t*>(w), i, n, f);
}

struct NormP {
  const uint16_t* x;
  const void* res;
  const void* w;
  void* h;      // optional, the residual's type
  uint16_t* y;  // optional
  uint8_t* q;   // QF != 0
  void* s;
  int T, H;
  float eps, inv_h;
  int w_fp32;
  int waves;  // waves per row
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

// RT: residual type, 0 none, 1 bf16, 2 fp32.  NV vectors per thread, `waves`
// waves per row; a workgroup of 256 threads takes 4 / waves rows where a row
// has fewer than 4 waves, else one row.
template <int NV, int QF, int RT>
__global__ void norm_kernel(NormP p) {
  const int lanes = p.waves * kWave;  // threads per row
  const int sub = threadIdx.x / lanes, tid = threadIdx.x - sub * lanes;
  const int rows = blockDim.x / lanes;
  const size_t row = (size_t)blockIdx.x * rows + sub;
  const bool live = row < (size_t)p.T;
  float h[NV][8];
  float ss = 0.f;
  if (live) {
    const uint16_t* x = p.x + row * p.H;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * lanes + tid) * kVec;
      load8(x, i, p.H, h[v]);
    }
    if (RT != 0) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int i = (v * lanes + tid) * kVec;
        float r[8];
        if (RT == 1)
          load8(static_cast<const uint16_t*>(p.res) + row * p.H, i, p.H, r);
        else
          load8(static_cast<const float*>(p.res) + row * p.H, i, p.H, r);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[v][j] += r[j];
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += h[v][j] * h[v][j];
  }
  float w[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) load_weight8(p.w, p.w_fp32, (v * lanes + tid) * kVec, p.H, w[v]);
  ss = wave_sum_u(ss);
  if (p.waves > 1) {
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
    const int i = (v * lanes + tid) * kVec;
    if (RT != 0 && p.h && i < p.H) {
      if (RT == 1)
        store8(static_cast<uint16_t*>(p.h) + row * p.H, i, p.H, h[v]);
      else
        store8(static_cast<float*>(p.h) + row * p.H, i, p.H, h[v]);
    }
    float y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = h[v][j] * r * w[v][j];
    if (p.y && i < p.H) store8(p.y + row * p.H, i, p.H, y);
    if (QF != 0) quant8<QF>(p, row, i, y);
  }
}

template <int NV, int QF>
void launch_norm_rt(const NormP& p, int rt, dim3 grid, int threads, hipStream_t s) {
  switch (rt) {
    case 0: norm_kernel<NV, QF, 0><<<grid, threads, 0, s>>>(p); break;
    case 1: norm_kernel<NV, QF, 1><<<grid, threads, 0, s>>>(p); break;
    default: norm_kernel<NV, QF, 2><<<grid, threads, 0, s>>>(p); break;
  }
}
template <int NV>
void launch_norm_q(const NormP& p, int qf, int rt, dim3 grid, int threads, hipStream_t s) {
  switch (qf) {
    case 0: launch_norm_rt<NV, 0>(p, rt, grid, threads, s); break;
    case 1: launch_norm_rt<NV, 1>(p, rt, grid, threads, s); break;
    default: launch_norm_rt<NV, 2>(p, rt, grid, threads, s); break;
  }
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
};

// One workgroup per row at a time, rows blockIdx.x, + gridDim.x, ...; a
// thread keeps the same columns for every row, so the weight and the weight
// gradient's sums stay in its registers.
template <int NV, bool HF32>
__global__ void norm_grad_kernel(NormGradP p) {
  typedef typename std::conditional<HF32, float, uint16_t>::type HT;
  const int lanes = blockDim.x, nw = lanes / kWave;
  __shared__ float part[2][2][16];
  float w[NV][8], dw[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    load_weight8(p.w, p.w_fp32, (v * lanes + threadIdx.x) * kVec, p.H, w[v]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[v][j] = 0.f;
  }
  int flip = 0;
  for (size_t row = blockIdx.x; row < (size_t)p.T; row += gridDim.x, flip ^= 1) {
    const size_t at = row * p.H;
    float h[NV][8], dy[NV][8];
    float ss = 0.f, gh = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * lanes + threadIdx.x) * kVec;
      load8(static_cast<const HT*>(p.h) + at, i, p.H, h[v]);
      load8(p.dy + at, i, p.H, dy[v]);
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss += h[v][j] * h[v][j];
        gh += dy[v][j] * w[v][j] * h[v][j];
      }
    ss = wave_sum_u(ss);
    gh = wave_sum_u(gh);
    if (nw > 1) {
      if ((threadIdx.x & 63) == 0) {
        part[flip][0][threadIdx.x >> 6] = ss;
        part[flip][1][threadIdx.x >> 6] = gh;
      }
      // one barrier a row: a wave writes the other half next time, and this
      // half again only after the next row's barrier
      __syncthreads();
      ss = gh = 0.f;
      for (int i = 0; i < nw; ++i) {
        ss += part[flip][0][i];
        gh += part[flip][1][i];
      }
    }
    const float r = rsqrtf(ss * p.inv_h + p.eps);
    const float c = r * r * r * (gh * p.inv_h);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * lanes + threadIdx.x) * kVec;
      float d[8];
      if (p.dh) load8(static_cast<const HT*>(p.dh) + at, i, p.H, d);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float n = r * (dy[v][j] * w[v][j]) - h[v][j] * c;
        d[j] = p.dh ? n + d[j] : n;
        dw[v][j] += dy[v][j] * (h[v][j] * r);
      }
      if (i < p.H) store8(static_cast<HT*>(p.dx) + at, i, p.H, d);
    }
  }
  if (p.part) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int i = (v * lanes + threadIdx.x) * kVec;
      if (i < p.H) store8(p.part + (size_t)blockIdx.x * p.H, i, p.H, dw[v]);
    }
  }
}

// out[c] = sum of n rows of part[., c], in a fixed order: 4 slices of the
// rows per workgroup of 64 columns, then the slices.  n = 0: zeros.
__global__ __launch_bounds__(256) void column_sum_kernel(const float* part, int n, int H, float* out) {
  __shared__ float s[16][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 15) * 4, slice = threadIdx.x >> 4;
  f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
  for (int r = slice; r < n; r += 16) {
    const float* row = part + (size_t)r * H;
    if (c + 4 <= H) {
      f32x4_t v;
      __builtin_memcpy(&v, row + c, 16);
      acc += v;
    } else {
      for (int j = 0; j < 4; ++j)
        if (c + j < H) acc[j] += row[c + j];
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) s[slice][(threadIdx.x & 15) * 4 + j] = acc[j];
  __syncthreads();
  const int col = blockIdx.x * 64 + threadIdx.x;
  if (threadIdx.x < 64 && col < H) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += s[i][threadIdx.x];
    out[col] = t;
  }
}

// Rows in flight of the backward pass; each leaves one fp32 row of weight
// gradient sums.
int norm_grad_groups(int T, int waves) {
  const int cap = 256 * (16 / waves > 4 ? 4 : 16 / waves > 0 ? 16 / waves : 1);
  return T < cap ? T : cap;
}
int norm_waves(int H, int nv) { return ceil_div(H, kWave * kVec * nv); }
int norm_grad_nv(int H) {
  if (norm_waves(H, 1) <= 1) return 1;
  return norm_waves(H, 2) <= 8 ? 2 : 4;
}

template <int NV>
void launch_grad_nv(const NormGradP& p, int h_fp32, int grid, int threads, hipStream_t s) {
  if (h_fp32)
    norm_grad_kernel<NV, true><<<grid, threads, 0, s>>>(p);
  else
    norm_grad_kernel<NV, false><<<grid, threads, 0, s>>>(p);
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
  const int nv = norm_waves(H, 1) <= 16 && T < 256 ? 1 : norm_waves(H, 2) <= 8 ? 2 : 4;
  p.waves = norm_waves(H, nv);
  if (p.waves == 3) p.waves = 4;  // rows of a workgroup: 4 / waves
  const int rows = p.waves >= 4 ? 1 : 4 / p.waves;
  const dim3 grid((unsigned)ceil_div(T, rows));
  if ((uint64_t)grid.x * rows * p.waves * kWave > 0xFFFFFFFFull) return MOE_E_UNSUPPORTED;  // HIP's limit of a grid
  const int threads = rows * p.waves * kWave, rt = !residual ? 0 : residual_is_fp32 ? 2 : 1;
  switch (nv) {
    case 1: launch_norm_q<1>(p, qformat, rt, grid, threads, stream); break;
    case 2: launch_norm_q<2>(p, qformat, rt, grid, threads, stream); break;
    default: launch_norm_q<4>(p, qformat, rt, grid, threads, stream); break;
  }
  MOE_CHECK_LAUNCH();
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
  const int waves = moe::norm_waves(H, moe::norm_grad_nv(H));
  return moe::kCtrlBytes + moe::align_up((size_t)moe::norm_grad_groups(T, waves) * H * sizeof(float), 256);
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
  const int nv = norm_grad_nv(H), waves = norm_waves(H, nv), grid = norm_grad_groups(T, waves);
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
  if (T > 0) {
    switch (nv) {
      case 1: launch_grad_nv<1>(p, h_is_fp32, grid, waves * kWave, stream); break;
      case 2: launch_grad_nv<2>(p, h_is_fp32, grid, waves * kWave, stream); break;
      default: launch_grad_nv<4>(p, h_is_fp32, grid, waves * kWave, stream); break;
    }
    MOE_CHECK_LAUNCH();
  }
  if (d_weight) {
    column_sum_kernel<<<ceil_div(H, 64), 256, 0, stream>>>(p.part, grid, H, d_weight);
    MOE_CHECK_LAUNCH();
  }
  return MOE_OK;
}
