// moe_gate_grad: the router's gradient from the logits to the hidden states
// and the gate,
//
//   dx[t, h]     = sum_e d_logits[t, e] gate[e, h] (+ dx_in[t, h])
//   d_gate[e, h] = sum_t d_logits[t, e] x[t, h]
//
// on the matrix cores.  The fp32 operands are split into bf16 planes that add
// up to them (hi: the value with its low 16 bits cleared, mid and lo: the
// same for what remains), every product of two planes is exact in fp32 and
// v_mfma_f32_16x16x32_bf16 accumulates in fp32:
//  * d_gate takes all three planes of d_logits against the bf16 x: the sums
//    are fp32 sums of exact products.
//  * dx is rounded to bf16 (2^-9 relative), so it takes two planes of
//    d_logits and of an fp32 gate, without the product of the two mid
//    planes: what is left out is below 2^-15 of each product.  A bf16 gate
//    is its own hi plane.
//
// A first launch writes the planes in the order the MFMA operands read them:
// fragments of 16 rows x 32 K values, 1 KiB each, lane l of a wave holding
// row l % 16, K values 8 (l / 16) .. + 7 at byte 16 l.  A fragment is then
// one contiguous copy into LDS and one conflict-free 16-byte read per lane.

#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kFrag = 512;  // bf16 values of a fragment (1 KiB)
constexpr int kMaxMf = 4;   // 16-row fragments of experts per wave of the d_gate kernel

typedef __attribute__((address_space(1))) void gmem_t;
typedef __attribute__((address_space(3))) void lmem_t;

// 64 lanes x 16 contiguous bytes from g + 16 lane to the wave-uniform LDS
// address + 16 lane
__device__ __forceinline__ void copy_frag(const uint16_t* g, uint16_t* lds, int lane) {
  __builtin_amdgcn_global_load_lds((gmem_t*)(g + lane * 8), (lmem_t*)lds, 16, 0, 0);
}

// v = hi + mid + lo, each a bf16 (the upper 16 bits of an fp32); a value that
// is not finite is its own hi plane
__device__ __forceinline__ void split3(float v, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
  const uint32_t u = __float_as_uint(v);
  const uint32_t h = u & 0xFFFF0000u;
  const float r = v - __uint_as_float(h);
  const uint32_t m = __float_as_uint(r) & 0xFFFF0000u;
  const float l = r - __uint_as_float(m);
  hi = h >> 16;
  mid = m >> 16;
  lo = __float_as_uint(l) >> 16;
  if ((u & 0x7F800000u) == 0x7F800000u) {
    hi |= (u & 0x7FFFFFu) ? 0x40u : 0u;
    mid = lo = 0u;
  }
}

struct GateGradP {
  const uint16_t* x;
  const void* gate;
  const float* dl;
  const uint16_t* dx_in;
  uint16_t* dx;
  float* d_gate;
  int T, H, E, gate_fp32;
  int Kf;       // K fragments of dx: E / 32 rounded up
  int tiles_t;  // 128-token tiles
  int nt32;     // K steps of d_gate: T / 32 rounded up
  int Ef;       // 16-expert fragments of d_gate, all M tiles
  int mtiles, mf;  // M tiles of d_gate, of 4 mf fragments each
  int splits, steps;  // K splits of d_gate, steps of each
  uint16_t* dxa;  // [tiles_t][Kf][2][8][kFrag]   d_logits, rows t
  uint16_t* dxb;  // [H / 128][Kf][1 or 2][8][kFrag]  gate, rows h
  uint16_t* dga;  // [nt32][3][Ef][kFrag]  d_logits, rows e
  float* part;    // [splits][E][H]
};

// d_logits -> its planes for both products: a workgroup takes 32 tokens x 64
// experts through LDS.
__global__ __launch_bounds__(256) void split_logits_kernel(GateGradP p) {
  __shared__ float tile[32][65];
  const int t0 = blockIdx.x * 32, e0 = blockIdx.y * 64;
  {
    const int t = t0 + threadIdx.x / 8, e = e0 + (threadIdx.x % 8) * 8;
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = t < p.T && e + i < p.E ? p.dl[(size_t)t * p.E + e + i] : 0.f;
      tile[threadIdx.x / 8][(threadIdx.x % 8) * 8 + i] = v;
      split3(v, h[i], m[i], l[i]);
    }
    if (p.dxa && e / 32 < p.Kf) {  // t0 < 128 tiles_t by the grid
      const int lane = t % 16 + 16 * ((e % 32) / 8);
      uint16_t* at = p.dxa + (((size_t)(t / 128) * p.Kf + e / 32) * 2 * 8 + (t % 128) / 16) * kFrag + lane * 8;
      *reinterpret_cast<u32x4_t*>(at) =
          u32x4_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
      *reinterpret_cast<u32x4_t*>(at + 8 * kFrag) =
          u32x4_t{m[0] | (m[1] << 16), m[2] | (m[3] << 16), m[4] | (m[5] << 16), m[6] | (m[7] << 16)};
    }
  }
  __syncthreads();
  const int c = threadIdx.x % 64, tg = threadIdx.x / 64, e = e0 + c;
  if (p.dga && e / 16 < p.Ef && (int)blockIdx.x < p.nt32) {
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(tile[tg * 8 + i][c], h[i], m[i], l[i]);
    const int lane = e % 16 + 16 * tg;
    uint16_t* at = p.dga + ((size_t)blockIdx.x * 3 * p.Ef + e / 16) * kFrag + lane * 8;
    const size_t plane = (size_t)p.Ef * kFrag;
    *reinterpret_cast<u32x4_t*>(at) =
        u32x4_t{h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16), h[6] | (h[7] << 16)};
    *reinterpret_cast<u32x4_t*>(at + plane) =
        u32x4_t{m[0] | (m[1] << 16), m[2] | (m[3] << 16), m[4] | (m[5] << 16), m[6] | (m[7] << 16)};
    *reinterpret_cast<u32x4_t*>(at + 2 * plane) =
        u32x4_t{l[0] | (l[1] << 16), l[2] | (l[3] << 16), l[4] | (l[5] << 16), l[6] | (l[7] << 16)};
  }
}

// The gate's planes with rows h: a workgroup takes 32 experts x 64 columns.
__global__ __launch_bounds__(256) void split_gate_kernel(GateGradP p) {
  __shared__ float tile[32][65];
  const int e0 = blockIdx.x * 32, h0 = blockIdx.y * 64;
  {
    const int e = e0 + threadIdx.x / 8, h = h0 + (threadIdx.x % 8) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = 0.f;
      if (e < p.E) {
        const size_t at = (size_t)e * p.H + h + i;
        v = p.gate_fp32 ? static_cast<const float*>(p.gate)[at]
                        : bf16_to_f32(static_cast<const uint16_t*>(p.gate)[at]);
      }
      tile[threadIdx.x / 8][(threadIdx.x % 8) * 8 + i] = v;
    }
  }
  __syncthreads();
  const int c = threadIdx.x % 64, eg = threadIdx.x / 64, h = h0 + c;
  uint32_t a[8], m[8], l[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) split3(tile[eg * 8 + i][c], a[i], m[i], l[i]);
  const int planes = p.gate_fp32 ? 2 : 1, lane = h % 16 + 16 * eg;
  uint16_t* at =
      p.dxb + (((size_t)(h / 128) * p.Kf + blockIdx.x) * planes * 8 + (h % 128) / 16) * kFrag + lane * 8;
  *reinterpret_cast<u32x4_t*>(at) =
      u32x4_t{a[0] | (a[1] << 16), a[2] | (a[3] << 16), a[4] | (a[5] << 16), a[6] | (a[7] << 16)};
  if (planes == 2)
    *reinterpret_cast<u32x4_t*>(at + 8 * kFrag) =
        u32x4_t{m[0] | (m[1] << 16), m[2] | (m[3] << 16), m[4] | (m[5] << 16), m[6] | (m[7] << 16)};
}

__device__ __forceinline__ bf16x8_t frag(const uint16_t* lds, int lane) {
  return *reinterpret_cast<const bf16x8_t*>(lds + lane * 8);
}

// dx: 128 columns x 128 tokens per workgroup, 2 x 2 waves of 64 x 64.  The
// gate is the MFMA's row operand, so a lane holds 4 consecutive columns of a
// token.  GP planes of the gate.
template <int GP>
__global__ __launch_bounds__(256) void dx_kernel(GateGradP p) {
  constexpr int AF = 2 * 8, BF = GP * 8;  // fragments per K step
  __shared__ __align__(16) uint16_t lds[2][(AF + BF) * kFrag];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wh = wave & 1, wt = wave >> 1;
  const uint16_t* ga = nullptr;
  const uint16_t* gb = p.dxb + (size_t)blockIdx.x * p.Kf * BF * kFrag;
  auto copy = [&](int s) {
    uint16_t* to = lds[s & 1];
    for (int f = wave; f < AF + BF; f += 4)
      copy_frag(f < AF ? ga + ((size_t)s * AF + f) * kFrag : gb + ((size_t)s * BF + f - AF) * kFrag, to + f * kFrag,
                lane);
  };
  for (int ty = blockIdx.y; ty < p.tiles_t; ty += gridDim.y) {
    ga = p.dxa + (size_t)ty * p.Kf * AF * kFrag;
    f32x4_t acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    copy(0);
    for (int s = 0; s < p.Kf; ++s) {
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

// d_gate: 64 MF experts x 128 columns per workgroup and K split, 4 x 2 waves
// of 16 MF x 64.  x comes with its rows along K: a thread loads 8 columns of
// a token and stores them into the fragments one value at a time.  The 16-byte slot of a
// fragment is XORed with the fragment's number, so that the 16 threads of a
// token, which write to 8 fragments, meet different banks.
template <int MF>
__global__ __launch_bounds__(512) void d_gate_kernel(GateGradP p) {
  constexpr int AF = 3 * 4 * MF;
  __shared__ __align__(16) uint16_t lds[2][(AF + 8) * kFrag];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wm = wave & 3, wn = wave >> 2;
  const int h0 = blockIdx.x * 128, mt = blockIdx.y;
  const int s0 = blockIdx.z * p.steps, s1 = min(p.nt32, s0 + p.steps);
  auto copy_a = [&](int s, int buf) {
    for (int f = wave; f < AF; f += 8) {
      const int plane = f / (4 * MF), i = f % (4 * MF);
      copy_frag(p.dga + (((size_t)s * 3 + plane) * p.Ef + mt * 4 * MF + i) * kFrag, lds[buf] + f * kFrag, lane);
    }
  };
  const int xt = tid / 16, xh = tid % 16;  // this thread's token and 8 columns of a step
  auto load_x = [&](int s) {
    const int t = s * 32 + xt;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (t < p.T) v = *reinterpret_cast<const u32x4_t*>(p.x + (size_t)t * p.H + h0 + xh * 8);
    return v;
  };
  auto store_x = [&](const u32x4_t& v, int buf) {
    uint16_t* B = lds[buf] + AF * kFrag + (xh / 2) * kFrag;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int slot = ((xt / 8) * 16 + (xh & 1) * 8 + i) ^ (xh / 2);
      B[slot * 8 + xt % 8] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
    }
  };
  f32x4_t acc[MF][4];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  u32x4_t xv = {0u, 0u, 0u, 0u};
  if (s0 < s1) {
    copy_a(s0, 0);
    store_x(load_x(s0), 0);
  }
  for (int s = s0; s < s1; ++s) {
    const int buf = (s - s0) & 1;
    if (s + 1 < s1) xv = load_x(s + 1);
    __syncthreads();  // step s is in LDS; the other buffer is read
    if (s + 1 < s1) copy_a(s + 1, buf ^ 1);
    const uint16_t* A = lds[buf];
    const uint16_t* B = A + AF * kFrag;
    bf16x8_t b[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b[j] = frag(B + (wn * 4 + j) * kFrag, lane ^ (wn * 4 + j));
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const bf16x8_t a = frag(A + (q * 4 * MF + wm * MF + i) * kFrag, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = mfma_16x16x32_bf16(a, b[j], acc[i][j]);
      }
    if (s + 1 < s1) store_x(xv, buf ^ 1);
  }
  float* out = p.splits > 1 ? p.part + (size_t)blockIdx.z * p.E * p.H : p.d_gate;
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int e = (mt * 4 * MF + wm * MF + i) * 16 + 4 * (lane / 16) + r;
      if (e >= p.E) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) out[(size_t)e * p.H + h0 + wn * 64 + j * 16 + lane % 16] = acc[i][j][r];
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
  p.mtiles = ceil_div(E, 64 * kMaxMf);
  p.mf = ceil_div(ceil_div(E, p.mtiles), 64);
  p.Ef = p.mtiles * 4 * p.mf;
  // about one workgroup per CU, at least 4 steps each
  const int tiles = (H / 128) * p.mtiles;
  int splits = 256 / tiles;
  const int most = ceil_div(p.nt32, 4);
  if (splits > most) splits = most;
  if (splits < 1) splits = 1;
  p.steps = ceil_div(p.nt32 > 0 ? p.nt32 : 1, splits);
  p.splits = ceil_div(p.nt32 > 0 ? p.nt32 : 1, p.steps);
  size_t off = kCtrlBytes;  // the control block stays as it is
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  const size_t fb = (size_t)kFrag * 2;
  L.dxa = take((size_t)p.tiles_t * p.Kf * 16 * fb);
  L.dxb = take((size_t)(H / 128) * p.Kf * 16 * fb);
  L.dga = take((size_t)p.nt32 * 3 * p.Ef * fb);
  L.part = take(p.splits > 1 ? (size_t)p.splits * E * H * sizeof(float) : 0);
  L.total = off;
  return L;
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
  split_logits_kernel<<<dim3((unsigned)p.tiles_t * 4, (unsigned)ceil_div(cols, 64)), 256, 0, stream>>>(p);
  MOE_CHECK_LAUNCH();
  if (dx) {
    split_gate_kernel<<<dim3((unsigned)p.Kf, (unsigned)(H / 64)), 256, 0, stream>>>(p);
    MOE_CHECK_LAUNCH();
    const dim3 grid((unsigned)(H / 128), (unsigned)(p.tiles_t < 65535 ? p.tiles_t : 65535));
    if (gate_is_fp32)
      dx_kernel<2><<<grid, 256, 0, stream>>>(p);
    else
      dx_kernel<1><<<grid, 256, 0, stream>>>(p);
    MOE_CHECK_LAUNCH();
  }
  if (d_gate) {
    const dim3 grid((unsigned)(H / 128), (unsigned)p.mtiles, (unsigned)p.splits);
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
