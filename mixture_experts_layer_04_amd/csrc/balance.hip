// moe_balance_loss and moe_route_grad: the router's training side.
//
// With sc the scores of a token's logits (softmax, sigmoid or
// sqrt(softplus), as moe_route takes them), p = sc / sum(sc) (softmax: p =
// sc), c[s, e] the assignments of sequence s to expert e, n_s its tokens and
// S' the sequences that have any:
//
//   balance = 1/S' sum_s sum_e (E c[s,e] / (k n_s)) (1/n_s sum_t p[t,e])
//   z       = 1/N sum_t logsumexp(l_t)^2            (N = sum_s n_s)
//
// Gradient to the logits, with gb = d_balance E c / (k n_s^2 S') (the counts
// carry no gradient) and gw the gradient of the routing weights w_j =
// scale sc_j / (sum_sel sc + 1e-20) (or scale sc_j) on the scores:
//
//   softmax:    d = p (g - sum p g),  g = gb + gw
//   the others: d = sc' ((gb - sum p gb) / sum(sc) + gw)
//   both:       d += d_z 2/N lse softmax(l)
//
// A token's E logits sit in the registers of 16 neighbouring lanes (32 or 64
// for many experts), so the row sums are four DPP steps and a wave holds four
// tokens.  The column sums of the loss are accumulated per lane over the
// tokens of a run, then added across lanes, waves and runs in a fixed order;
// only integer counts use atomics, so every result is the same in every run.
//
// Both read their logits once.  Measured: the loss of 131072 x 256 sigmoid
// scores in 37 sequences 35.8 us, 28 of them the pass over the 134 MB of
// logits (4.8 TB/s), the gradient of 65536 x 128 softmax scores 15.2 us (4.7
// TB/s, as much held by its 84 vector instructions a token as by memory).

#include <cmath>

#include "common.h"
#include "launch.h"

namespace moe {

namespace {

constexpr int kMaxSeqs = 1 << 20;
constexpr float kTiny = 1e-20f;  // the guard of the router's own renormalisation
constexpr float kNegInf = -__builtin_huge_valf();

typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));

// 4 logits from expert e on; -inf (a score of zero) past the last expert.
// ONCE: with the hint that nobody reads them again soon.
template <bool ONCE>
__device__ __forceinline__ void load4(const float* row, int e, int E, float* l) {
  if (e + 4 <= E) {
    const f32x4_any_t* at = reinterpret_cast<const f32x4_any_t*>(row + e);
    f32x4_t v;
    if constexpr (ONCE)
      v = __builtin_nontemporal_load(at);
    else
      v = *at;
#pragma unroll
    for (int j = 0; j < 4; ++j) l[j] = v[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) l[j] = e + j < E ? row[e + j] : kNegInf;
  }
}

// exp2, log2, 1 / x and sqrt are the hardware's (about 1 ulp each); the
// exponent l log2(e) - m log2(e) is one fma.
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float rcp_(float x) { return __builtin_amdgcn_rcpf(x); }

// log(1 + x) for x >= 0: the rounding of 1 + x is put back where it counts
// (below x = 1; above, it is within 1 ulp of the logarithm)
__device__ __forceinline__ float log1p_(float x) {
  const float w = 1.f + x;
  return __builtin_amdgcn_logf(w) * kLn2 + (x < 1.f ? x - (w - 1.f) : 0.f);
}

// The scores of a row from a = exp(l - m), m its largest logit, which the
// softmax and the z loss need anyway: with c = exp(-m), sigmoid(l) = a /
// (a + c), its complement c / (a + c) and exp(l) = a / c, one exponential
// for all.  Holds while c neither overflows nor vanishes, |m| <= 60 (scores
// below exp(m - 87) become 0); other rows take the functions of l itself,
// with t = exp(-|l|) <= 1.
constexpr float kSafeMax = 60.f;
struct RowScale {
  float c, ec;  // exp(-m), exp(m)
  bool safe;
};
__device__ __forceinline__ RowScale row_scale(float m) {
  return RowScale{exp2_(-m * kLog2e), exp2_(m * kLog2e), fabsf(m) <= kSafeMax};
}
template <int SC>
__device__ __forceinline__ float score(float a, const RowScale& r) {
  if (SC == MOE_SIGMOID) return a * rcp_(a + r.c);
  return __builtin_amdgcn_sqrtf(log1p_(a * r.ec));
}
template <int SC>
__device__ __forceinline__ float score_and_slope(float a, const RowScale& r, float& slope) {
  const float q = rcp_(a + r.c), sig = a * q;
  if (SC == MOE_SIGMOID) {
    slope = sig * (r.c * q);
    return sig;
  }
  const float s = __builtin_amdgcn_sqrtf(log1p_(a * r.ec));
  slope = s > 0.f ? sig * 0.5f * rcp_(s) : 0.f;
  return s;
}
template <int SC>
__device__ __forceinline__ float far_score_and_slope(float l, float& slope) {
  const float t = expf(-fabsf(l)), r = 1.f / (1.f + t);
  if (SC == MOE_SIGMOID) {
    slope = t * r * r;
    return l >= 0.f ? r : t * r;
  }
  const float s = sqrtf(fmaxf(l, 0.f) + log1pf(t));
  slope = s > 0.f ? (l >= 0.f ? r : t * r) / (2.f * s) : 0.f;
  return s;
}

// Sequence boundaries are read on the device and clamped to the batch, so
// that no value of theirs leads outside a buffer.
__device__ __forceinline__ int seq_at(const int32_t* off, int s, int T) {
  const int v = off[s];
  return v < 0 ? 0 : v > T ? T : v;
}
// first s of [0, S) whose end lies past row t (S - 1 if none does)
__device__ __forceinline__ int seq_of(const int32_t* off, int S, int T, int t) {
  int lo = 0, hi = S - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_at(off, mid + 1, T) > t)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

struct BalanceP {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* off;
  int T, E, k, ks, S;
  int chunk, chunks;  // rows per workgroup, and how many
  int Ep;             // E padded to 64: row length of the partial sums
  // per piece (a run of one sequence's rows inside one chunk; piece (c, s)
  // has slot c + s, no two pieces the same one)
  float* psum;    // [slots][Ep]
  int32_t* csum;  // [slots][Ep]
  float* zsum;    // [slots]
  int32_t* nsum;  // [slots]
  // per sequence
  float* dot;    // [S][Ep / 64]
  float* zseq;   // [S]
  int32_t* nseq;  // [S]: the tokens output
  float* losses;
  int32_t* counts;
  float* probs;
};

// One workgroup per chunk of rows: the pieces of the sequences in it.
// Token t's logits, its slots' ids and its mask are on their way while the
// tokens before it are worked on (logits and ids one token of the lane group
// ahead, the mask two).
// ALL: one workgroup for a small batch of one sequence, which writes the
// results itself (one launch instead of three).
template <int LANES, int NV, int SC, int NT, bool ALL, bool ONCE>
__global__ __launch_bounds__(NT) void balance_kernel(BalanceP p) {
  constexpr int V = 4 * NV, GROUPS = NT / LANES, WAVES = NT / kWave;
  extern __shared__ float lds[];  // [WAVES][Ep] column sums per wave, then [Ep] counts
  int32_t* hist = reinterpret_cast<int32_t*>(lds + WAVES * p.Ep);
  __shared__ float zw[WAVES], dw[WAVES];
  __shared__ int nw[WAVES];
  const int j = threadIdx.x % LANES, g = threadIdx.x / LANES, wave = threadIdx.x >> 6;
  const int a = blockIdx.x * p.chunk, b = min(p.T, a + p.chunk);
  int s = p.off ? seq_of(p.off, p.S, p.T, a) : 0;
  for (; s < p.S; ++s) {
    const int lo = p.off ? max(a, seq_at(p.off, s, p.T)) : a;
    const int hi = p.off ? min(b, seq_at(p.off, s + 1, p.T)) : b;
    if (!ALL && lo >= b) break;
    if (!ALL && lo >= hi) continue;
    for (int e = threadIdx.x; e < p.Ep; e += NT) hist[e] = 0;
    __syncthreads();
    float acc[V], z = 0.f;
    int n = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    auto live = [&](int t) { return t < hi && (!p.mask || p.mask[t]); };
    float l[V], ln[V];
    int id = -1, idn = -1;
    auto load = [&](int t, bool on, float(&to)[V], int& slot) {
      slot = -1;
      if (!on) return;
      if (j < p.k) slot = p.ids[(size_t)t * p.ks + j];
#pragma unroll
      for (int v = 0; v < NV; ++v) load4<ONCE>(p.logits + (size_t)t * p.E, (v * LANES + j) * 4, p.E, to + 4 * v);
    };
    bool on = live(lo + g), next = live(lo + g + GROUPS);
    load(lo + g, on, l, id);
    for (int t = lo + g; t < hi; t += GROUPS) {
      load(t + GROUPS, next, ln, idn);
      const bool after = live(t + 2 * GROUPS);
      if (on) {
        if (id >= 0 && id < p.E) atomicAdd(&hist[id], 1);
        float m = kNegInf;
#pragma unroll
        for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
        m = group_max<LANES>(m);
        if (m == kNegInf) m = 0.f;  // every logit -inf: the sum below is zero
        const float ml = m * kLog2e;
        float e[V], es = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          e[i] = exp2_(fmaf(l[i], kLog2e, -ml));
          es += e[i];
        }
        es = group_sum<LANES>(es);
        float tot = es;
        if (SC != MOE_SOFTMAX) {
          const RowScale r = row_scale(m);
          tot = 0.f;
          if (r.safe) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              e[i] = score<SC>(e[i], r);
              tot += e[i];
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              float slope;
              e[i] = far_score_and_slope<SC>(l[i], slope);
              tot += e[i];
            }
          }
          tot = group_sum<LANES>(tot) + kTiny;
        }
        const float inv = tot == 0.f ? 0.f : rcp_(tot);
        const float lse = es == 0.f ? 0.f : (ml + __builtin_amdgcn_logf(es)) * kLn2;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = fmaf(e[i], inv, acc[i]);
        z += lse * lse;
        ++n;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) l[i] = ln[i];
      id = idn;
      on = next;
      next = after;
    }
#pragma unroll
    for (int off = LANES; off < kWave; off *= 2) {  // the wave's tokens
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += __shfl_xor(acc[i], off, kWave);
      z += __shfl_xor(z, off, kWave);
      n += __shfl_xor(n, off, kWave);
    }
    if ((threadIdx.x & 63) < LANES) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int e = (v * LANES + j) * 4;
        if (e < p.Ep)
          *reinterpret_cast<f32x4_t*>(lds + wave * p.Ep + e) =
              f32x4_t{acc[4 * v], acc[4 * v + 1], acc[4 * v + 2], acc[4 * v + 3]};
      }
      if (j == 0) {
        zw[wave] = z;
        nw[wave] = n;
      }
    }
    __syncthreads();
    z = 0.f;
    n = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      z += zw[w];
      n += nw[w];
    }
    const size_t slot = (size_t)blockIdx.x + s;
    float dot = 0.f;
    for (int e = threadIdx.x; e < p.Ep; e += NT) {
      float P = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) P += lds[w * p.Ep + e];
      const int c = hist[e];
      if (!ALL) {
        p.psum[slot * p.Ep + e] = P;
        p.csum[slot * p.Ep + e] = c;
      } else if (e < p.E) {
        P = n > 0 ? P / (float)n : 0.f;
        p.probs[e] = P;
        p.counts[e] = c;
        dot += n > 0 ? (float)c / (float)n * ((float)p.E / (float)p.k) * P : 0.f;
      }
    }
    if (!ALL) {
      if (threadIdx.x == 0) {
        p.zsum[slot] = z;
        p.nsum[slot] = n;
      }
    } else {
      dot = wave_sum(dot);
      if ((threadIdx.x & 63) == 0) dw[wave] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        dot = 0.f;
        for (int w = 0; w < WAVES; ++w) dot += dw[w];
        p.losses[0] = dot;
        p.losses[1] = n > 0 ? z / (float)n : 0.f;
        p.nseq[0] = p.nseq[1] = n;
        p.nseq[2] = n > 0;
      }
    }
    __syncthreads();
  }
}

// Adds the pieces of sequence s for the 64 experts of a tile (NT / 16 slices
// of the pieces, then the slices) and writes its counts and mean
// probabilities; in wave 0, dot: the tile's share of sum_e (E c / (k n)) P.
template <int NT>
struct SeqSums {
  float ps[NT / 16][64];
  int32_t cs[NT / 16][64];
  float zs[NT / kWave];
  int ns[NT / kWave];
};
template <int NT>
__device__ __forceinline__ void add_pieces(const BalanceP& p, SeqSums<NT>& sh, int s, int tile, float& dot, float& z,
                                           int& n) {
  const int lo = p.off ? seq_at(p.off, s, p.T) : 0, hi = p.off ? seq_at(p.off, s + 1, p.T) : p.T;
  const int first = lo / p.chunk, last = hi > lo ? (hi - 1) / p.chunk : first - 1;
  const int quad = threadIdx.x & 15, slice = threadIdx.x >> 4;
  f32x4_t pa = {0.f, 0.f, 0.f, 0.f};
  i32x4_t ca = {0, 0, 0, 0};
  for (int c = first + slice; c <= last; c += NT / 16) {
    const size_t at = (size_t)(c + s) * p.Ep + tile * 64 + quad * 4;
    pa += *reinterpret_cast<const f32x4_t*>(p.psum + at);
    ca += *reinterpret_cast<const i32x4_t*>(p.csum + at);
  }
  z = 0.f;
  n = 0;
  for (int c = first + (int)threadIdx.x; c <= last; c += NT) {
    z += p.zsum[c + s];
    n += p.nsum[c + s];
  }
  z = wave_sum(z);
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) n += __shfl_xor(n, off, kWave);
  if ((threadIdx.x & 63) == 0) {
    sh.zs[threadIdx.x >> 6] = z;
    sh.ns[threadIdx.x >> 6] = n;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    sh.ps[slice][quad * 4 + i] = pa[i];
    sh.cs[slice][quad * 4 + i] = ca[i];
  }
  __syncthreads();
  dot = 0.f;
  if (threadIdx.x < 64) {
    n = 0;
    z = 0.f;
    for (int i = 0; i < NT / kWave; ++i) {
      n += sh.ns[i];
      z += sh.zs[i];
    }
    float P = 0.f;
    int c = 0;
#pragma unroll 8
    for (int i = 0; i < NT / 16; ++i) {
      P += sh.ps[i][threadIdx.x];
      c += sh.cs[i][threadIdx.x];
    }
    P = n > 0 ? P / (float)n : 0.f;
    const int e = tile * 64 + threadIdx.x;
    if (e < p.E) {
      p.probs[(size_t)s * p.E + e] = P;
      p.counts[(size_t)s * p.E + e] = c;
    }
    dot = wave_sum(n > 0 ? (float)c / (float)n * ((float)p.E / (float)p.k) * P : 0.f);
  }
}

// The sums over the sequences (in 64 bits), and what the losses are of them.
struct Totals {
  double b, z;
  int n, full;
  __device__ __forceinline__ void write(const BalanceP& p) const {
    p.losses[0] = full ? (float)(b / full) : 0.f;
    p.losses[1] = n ? (float)(z / n) : 0.f;
    p.nseq[p.S] = n;
    p.nseq[p.S + 1] = full;
  }
};

// Grid (sequences, tiles), and then one workgroup for the totals.  Slower:
// totals by the workgroup that arrives last, instead of a launch of their own
// (every arrival is an L2 write-back, 10.3 against 4.8 + 3.5 us at 37
// sequences of 256 experts), and one workgroup for all of it in small batches
// (about 4 us a tile: 23 against 14 us at 4096 x 256).  Not kept either: a
// wave per sequence and tile with its totals by the last of at most 64
// workgroups (1 to 2 us less below 8192 rows of one sequence, 3 to 4 more at
// 131072 x 256 in 37 or 150).
template <int NT>
__global__ __launch_bounds__(NT) void balance_seq_kernel(BalanceP p) {
  __shared__ SeqSums<NT> sh;
  float dot, z;
  int n;
  add_pieces<NT>(p, sh, blockIdx.x, blockIdx.y, dot, z, n);
  if (threadIdx.x == 0) {
    p.dot[(size_t)blockIdx.x * gridDim.y + blockIdx.y] = dot;
    if (blockIdx.y == 0) {
      p.zseq[blockIdx.x] = z;
      p.nseq[blockIdx.x] = n;
    }
  }
}
__global__ __launch_bounds__(256) void balance_total_kernel(BalanceP p, int tiles) {
  __shared__ Totals sh[4];
  Totals a = {0.0, 0.0, 0, 0};
  for (int s = threadIdx.x; s < p.S; s += 256) {
    for (int i = 0; i < tiles; ++i) a.b += (double)p.dot[(size_t)s * tiles + i];
    a.z += (double)p.zseq[s];
    a.n += p.nseq[s];
    a.full += p.nseq[s] > 0;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) {
    a.b += __shfl_xor(a.b, off, kWave);
    a.z += __shfl_xor(a.z, off, kWave);
    a.n += __shfl_xor(a.n, off, kWave);
    a.full += __shfl_xor(a.full, off, kWave);
  }
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = a;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 4; ++w) {
      a.b += sh[w].b;
      a.z += sh[w].z;
      a.n += sh[w].n;
      a.full += sh[w].full;
    }
    a.write(p);
  }
}
struct RouteGradP {
  const float* logits;
  const int32_t* ids;
  const uint8_t* mask;
  const int32_t* off;
  const float* d_weights;  // optional [T][ks]
  const float* d_losses;   // optional [2]
  const int32_t* counts;
  const int32_t* tokens;
  float* out;
  int T, E, k, ks, S, renorm;
  int rows;  // tokens per workgroup
  float scale;
};

// Value of lane i < 16 of the caller's group, for its first 16 lanes.
template <int LANES, int I>
__device__ __forceinline__ int group_bcast(int v) {
  if (LANES < 64) return __builtin_amdgcn_update_dpp(v, v, 0x150 + I, 0xF, 0xF, false);  // row_newbcast
  return __builtin_amdgcn_readlane(v, I);
}
// sum over the slots i < k that hold this lane's id, of their values, in order
template <int LANES, int I>
__device__ __forceinline__ float same_id_sum(int id, float v, int k, float sum) {
  if (I < k) {
    const int oid = group_bcast<LANES, I>(id);
    const float ov = __builtin_bit_cast(float, group_bcast<LANES, I>(__builtin_bit_cast(int, v)));
    sum += oid == id ? ov : 0.f;
    if constexpr (I + 1 < 16) return same_id_sum<LANES, I + 1>(id, v, k, sum);
  }
  return sum;
}

// One workgroup per run of `rows` tokens; a lane group takes every GROUPS-th
// of them, with the next one's logits and slots on their way.
template <int LANES, int NV, int SC>
__global__ __launch_bounds__(256) void route_grad_kernel(RouteGradP p) {
  constexpr int V = 4 * NV, GROUPS = 256 / LANES, ROW = NV * LANES * 4;
  __shared__ float gwbuf[GROUPS * ROW];  // gradient of the chosen scores, by expert; zero between tokens
  const int j = threadIdx.x % LANES, g = threadIdx.x / LANES;
  float* gwrow = gwbuf + g * ROW;
#pragma unroll
  for (int v = 0; v < NV; ++v) *reinterpret_cast<f32x4_t*>(gwrow + (v * LANES + j) * 4) = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int a = blockIdx.x * p.rows, b = min(p.T, a + p.rows);
  const bool losses = p.d_losses != nullptr, wants = p.d_weights != nullptr;
  float da = 0.f, dz = 0.f;
  if (losses) {
    const float total = (float)p.tokens[p.S], full = (float)p.tokens[p.S + 1];
    da = p.d_losses[0] * ((float)p.E / (float)p.k) / full;
    dz = p.d_losses[1] * 2.f / total;
  }
  // the sequence of the group's token, its rows [lo, hi) and its gradient to
  // the probabilities, kept while the tokens stay in it
  int s = losses && p.off ? seq_of(p.off, p.S, p.T, a) : 0, lo = 0, hi = p.T;
  if (losses && p.off) {
    lo = seq_at(p.off, s, p.T);
    hi = seq_at(p.off, s + 1, p.T);
  }
  int have = -1;
  float gb[V];
#pragma unroll
  for (int i = 0; i < V; ++i) gb[i] = 0.f;

  float l[V], ln[V];
  int id = -1, idn = -1;
  float dw = 0.f, dwn = 0.f;
  bool on = false, onn = false;
  auto load = [&](int t, float(&to)[V], int& slot, float& w, bool& keep) {
    slot = -1;
    w = 0.f;
    keep = false;
    if (t >= b) return;
    keep = !p.mask || p.mask[t];
    if (wants && j < p.k) {
      slot = p.ids[(size_t)t * p.ks + j];
      w = p.d_weights[(size_t)t * p.ks + j];
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) load4<false>(p.logits + (size_t)t * p.E, (v * LANES + j) * 4, p.E, to + 4 * v);
  };
  load(a + g, l, id, dw, on);
  for (int t = a + g; t < b; t += GROUPS) {
    load(t + GROUPS, ln, idn, dwn, onn);
    const float* row = p.logits + (size_t)t * p.E;
    if (id < 0 || id >= p.E) {
      id = -1;
      dw = 0.f;
    }
    const float lsel = id >= 0 ? row[id] : 0.f;
    dw *= p.scale;
    const bool weights = wants && group_max<LANES>(dw != 0.f ? 1.f : 0.f) > 0.f;  // NaN counts
    bool loss = losses && on;
    if (loss && p.off) {
      while (t >= hi && s + 1 < p.S) {
        ++s;
        lo = hi;
        hi = seq_at(p.off, s + 1, p.T);
      }
      loss = lo <= t && t < hi;
    }
    float d[V];
    if (!loss && !weights) {
#pragma unroll
      for (int i = 0; i < V; ++i) d[i] = 0.f;
    } else {
      float m = kNegInf;
#pragma unroll
      for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
      m = group_max<LANES>(m);
      if (m == kNegInf) m = 0.f;
      const float ml = m * kLog2e;
      float soft[V], es = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        soft[i] = exp2_(fmaf(l[i], kLog2e, -ml));
        es += soft[i];
      }
      es = group_sum<LANES>(es);
      const float einv = es == 0.f ? 0.f : rcp_(es);
      const float beta = loss && es != 0.f ? dz * (ml + __builtin_amdgcn_logf(es)) * kLn2 : 0.f;
      float sel = id >= 0 ? exp2_(fmaf(lsel, kLog2e, -ml)) : 0.f;
      float sc[V], slope[V], tinv = 1.f;
      if (SC == MOE_SOFTMAX) {
        sel *= einv;
#pragma unroll
        for (int i = 0; i < V; ++i) soft[i] *= einv;
      } else {
        const RowScale r = row_scale(m);
        float tot = 0.f;
        if (r.safe) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            sc[i] = score_and_slope<SC>(soft[i], r, slope[i]);
            tot += sc[i];
          }
          sel = id >= 0 ? score<SC>(sel, r) : 0.f;
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            sc[i] = far_score_and_slope<SC>(l[i], slope[i]);
            tot += sc[i];
          }
          float unused;
          sel = id >= 0 ? far_score_and_slope<SC>(lsel, unused) : 0.f;
        }
        tinv = rcp_(group_sum<LANES>(tot) + kTiny);
      }
      float gw[V];
#pragma unroll
      for (int i = 0; i < V; ++i) gw[i] = 0.f;
      if (weights) {
        float ds = dw;
        if (p.renorm) {
          const float inv = rcp_(group_sum<LANES>(sel) + kTiny);
          ds = (dw - group_sum<LANES>(id >= 0 ? dw * sel : 0.f) * inv) * inv;
        }
        // slots that chose the same expert: each gets the sum of all of them
        const float sum = same_id_sum<LANES, 0>(id, ds, p.k, 0.f);
        if (id >= 0) gwrow[id] = sum;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const f32x4_t x = *reinterpret_cast<const f32x4_t*>(gwrow + (v * LANES + j) * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) gw[4 * v + i] = x[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (id >= 0) gwrow[id] = 0.f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      if (loss && have != s) {
        have = s;
        const float n = (float)p.tokens[s], alpha = da / (n * n);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = (v * LANES + j) * 4;
          i32x4_t c = {0, 0, 0, 0};
          const int32_t* at = p.counts + (size_t)s * p.E + e;
          if (e + 4 <= p.E) {
            __builtin_memcpy(&c, at, 16);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (e + i < p.E) c[i] = at[i];
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) gb[4 * v + i] = alpha * (float)c[i];
        }
      }
      const float on_loss = loss ? 1.f : 0.f;
      float dot = 0.f;
      if (SC == MOE_SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          gw[i] = fmaf(gb[i], on_loss, gw[i]);
          dot = fmaf(soft[i], gw[i], dot);
        }
        const float shift = beta - group_sum<LANES>(dot);
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = soft[i] * (gw[i] + shift);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) dot = fmaf(sc[i], gb[i], dot);
        dot = group_sum<LANES>(dot) * tinv;
        const float scale = tinv * on_loss, zs = beta * einv;
#pragma unroll
        for (int i = 0; i < V; ++i) d[i] = slope[i] * fmaf(gb[i] - dot, scale, gw[i]) + zs * soft[i];
      }
    }
    float* out = p.out + (size_t)t * p.E;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = (v * LANES + j) * 4;
      if (e + 4 <= p.E) {
        const f32x4_t x = {d[4 * v], d[4 * v + 1], d[4 * v + 2], d[4 * v + 3]};
        __builtin_memcpy(out + e, &x, 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (e + i < p.E) out[e + i] = d[4 * v + i];
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) l[i] = ln[i];
    id = idn;
    dw = dwn;
    on = onn;
  }
}

// Rows per workgroup of the loss, a multiple of 16: at most 512 chunks, 1024
// in large batches (65536 x 64: 17.9 / 20.1 us with 512 / 1024; 131072 x 256:
// 39.2 / 37.1).
int balance_chunk(int T) { return ceil_div(T > 0 ? T : 1, 16 * (T <= 65536 ? 512 : 1024)) * 16; }

struct BalanceLayout {
  size_t psum, csum, zsum, nsum, dot, zseq, total;
};
bool balance_in_one(int T, int E, int S);
BalanceLayout balance_layout(int T, int E, int S) {
  const size_t Ep = align_up((size_t)E, 64);
  const size_t slots = (size_t)ceil_div(T, balance_chunk(T)) + S;
  BalanceLayout L;
  size_t off = kCtrlBytes;  // the control block stays as it is
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, 256);
    return at;
  };
  L.total = 0;
  if (balance_in_one(T, E, S)) return L;  // no scratch memory
  L.psum = take(slots * Ep * 4);
  L.csum = take(slots * Ep * 4);
  L.zsum = take(slots * 4);
  L.nsum = take(slots * 4);
  L.dot = take((size_t)S * (Ep / 64) * 4);
  L.zseq = take((size_t)S * 4);
  L.total = off;
  return L;
}

moe_status router_shape(int T, int E, int k, int n_shared, int n_seq, int scoring) {
  if (T < 0 || T > (1 << 24) || E < 1 || E > 1024 || k < 1 || k > E || k > 16) return MOE_E_INVAL;
  if (n_shared < 0 || n_shared > 1 || k + n_shared > 16) return MOE_E_INVAL;
  if (n_seq < 1 || n_seq > kMaxSeqs) return MOE_E_INVAL;
  if (scoring != MOE_SOFTMAX && scoring != MOE_SIGMOID && scoring != MOE_SQRTSOFTPLUS) return MOE_E_INVAL;
  return MOE_OK;
}

// One workgroup of 16 waves for a small batch of one sequence.
bool balance_in_one(int T, int E, int S) { return S == 1 && T <= 256 && E <= 256; }

template <int LANES, int NV, int SC>
void balance_launch_sc(const BalanceP& p, bool one, hipStream_t s) {
  if constexpr (LANES == 16 && NV <= 4) {
    if (one) {
      balance_kernel<LANES, NV, SC, 1024, true, false><<<1, 1024, (size_t)17 * p.Ep * 4, s>>>(p);
      return;
    }
  }
  // Logits of more than 64 MiB are not in the caches any more, nor is there
  // room for them beside what is: read with the non-temporal hint (us without
  // / with it, the whole call: 131072 x 256 39.2 / 36.0, 262144 x 128 37.2 /
  // 34.0; below, where they may be there still, 65536 x 256 22.3 / 23.4,
  // 131072 x 64 17.2 / 18.5)
  const size_t lds = (size_t)5 * p.Ep * 4;
  if ((uint64_t)p.T * p.E * 4 > (64ull << 20))
    balance_kernel<LANES, NV, SC, 256, false, true><<<p.chunks, 256, lds, s>>>(p);
  else
    balance_kernel<LANES, NV, SC, 256, false, false><<<p.chunks, 256, lds, s>>>(p);
}
template <int LANES, int NV>
void balance_launch(const BalanceP& p, bool one, int scoring, hipStream_t s) {
  switch (scoring) {
    case MOE_SOFTMAX: balance_launch_sc<LANES, NV, MOE_SOFTMAX>(p, one, s); break;
    case MOE_SIGMOID: balance_launch_sc<LANES, NV, MOE_SIGMOID>(p, one, s); break;
    default: balance_launch_sc<LANES, NV, MOE_SQRTSOFTPLUS>(p, one, s); break;
  }
}
template <int LANES, int NV>
void route_grad_launch(RouteGradP p, int scoring, hipStream_t s) {
  // one token per lane group until the chip is full, then three, with the
  // next one's loads under way (us with 1 / 2 / 3 / 4: 16384 x 128 7.0 / 7.4 /
  // 8.7 / 9.4, 65536 x 128 17.1 / 17.1 / 15.8 / 16.0, 131072 x 256 68.5 /
  // 61.5 / 61.7 / 62.1)
  constexpr int GROUPS = 256 / LANES;
  p.rows = GROUPS * (ceil_div64(p.T, GROUPS) <= 2048 ? 1 : 3);
  const int grid = ceil_div(p.T, p.rows);
  switch (scoring) {
    case MOE_SOFTMAX: route_grad_kernel<LANES, NV, MOE_SOFTMAX><<<grid, 256, 0, s>>>(p); break;
    case MOE_SIGMOID: route_grad_kernel<LANES, NV, MOE_SIGMOID><<<grid, 256, 0, s>>>(p); break;
    default: route_grad_kernel<LANES, NV, MOE_SQRTSOFTPLUS><<<grid, 256, 0, s>>>(p); break;
  }
}

// 16 lanes per token up to 320 experts, 32 above, and MANY above 640: 32 for
// the loss, 64 for the gradient, which has more per logit in registers.
// Measured with 16 / 32 / 64 lanes (us, sigmoid): the loss of 65536 tokens and 320
// experts 28.9 / 35.1 / -, of 448 34.8 / 37.8 / 49.3, of 384 31.7 / 33.0 /
// 48.6, of 512 34.6 / 33.3 / 42.0 (softmax), of 32768 and 640 - / 29.0 / 36.0,
// of 1024 - / 37.2 / 39.0; the gradient of 65536 and 128 15.8 / 19.4 / -, of
// 384 52 / 43 / 58, of 512 78 / 55 / 55, of 16384 and 640 - / 18.1 / 22.2, of
// 768 - / 23.8 / 23.5, of 32768 and 1024 - / 79 / 53.
#define MOE_BY_EXPERTS(FN, MANY, E, ...)                                  \
  do {                                                                    \
    switch (ceil_div(E, 64)) {                                            \
      case 1: FN<16, 1>(__VA_ARGS__); break;                              \
      case 2: FN<16, 2>(__VA_ARGS__); break;                              \
      case 3: FN<16, 3>(__VA_ARGS__); break;                              \
      case 4: FN<16, 4>(__VA_ARGS__); break;                              \
      case 5: FN<16, 5>(__VA_ARGS__); break;                              \
      case 6: FN<32, 3>(__VA_ARGS__); break;                              \
      case 7: case 8: FN<32, 4>(__VA_ARGS__); break;                      \
      case 9: case 10: FN<32, 5>(__VA_ARGS__); break;                     \
      case 11: case 12: FN<MANY, 192 / MANY>(__VA_ARGS__); break;         \
      default: FN<MANY, 256 / MANY>(__VA_ARGS__); break;                  \
    }                                                                     \
  } while (0)

}  // namespace

}  // namespace moe

extern "C" size_t moe_balance_loss_workspace_size(int T, int E, int n_seq) {
  if (T < 0 || T > (1 << 24) || E < 1 || E > 1024 || n_seq < 1 || n_seq > moe::kMaxSeqs) return 0;
  return moe::balance_layout(T, E, n_seq).total;
}

extern "C" moe_status moe_balance_loss(const float* logits, const int32_t* topk_ids, const uint8_t* token_mask,
                                       const int32_t* seq_offsets, int T, int E, int k, int n_shared, int n_seq,
                                       int scoring, float* losses, int32_t* counts, float* probs, int32_t* tokens,
                                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  using namespace moe;
  const moe_status st = router_shape(T, E, k, n_shared, n_seq, scoring);
  if (st != MOE_OK) return st;
  if (!seq_offsets && n_seq != 1) return MOE_E_INVAL;
  if (T > 0 && (!logits || !topk_ids)) return MOE_E_INVAL;
  if (!losses || !counts || !probs || !tokens) return MOE_E_INVAL;
  const BalanceLayout L = balance_layout(T, E, n_seq);
  if (L.total > 0 && (!workspace || !aligned(workspace, 16))) return MOE_E_INVAL;
  if (workspace_bytes < L.total) return MOE_E_WORKSPACE;
  char* b = static_cast<char*>(workspace);
  BalanceP p;
  p.logits = logits;
  p.ids = topk_ids;
  p.mask = token_mask;
  p.off = seq_offsets;
  p.T = T;
  p.E = E;
  p.k = k;
  p.ks = k + n_shared;
  p.S = n_seq;
  p.chunk = balance_chunk(T);
  p.chunks = ceil_div(T, p.chunk);
  p.Ep = (int)align_up((size_t)E, 64);
  p.psum = reinterpret_cast<float*>(b + L.psum);
  p.csum = reinterpret_cast<int32_t*>(b + L.csum);
  p.zsum = reinterpret_cast<float*>(b + L.zsum);
  p.nsum = reinterpret_cast<int32_t*>(b + L.nsum);
  p.dot = reinterpret_cast<float*>(b + L.dot);
  p.zseq = reinterpret_cast<float*>(b + L.zseq);
  p.nseq = tokens;
  p.losses = losses;
  p.counts = counts;
  p.probs = probs;
  const bool one = balance_in_one(T, E, n_seq);
  if (one) {
    p.chunk = T > 0 ? T : 1;
    p.chunks = 1;
  }
  if (T > 0 || one) {
    MOE_BY_EXPERTS(balance_launch, 32, E, p, one, scoring, stream);
    MOE_CHECK_LAUNCH();
  }
  if (one) return MOE_OK;
  const dim3 grid((unsigned)n_seq, (unsigned)(p.Ep / 64));
  if (p.chunks / n_seq > 64)  // pieces of an average sequence
    balance_seq_kernel<1024><<<grid, 1024, 0, stream>>>(p);
  else
    balance_seq_kernel<256><<<grid, 256, 0, stream>>>(p);
  MOE_CHECK_LAUNCH();
  balance_total_kernel<<<1, 256, 0, stream>>>(p, p.Ep / 64);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}

extern "C" moe_status moe_route_grad(const float* logits, const int32_t* topk_ids, const uint8_t* token_mask,
                                     const int32_t* seq_offsets, int T, int E, int k, int n_shared, int n_seq,
                                     int scoring, int renormalize, float routed_scale, const float* d_weights,
                                     const float* d_losses, const int32_t* counts, const int32_t* tokens,
                                     float* d_logits, hipStream_t stream) {
  using namespace moe;
  const moe_status st = router_shape(T, E, k, n_shared, n_seq, scoring);
  if (st != MOE_OK) return st;
  if (!seq_offsets && n_seq != 1) return MOE_E_INVAL;
  if (!d_weights && !d_losses) return MOE_E_INVAL;
  if (d_losses && (!counts || !tokens)) return MOE_E_INVAL;
  if (T == 0) return MOE_OK;
  if (!logits || !topk_ids || !d_logits) return MOE_E_INVAL;
  RouteGradP p;
  p.logits = logits;
  p.ids = topk_ids;
  p.mask = token_mask;
  p.off = seq_offsets;
  p.d_weights = d_weights;
  p.d_losses = d_losses;
  p.counts = counts;
  p.tokens = tokens;
  p.out = d_logits;
  p.T = T;
  p.E = E;
  p.k = k;
  p.ks = k + n_shared;
  p.S = n_seq;
  p.renorm = renormalize != 0;
  p.scale = routed_scale;
  MOE_BY_EXPERTS(route_grad_launch, 64, E, p, scoring, stream);
  MOE_CHECK_LAUNCH();
  return MOE_OK;
}
