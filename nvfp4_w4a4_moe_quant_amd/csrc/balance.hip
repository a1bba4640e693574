// Balance loss of an MoE router: per-expert counts and mean probabilities, the
// balance loss and the z-loss, and the gradient of the logits.
//
// Per counted row, p = softmax(l) and lse = m + ln sum e^(l - m).  A row is held by
// LPR lanes, V logits to a load, so that a wave works on 64 / LPR rows at a time
// with the next ones in flight.  Forward, a lane keeps the sums of its experts'
// probabilities over the rows of its wave, in FP32 over 64 rows at a time and in
// FP64 beyond, and lse^2 in FP64; workgroups write partial sums, and a
// second launch joins them, a workgroup for 32 experts each, the last of them
// adding up the loss.  Few rows take one launch of one workgroup.
// Backward needs the counts alone besides the row itself:
//   grad_j = p_j (a (c_j - sum_e c_e p_e) + b lse).
// The counts enter centred, c_j - (sum c) / E, which changes nothing since the p
// sum to one and keeps the difference small where the experts are balanced.
//
// What bounds it (times of a trace, which adds about a microsecond to a kernel): few
// rows the latency of a chain of loads, reductions and the join (8192 x 256 FP32:
// forward 5.1 + 7.7 us, backward 7.6 us, for 8 MB read once; in a graph 11.6 and
// 6.3), many rows memory (65536 x 256 FP32 with inputs beyond the last-level cache
// in turn: forward 22 + 6 us for 67 MB, backward 24 us for 134 MB, of which the
// forward call left the logits in that cache) or, in bf16, as much the arithmetic
// (65536 x 128: 8.8 + 6.1 us and 15 us for 34 MB).  A wave for a row with one logit
// to a load, and one workgroup to join: 10.5 + 80 us for the forward of 8192 x 256,
// 77 + 83 us for that of 65536 x 128.

#include <type_traits>

#include "common.h"

namespace {

constexpr int kMaxE = 1024;
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kFwdWaves = 16;
constexpr int kFwdBlocks = 256;   // workgroups (partial sums) at most
// One workgroup alone takes rows that are at most so many lanes' work, five rows
// of a lane (128 experts: 64 rows 5.0 us for 7.9 in two launches, 128 rows 6.7 for
// 8.0, 192 rows 8.6 for 8.0; 256 experts: 64 rows 7.1 for 8.5, 128 rows 11.1 for
// 8.7; 32 experts: 512 rows 6.4 for 7.7).
constexpr int64_t kOneBlock = 5 * 64 * kFwdWaves;
constexpr int kJoinCols = 32, kJoinParts = 32;
// Probabilities are added in FP32 over so many rows of a lane, then in FP64: 2^24
// rows of five experts, 1024 to a lane, drift by 161 half-steps in FP32 alone.
constexpr int kChain = 64;

struct BalParams {
  const void* logits;
  int64_t T, ld, k;
  int E;
  const uint8_t* mask;
  const int32_t* ids;
  int32_t* counts;
  int32_t* tokens;
  float* mean;
  float* losses;
  // partial sums of nblk workgroups, and what the joining ones share
  double* part_z;    // [nblk]
  float* part_p;     // [nblk][E]
  int32_t* part_c;   // [nblk][E]
  int32_t* part_n;   // [nblk]
  double* dots;      // [E / 32]
  uint32_t* joined;
  const float* grad_losses;
  void* grad;
  int64_t ldg;
};

template <int CTRL>
__device__ __forceinline__ float bal_dpp(float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}

// op over the LPR lanes of a row, in every lane of it: neighbours and quads by
// quad_perm, 8 and 16 lanes by the half and whole row mirrored, 32 and 64 by the
// lane swaps.
template <int LPR, class Op>
__device__ __forceinline__ float bal_reduce(float v, Op op) {
  v = op(v, bal_dpp<0xB1>(v));
  v = op(v, bal_dpp<0x4E>(v));
  v = op(v, bal_dpp<0x141>(v));
  if constexpr (LPR >= 16) v = op(v, bal_dpp<0x140>(v));
  if constexpr (LPR >= 32) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  if constexpr (LPR >= 64) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  }
  return v;
}
struct BalAdd {
  __device__ float operator()(float a, float b) const { return a + b; }
};
struct BalMax {
  __device__ float operator()(float a, float b) const { return __builtin_fmaxf(a, b); }
};

// One row group's share of a lane: V logits of PER pieces, piece j of the row at
// expert (j LPR + lane) V.  V > 1: rows start on 16 bytes and a piece is 16
// bytes; the piece that holds the last expert is read whole (its other bytes lie
// in the same 16) and what is behind E is taken out.
template <bool BF16, int V, int LPR, int PER>
struct BalRow {
  static constexpr int RPW = 64 / LPR;  // rows of a wave
  uint4 raw[V > 1 ? PER : 1];
  float one[V > 1 ? 1 : PER];
  int32_t id;  // the lane's first slot
  bool on;     // the row is there and the mask takes it

  __device__ __forceinline__ void load(const BalParams& p, int64_t t, int lir, bool want_ids) {
    on = t < p.T && (!p.mask || p.mask[t]);
    const int64_t at = on ? t * p.ld : 0;
    id = on && want_ids && lir < p.k ? p.ids[t * p.k + lir] : -1;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = (j * LPR + lir) * V;
      if constexpr (V > 1) {
        constexpr int SIZE = BF16 ? 2 : 4;
        raw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (on && e < p.E)
          raw[j] = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p.logits) + (at + e) * SIZE);
      } else {
        one[j] = 0.0f;
        if (on && e < p.E) {
          if constexpr (BF16)
            one[j] = nv_bf16_to_f32(reinterpret_cast<const uint16_t*>(p.logits)[at + e]);
          else
            one[j] = reinterpret_cast<const float*>(p.logits)[at + e];
        }
      }
    }
  }

  // The probabilities, the log-sum, and whether the row counts (uniform in the
  // row's lanes).  The maximum passes over a NaN, which reaches the sums by itself.
  // l - m comes before the factor log2 e: a mask of the type's lowest value stays
  // the number that it is.
  __device__ __forceinline__ bool softmax(const BalParams& p, int lir, float (&l)[PER * V], float& lse) {
    const float none = -__builtin_inff();
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if constexpr (V > 1) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (BF16) {
            l[j * V + 2 * i] = __uint_as_float(w[i] << 16);
            l[j * V + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
          } else {
            l[j * V + i] = __uint_as_float(w[i]);
          }
        }
      } else {
        l[j] = one[j];
      }
    }
    if (p.E != LPR * PER * V)  // uniform: places without an expert
#pragma unroll
      for (int j = 0; j < PER; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i)
          if ((j * LPR + lir) * V + i >= p.E) l[j * V + i] = none;
    float m = none;
#pragma unroll
    for (int i = 0; i < PER * V; ++i) m = __builtin_fmaxf(m, l[i]);
    m = bal_reduce<LPR>(m, BalMax());
    float real = 1.0f;
    if (__ballot(m == none)) {  // a row of nothing but -inf, or of NaN and -inf
      real = 0.0f;
#pragma unroll
      for (int i = 0; i < PER * V; ++i) real = l[i] == none ? real : 1.0f;
      real = bal_reduce<LPR>(real, BalMax());
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < PER * V; ++i) {
      l[i] = __builtin_amdgcn_exp2f((l[i] - m) * kLog2E);
      s += l[i];
    }
    s = bal_reduce<LPR>(s, BalAdd());
    const float r = 1.0f / s;
#pragma unroll
    for (int i = 0; i < PER * V; ++i) l[i] *= r;
    lse = m + __builtin_amdgcn_logf(s) * kLn2;
    return on && real != 0.0f;
  }
};

// dot = sum over the experts of counts and mean probabilities; the outputs.
__device__ __forceinline__ void bal_finish(const BalParams& p, double dot, double z, int64_t n) {
  const double inv = n > 0 ? 1.0 / (double)n : 0.0;
  p.tokens[0] = (int32_t)n;
  p.losses[0] = (float)(dot * inv * (double)p.E / (double)p.k);
  p.losses[1] = (float)(z * inv);
}

template <bool BF16, int V, int LPR, int PER, bool ONE>
__global__ __launch_bounds__(64 * kFwdWaves) void k_balance(BalParams p) {
  using Row = BalRow<BF16, V, LPR, PER>;
  constexpr int COLS = LPR * PER * V, NT = 64 * kFwdWaves;
  __shared__ int32_t hist[COLS];
  __shared__ float sp[kFwdWaves][COLS];
  __shared__ double sz[kFwdWaves];
  __shared__ int32_t sn[kFwdWaves];
  __shared__ double sd[kFwdWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lir = lane % LPR, slot = lane / LPR;
  for (int e = tid; e < COLS; e += NT) hist[e] = 0;
  if (!ONE && blockIdx.x == 0 && tid == 0) *p.joined = 0u;
  __syncthreads();
  float sum[PER * V];
  double far[PER * V];  // of the chains behind
  double z = 0.0;  // an lse of 2^64 has a square beyond FP32's range
  int n = 0;
#pragma unroll
  for (int i = 0; i < PER * V; ++i) {
    sum[i] = 0.0f;
    far[i] = 0.0;
  }
  int chain = 0;
  const int64_t stride = (int64_t)gridDim.x * kFwdWaves * Row::RPW;
  int64_t t = ((int64_t)blockIdx.x * kFwdWaves + wave) * Row::RPW + slot;
  Row cur, nxt;
  cur.load(p, t, lir, true);
  for (; t - slot < p.T; t += stride) {
    nxt.load(p, t + stride, lir, true);
    float l[PER * V], lse;
    if (cur.softmax(p, lir, l, lse)) {
#pragma unroll
      for (int i = 0; i < PER * V; ++i) sum[i] += l[i];
      if (lir == 0) {
        z = __builtin_fma((double)lse, (double)lse, z);
        ++n;
      }
      if ((uint32_t)cur.id < (uint32_t)p.E) atomicAdd(&hist[cur.id], 1);
      for (int64_t s = lir + LPR; s < p.k; s += LPR) {
        const uint32_t e = (uint32_t)p.ids[t * p.k + s];
        if (e < (uint32_t)p.E) atomicAdd(&hist[e], 1);
      }
    }
    cur = nxt;
    if (!ONE && ++chain == kChain) {  // ONE: five rows of a lane
      chain = 0;
#pragma unroll
      for (int i = 0; i < PER * V; ++i) {
        far[i] += (double)sum[i];
        sum[i] = 0.0f;
      }
    }
  }
  if constexpr (!ONE)
#pragma unroll
    for (int i = 0; i < PER * V; ++i) sum[i] = (float)(far[i] + (double)sum[i]);
  // the wave's row slots, then the waves
#pragma unroll
  for (int o = LPR; o < 64; o <<= 1) {
#pragma unroll
    for (int i = 0; i < PER * V; ++i) sum[i] += __shfl_xor(sum[i], o, 64);
    z += __shfl_xor(z, o, 64);
    n += __shfl_xor(n, o, 64);
  }
  if (slot == 0)
#pragma unroll
    for (int j = 0; j < PER; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) sp[wave][(j * LPR + lir) * V + i] = sum[j * V + i];
  if (lane == 0) {
    sz[wave] = z;
    sn[wave] = n;
  }
  __syncthreads();
  const int64_t b = blockIdx.x;
  if constexpr (ONE) {
    int64_t all = 0;
    for (int w = 0; w < kFwdWaves; ++w) all += sn[w];
    const double inv = all > 0 ? 1.0 / (double)all : 0.0;
    double dot = 0.0;
    for (int e = tid; e < p.E; e += NT) {
      double s = 0.0;
      for (int w = 0; w < kFwdWaves; ++w) s += sp[w][e];
      p.counts[e] = hist[e];
      if (p.mean) p.mean[e] = (float)(s * inv);
      dot += (double)hist[e] * (s * inv);
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
    if (lane == 0) sd[wave] = dot;
    __syncthreads();
    if (tid == 0) {
      double d = 0.0, zz = 0.0;
      for (int w = 0; w < kFwdWaves; ++w) {
        d += sd[w];
        zz += sz[w];
      }
      bal_finish(p, d, zz, all);
    }
  } else {
    for (int e = tid; e < p.E; e += NT) {
      float s = sp[0][e];
      for (int w = 1; w < kFwdWaves; ++w) s += sp[w][e];
      p.part_p[b * p.E + e] = s;
      p.part_c[b * p.E + e] = hist[e];
    }
    if (tid == 0) {
      double s = sz[0];
      int c = sn[0];
      for (int w = 1; w < kFwdWaves; ++w) {
        s += sz[w];
        c += sn[w];
      }
      p.part_z[b] = s;
      p.part_n[b] = c;
    }
  }
}

// Adds the partial sums of 32 experts in 64 bits, always in the same order.  The
// workgroup that comes last adds up the loss, from all workgroups' shares in
// their order.  The counter was cleared by the launch before.
__global__ __launch_bounds__(kJoinCols* kJoinParts) void k_balance_join(BalParams p, int nblk) {
  // two parts to a wave, whose sums meet in registers
  constexpr int WAVES = kJoinCols * kJoinParts / 64;
  static_assert(kJoinCols == 32 && WAVES == 16 && kFwdBlocks <= 256, "lanes below");
  __shared__ double rs[WAVES][kJoinCols];
  __shared__ int32_t rc[WAVES][kJoinCols];
  __shared__ double wz[4];
  __shared__ int32_t wn[4];
  const int tid = threadIdx.x, col = tid % kJoinCols, part = tid / kJoinCols;
  const int e = blockIdx.x * kJoinCols + col;
  double s = 0.0;
  int c = 0;
  if (e < p.E) {
#pragma unroll
    for (int i = 0; i < kFwdBlocks / kJoinParts; ++i) {
      const int b = i * kJoinParts + part;
      if (b < nblk) {
        s += p.part_p[(int64_t)b * p.E + e];
        c += p.part_c[(int64_t)b * p.E + e];
      }
    }
  }
  if (tid < 256) {  // nblk <= 256
    double z = tid < nblk ? p.part_z[tid] : 0.0;
    int n = tid < nblk ? p.part_n[tid] : 0;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      z += __shfl_xor(z, o, 64);
      n += __shfl_xor(n, o, 64);
    }
    if ((tid & 63) == 0) {
      wz[tid >> 6] = z;
      wn[tid >> 6] = n;
    }
  }
  s += __shfl_xor(s, 32, 64);
  c += __shfl_xor(c, 32, 64);
  if ((tid & 32) == 0) {
    rs[tid >> 6][col] = s;
    rc[tid >> 6][col] = c;
  }
  __syncthreads();
  if (tid >= 64) return;
  const int64_t n = (int64_t)wn[0] + wn[1] + wn[2] + wn[3];
  const double inv = n > 0 ? 1.0 / (double)n : 0.0;
  s = 0.0;
  c = 0;
#pragma unroll
  for (int i = 0; i < WAVES / 2; ++i) {
    s += rs[part * (WAVES / 2) + i][col];
    c += rc[part * (WAVES / 2) + i][col];
  }
  s += __shfl_xor(s, 32, 64);
  c += __shfl_xor(c, 32, 64);
  double dot = 0.0;
  if (part == 0 && e < p.E) {
    p.counts[e] = c;
    if (p.mean) p.mean[e] = (float)(s * inv);
    dot = (double)c * (s * inv);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
  if (tid != 0) return;
  __hip_atomic_store(&p.dots[blockIdx.x], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t before =
      __hip_atomic_fetch_add(p.joined, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
  if (before + 1 != gridDim.x) return;
  dot = 0.0;
  for (uint32_t i = 0; i < gridDim.x; ++i)
    dot += __hip_atomic_load(&p.dots[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  bal_finish(p, dot, wz[0] + wz[1] + wz[2] + wz[3], n);
}

// VOUT: gradient rows start on 16 bytes too, and are written in 16-byte pieces
// but for one that is not whole.
template <bool BF16, int V, int LPR, int PER, bool VOUT>
__global__ __launch_bounds__(256) void k_balance_bwd(BalParams p) {
  using Row = BalRow<BF16, V, LPR, PER>;
  constexpr int SIZE = BF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, lir = lane % LPR, slot = lane / LPR;
  const int64_t stride = (int64_t)gridDim.x * 4 * Row::RPW;
  int64_t t = ((int64_t)blockIdx.x * 4 + (threadIdx.x >> 6)) * Row::RPW + slot;
  Row cur, nxt;
  cur.load(p, t, lir, false);
  float c[PER * V];
  int total = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (j * LPR + lir) * V + i;
      const int n = e < p.E ? p.counts[e] : 0;
      c[j * V + i] = __int_as_float(n);
      total += n;
    }
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  const double mean = (double)total / (double)p.E;
#pragma unroll
  for (int i = 0; i < PER * V; ++i) c[i] = (float)((double)__float_as_int(c[i]) - mean);
  const double n = (double)p.tokens[0], inv = n > 0.0 ? 1.0 / n : 0.0;
  const float a = (float)((double)p.grad_losses[0] * (double)p.E / (double)p.k * inv * inv);
  const float b = (float)((double)p.grad_losses[1] * 2.0 * inv);
#pragma unroll
  for (int i = 0; i < PER * V; ++i) c[i] *= a;
  for (; t - slot < p.T; t += stride) {
    nxt.load(p, t + stride, lir, false);
    float l[PER * V], lse;
    const bool live = cur.softmax(p, lir, l, lse);
    float cp = 0.0f;
#pragma unroll
    for (int i = 0; i < PER * V; ++i) cp += c[i] * l[i];
    cp = b * lse - bal_reduce<LPR>(cp, BalAdd());
    if (live) {
#pragma unroll
      for (int i = 0; i < PER * V; ++i) l[i] *= c[i] + cp;
    } else {
#pragma unroll
      for (int i = 0; i < PER * V; ++i) l[i] = 0.0f;
    }
    if (t < p.T) {
      char* out = reinterpret_cast<char*>(p.grad) + t * p.ldg * SIZE;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const int e = (j * LPR + lir) * V;
        if (VOUT && e + V <= p.E) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if constexpr (BF16)
              w[i] = __builtin_bit_cast(uint16_t, (__bf16)l[(j * V + 2 * i) % (PER * V)]) |
                     (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)l[(j * V + 2 * i + 1) % (PER * V)]) << 16;
            else
              w[i] = __float_as_uint(l[(j * V + i) % (PER * V)]);
          }
          *reinterpret_cast<uint4*>(out + e * SIZE) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (e + i < p.E) {
              if constexpr (BF16)
                reinterpret_cast<uint16_t*>(out)[e + i] = __builtin_bit_cast(uint16_t, (__bf16)l[j * V + i]);
              else
                reinterpret_cast<float*>(out)[e + i] = l[j * V + i];
            }
        }
      }
    }
    cur = nxt;
  }
}

int fwd_blocks(int64_t T, int rpw) {
  const int64_t n = (T + kFwdWaves * rpw - 1) / (kFwdWaves * rpw);
  return (int)(n < 1 ? 1 : n < kFwdBlocks ? n : kFwdBlocks);
}

template <bool BF16, int V, int LPR, int PER>
int launch(const BalParams& p, bool backward, bool vout, hipStream_t s) {
  if (!backward) {
    const int nblk = fwd_blocks(p.T, 64 / LPR);
    const dim3 grid((unsigned)nblk), block(64 * kFwdWaves);
    if (p.T * LPR <= kOneBlock) {
      hipLaunchKernelGGL((k_balance<BF16, V, LPR, PER, true>), dim3(1), block, 0, s, p);
      return nv_launch_status();
    }
    hipLaunchKernelGGL((k_balance<BF16, V, LPR, PER, false>), grid, block, 0, s, p);
    hipLaunchKernelGGL(k_balance_join, dim3((unsigned)((p.E + kJoinCols - 1) / kJoinCols)),
                       dim3(kJoinCols * kJoinParts), 0, s, p, nblk);
    return nv_launch_status();
  }
  const int64_t n = (p.T * LPR + 255) / 256;
  const dim3 grid((unsigned)(n < 2048 ? n : 2048)), block(256);
  if (vout)
    hipLaunchKernelGGL((k_balance_bwd<BF16, V, LPR, PER, V != 1>), grid, block, 0, s, p);
  else
    hipLaunchKernelGGL((k_balance_bwd<BF16, V, LPR, PER, false>), grid, block, 0, s, p);
  return nv_launch_status();
}

// 16-byte pieces where the rows of logits start on 16 bytes, else single logits.
template <bool BF16>
int launch_by_experts(const BalParams& p, bool backward, hipStream_t s) {
  constexpr int SIZE = BF16 ? 2 : 4, V = 16 / SIZE;
  auto whole = [](const void* x, int64_t ld) { return nv_aligned16(x) && ld * SIZE % 16 == 0; };
  const bool vin = whole(p.logits, p.ld), vout = backward && whole(p.grad, p.ldg);
  if (!vin) {
    if (p.E <= 16) return launch<BF16, 1, 16, 1>(p, backward, false, s);
    if (p.E <= 64) return launch<BF16, 1, 64, 1>(p, backward, false, s);
    if (p.E <= 128) return launch<BF16, 1, 64, 2>(p, backward, false, s);
    if (p.E <= 256) return launch<BF16, 1, 64, 4>(p, backward, false, s);
    if (p.E <= 512) return launch<BF16, 1, 64, 8>(p, backward, false, s);
    return launch<BF16, 1, 64, 16>(p, backward, false, s);
  }
  if (p.E <= 8 * V) return launch<BF16, V, 8, 1>(p, backward, vout, s);
  if (p.E <= 16 * V) return launch<BF16, V, 16, 1>(p, backward, vout, s);
  if (p.E <= 32 * V) return launch<BF16, V, 32, 1>(p, backward, vout, s);
  if (p.E <= 64 * V) return launch<BF16, V, 64, 1>(p, backward, vout, s);
  if constexpr (!BF16)
    if (p.E > 128 * V) return launch<BF16, V, 64, 4>(p, backward, vout, s);
  return launch<BF16, V, 64, 2>(p, backward, vout, s);
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

bool bad_shape(int64_t T, int64_t E, int64_t k, int64_t ld) {
  return T < 0 || E < 1 || E > kMaxE || k < 1 || k > E || ld < E || T > 0x7fffffff ||
         T * k > 0x7fffffff;
}

}  // namespace

extern "C" {

size_t moe_balance_loss_workspace_size(int64_t T, int64_t E) {
  if (T < 0 || E < 1 || E > kMaxE) return 0;
  // the loss's shares and the counter, then the partial sums
  return nv_round256(512 + (T * 64 <= kOneBlock ? 0 : (size_t)fwd_blocks(T, 1) * (size_t)(8 * E + 12)));
}

int moe_balance_loss(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                     const int32_t* topk_ids, int64_t k, const uint8_t* mask, int32_t* counts,
                     int32_t* tokens, float* mean_probs, float* losses, void* ws,
                     size_t ws_bytes, void* stream) {
  NV_RETURN_IF(dtype != NVFP4_IN_F32 && dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(bad_shape(T, E, k, ld), NVFP4_ERR_SHAPE);
  NV_RETURN_IF(!counts || !tokens || !losses || (T > 0 && (!logits || !topk_ids)), NVFP4_ERR_NULL);
  NV_RETURN_IF(misaligned(logits, dtype == NVFP4_IN_F32 ? 4 : 2) || misaligned(topk_ids, 4) ||
                   misaligned(counts, 4) || misaligned(tokens, 4) || misaligned(mean_probs, 4) ||
                   misaligned(losses, 4),
               NVFP4_ERR_ALIGN);
  NV_RETURN_IF(!ws || ws_bytes < moe_balance_loss_workspace_size(T, E) || misaligned(ws, 8),
               NVFP4_ERR_WORKSPACE);
  const int64_t nblk = fwd_blocks(T, 1);
  BalParams p{};
  p.logits = logits;
  p.T = T;
  p.E = (int)E;
  p.ld = ld;
  p.k = k;
  p.mask = mask;
  p.ids = topk_ids;
  p.counts = counts;
  p.tokens = tokens;
  p.mean = mean_probs;
  p.losses = losses;
  p.dots = reinterpret_cast<double*>(ws);
  p.joined = reinterpret_cast<uint32_t*>(p.dots + kMaxE / kJoinCols);
  p.part_z = p.dots + 64;
  p.part_p = reinterpret_cast<float*>(p.part_z + nblk);
  p.part_c = reinterpret_cast<int32_t*>(p.part_p + nblk * E);
  p.part_n = p.part_c + nblk * E;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == NVFP4_IN_BF16 ? launch_by_experts<true>(p, false, s)
                                : launch_by_experts<false>(p, false, s);
}

int moe_balance_loss_backward(const void* logits, int dtype, int64_t T, int64_t E, int64_t ld,
                              int64_t k, const uint8_t* mask, const int32_t* counts,
                              const int32_t* tokens, const float* grad_losses, void* grad_logits,
                              int64_t ldg, void* stream) {
  NV_RETURN_IF(dtype != NVFP4_IN_F32 && dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(bad_shape(T, E, k, ld) || ldg < E, NVFP4_ERR_SHAPE);
  if (T == 0) return NVFP4_OK;
  NV_RETURN_IF(!logits || !counts || !tokens || !grad_losses || !grad_logits, NVFP4_ERR_NULL);
  NV_RETURN_IF(grad_logits == logits && ldg != ld && T > 1, NVFP4_ERR_SHAPE);
  const unsigned size = dtype == NVFP4_IN_F32 ? 4 : 2;
  NV_RETURN_IF(misaligned(logits, size) || misaligned(grad_logits, size) ||
                   misaligned(counts, 4) || misaligned(tokens, 4) || misaligned(grad_losses, 4),
               NVFP4_ERR_ALIGN);
  BalParams p{};
  p.logits = logits;
  p.T = T;
  p.E = (int)E;
  p.ld = ld;
  p.k = k;
  p.mask = mask;
  p.counts = const_cast<int32_t*>(counts);
  p.tokens = const_cast<int32_t*>(tokens);
  p.grad_losses = grad_losses;
  p.grad = grad_logits;
  p.ldg = ldg;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == NVFP4_IN_BF16 ? launch_by_experts<true>(p, true, s)
                                : launch_by_experts<false>(p, true, s);
}

}  // extern "C"
