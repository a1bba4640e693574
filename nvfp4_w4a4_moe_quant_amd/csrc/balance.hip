// Balance loss of an MoE router: per-expert counts and mean probabilities, the
// balance loss and the z-loss, and the gradient of the logits.
//
// Per counted row, p = softmax(l) and lse = m + ln sum e^(l - m).  Forward, a
// lane keeps the sums of its experts' probabilities over the rows of its wave,
// which never leave registers; workgroups write partial sums and a second
// launch joins them.  Backward needs the counts alone besides the row itself:
//   grad_j = p_j (a (c_j - sum_e c_e p_e) + b lse).
// The counts enter centred, c_j - (sum c) / E, which changes nothing since the p
// sum to one and keeps the difference small where the experts are balanced.

#include <type_traits>

#include "common.h"

namespace {

constexpr int kMaxE = 1024;
constexpr float kLog2E = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kFwdWaves = 4;
constexpr int kFwdBlocks = 256;  // workgroups (partial sums) at most

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
  // partial sums: float p[nblk][E], z[nblk]; int32 counts[nblk][E], n[nblk]
  float* part_p;
  float* part_z;
  int32_t* part_c;
  int32_t* part_n;
  const float* grad_losses;
  void* grad;
  int64_t ldg;
};

template <bool BF16>
__device__ __forceinline__ float bal_load(const void* x, int64_t i) {
  if constexpr (BF16) return nv_bf16_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
  return reinterpret_cast<const float*>(x)[i];
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Logits of row t in registers (lane + 64 j), and whether the row counts.  m is
// the largest logit; a NaN does not enter it, and reaches the sums by itself.
template <bool BF16, int PER>
__device__ __forceinline__ bool bal_row(const BalParams& p, int64_t t, float (&l)[PER], float& m) {
  if (p.mask && !p.mask[t]) return false;
  const int lane = threadIdx.x & 63;
  m = -__builtin_inff();
  bool real = false;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 64 * j;
    l[j] = e < p.E ? bal_load<BF16>(p.logits, t * p.ld + e) : -__builtin_inff();
    real |= !(l[j] == -__builtin_inff());
    m = __builtin_fmaxf(m, l[j]);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = __builtin_fmaxf(m, __shfl_xor(m, o, 64));
  return __ballot(real) != 0;
}

// p = e^(l - m) / sum in place, the log-sum returned.  l - m before the factor
// log2 e: a mask of the type's lowest value stays the number that it is.
template <int PER>
__device__ __forceinline__ float bal_softmax(float (&l)[PER], float m) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    l[j] = __builtin_amdgcn_exp2f((l[j] - m) * kLog2E);
    s += l[j];
  }
  s = wave_sum(s);
  const float r = 1.0f / s;
#pragma unroll
  for (int j = 0; j < PER; ++j) l[j] *= r;
  return m + __builtin_amdgcn_logf(s) * kLn2;
}

template <bool BF16, int PER>
__global__ __launch_bounds__(64 * kFwdWaves) void k_balance(BalParams p) {
  __shared__ int32_t hist[kMaxE];
  __shared__ float sp[kFwdWaves][kMaxE];
  __shared__ float sz[kFwdWaves];
  __shared__ int32_t sn[kFwdWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  for (int e = tid; e < p.E; e += 64 * kFwdWaves) hist[e] = 0;
  __syncthreads();
  float sum[PER], z = 0.0f;
  int n = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) sum[j] = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kFwdWaves + wave; t < p.T;
       t += (int64_t)gridDim.x * kFwdWaves) {
    float l[PER], m;
    if (!bal_row<BF16, PER>(p, t, l, m)) continue;
    const float lse = bal_softmax<PER>(l, m);
    z += lse * lse;
    ++n;
#pragma unroll
    for (int j = 0; j < PER; ++j) sum[j] += l[j];
    for (int64_t s = lane; s < p.k; s += 64) {
      const uint32_t e = (uint32_t)p.ids[t * p.k + s];
      if (e < (uint32_t)p.E) atomicAdd(&hist[e], 1);
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (lane + 64 * j < p.E) sp[wave][lane + 64 * j] = sum[j];
  if (lane == 0) {
    sz[wave] = z;
    sn[wave] = n;
  }
  __syncthreads();
  const int64_t b = blockIdx.x;
  for (int e = tid; e < p.E; e += 64 * kFwdWaves) {
    float s = sp[0][e];
    for (int w = 1; w < kFwdWaves; ++w) s += sp[w][e];
    p.part_p[b * p.E + e] = s;
    p.part_c[b * p.E + e] = hist[e];
  }
  if (tid == 0) {
    float s = sz[0];
    int c = sn[0];
    for (int w = 1; w < kFwdWaves; ++w) {
      s += sz[w];
      c += sn[w];
    }
    p.part_z[b] = s;
    p.part_n[b] = c;
  }
}

// One workgroup adds the partial sums, in their order, in 64 bits.
__global__ __launch_bounds__(kMaxE) void k_balance_join(BalParams p, int nblk) {
  __shared__ double red[kMaxE / 64];
  const int e = threadIdx.x, lane = e & 63, w = e >> 6;
  double z = 0.0;
  int64_t n = 0;
  for (int b = 0; b < nblk; ++b) {
    z += p.part_z[b];
    n += p.part_n[b];
  }
  const double inv = n > 0 ? 1.0 / (double)n : 0.0;
  double dot = 0.0;
  if (e < p.E) {
    double s = 0.0;
    int c = 0;
    for (int b = 0; b < nblk; ++b) {
      s += p.part_p[(int64_t)b * p.E + e];
      c += p.part_c[(int64_t)b * p.E + e];
    }
    p.counts[e] = c;
    if (p.mean) p.mean[e] = (float)(s * inv);
    dot = (double)c * (s * inv);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o, 64);
  if (lane == 0) red[w] = dot;
  __syncthreads();
  if (e == 0) {
    double d = 0.0;
    for (int i = 0; i < kMaxE / 64; ++i) d += red[i];
    p.tokens[0] = (int32_t)n;
    p.losses[0] = (float)(d * inv * (double)p.E / (double)p.k);
    p.losses[1] = (float)(z * inv);
  }
}

template <bool BF16, int PER>
__global__ __launch_bounds__(256) void k_balance_bwd(BalParams p) {
  const int lane = threadIdx.x & 63;
  float c[PER];
  int total = 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 64 * j;
    total += e < p.E ? p.counts[e] : 0;
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) total += __shfl_xor(total, o, 64);
  const double mean = (double)total / (double)p.E;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 64 * j;
    c[j] = e < p.E ? (float)((double)p.counts[e] - mean) : 0.0f;
  }
  const double n = (double)p.tokens[0], inv = n > 0.0 ? 1.0 / n : 0.0;
  const float a = (float)((double)p.grad_losses[0] * (double)p.E / (double)p.k * inv * inv);
  const float b = (float)((double)p.grad_losses[1] * 2.0 * inv);
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < p.T;
       t += (int64_t)gridDim.x * 4) {
    float l[PER], m;
    if (bal_row<BF16, PER>(p, t, l, m)) {
      const float lse = bal_softmax<PER>(l, m);
      float cp = 0.0f;
#pragma unroll
      for (int j = 0; j < PER; ++j) cp += c[j] * l[j];
      cp = wave_sum(cp);
#pragma unroll
      for (int j = 0; j < PER; ++j) l[j] *= a * (c[j] - cp) + b * lse;
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) l[j] = 0.0f;
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int e = lane + 64 * j;
      if (e < p.E) {
        if constexpr (BF16)
          reinterpret_cast<uint16_t*>(p.grad)[t * p.ldg + e] =
              __builtin_bit_cast(uint16_t, (__bf16)l[j]);
        else
          reinterpret_cast<float*>(p.grad)[t * p.ldg + e] = l[j];
      }
    }
  }
}

int fwd_blocks(int64_t T) {
  const int64_t n = (T + kFwdWaves - 1) / kFwdWaves;
  return (int)(n < 1 ? 1 : n < kFwdBlocks ? n : kFwdBlocks);
}

template <bool BF16>
int launch_fwd(const BalParams& p, hipStream_t s) {
  const int nblk = fwd_blocks(p.T);
  const dim3 grid((unsigned)nblk), block(64 * kFwdWaves);
  if (p.E <= 64) hipLaunchKernelGGL((k_balance<BF16, 1>), grid, block, 0, s, p);
  else if (p.E <= 128) hipLaunchKernelGGL((k_balance<BF16, 2>), grid, block, 0, s, p);
  else if (p.E <= 256) hipLaunchKernelGGL((k_balance<BF16, 4>), grid, block, 0, s, p);
  else if (p.E <= 512) hipLaunchKernelGGL((k_balance<BF16, 8>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_balance<BF16, 16>), grid, block, 0, s, p);
  hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(kMaxE), 0, s, p, nblk);
  return nv_launch_status();
}

template <bool BF16>
int launch_bwd(const BalParams& p, hipStream_t s) {
  const int64_t n = (p.T + 3) / 4;
  const dim3 grid((unsigned)(n < 2048 ? n : 2048)), block(256);
  if (p.E <= 64) hipLaunchKernelGGL((k_balance_bwd<BF16, 1>), grid, block, 0, s, p);
  else if (p.E <= 128) hipLaunchKernelGGL((k_balance_bwd<BF16, 2>), grid, block, 0, s, p);
  else if (p.E <= 256) hipLaunchKernelGGL((k_balance_bwd<BF16, 4>), grid, block, 0, s, p);
  else if (p.E <= 512) hipLaunchKernelGGL((k_balance_bwd<BF16, 8>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((k_balance_bwd<BF16, 16>), grid, block, 0, s, p);
  return nv_launch_status();
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
  return nv_round256(8 * (size_t)fwd_blocks(T) * (size_t)(E + 1));
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
  NV_RETURN_IF(!ws || ws_bytes < moe_balance_loss_workspace_size(T, E) || misaligned(ws, 4),
               NVFP4_ERR_WORKSPACE);
  const int64_t nblk = fwd_blocks(T);
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
  p.part_p = reinterpret_cast<float*>(ws);
  p.part_z = p.part_p + nblk * E;
  p.part_c = reinterpret_cast<int32_t*>(p.part_z + nblk);
  p.part_n = p.part_c + nblk * E;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return dtype == NVFP4_IN_BF16 ? launch_fwd<true>(p, s) : launch_fwd<false>(p, s);
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
  return dtype == NVFP4_IN_BF16 ? launch_bwd<true>(p, s) : launch_bwd<false>(p, s);
}

}  // extern "C"
