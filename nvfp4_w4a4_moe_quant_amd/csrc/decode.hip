// A whole MoE FFN layer for a few tokens on the NVFP4 expert weights.
//
// QUADS blog post, section "Two fixes, on two different sides": the trainer
// fake-quantizes its weights and leaves its activations alone.  For a handful
// of tokens the layer costs the bytes of the routed experts' weights whatever
// the activations are, so this path multiplies unquantized activations and
// needs neither the quantizer nor the residual pass.
#include "common.h"

namespace {

constexpr int kDcMaxT = 64;
constexpr int kDcMaxE = 1024;
constexpr int kDcMaxK = 16;
constexpr int kDcMaxDim = 65536;

struct DecodeParams {
  int T, E, k, H, I;
  const void* x;
  int64_t ldx;
  const float* logits;
  int64_t ldl;
  const uint8_t *gu_codes, *gu_scales;
  const float* gu_ts;
  const uint8_t *d_codes, *d_scales;
  const float* d_ts;
  void* out;
  int64_t ldo;
  int32_t *user_ids, *ids;  // caller's (nullable), workspace's
  float *user_wts, *wts;
  float* h;  // [T k, I]
};

__device__ __forceinline__ float dc_logit(float l) { return l != l ? -__builtin_inff() : l; }

// One wave per token: k rounds of a wave arg-max.
__global__ __launch_bounds__(64) void k_dc_route(DecodeParams p) {
  const int t = blockIdx.x, lane = threadIdx.x;
  const float* row = p.logits + t * p.ldl;
  float pv = __builtin_inff(), mx = 0.0f, den = 0.0f;
  int pi = -1;
  for (int s = 0; s < p.k; ++s) {
    float bv = -__builtin_inff();
    int bi = 0x7fffffff;
    for (int e = lane; e < p.E; e += 64) {
      const float l = dc_logit(row[e]);
      const bool left = pi < 0 || pv > l || (pv == l && pi < e);
      if (left && (l > bv || (l == bv && e < bi))) {
        bv = l;
        bi = e;
      }
    }
    for (int o = 32; o > 0; o >>= 1) {
      const float ov = __shfl_xor(bv, o, 64);
      const int oi = __shfl_xor(bi, o, 64);
      if (ov > bv || (ov == bv && oi < bi)) {
        bv = ov;
        bi = oi;
      }
    }
    if (s == 0) {
      mx = bv;
      for (int e = lane; e < p.E; e += 64) den += __expf(dc_logit(row[e]) - mx);
      for (int o = 32; o > 0; o >>= 1) den += __shfl_xor(den, o, 64);
    }
    pv = bv;
    pi = bi;
    if (lane == 0) {
      const float w = bv == -__builtin_inff() ? 0.0f : __expf(bv - mx) / den;
      p.ids[t * p.k + s] = bi;
      p.wts[t * p.k + s] = w;
      if (p.user_ids) p.user_ids[t * p.k + s] = bi;
      if (p.user_wts) p.user_wts[t * p.k + s] = w;
    }
  }
}

// Dot product of W row (codes, scales) with v over K, spread over a wave.
template <typename F>
__device__ __forceinline__ float dc_dot(const uint8_t* codes, const uint8_t* scales, int K, F v) {
  float acc = 0.0f;
  for (int k = (threadIdx.x & 63) * 8; k < K; k += 512) {
    float g[8], s = 0.0f;
    nv_decode8(*reinterpret_cast<const uint32_t*>(codes + (k >> 1)), g);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __builtin_fmaf(g[i], v(k + i), s);
    acc = __builtin_fmaf(s, nv_e4m3_to_f32(scales[k >> 4]), acc);
  }
  for (int o = 32; o > 0; o >>= 1) acc += __shfl_xor(acc, o, 64);
  return acc;
}

// One wave per (pair, intermediate column).
template <bool kBf16>
__global__ __launch_bounds__(256) void k_dc_gate_up(DecodeParams p) {
  const int pair = blockIdx.y, i = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= p.I || !(p.wts[pair] > 0.0f)) return;
  const int e = p.ids[pair];
  const int64_t row = (int64_t)(pair / p.k) * p.ldx;
  auto x = [&](int k) -> float {
    return kBf16 ? nv_bf16_to_f32(reinterpret_cast<const uint16_t*>(p.x)[row + k])
                 : reinterpret_cast<const float*>(p.x)[row + k];
  };
  float y[2];
  for (int half = 0; half < 2; ++half) {
    const int64_t n = (int64_t)e * 2 * p.I + half * p.I + i;
    y[half] = p.gu_ts[e] * dc_dot(p.gu_codes + n * (p.H >> 1), p.gu_scales + n * (p.H >> 4), p.H, x);
  }
  if ((threadIdx.x & 63) == 0) p.h[(int64_t)pair * p.I + i] = y[0] / (1.0f + __expf(-y[0])) * y[1];
}

// One wave per (token, output column).
template <bool kBf16>
__global__ __launch_bounds__(256) void k_dc_down(DecodeParams p) {
  const int t = blockIdx.y, n = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (n >= p.H) return;
  float acc = 0.0f;
  for (int s = 0; s < p.k; ++s) {
    const int pair = t * p.k + s;
    const float w = p.wts[pair];
    if (!(w > 0.0f)) continue;
    const int e = p.ids[pair];
    const int64_t r = (int64_t)e * p.H + n;
    const float* h = p.h + (int64_t)pair * p.I;
    const float y = dc_dot(p.d_codes + r * (p.I >> 1), p.d_scales + r * (p.I >> 4), p.I,
                           [&](int k) { return h[k]; });
    acc += w * (p.d_ts[e] * y);
  }
  if ((threadIdx.x & 63) == 0) {
    if (kBf16)
      reinterpret_cast<uint16_t*>(p.out)[t * p.ldo + n] =
          acc != acc ? (uint16_t)0x7FC0 : (uint16_t)nv_f32_to_bf16(acc);
    else
      reinterpret_cast<float*>(p.out)[t * p.ldo + n] = acc;
  }
}

}  // namespace

extern "C" {

size_t nvfp4_moe_decode_workspace_size(const nvfp4_moe_decode_args_t* a) {
  if (!a || a->T < 0 || a->T > kDcMaxT || a->k < 1 || a->k > kDcMaxK || a->I < 0 ||
      a->I > kDcMaxDim)
    return 0;
  const size_t P = (size_t)(a->T * a->k);
  return 2 * nv_round256(P * 4) + nv_round256(P * (size_t)a->I * 4);
}

int nvfp4_moe_decode(const nvfp4_moe_decode_args_t* a, void* ws, size_t ws_bytes, void* stream) {
  NV_RETURN_IF(!a, NVFP4_ERR_NULL);
  NV_RETURN_IF(a->x_dtype != NVFP4_IN_F32 && a->x_dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(a->T < 0 || a->T > kDcMaxT || a->E < 1 || a->E > kDcMaxE || a->k < 1 ||
                   a->k > a->E || a->k > kDcMaxK || a->H < 32 || a->H > kDcMaxDim || a->H % 32 ||
                   a->I < 32 || a->I > kDcMaxDim || a->I % 32 || a->ldx < a->H ||
                   a->ldo < a->H || a->ld_logits < a->E,
               NVFP4_ERR_SHAPE);
  if (a->T == 0) return NVFP4_OK;
  NV_RETURN_IF(!a->x || !a->logits || !a->gu_codes || !a->gu_scales || !a->gu_tscale ||
                   !a->d_codes || !a->d_scales || !a->d_tscale || !a->out,
               NVFP4_ERR_NULL);
  NV_RETURN_IF(!nv_aligned16(a->x) || !nv_aligned16(a->out) || !nv_aligned16(a->gu_codes) ||
                   !nv_aligned16(a->gu_scales) || !nv_aligned16(a->d_codes) ||
                   !nv_aligned16(a->d_scales) || a->ldx % 8 || a->ldo % 8 ||
                   (reinterpret_cast<uintptr_t>(a->logits) & 3) ||
                   (reinterpret_cast<uintptr_t>(a->gu_tscale) & 3) ||
                   (reinterpret_cast<uintptr_t>(a->d_tscale) & 3) ||
                   (reinterpret_cast<uintptr_t>(a->topk_ids) & 3) ||
                   (reinterpret_cast<uintptr_t>(a->topk_weights) & 3),
               NVFP4_ERR_ALIGN);
  NV_RETURN_IF(!ws || ws_bytes < nvfp4_moe_decode_workspace_size(a) || !nv_aligned16(ws),
               NVFP4_ERR_WORKSPACE);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const size_t P = (size_t)(a->T * a->k);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  DecodeParams p{(int)a->T, (int)a->E, (int)a->k, (int)a->H, (int)a->I, a->x, a->ldx,
                 a->logits, a->ld_logits, a->gu_codes, a->gu_scales, a->gu_tscale,
                 a->d_codes, a->d_scales, a->d_tscale, a->out, a->ldo,
                 a->topk_ids, reinterpret_cast<int32_t*>(w),
                 a->topk_weights, reinterpret_cast<float*>(w + nv_round256(P * 4)),
                 reinterpret_cast<float*>(w + 2 * nv_round256(P * 4))};
  const bool bf = a->x_dtype == NVFP4_IN_BF16;
  const dim3 g1((unsigned)((p.I + 3) / 4), (unsigned)P), g2((unsigned)((p.H + 3) / 4), (unsigned)p.T);
  hipLaunchKernelGGL(k_dc_route, dim3((unsigned)p.T), dim3(64), 0, s, p);
  if (bf) {
    hipLaunchKernelGGL(k_dc_gate_up<true>, g1, dim3(256), 0, s, p);
    hipLaunchKernelGGL(k_dc_down<true>, g2, dim3(256), 0, s, p);
  } else {
    hipLaunchKernelGGL(k_dc_gate_up<false>, g1, dim3(256), 0, s, p);
    hipLaunchKernelGGL(k_dc_down<false>, g2, dim3(256), 0, s, p);
  }
  return nv_launch_status();
}

}  // extern "C"
