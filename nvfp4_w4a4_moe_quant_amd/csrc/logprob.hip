// Token log-probabilities, entropies and top alternatives of vocabulary
// logits, and their gradient.
//
// The QUADS pages judge a rollout by the gap between its log-probabilities
// and the trainer's (blog post, section "What it buys"); these kernels compute
// the two sides of that gap.  With c = inv_temperature * log2 e, m = max_j l_j
// and d_j = (l_j - m) c:
//   S = sum 2^d_j,  Q = sum d_j 2^d_j,  log2 p_j = d_j - log2 S,
//   entropy = ln 2 (log2 S - Q / S).
// Base 2 saves the multiplication inside every exponential.  The difference
// comes before the product, so that logits at the type's lowest value (a mask
// that is a number) do not overflow.  Reported log-probabilities are
// (l_j - m) inv_temperature - ln 2 log2 S.
#include "common.h"

namespace {

constexpr int kLpMaxTop = 32;
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

__device__ __forceinline__ float lp_load(const float* p) { return *p; }
__device__ __forceinline__ float lp_load(const uint16_t* p) { return nv_bf16_to_f32(*p); }

__device__ __forceinline__ bool lp_better(float va, int ia, float vb, int ib) {
  return va > vb || (va == vb && ia < ib);
}

// log p of a logit from the row's maximum m and L = log2 S.
__device__ __forceinline__ float lp_value(float l, float m, float it, float L) {
  return l == -kInf ? l : __builtin_fmaf(-kLn2, L, (l - m) * it);
}

// One workgroup per row; top_k further passes for the alternatives.
template <typename E>
__global__ __launch_bounds__(256) void k_logprob(const E* __restrict__ logits, int V, int64_t ld,
                                                 const int64_t* __restrict__ targets,
                                                 const float* __restrict__ inv_t, int top_k,
                                                 float* __restrict__ logprobs,
                                                 float* __restrict__ entropy,
                                                 float* __restrict__ norm,
                                                 int32_t* __restrict__ top_ids,
                                                 float* __restrict__ top_lp) {
  __shared__ float sa[256], sb[256];
  __shared__ int si[256];
  const int64_t t = blockIdx.x;
  const E* row = logits + t * ld;
  const float it = inv_t ? inv_t[t] : 1.0f, c = it * kLog2e;
  const int tid = threadIdx.x;
  float m = -kInf;
  bool bad = false;
  for (int j = tid; j < V; j += 256) {
    const float l = lp_load(row + j);
    bad |= l != l;
    m = __builtin_fmaxf(m, l);
  }
  sa[tid] = bad ? __builtin_nanf("") : m;
  __syncthreads();
  m = -kInf;
  for (int i = 0; i < 256; ++i) m = (sa[i] != sa[i] || m != m) ? __builtin_nanf("") : __builtin_fmaxf(m, sa[i]);
  __syncthreads();
  const bool empty = m == -kInf;
  if (empty) m = 0.0f;
  float s = 0.0f, q = 0.0f;
  for (int j = tid; j < V; j += 256) {
    const float d = (lp_load(row + j) - m) * c;
    const float e = __builtin_amdgcn_exp2f(d);
    s += e;
    if (e > 0.0f || e != e) q = __builtin_fmaf(d, e, q);
  }
  sa[tid] = s;
  sb[tid] = q;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (tid < o) {
      sa[tid] += sa[tid + o];
      sb[tid] += sb[tid + o];
    }
    __syncthreads();
  }
  s = sa[0];
  q = sb[0];
  const float L = empty ? -kInf : __builtin_log2f(s);
  __syncthreads();
  if (tid == 0) {
    if (logprobs) {
      const int64_t y = targets[t];
      float lp = 0.0f;
      if (y >= V) lp = __builtin_nanf("");
      else if (y >= 0) {
        lp = lp_value(lp_load(row + y), m, it, L);
      }
      logprobs[t] = lp;
    }
    if (entropy) entropy[t] = empty ? 0.0f : (L - q / s) * kLn2;
    if (norm) {
      norm[2 * t] = m;
      norm[2 * t + 1] = L;
    }
  }
  float pv = kInf;
  int pi = -1;  // the last alternative written
  for (int k = 0; k < top_k; ++k) {
    float bv = -kInf;
    int bi = 0x7fffffff;
    for (int j = tid; j < V; j += 256) {
      float l = lp_load(row + j);
      if (l != l) l = -kInf;
      const bool left = pi < 0 || lp_better(pv, pi, l, j);  // ranked after the last one
      if (left && lp_better(l, j, bv, bi)) {
        bv = l;
        bi = j;
      }
    }
    sa[tid] = bv;
    si[tid] = bi;
    __syncthreads();
    for (int i = 0; i < 256; ++i)
      if (lp_better(sa[i], si[i], bv, bi)) {
        bv = sa[i];
        bi = si[i];
      }
    __syncthreads();
    pv = bv;
    pi = bi;
    if (tid == 0) {
      top_ids[t * top_k + k] = bi;
      top_lp[t * top_k + k] = s == s ? lp_value(bv, m, it, L) : s;
    }
  }
}

__device__ __forceinline__ void lp_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void lp_store(uint16_t* p, float v) {
  *p = v != v ? (uint16_t)0x7FC0 : (uint16_t)nv_f32_to_bf16(v);
}

template <typename E>
__global__ __launch_bounds__(256) void k_logprob_bwd(
    const E* logits, int V, int64_t ld, const int64_t* __restrict__ targets,
    const float* __restrict__ inv_t, const float* __restrict__ norm,
    const float* __restrict__ entropy, const float* __restrict__ g_lp,
    const float* __restrict__ g_ent, E* grad, int64_t ldg) {
  const int64_t t = blockIdx.x;
  const float it = inv_t ? inv_t[t] : 1.0f;
  const float m = norm[2 * t], L = norm[2 * t + 1], c = it * kLog2e;
  const bool empty = L == -kInf;
  const int64_t y = targets ? targets[t] : -1;
  float a = (g_lp && y >= 0 && !empty) ? g_lp[t] : 0.0f;
  if (g_lp && y >= V) a = __builtin_nanf("");
  const float b = g_ent ? g_ent[t] : 0.0f, h = g_ent ? entropy[t] : 0.0f;
  for (int j = threadIdx.x; j < V; j += 256) {
    const float d = empty ? -kInf : (lp_load(logits + t * ld + j) - m) * c - L;
    const float p = __builtin_amdgcn_exp2f(d);
    float g = (j == y ? a : 0.0f) - p * a;
    if (p > 0.0f) g -= b * p * (d * kLn2 + h);
    lp_store(grad + t * ldg + j, it * g);
  }
}

}  // namespace

extern "C" {

size_t token_logprobs_workspace_size(int64_t, int64_t, int64_t) { return 256; }

int token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                   const int64_t* targets, const float* inv_temperature, int64_t top_k,
                   float* logprobs, float* entropy, float* norm, int32_t* top_ids,
                   float* top_logprobs, void* ws, size_t ws_bytes, void* stream) {
  NV_RETURN_IF(dtype != NVFP4_IN_F32 && dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(T < 0 || T > INT32_MAX || V < 1 || V > INT32_MAX || ld < V || top_k < 0 ||
                   top_k > kLpMaxTop || top_k > V,
               NVFP4_ERR_SHAPE);
  if (T == 0) return NVFP4_OK;
  NV_RETURN_IF(!logits || (targets == nullptr) != (logprobs == nullptr) ||
                   (top_k > 0 && (!top_ids || !top_logprobs)),
               NVFP4_ERR_NULL);
  NV_RETURN_IF((reinterpret_cast<uintptr_t>(logits) & (dtype == NVFP4_IN_F32 ? 3 : 1)),
               NVFP4_ERR_ALIGN);
  NV_RETURN_IF(!ws || ws_bytes < token_logprobs_workspace_size(T, V, top_k) ||
                   (reinterpret_cast<uintptr_t>(ws) & 15),
               NVFP4_ERR_WORKSPACE);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)T);
  if (dtype == NVFP4_IN_F32)
    hipLaunchKernelGGL(k_logprob<float>, grid, dim3(256), 0, s, (const float*)logits, (int)V, ld,
                       targets, inv_temperature, (int)top_k, logprobs, entropy, norm, top_ids,
                       top_logprobs);
  else
    hipLaunchKernelGGL(k_logprob<uint16_t>, grid, dim3(256), 0, s, (const uint16_t*)logits, (int)V,
                       ld, targets, inv_temperature, (int)top_k, logprobs, entropy, norm, top_ids,
                       top_logprobs);
  return nv_launch_status();
}

int token_logprobs_backward(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                            const int64_t* targets, const float* inv_temperature,
                            const float* norm, const float* entropy, const float* grad_logprobs,
                            const float* grad_entropy, void* grad_logits, int64_t ldg,
                            void* stream) {
  NV_RETURN_IF(dtype != NVFP4_IN_F32 && dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(T < 0 || T > INT32_MAX || V < 1 || V > INT32_MAX || ld < V || ldg < V ||
                   (logits == grad_logits && ld != ldg),
               NVFP4_ERR_SHAPE);
  if (T == 0) return NVFP4_OK;
  NV_RETURN_IF(!logits || !norm || !grad_logits || (grad_logprobs && !targets) ||
                   (grad_entropy && !entropy),
               NVFP4_ERR_NULL);
  const uintptr_t mask = dtype == NVFP4_IN_F32 ? 3 : 1;
  NV_RETURN_IF((reinterpret_cast<uintptr_t>(logits) & mask) ||
                   (reinterpret_cast<uintptr_t>(grad_logits) & mask),
               NVFP4_ERR_ALIGN);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)T);
  if (dtype == NVFP4_IN_F32)
    hipLaunchKernelGGL(k_logprob_bwd<float>, grid, dim3(256), 0, s, (const float*)logits, (int)V,
                       ld, targets, inv_temperature, norm, entropy, grad_logprobs, grad_entropy,
                       (float*)grad_logits, ldg);
  else
    hipLaunchKernelGGL(k_logprob_bwd<uint16_t>, grid, dim3(256), 0, s, (const uint16_t*)logits,
                       (int)V, ld, targets, inv_temperature, norm, entropy, grad_logprobs,
                       grad_entropy, (uint16_t*)grad_logits, ldg);
  return nv_launch_status();
}

}  // extern "C"
