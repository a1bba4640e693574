// INT8 W8A8 comparator: per-row quantizer and grouped GEMM.
//
// One FP32 scale per activation row (at run time) and per weight output
// channel: s = RN32(amax / 127), r = RN32(1 / s), code = the nearest integer to
// RN32(x r).  A product is y = s_a s_w sum_k a_k w_k with the sum exact in 32-bit
// integers (K <= 131056), whatever its order.

#include <type_traits>

#include "common.h"

namespace {

typedef int int4v __attribute__((ext_vector_type(4)));

constexpr int64_t kMaxK = 131056;  // 128^2 K < 2^31

__device__ __forceinline__ uint16_t i8_bf16(float f) {  // nearest even; a NaN stays one
  return __builtin_bit_cast(uint16_t, (__bf16)f);
}

// ------------------------------------------------------------------ quantizer

// 8 consecutive inputs at element offset `off` (16-byte aligned).
template <bool BF16>
__device__ __forceinline__ void i8_load8(const void* x, int64_t off, float* v) {
  if constexpr (BF16) {
    const uint4 a = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(x) + off);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const float4* q = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(x) + off);
    const float4 a = q[0], b = q[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
}

// |x| as an integer orders like |x|, with infinities and NaN above all numbers.
__device__ __forceinline__ uint32_t i8_mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t i8_wave_max(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const uint32_t w = (uint32_t)__shfl_xor((int)v, o, 64);
    v = v > w ? v : w;
  }
  return v;
}

// Scale and reciprocal of a row from the largest magnitude.  The floor of
// 2^-126 keeps 1 / s finite and the codes of a row of subnormals in range.
// r = 0 (a zero or non-finite row) gives codes 0.
__device__ __forceinline__ void i8_row_scale(uint32_t mag, float& s, float& r) {
  if (mag >= 0x7F800000u) {
    s = __uint_as_float(0x7FC00000u);
    r = 0.0f;
  } else if (mag == 0u) {
    s = r = 0.0f;
  } else {
    s = __builtin_fmaxf((float)((double)__uint_as_float(mag) / 127.0), 0x1p-126f);
    r = (float)(1.0 / (double)s);
  }
}

// 8 values times r -> 8 codes.  Adding 1.5 * 2^23 leaves the nearest integer
// (ties to even) in the sum's low bits, whose lowest byte is the code; |x r|
// is at most 127 (1 + 2^-22).  With r = 0 the values may be infinite or NaN
// and are not used.
__device__ __forceinline__ uint2 i8_encode8(const float* v, float r) {
  if (r == 0.0f) return make_uint2(0u, 0u);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i] = __float_as_uint(v[i] * r + 12582912.0f);
  uint2 o;
  o.x = (c[0] & 255u) | ((c[1] & 255u) << 8) | ((c[2] & 255u) << 16) | (c[3] << 24);
  o.y = (c[4] & 255u) | ((c[5] & 255u) << 8) | ((c[6] & 255u) << 16) | (c[7] << 24);
  return o;
}

// One wave per row, four rows per workgroup; the row is read twice (the
// second read hits the caches).
template <bool BF16>
__global__ __launch_bounds__(256) void k_i8_rows(const void* x, int64_t rows, int K, int64_t ldx,
                                                 int8_t* codes, float* scales) {
  const int lane = threadIdx.x & 63;
  const int nv = K >> 3;
  for (int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); row < rows;
       row += (int64_t)gridDim.x * 4) {
    uint32_t mag = 0;
    for (int c = lane; c < nv; c += 64) {
      float v[8];
      i8_load8<BF16>(x, row * ldx + 8 * c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) mag = max(mag, i8_mag(v[e]));
    }
    float s, r;
    i8_row_scale(i8_wave_max(mag), s, r);
    for (int c = lane; c < nv; c += 64) {
      float v[8];
      i8_load8<BF16>(x, row * ldx + 8 * c, v);
      *reinterpret_cast<uint2*>(codes + row * (int64_t)K + 8 * c) = i8_encode8(v, r);
    }
    if (lane == 0) scales[row] = s;
  }
}

// ----------------------------------------------------------------------- GEMM

struct I8Params {
  int G, N, K, total_rows;
  const int32_t* offsets;  // NULL: one group
  const int32_t* gather;
  const int8_t* a_codes;
  const float* a_scales;
  const int8_t* w_codes;
  const float* w_scales;
  void* out;
};

// silu(g) * u in FP32 with the hardware exp and reciprocal.
__device__ __forceinline__ float i8_silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// A wave computes 16 rows of one group by 16 output columns (with SiLU*mul 16
// gate and the 16 up columns) over the whole of K, its operands read from
// memory in v_mfma_i32_16x16x64_i8's layout: lane l feeds row (or column) l % 16
// with the 16 bytes k = 16 (l / 16) + 0..15 of a 64-k step.  Workgroups of four
// waves (64 columns), grid (column blocks, groups).
template <int EPI, bool GATHER>
__global__ __launch_bounds__(256) void k_i8_direct(I8Params p) {
  constexpr bool SILU = EPI == NVFP4_EPI_SILU_MUL_BF16;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int cols = SILU ? p.N >> 1 : p.N;
  const int n0 = (int)(blockIdx.x * 4 + wave) * 16;
  if (n0 >= cols) return;
  const int nw = min(n0 + c, cols - 1);
  for (int grp = (int)blockIdx.y; grp < p.G; grp += (int)gridDim.y) {
    const int beg = p.offsets ? p.offsets[grp] : 0;
    const int end = p.offsets ? p.offsets[grp + 1] : p.total_rows;
    const int64_t wrow = (int64_t)grp * p.N + nw;
    const int8_t* w0 = p.w_codes + wrow * p.K;
    const int8_t* w1 = w0 + (SILU ? (int64_t)cols * p.K : 0);
    for (int m0 = beg; m0 < end; m0 += 16) {
      const int m = min(m0 + c, end - 1);
      const int64_t src = GATHER ? (int64_t)p.gather[m] : (int64_t)m;
      const int8_t* a = p.a_codes + src * p.K;
      int4v acc = {0, 0, 0, 0}, acc1 = {0, 0, 0, 0};
      for (int k = 0; k < p.K; k += 64) {
        const int kk = k + 16 * q;
        int4v av = {0, 0, 0, 0}, wv = {0, 0, 0, 0}, uv = {0, 0, 0, 0};
        if (kk < p.K) {
          av = *reinterpret_cast<const int4v*>(a + kk);
          wv = *reinterpret_cast<const int4v*>(w0 + kk);
          if constexpr (SILU) uv = *reinterpret_cast<const int4v*>(w1 + kk);
        }
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, wv, acc, 0, 0, 0);
        if constexpr (SILU) acc1 = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, uv, acc1, 0, 0, 0);
      }
      // element i of lane (c, q): row m0 + 4 q + i, column n0 + c
      if (n0 + c >= cols) continue;
      const float sw = p.w_scales[wrow];
      const float su = SILU ? p.w_scales[wrow + cols] : 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = m0 + 4 * q + i;
        if (row >= end) break;
        const float sa = p.a_scales[GATHER ? (int64_t)p.gather[row] : (int64_t)row];
        const float y = (sa * sw) * (float)acc[i];
        const int64_t o = (int64_t)row * cols + n0 + c;
        if constexpr (SILU)
          reinterpret_cast<uint16_t*>(p.out)[o] = i8_bf16(i8_silu_mul(y, (sa * su) * (float)acc1[i]));
        else if constexpr (EPI == NVFP4_EPI_BF16)
          reinterpret_cast<uint16_t*>(p.out)[o] = i8_bf16(y);
        else
          reinterpret_cast<float*>(p.out)[o] = y;
      }
    }
  }
}

template <int EPI>
int launch_direct(const I8Params& p, hipStream_t s) {
  const int cols = EPI == NVFP4_EPI_SILU_MUL_BF16 ? p.N / 2 : p.N;
  const dim3 grid((unsigned)((cols + 63) / 64), (unsigned)min(p.G, 65535));
  if (p.gather)
    hipLaunchKernelGGL((k_i8_direct<EPI, true>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((k_i8_direct<EPI, false>), grid, dim3(256), 0, s, p);
  return nv_launch_status();
}

int launch_rows(const void* x, int64_t dtype, int64_t rows, int K, int64_t ldx, int8_t* codes,
                float* scales, hipStream_t s) {
  const int64_t wgs = (rows + 3) / 4;
  const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20)));
  if (dtype == NVFP4_IN_BF16)
    hipLaunchKernelGGL(k_i8_rows<true>, grid, dim3(256), 0, s, x, rows, K, ldx, codes, scales);
  else
    hipLaunchKernelGGL(k_i8_rows<false>, grid, dim3(256), 0, s, x, rows, K, ldx, codes, scales);
  return nv_launch_status();
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The checks shared by the workspace size and the call.
int check_gemm(const int8_gemm_args_t* a) {
  NV_RETURN_IF(!a, NVFP4_ERR_NULL);
  NV_RETURN_IF(a->epilogue != NVFP4_EPI_F32 && a->epilogue != NVFP4_EPI_SILU_MUL_BF16 &&
                   a->epilogue != NVFP4_EPI_BF16,
               NVFP4_ERR_DTYPE);
  NV_RETURN_IF(a->num_groups < 1 || a->num_groups > (1 << 20) || a->total_rows < 0 ||
                   a->total_rows > 0x7fffffff || a->N < 1 || a->N > (1 << 24) || a->K < 16 ||
                   a->K % 16 || a->K > kMaxK ||
                   (a->epilogue == NVFP4_EPI_SILU_MUL_BF16 && a->N % 2),
               NVFP4_ERR_SHAPE);
  if (a->x) {
    NV_RETURN_IF(a->x_dtype != NVFP4_IN_F32 && a->x_dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
    NV_RETURN_IF(a->src_rows < 0 || a->src_rows > 0x7fffffff || a->ldx < a->K ||
                     (!a->gather_rows && a->src_rows < a->total_rows) ||
                     (a->src_rows == 0 && a->total_rows > 0),
                 NVFP4_ERR_SHAPE);
  }
  return NVFP4_OK;
}

}  // namespace

extern "C" {

int int8_quantize_rows(const void* x, int in_dtype, int64_t rows, int64_t K, int64_t ldx,
                       int8_t* codes, float* row_scales, void* stream) {
  NV_RETURN_IF(in_dtype != NVFP4_IN_F32 && in_dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(rows < 0 || K <= 0 || K % 16 || K > (1 << 24) || rows > 0x7fffffffLL || ldx < K,
               NVFP4_ERR_SHAPE);
  if (rows == 0) return NVFP4_OK;
  NV_RETURN_IF(!x || !codes || !row_scales, NVFP4_ERR_NULL);
  NV_RETURN_IF(misaligned(x, 16) || misaligned(codes, 16) || misaligned(row_scales, 4) || ldx % 8,
               NVFP4_ERR_ALIGN);
  return launch_rows(x, in_dtype, rows, (int)K, ldx, codes, row_scales,
                     reinterpret_cast<hipStream_t>(stream));
}

size_t int8_grouped_gemm_workspace_size(const int8_gemm_args_t* a) {
  if (check_gemm(a) != NVFP4_OK || !a->x || a->total_rows == 0) return 0;
  return nv_round256((size_t)a->src_rows * (size_t)a->K) + nv_round256(4 * (size_t)a->src_rows);
}

int int8_grouped_gemm(const int8_gemm_args_t* a, void* ws, size_t ws_bytes, void* stream) {
  const int bad = check_gemm(a);
  if (bad != NVFP4_OK) return bad;
  NV_RETURN_IF(!a->w_codes || !a->w_scales || (!a->group_offsets && a->num_groups > 1),
               NVFP4_ERR_NULL);
  if (a->total_rows == 0) return NVFP4_OK;
  NV_RETURN_IF(!a->out || (!a->x && (!a->a_codes || !a->a_scales)), NVFP4_ERR_NULL);
  NV_RETURN_IF(a->x && (a->a_codes || a->a_scales), NVFP4_ERR_SHAPE);
  const unsigned esize = a->epilogue == NVFP4_EPI_F32 ? 4 : 2;
  NV_RETURN_IF(misaligned(a->w_codes, 16) || misaligned(a->w_scales, 4) ||
                   misaligned(a->group_offsets, 4) || misaligned(a->gather_rows, 4) ||
                   misaligned(a->out, esize) || misaligned(a->a_codes, 16) ||
                   misaligned(a->a_scales, 4) || (a->x && (misaligned(a->x, 16) || a->ldx % 8)),
               NVFP4_ERR_ALIGN);
  const size_t need = int8_grouped_gemm_workspace_size(a);
  NV_RETURN_IF(need && (!ws || ws_bytes < need || misaligned(ws, 16)), NVFP4_ERR_WORKSPACE);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  I8Params p{};
  p.G = (int)a->num_groups;
  p.N = (int)a->N;
  p.K = (int)a->K;
  p.total_rows = (int)a->total_rows;
  p.offsets = a->group_offsets;
  p.gather = a->gather_rows;
  p.a_codes = a->a_codes;
  p.a_scales = a->a_scales;
  p.w_codes = a->w_codes;
  p.w_scales = a->w_scales;
  p.out = a->out;
  if (a->x) {
    int8_t* codes = reinterpret_cast<int8_t*>(ws);
    float* scales = reinterpret_cast<float*>(codes + nv_round256((size_t)a->src_rows * p.K));
    p.a_codes = codes;
    p.a_scales = scales;
    const int st = launch_rows(a->x, a->x_dtype, a->src_rows, p.K, a->ldx, codes, scales, s);
    if (st != NVFP4_OK) return st;
  }
  if (a->epilogue == NVFP4_EPI_SILU_MUL_BF16) return launch_direct<NVFP4_EPI_SILU_MUL_BF16>(p, s);
  if (a->epilogue == NVFP4_EPI_BF16) return launch_direct<NVFP4_EPI_BF16>(p, s);
  return launch_direct<NVFP4_EPI_F32>(p, s);
}

}  // extern "C"
