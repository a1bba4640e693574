// A whole MoE FFN layer for a few tokens on the NVFP4 expert weights.
//
// QUADS blog post, section "Two fixes, on two different sides": the trainer
// fake-quantizes its weights and leaves its activations alone.  For a handful
// of tokens the layer costs the bytes of the routed experts' weights whatever
// the activations are, so this path multiplies unquantized activations and
// needs neither the quantizer nor the residual pass.
//
//   k_dc_route    one wave per token: top-k, softmax weights (where the
//                 gate/up kernel does not route by itself)
//   k_dc_gate_up  tables of the routed rows by expert, then h = silu(g) u of
//                 every routed (token, slot) pair, to the workspace
//   k_dc_down     the down product, weighted and summed over each token's
//                 experts, to the output
//
// Both products stream W, 0.5625 bytes a weight, once for every 16 rows of an
// expert, and with few rows an expert that is what bounds them: 16 tokens of a
// layer of 256 experts, H 7168, I 2048 (103 experts, 1.70 and 0.85 GB) take 285
// (279-298) and 158 (151-173) us, 6.0 and 5.4 TB/s where a large copy reaches 4.9
// on this card; the same with the arithmetic taken out takes as long.  (Medians
// and ranges of settled calls: the first 40 after an idle time are up to a
// third slower.)  One token (8 experts) takes 27 and 20 us: some 8 us of the
// first and 5 us of the second pass before the stream runs (routing 3, first
// loads 4), and the join of the parts is another 4 us of the second, which is
// all of it in small layers (128 experts, H 2048, I 768: 10 and 9 us, 16 tokens 67
// us for 47 us of bytes).  With more than 16 rows an expert W is read again: 64
// tokens of 16 experts, top-8, H 4096, I 2048 (39 tiles of rows) take 163 us for
// 46 us of bytes.
//
// v_mfma_f32_16x16x32_f16 (16 tokens x 16 columns): lane (c, q) of a wave
// takes column c and, of each group of 128 k, the 16 code bytes of k = 32 q ..
// 32 q + 31 for four MFMA steps of 8 k -- the same permutation of k for both
// operands.  g * s_b is exact in fp16.  Activations enter as fp16 pieces: a
// row's values in one K range are scaled by a power of two to just below
// 2^15, so that one piece holds a bf16 value exactly (down to 2^-29 of the
// largest) and two hold 22 bits of an FP32 value; the FP32 sums of the range
// are scaled back.  h goes from one product to the other in the same form
// (rounded to 11 bits for bf16, an eighth of bf16's step; to 22 for FP32).  A
// wave keeps the fragments of its rows in registers for every column of its
// work; W loads run two column slabs ahead of their use.
#include <cmath>

#include "common.h"

namespace {

typedef _Float16 half8 __attribute__((ext_vector_type(8)));
typedef _Float16 half2v __attribute__((ext_vector_type(2)));
typedef float float4v __attribute__((ext_vector_type(4)));
typedef uint32_t word4 __attribute__((ext_vector_type(4)));

constexpr int kDcMaxT = 64;
constexpr int kDcMaxE = 1024;
constexpr int kDcMaxK = 16;
constexpr int kDcMaxDim = 65536;
constexpr int kDcMaxPairs = kDcMaxT * kDcMaxK;
constexpr int kDcMaxTiles = kDcMaxPairs;  // 16-row tiles: at most one per pair
constexpr int kDcThreads = 256;
constexpr int kDcWaves = kDcThreads / 64;
constexpr int kDcGrid = 512;     // two workgroups on each of 256 CUs
// The gate/up kernel routes by itself for few tokens (every workgroup does
// it all): 1 token of the 128-expert layer 21.4 against 22.2 us with a launch
// before it, 4 tokens 38.9 / 39.9, 8 tokens 53.3 / 51.9.
constexpr int kDcInlineT = 4;
constexpr int kDcInlineE = 256;
constexpr int kDcRow = 1024 + 16;  // bytes of a staged row: 512 k x 1 piece or 256 k x 2, padded
constexpr int kDcStageRows = 8;
constexpr int kDcAcc = 2048;       // output sums of a wave of k_dc_down
constexpr int kDcMaxParts = 16;
__host__ __device__ inline int dc_pad(int I) { return (I + 127) & ~127; }

struct DcRows;
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
  // h of a pair as fp16 pieces [T k, pieces, Ip] and an exponent byte per 16
  // columns [T k, Ip / 16]; Ip is I rounded up to whole groups of 128
  uint16_t* h;
  uint8_t* hexp;
  float* part;  // [parts, T, H]
  int32_t* count;  // per column block of k_dc_down
  DcRows* rows;  // the row tables for k_dc_down
  int blocks;      // column blocks
  int ks_up, ks_down;  // waves that share K (the others share the columns)
};

// What the lanes of a wave wrote to LDS before it, all of them read after it.
__device__ __forceinline__ void dc_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// ---------------------------------------------------------------- routing
// Float order as unsigned order; a NaN counts as -inf, and 0 is below both.
__device__ __forceinline__ uint32_t dc_key(float l) {
  if (l != l) l = -__builtin_inff();
  const uint32_t u = __float_as_uint(l + 0.0f);  // -0 equals +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float dc_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// Maximum over the wave: four steps within rows of 16 lanes, then the four
// rows' values on the scalar unit.
__device__ __forceinline__ uint32_t dc_wave_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));   // xor 1
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));   // xor 2
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // half mirror
  v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // mirror
  const uint32_t a = __builtin_amdgcn_readlane((int)v, 0), b = __builtin_amdgcn_readlane((int)v, 16);
  const uint32_t c = __builtin_amdgcn_readlane((int)v, 32), d = __builtin_amdgcn_readlane((int)v, 48);
  return max(max(a, b), max(c, d));
}

// Maximum over each row of 16 lanes.
__device__ __forceinline__ float dc_row_max(float v) {
  auto step = [](float a, int b) { return __builtin_fmaxf(a, __builtin_bit_cast(float, b)); };
  v = step(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false));
  v = step(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false));
  v = step(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false));
  return step(v, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false));
}

// Top-k of token t by one wave, PER logits per lane (E <= 64 PER).  The ids
// and weights go to sid / swt, and to the workspace and the caller's arrays if
// `store`.
template <int PER>
__device__ __forceinline__ void dc_route_token(const DecodeParams& p, int t, int32_t* sid,
                                               float* swt, bool store) {
  const int lane = threadIdx.x & 63;
  const float* row = p.logits + t * p.ldl;
  uint32_t key[PER];
  float l[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int e = lane + 64 * j;
    l[j] = e < p.E ? row[e] : -__builtin_inff();
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) key[j] = lane + 64 * j < p.E ? dc_key(l[j]) : 0u;
  uint32_t mx = 0u, mine = 0u;  // lane s keeps the s-th choice
  int id = 0;
  float den = 0.0f;
  for (int s = 0; s < p.k; ++s) {
    uint32_t b = 0u;
#pragma unroll
    for (int j = 0; j < PER; ++j) b = max(b, key[j]);
    b = dc_wave_max(b);
    int e = 0;
    bool found = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const uint64_t at = __ballot(key[j] == b);
      if (!found && at) {
        const int who = __ffsll((unsigned long long)at) - 1;
        e = 64 * j + who;
        if (lane == who) key[j] = 0u;
        found = true;
      }
    }
    if (s == 0) {
      mx = b;
      const float m = dc_unkey(b);
#pragma unroll
      for (int j = 0; j < PER; ++j)
        if (lane + 64 * j < p.E && l[j] == l[j]) den += __expf(l[j] - m);
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) den += __shfl_xor(den, o, 64);
    }
    if (lane == s) {
      mine = b;
      id = e;
    }
  }
  if (lane < p.k) {
    const float v = dc_unkey(mine);
    const float w = v == -__builtin_inff() ? 0.0f : __expf(v - dc_unkey(mx)) / den;
    const int i = t * p.k + lane;
    if (sid) {
      sid[i] = id;
      swt[i] = w;
    }
    if (store) {
      p.ids[i] = id;
      p.wts[i] = w;
      if (p.user_ids) p.user_ids[i] = id;
      if (p.user_wts) p.user_wts[i] = w;
    }
  }
}

template <int PER>
__global__ __launch_bounds__(64) void k_dc_route(DecodeParams p) {
  dc_route_token<PER>(p, blockIdx.x, nullptr, nullptr, true);
}

// --------------------------------------------------------- rows by expert
// Every workgroup of the gate/up kernel builds the same tables in LDS: the pairs with a weight, in
// (expert, token) order, cut into tiles of at most 16 rows of one expert.
struct DcTables {
  uint32_t tile[kDcMaxTiles];   // expert << 16 | first row
  uint16_t pair[kDcMaxPairs];   // row -> (t * k + s) << 6 | t
  int ntile, nrow;
  __device__ __forceinline__ int token(int row) const { return pair[row] & 63; }
  __device__ __forceinline__ int pair_of(int row) const { return pair[row] >> 6; }
};
// The same for k_dc_down, from the gate/up kernel's first workgroup.
struct DcRows {
  DcTables tb;
  float wt[kDcMaxPairs];  // of a row: its weight times its expert's tensor scale
};
struct DcBuild {  // while building
  unsigned long long mask[kDcMaxE];  // tokens of an expert
  uint16_t base[kDcMaxE];            // its first row
  int wave_rows[kDcWaves], wave_tiles[kDcWaves];
};

// ids and weights: LDS or the workspace.
__device__ __forceinline__ void dc_build(const DecodeParams& p, const int32_t* ids,
                                         const float* wts, DcTables& tb, DcBuild& bd) {
  const bool publish = blockIdx.x == 0;
  DcRows* pub = p.rows;
  const int tid = threadIdx.x, P = p.T * p.k;
  if (p.T == 1) {  // a row and a tile for each slot, in slot order
    if (tid < 64) {
      const bool on = tid < P && wts[tid] > 0.0f;
      const uint64_t bal = __ballot(on);
      if (on) {
        const int row = __popcll(bal & ((1ull << tid) - 1)), e = ids[tid];
        tb.tile[row] = ((uint32_t)e << 16) | (uint32_t)row;
        tb.pair[row] = (uint16_t)(tid << 6);
        if (publish) {
          pub->tb.tile[row] = tb.tile[row];
          pub->tb.pair[row] = tb.pair[row];
          pub->wt[row] = wts[tid] * p.d_ts[e];
        }
      }
      if (tid == 0) {
        tb.ntile = tb.nrow = __popcll(bal);
        if (publish) pub->tb.ntile = pub->tb.nrow = __popcll(bal);
      }
    }
    __syncthreads();
    return;
  }
  for (int e = tid; e < p.E; e += kDcThreads) bd.mask[e] = 0ull;
  __syncthreads();
  int e_of[kDcMaxPairs / kDcThreads];
#pragma unroll
  for (int j = 0; j < kDcMaxPairs / kDcThreads; ++j) {
    const int i = tid + j * kDcThreads;
    e_of[j] = -1;
    if (i < P && wts[i] > 0.0f) {
      e_of[j] = ids[i];
      atomicOr(&bd.mask[e_of[j]], 1ull << (i / p.k));
    }
  }
  __syncthreads();
  // thread tid owns experts 4 tid .. 4 tid + 3: rows and tiles, scanned
  constexpr int kPer = kDcMaxE / kDcThreads;
  int rows[kPer], mr = 0, mt = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    rows[j] = e < p.E ? __popcll(bd.mask[e]) : 0;
    mr += rows[j];
    mt += (rows[j] + 15) >> 4;
  }
  const int lane = tid & 63, w = tid >> 6;
  int ir = mr, it = mt;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(ir, o, 64), b = __shfl_up(it, o, 64);
    if (lane >= o) {
      ir += a;
      it += b;
    }
  }
  if (lane == 63) {
    bd.wave_rows[w] = ir;
    bd.wave_tiles[w] = it;
  }
  __syncthreads();
  int r = ir - mr, t = it - mt;
  for (int i = 0; i < w; ++i) {
    r += bd.wave_rows[i];
    t += bd.wave_tiles[i];
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int e = tid * kPer + j;
    if (e < p.E) bd.base[e] = (uint16_t)r;
    for (int i = 0; i < rows[j]; i += 16) {
      const uint32_t tile = ((uint32_t)e << 16) | (uint32_t)(r + i);
      if (publish) pub->tb.tile[t] = tile;
      tb.tile[t++] = tile;
    }
    r += rows[j];
  }
  if (tid == kDcThreads - 1) {
    tb.ntile = t;
    tb.nrow = r;
    if (publish) {
      pub->tb.ntile = t;
      pub->tb.nrow = r;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kDcMaxPairs / kDcThreads; ++j) {
    const int i = tid + j * kDcThreads, e = e_of[j];
    if (e >= 0) {
      const unsigned long long before = (1ull << (i / p.k)) - 1;
      const int row = bd.base[e] + __popcll(bd.mask[e] & before);
      tb.pair[row] = (uint16_t)((i << 6) | (i / p.k));
      if (publish) {
        pub->tb.pair[row] = tb.pair[row];
        pub->wt[row] = wts[i] * p.d_ts[e];
      }
    }
  }
  __syncthreads();
}

// Rows of tile j: until the next tile's first row.
__device__ __forceinline__ int dc_tile_rows(const DcTables& tb, int j) {
  const int first = tb.tile[j] & 0xFFFF;
  const int end = j + 1 < tb.ntile ? (int)(tb.tile[j + 1] & 0xFFFF) : tb.nrow;
  return end - first;
}

// ------------------------------------------------------------- products
// 8 E2M1 codes times an E4M3 scale -> 8 exact fp16 values.
__device__ __forceinline__ half8 dc_dequant8(uint32_t codes, half2v s2) {
  half2v p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 0);
  half2v p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 1);
  half2v p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 2);
  half2v p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(codes, 1.0f, 3);
  p0 *= s2;
  p1 *= s2;
  p2 *= s2;
  p3 *= s2;
  return __builtin_shufflevector(__builtin_shufflevector(p0, p1, 0, 1, 2, 3),
                                 __builtin_shufflevector(p2, p3, 0, 1, 2, 3), 0, 1, 2, 3, 4,
                                 5, 6, 7);
}

// Power of two that brings amax to [2^14, 2^15), and its inverse.  Rows of
// zeros and of values beyond the FP32 exponent's reach take the nearest.
__device__ __forceinline__ int dc_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xFF) - 127;
  return e < -106 ? -106 : e;
}
__device__ __forceinline__ float dc_row_scale(float amax, float* inv) {
  const int e = dc_exponent(amax);
  *inv = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
  return __uint_as_float((uint32_t)(14 - e + 127) << 23);
}

template <int PIECES>
struct DcShape {
  static constexpr int NG = PIECES == 1 ? 4 : 2;  // 128-k groups of a K range
};

// One K range of a wave: up to NG groups of 128 k from group g.
template <int PIECES>
struct DcFrags {
  half8 a[PIECES][DcShape<PIECES>::NG][4];
};

// Rows r0 .. r0 + 3 of a tile on the four lane quarters: 16 lanes load a
// row's values of the K range, 8 consecutive k to a lane.
template <bool F32, int PIECES>
struct DcRaw {
  static constexpr int NL = DcShape<PIECES>::NG;  // 128-k pieces of a row
  word4 v[NL][F32 ? 2 : 1];
};
// Loads without a branch, so that waits for older loads stay exact: lanes past
// kend (a multiple of 32) read the last values before it and get zeros.
template <bool F32, int PIECES>
__device__ __forceinline__ void dc_fetch_rows(DcRaw<F32, PIECES>& raw, const void* src,
                                              int64_t row_off, int k0, int kend) {
  const int l16 = threadIdx.x & 15;
#pragma unroll
  for (int j = 0; j < DcRaw<F32, PIECES>::NL; ++j) {
    const int k = min(k0 + j * 128 + l16 * 8, kend - 8);
    if constexpr (F32) {
      const word4* at = reinterpret_cast<const word4*>(reinterpret_cast<const float*>(src) + row_off + k);
      raw.v[j][0] = at[0];
      raw.v[j][1] = at[1];
    } else {
      raw.v[j][0] = *reinterpret_cast<const word4*>(reinterpret_cast<const uint16_t*>(src) + row_off + k);
    }
  }
}

// Scales the rows and writes their fp16 pieces to the wave's buffer (row
// `slot` of the quarter) and the inverse scale to inv[slot].
template <bool F32, int PIECES>
__device__ __forceinline__ void dc_stage_rows(DcRaw<F32, PIECES>& raw, int k0, int kend,
                                              uint8_t* buf, float* inv, int slot, int inv_slot) {
  constexpr int NL = DcRaw<F32, PIECES>::NL;
  const int l16 = threadIdx.x & 15;
  auto get = [&](int j, int i) -> float {
    if constexpr (F32) {
      const word4& v = raw.v[j][i >> 2];
      const int e = i & 3;
      return __uint_as_float(e == 0 ? v.x : e == 1 ? v.y : e == 2 ? v.z : v.w);
    } else {
      const word4& v = raw.v[j][0];
      const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
      return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
  };
  if (k0 + NL * 128 > kend) {
#pragma unroll
    for (int j = 0; j < NL; ++j)
      if (k0 + j * 128 + l16 * 8 >= kend) {
#pragma unroll
        for (int i = 0; i < (F32 ? 2 : 1); ++i) raw.v[j][i] = word4{0u, 0u, 0u, 0u};
      }
  }
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < NL; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = __builtin_fmaxf(amax, __builtin_fabsf(get(j, i)));
  amax = dc_row_max(amax);
  float back;
  const float s = dc_row_scale(amax, &back);
#pragma unroll
  for (int j = 0; j < NL; ++j) {
    half8 hi, lo;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float v = get(j, i) * s;
      hi[i] = (_Float16)v;  // nearest even
      if constexpr (PIECES == 2) lo[i] = (_Float16)(v - (float)hi[i]);
    }
    uint8_t* at = buf + slot * kDcRow + j * 256 + l16 * 16;
    *reinterpret_cast<half8*>(at) = hi;
    if constexpr (PIECES == 2) *reinterpret_cast<half8*>(at + NL * 256) = lo;
  }
  if (l16 == 0) inv[inv_slot] = back;
}

// The fragments of a tile's rows in one K range.  `row_off(r)` is the source
// offset of row r.  raw holds rows 0 .. 3, fetched before.  Rows past the tile
// are copies of its last one: they only enter sums that nobody reads.
template <bool F32, int PIECES, typename RowOff>
__device__ __forceinline__ void dc_fill(DcFrags<PIECES>& fr, DcRaw<F32, PIECES>& raw,
                                        const void* src, RowOff row_off, int nrows, int k0,
                                        int kend, uint8_t* buf, float* inv) {
  constexpr int NG = DcShape<PIECES>::NG;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  auto rows4 = [&](int r0, int p0, bool fetched) {  // rows r0 .. r0 + 3
    const int r = r0 + q;
    if (!fetched) dc_fetch_rows<F32, PIECES>(raw, src, row_off(min(r, nrows - 1)), k0, kend);
    if (r < nrows) dc_stage_rows<F32, PIECES>(raw, k0, kend, buf, inv, r - p0, r);
  };
  auto take = [&](int p0) {
    dc_wave_sync();
    const int row = min(c, nrows - 1) - p0;
    if (row >= 0 && row < kDcStageRows) {
#pragma unroll
      for (int pc = 0; pc < PIECES; ++pc)
#pragma unroll
        for (int g = 0; g < NG; ++g)
#pragma unroll
          for (int st = 0; st < 4; ++st)
            fr.a[pc][g][st] = *reinterpret_cast<const half8*>(
                buf + row * kDcRow + pc * NG * 256 + g * 256 + q * 64 + st * 16);
    }
    dc_wave_sync();
  };
  rows4(0, 0, true);
  if (nrows > 4) rows4(4, 0, false);
  take(0);
  if (nrows > 8) {
    rows4(8, 8, false);
    if (nrows > 12) rows4(12, 8, false);
    take(8);
  }
}

// W of one 16-column slab in one K range of NG groups: NG KiB of codes and
// their block scales.  A matrix-core fragment wants column c in lane c, so
// fragments loaded straight from memory take every lane's 16 bytes from
// another row, and what bounds the kernel then is the number of such pieces
// (16 tokens of the 256-expert layer: 583 us, and in proportion to the
// pieces).  So a wave loads whole runs of a row into neighbouring lanes, holds
// them in registers while they are in flight, and turns them round through a
// slot of LDS of its own.  Slots are swizzled by row: the 16 rows of a
// fragment read lie in different banks.  All of it without branches, so that
// waits for older loads stay exact: past the end of the work a wave loads its
// last slab again, past the end of K the last pieces (activations are 0 there).
// Codes are not kept in the caches, which the scales' short runs and the rows
// then have to themselves: 16 tokens of the 256-expert layer 442 against 474 us,
// 4 tokens 139 / 151; 16 tokens of the 128-expert layer, which the last-level
// cache would hold from one call to the next, 67.5 / 66.2.  Where experts have
// several tiles of rows the second reading of their codes finds less in the
// caches: H 4096, I 2048, 64 tokens of 10 experts, top-10 (40 tiles) 169 against
// 157 us, of 16 experts, top-8 (39) 163 / 149, of 32 (44) 178 / 173; of 8, top-2,
// I 14336 (10) 282 / 282.  With the scales loaded past the caches too the first
// takes 484 us.  Rows that are not whole 64-byte
// pieces share them between runs and do go through the caches (8 tokens of 19
// experts, H 6112: 54.5 us, 60.6 past them).
template <int NG>
struct DcSlab {
  word4 code[NG];
  uint32_t scale[NG / 2];
};

template <int NG>
struct DcSlot {
  static constexpr int kRow = NG * 64;  // code bytes of a row
  static constexpr int kScales = 16 * kRow, kBytes = kScales + 16 * NG * 8;
  static constexpr int kPieces = NG * 4;  // 16-byte pieces of a row
  static __device__ __forceinline__ int swizzle(int row) {
    return kPieces == 16 ? row & 15 : (row >> 1) & 7;
  }
};

// WHOLE: K a multiple of 128, so that a row's block scales are whole groups.
template <int NG, bool WHOLE>
struct DcWalk {
  typedef DcSlot<NG> Slot;
  static constexpr int kRows = 64 / Slot::kPieces;  // rows of one load
  int K2, K16, ng;  // bytes of a row of codes and scales, groups
  __device__ __forceinline__ explicit DcWalk(int K) : K2(K >> 1), K16(K >> 4), ng((K + 127) >> 7) {}
  // the slab at W row `row`, from group g on
  __device__ __forceinline__ void load(DcSlab<NG>& s, const uint8_t* codes, const uint8_t* scales,
                                       int64_t row, int g) const {
    const int lane = threadIdx.x & 63;
    const int piece = min(g * 4 + lane % Slot::kPieces, (K2 >> 4) - 1);
    const uint32_t oc = (lane / Slot::kPieces) * K2 + piece * 16;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const word4* at = reinterpret_cast<const word4*>(codes + (row + i * kRows) * K2 + oc);
      if constexpr (WHOLE) s.code[i] = __builtin_nontemporal_load(at);
      else s.code[i] = *at;
    }
    const uint8_t* ps = scales + row * K16 + (uint32_t)((lane >> 2) * K16);
    const int os = g * 8 + (lane & 3) * (2 * NG);
    if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < NG / 2; ++i)
        s.scale[i] = *reinterpret_cast<const uint16_t*>(ps + min(os + 4 * i, K16 - 2)) |
                     (uint32_t)*reinterpret_cast<const uint16_t*>(ps + min(os + 4 * i + 2, K16 - 2)) << 16;
    } else if constexpr (NG == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(ps + min(os, K16 - 8));
      s.scale[0] = v.x;
      s.scale[1] = v.y;
    } else {
      s.scale[0] = *reinterpret_cast<const uint32_t*>(ps + min(os, K16 - 4));
    }
  }
  static __device__ __forceinline__ void put(const DcSlab<NG>& s, uint8_t* slot) {
    const int lane = threadIdx.x & 63, piece = lane % Slot::kPieces;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const int r = i * kRows + lane / Slot::kPieces;
      *reinterpret_cast<word4*>(slot + r * Slot::kRow + (piece ^ Slot::swizzle(r)) * 16) = s.code[i];
    }
    uint8_t* ps = slot + Slot::kScales + lane * (2 * NG);
    if constexpr (NG == 4)
      *reinterpret_cast<uint2*>(ps) = make_uint2(s.scale[0], s.scale[1]);
    else
      *reinterpret_cast<uint32_t*>(ps) = s.scale[0];
  }
};

typedef unsigned dc_uint2 __attribute__((ext_vector_type(2)));

// Two bytes of each of NG groups (32 k: a lane quarter's share) from words
// that hold them by group: with four groups, quarter q has group q's eight
// bytes, two words for quarters 0 1 and 2 3.  Swapping the upper half-wave of
// the first word with the lower one of the second, then odd 16-lane rows of
// the result with even ones, leaves every row with the pair that holds its
// own.  With two groups, quarter q has half of group q / 2, for quarters 2 (q %
// 2) and the next.
template <int NG>
__device__ __forceinline__ void dc_by_quarter(const uint32_t (&w)[NG / 2], uint32_t (&r)[NG]) {
  const int q = (threadIdx.x & 63) >> 4;
  const int sh = (q & 1) * 16;
  const dc_uint2 h = __builtin_amdgcn_permlane32_swap(w[0], w[NG / 2 - 1], false, false);
  const dc_uint2 a = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
  const dc_uint2 b = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
  if constexpr (NG == 4) {
    r[0] = a[0] >> sh;
    r[1] = a[1] >> sh;
    r[2] = b[0] >> sh;
    r[3] = b[1] >> sh;
  } else {
    r[0] = (q >= 2 ? a[1] : a[0]) >> sh;
    r[1] = (q >= 2 ? b[1] : b[0]) >> sh;
  }
}

// The lane's fragments of a slab from its slot.
template <int NG>
struct DcCols {
  word4 code[NG];
  uint32_t scale[NG];
  __device__ __forceinline__ void take(const uint8_t* slot) {
    typedef DcSlot<NG> Slot;
    const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
    uint32_t w[NG / 2];
    const uint8_t* ps = slot + Slot::kScales + c * (NG * 8) + q * (NG * 2);
    if constexpr (NG == 4) {
      const uint2 v = *reinterpret_cast<const uint2*>(ps);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(ps);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g)
      code[g] = *reinterpret_cast<const word4*>(slot + c * Slot::kRow +
                                                ((4 * g + q) ^ Slot::swizzle(c)) * 16);
    dc_by_quarter<NG>(w, scale);
  }
};

template <int PIECES, int NG>
__device__ __forceinline__ void dc_mul(float4v& acc, const DcFrags<PIECES>& fr, const word4& code,
                                       uint32_t scale, int g) {
  const half2v sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(scale, 1.0f, false);
  const half2v s0 = __builtin_shufflevector(sc, sc, 0, 0), s1 = __builtin_shufflevector(sc, sc, 1, 1);
  const uint32_t w[4] = {code.x, code.y, code.z, code.w};
#pragma unroll
  for (int st = 0; st < 4; ++st) {
    const half8 b = dc_dequant8(w[st], st < 2 ? s0 : s1);
#pragma unroll
    for (int pc = 0; pc < PIECES; ++pc)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(fr.a[pc][g][st], b, acc, 0, 0, 0);
  }
}

__device__ __forceinline__ float dc_silu_mul(float g, float u) {
  return g / (1.0f + __expf(-g)) * u;
}

constexpr int kDcSlot = DcSlot<4>::kBytes;
static_assert(DcSlot<2>::kBytes <= kDcSlot, "a slot holds a slab of either shape");

struct DcGateUpShared {
  __attribute__((aligned(16))) uint8_t slot[kDcWaves][2][kDcSlot];
  DcTables tb;
  // a wave's rows while it fills its fragments, and its sums at the unit's end
  union Own {
    uint8_t buf[kDcStageRows * kDcRow];
    float4v red[4][64];
  };
  union {
    DcBuild bd;
    Own own[kDcWaves];
  };
  float inv[kDcWaves][16];
  int32_t sid[kDcInlineT * kDcMaxK];
  float swt[kDcInlineT * kDcMaxK];
};

// Units of (tile, column block): a wave takes NSH / 2 gate slabs and their up
// slabs over its share of K (ks of KS) and column share (cs of CS); the K
// shares meet in LDS at the unit's end, where h is computed, scaled by its
// largest value in 16 columns and stored where k_dc_down's lanes want it.
// Consecutive units of a workgroup mostly have the same rows, which stay in
// registers where K is one range.
template <bool F32, int PIECES, bool WHOLE, int NSH>
__device__ __forceinline__ void dc_gate_up(const DecodeParams& p, DcGateUpShared& sh, int KS,
                                           DcRaw<F32, PIECES>& raw) {
  constexpr int NG = DcShape<PIECES>::NG, SPW = NSH / 2;
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int ks = wave % KS, cs = wave / KS, CS = kDcWaves / KS;
  const DcWalk<NG, WHOLE> walk(p.H);
  const int nslab = p.I >> 4, SPU = SPW * CS, nblk = (nslab + SPU - 1) / SPU;
  // K range ph of the wave starts at group (ph KS + ks) NG: the shares lie
  // side by side, so that the waves read neighbouring runs of a row together
  const int nph = (walk.ng + NG * KS - 1) / (NG * KS);
  auto first_group = [&](int ph) { return min((ph * KS + ks) * NG, walk.ng); };
  const int units = sh.tb.ntile * nblk;
  const int Ip = dc_pad(p.I);
  const int u0 = (int)((int64_t)units * blockIdx.x / kDcGrid);
  const int u1 = (int)((int64_t)units * (blockIdx.x + 1) / kDcGrid);
  if (u0 >= u1) return;

  // where a unit's columns lie: its expert's first W row and the wave's slab
  struct Pos {
    int j, blk, n, first, slab, e;
    int64_t row;
  };
  auto pos = [&](int u) {
    Pos o;
    o.j = u / nblk;
    o.blk = u - o.j * nblk;
    const uint32_t tile = __builtin_amdgcn_readfirstlane((int)sh.tb.tile[o.j]);
    o.first = tile & 0xFFFF;
    o.n = __builtin_amdgcn_readfirstlane(dc_tile_rows(sh.tb, o.j));
    o.slab = o.blk * SPU + cs * SPW;
    o.e = tile >> 16;
    o.row = (int64_t)o.e * 2 * p.I;
    return o;
  };
  DcSlab<NG> w[2];
  auto load = [&](const Pos& o, int ph, int st) {
    walk.load(w[st & 1], p.gu_codes, p.gu_scales,
              o.row + ((st & 1) ? p.I : 0) + min(o.slab + (st >> 1), nslab - 1) * 16, first_group(ph));
  };
  uint8_t* slot = sh.slot[wave][0];
  auto row_off = [&](int row) { return (int64_t)sh.tb.token(row) * p.ldx; };
  auto fetch = [&](const Pos& o, int ph) {
    dc_fetch_rows<F32, PIECES>(raw, p.x, row_off(o.first + min(q, o.n - 1)),
                               first_group(ph) * 128, p.H);
  };
  DcFrags<PIECES> fr;
  Pos cur = pos(u0);
  if (p.T > 1) fetch(cur, 0);  // before W: loads return in order
  load(cur, 0, 0);
  load(cur, 0, 1);
  walk.put(w[0], slot);
  int held = -1;  // tile whose fragments are in registers (one K range only)
  for (int u = u0; u < u1; ++u) {
    const Pos next = pos(u + 1 < u1 ? u + 1 : u);
    const float ts = p.gu_ts[cur.e];
    float4v tot[NSH];
#pragma unroll
    for (int st = 0; st < NSH; ++st) tot[st] = float4v{0.0f, 0.0f, 0.0f, 0.0f};
    for (int ph = 0; ph < nph; ++ph) {
      const bool inside = ph + 1 < nph;
      const Pos& np = inside ? cur : next;
      const int nph_i = inside ? ph + 1 : 0;
      if (nph > 1 || held != cur.j)
        dc_fill<F32, PIECES>(
            fr, raw, p.x, [&](int r) { return row_off(cur.first + r); }, cur.n,
            first_group(ph) * 128, p.H, sh.own[wave].buf, sh.inv[wave]);
      held = cur.j;
      if (nph > 1 || next.j != cur.j) fetch(np, nph_i);
      const float4v back = *reinterpret_cast<const float4v*>(&sh.inv[wave][4 * q]);
#pragma unroll
      for (int st = 0; st < NSH; ++st) {
        float4v acc = {0.0f, 0.0f, 0.0f, 0.0f};
        // two stages ahead, into the registers put last; the next stage's
        // slot is filled half way through this one
        if (st + 2 < NSH) load(cur, ph, st + 2);
        else load(np, nph_i, st + 2 - NSH);
        __builtin_amdgcn_sched_barrier(0);
        dc_wave_sync();
        DcCols<NG> cols;
        cols.take(slot + (st & 1) * kDcSlot);
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          if (i == NG / 2) {
            __builtin_amdgcn_sched_barrier(0);
            walk.put(w[(st + 1) & 1], slot + ((st + 1) & 1) * kDcSlot);
            __builtin_amdgcn_sched_barrier(0);
          }
          dc_mul<PIECES, NG>(acc, fr, cols.code[i], cols.scale[i], i);
        }
        tot[st] += acc * back;
      }
    }
#pragma unroll
    for (int st = 0; st < NSH; ++st) sh.own[wave].red[st][lane] = tot[st];
    __syncthreads();
    // a wave takes rows i, 4 + i, 8 + i and 12 + i of a slab
    for (int it = wave; it < SPU * 4; it += kDcWaves) {
      const int s = it >> 2, i = it & 3, w0 = (s / SPW) * KS, st = 2 * (s % SPW);
      const int slab = cur.blk * SPU + s;
      if (slab >= nslab || i >= cur.n) continue;
      float g = 0.0f, up = 0.0f;
      for (int v = 0; v < KS; ++v) {
        g += sh.own[w0 + v].red[st][lane][i];
        up += sh.own[w0 + v].red[st + 1][lane][i];
      }
      // fp16 pieces scaled by the row's largest of these 16 columns, at the
      // place where k_dc_down's lane quarter and step find them
      auto place = [](int k) { return (k & ~127) + ((k >> 3) & 3) * 32 + ((k >> 5) & 3) * 8 + (k & 7); };
      const float h = dc_silu_mul(ts * g, ts * up);
      const float amax = dc_row_max(__builtin_fabsf(h));
      const int r = 4 * q + i, c = lane & 15;
      if (r >= cur.n) continue;
      const int64_t pair = sh.tb.pair_of(cur.first + r);
      const int e = dc_exponent(amax);
      const float v = h * __uint_as_float((uint32_t)(14 - e + 127) << 23);
      const _Float16 hi = (_Float16)v;
      uint16_t* out = p.h + pair * PIECES * Ip;
      uint8_t* ex = p.hexp + pair * (Ip >> 4);
      const int at = place(slab * 16 + c);
      out[at] = __builtin_bit_cast(uint16_t, hi);
      // an h beyond FP32's range stays an infinity: no second piece (inf - inf),
      // and the largest exponent byte instead of 256
      if constexpr (PIECES == 2) {
        const float lo = __builtin_fabsf(v) == __builtin_inff() ? 0.0f : v - (float)hi;
        out[Ip + at] = __builtin_bit_cast(uint16_t, (_Float16)lo);
      }
      if (c == 0) ex[slab] = (uint8_t)min(e + 128, 255);
      if (slab == nslab - 1) {  // zeros behind I, for the lanes that read them
        for (int z = p.I + c; z < Ip; z += 16) {
          out[place(z)] = 0;
          if constexpr (PIECES == 2) out[Ip + place(z)] = 0;
          if (c == 0) ex[z >> 4] = 0;
        }
      }
    }
    __syncthreads();
    cur = next;
  }
}

template <bool F32, int PIECES, bool WHOLE, bool ROUTE, int NSH>
__global__ __launch_bounds__(kDcThreads, 2) void k_dc_gate_up(DecodeParams p) {
  __shared__ DcGateUpShared sh;
  // one token: its row does not wait for the routing
  DcRaw<F32, PIECES> raw;
  if (p.T == 1) {
    constexpr int NG = DcShape<PIECES>::NG;
    const int ks = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % p.ks_up;
    dc_fetch_rows<F32, PIECES>(raw, p.x, 0, min(ks * NG, (p.H + 127) >> 7) * 128, p.H);
  }
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < p.blocks; i += kDcThreads) p.count[i] = 0;
  if constexpr (ROUTE) {
    for (int t = threadIdx.x >> 6; t < p.T; t += kDcWaves)
      dc_route_token<kDcInlineE / 64>(p, t, sh.sid, sh.swt, blockIdx.x == 0);
    __syncthreads();
    dc_build(p, sh.sid, sh.swt, sh.tb, sh.bd);
  } else {
    dc_build(p, p.ids, p.wts, sh.tb, sh.bd);
  }
  dc_gate_up<F32, PIECES, WHOLE, NSH>(p, sh, p.ks_up, raw);
}

// ------------------------------------------------------------------- down
// A workgroup owns a block of output columns and walks the row tiles of its
// part: W streams without a break, a tile's sums go to the tokens' rows of an
// LDS accumulator of each wave, and nothing is synchronized until the end.
// Where the column blocks alone do not fill the chip the tiles are split into
// parts, and the last workgroup of a block adds the parts in their order.
constexpr int kDcDownRows = 4;   // rows staged at a time
constexpr int kDcDownAhead = 2;  // rows in flight a tile ahead
struct DcDownShared {
  __attribute__((aligned(16))) uint8_t slot[kDcWaves][kDcSlot];
  uint8_t buf[kDcWaves][kDcDownRows * kDcRow];
  DcTables tb;
  float wt[kDcMaxPairs];  // of a row
  __attribute__((aligned(16))) float acc[kDcWaves][kDcAcc];  // [token][NS * 16]
  int last;
};
static_assert(2 * sizeof(DcDownShared) <= 160 * 1024 && 2 * sizeof(DcGateUpShared) <= 160 * 1024,
              "two workgroups on a CU");

template <int PIECES, bool WHOLE, int NS, bool BF16>
__global__ __launch_bounds__(kDcThreads, 2) void k_dc_down(DecodeParams p) {
  constexpr int NG = DcShape<PIECES>::NG;
  __shared__ DcDownShared sh;
  for (int i = threadIdx.x; i < p.T * p.k; i += kDcThreads) {  // no more rows or tiles than pairs
    sh.tb.tile[i] = p.rows->tb.tile[i];
    sh.tb.pair[i] = p.rows->tb.pair[i];
    sh.wt[i] = p.rows->wt[i];
  }
  if (threadIdx.x == 0) {
    sh.tb.ntile = p.rows->tb.ntile;
    sh.tb.nrow = p.rows->tb.nrow;
  }
  __syncthreads();
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int KS = p.ks_down, ks = wave % KS, cs = wave / KS, CS = kDcWaves / KS;
  const DcWalk<NG, WHOLE> walk(p.I);
  const int nslab = p.H >> 4, SPU = NS * CS, nblk = p.blocks;
  const int nph = (walk.ng + NG * KS - 1) / (NG * KS), ntile = sh.tb.ntile, g1 = walk.ng;
  auto first_group = [&](int ph) { return min((ph * KS + ks) * NG, walk.ng); };
  const int parts = max(1, min(min(ntile, kDcMaxParts), kDcGrid / nblk));
  float* mine = sh.acc[wave];
  const int Ip = dc_pad(p.I);

  for (int id = blockIdx.x; id < nblk * parts; id += kDcGrid) {
    const int part = id / nblk, blk = id - part * nblk;
    const int j0 = ntile * part / parts, j1 = ntile * (part + 1) / parts;
    for (int i = lane; i < p.T * NS * 16; i += 64) mine[i] = 0.0f;
    struct Pos {
      int first, n;
      int64_t row;
    };
    auto pos = [&](int j) {
      Pos o;
      const uint32_t tile = __builtin_amdgcn_readfirstlane((int)sh.tb.tile[j]);
      o.first = tile & 0xFFFF;
      o.n = __builtin_amdgcn_readfirstlane(dc_tile_rows(sh.tb, j));
      o.row = (int64_t)(tile >> 16) * p.H;
      return o;
    };
    DcSlab<NG> w[2];
    auto load = [&](const Pos& o, int ph, int st) {
      walk.load(w[st & 1], p.d_codes, p.d_scales, o.row + min(blk * SPU + cs * NS + st, nslab - 1) * 16,
                first_group(ph));
    };
    uint8_t* slot = sh.slot[wave];
    // Rows of the tile: a row's K range is 64 lanes of 16 bytes, the first two
    // rows in flight a tile ahead (sparse batches have no more; with eight, 16
    // tokens of the 128-expert layer take 67.8 us for 66.2, 64 tokens of the
    // 256-expert layer 1129 for 1114); through LDS, lane (c, q) takes row c (rows
    // past the tile are copies of its last one, whose sums nobody reads) and
    // quarter q also the exponent bytes of group q, as the block scales of W.
    struct Ahead {
      word4 v[kDcDownAhead];
      uint32_t exps[NG / 2];
    };
    constexpr int kLanes = 64 / PIECES;  // of one piece of a row
    auto fetch_row = [&](const Pos& o, int r, int gf) -> word4 {
      const int pair = sh.tb.pair_of(o.first + min(r, o.n - 1));
      const int k = min(gf * 128 + (lane % kLanes) * 8, Ip - 8);
      return *reinterpret_cast<const word4*>(p.h + ((int64_t)pair * PIECES + lane / kLanes) * Ip + k);
    };
    auto fetch = [&](Ahead& nx, const Pos& o, int ph) {
      const int gf = first_group(ph);
#pragma unroll
      for (int r = 0; r < kDcDownAhead; ++r) nx.v[r] = fetch_row(o, r, gf);
      const int pair = sh.tb.pair_of(o.first + min(c, o.n - 1));
      const uint8_t* ex = p.hexp + (int64_t)pair * (Ip >> 4);
      if constexpr (NG == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(ex + min(gf + q, g1 - 1) * 8);
        nx.exps[0] = v.x;
        nx.exps[1] = v.y;
      } else {
        nx.exps[0] = *reinterpret_cast<const uint32_t*>(ex + min(gf + (q >> 1), g1 - 1) * 8 + (q & 1) * 4);
      }
    };
    struct Rows {
      DcFrags<PIECES> fr;
      uint32_t exps[NG / 2];
    };
    auto stage = [&](Rows& rw, const auto& v, int p0, int n) {  // rows p0 and on
      constexpr int kCount = sizeof(v) / sizeof(word4);
      uint8_t* buf = sh.buf[wave];
#pragma unroll
      for (int r = 0; r < kCount; ++r)
        *reinterpret_cast<word4*>(buf + r * kDcRow + lane * 16) = v[r];
      dc_wave_sync();
      const int row = min(c, n - 1) - p0;
      if (row >= 0 && row < kCount) {
#pragma unroll
        for (int pc = 0; pc < PIECES; ++pc)
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int st = 0; st < 4; ++st)
              rw.fr.a[pc][g][st] = *reinterpret_cast<const half8*>(
                  buf + row * kDcRow + pc * NG * 256 + g * 256 + st * 64 + q * 16);
      }
      dc_wave_sync();
    };
    auto fill = [&](Rows& rw, const Ahead& nx, const Pos& o, int ph) {
      stage(rw, nx.v, 0, o.n);
      for (int p0 = kDcDownAhead; p0 < o.n; p0 += kDcDownRows) {
        word4 v[kDcDownRows];
#pragma unroll
        for (int r = 0; r < kDcDownRows; ++r) v[r] = fetch_row(o, p0 + r, first_group(ph));
        stage(rw, v, p0, o.n);
      }
#pragma unroll
      for (int i = 0; i < NG / 2; ++i) rw.exps[i] = nx.exps[i];
    };
    auto scale_group = [&](Rows& rw, int g, uint32_t f0, uint32_t f1) {
      const half2v lo = __builtin_bit_cast(half2v, f0 | (f0 << 16));
      const half2v hi = __builtin_bit_cast(half2v, f1 | (f1 << 16));
      const half8 a0 = __builtin_shufflevector(lo, lo, 0, 1, 0, 1, 0, 1, 0, 1);
      const half8 a1 = __builtin_shufflevector(hi, hi, 0, 1, 0, 1, 0, 1, 0, 1);
#pragma unroll
      for (int pc = 0; pc < PIECES; ++pc)
#pragma unroll
        for (int st = 0; st < 4; ++st) rw.fr.a[pc][g][st] *= st < 2 ? a0 : a1;
    };
    // Brings the row to one exponent in this K range (the largest of its
    // bytes) and groups past the wave's share to zero; returns the inverse
    // scale of the lane's four result rows.
    auto settle = [&](Rows& rw, int left) -> float4v {
      uint32_t b[NG];
      dc_by_quarter<NG>(rw.exps, b);
      uint32_t top = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        b[g] = g < left ? b[g] & 0xFFFFu : 0u;
        top = max(top, max(b[g] & 0xFFu, b[g] >> 8));
      }
      top = max(top, (uint32_t)__shfl_xor((int)top, 16, 64));
      top = max(top, (uint32_t)__shfl_xor((int)top, 32, 64));
      // 2^(e - top) in a normal factor of at least 2^-14, and in rows of more
      // than that range a second one, 0 for what is below 2^-38 of the largest
      int below = 0;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int d0 = (int)top - (int)(b[g] & 0xFFu), d1 = (int)top - (int)(b[g] >> 8);
        const uint32_t f0 = g < left ? (uint32_t)(15 - min(d0, 14)) << 10 : 0u;
        const uint32_t f1 = g < left ? (uint32_t)(15 - min(d1, 14)) << 10 : 0u;
        if (g < left) below = max(below, max(d0, d1));
        scale_group(rw, g, f0, f1);
      }
      if (__ballot(below > 14)) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int d0 = (int)top - (int)(b[g] & 0xFFu) - 14, d1 = (int)top - (int)(b[g] >> 8) - 14;
          auto more = [&](int d) -> uint32_t {
            return d <= 0 ? 15u << 10 : d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u;
          };
          scale_group(rw, g, more(d0), more(d1));
        }
      }
      float4v back;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = max(__shfl((int)top, 4 * q + i, 64), 22);
        back[i] = __uint_as_float((uint32_t)(e - 128 - 14 + 127) << 23);
      }
      return back;
    };

    Rows rw;
    Ahead nx;
    if (j0 < j1) {
      Pos cur = pos(j0);
      fetch(nx, cur, 0);  // before W: loads return in order
      load(cur, 0, 0);
      load(cur, 0, 1);
      dc_wave_sync();
      walk.put(w[0], slot);
      for (int j = j0, ph = 0; j < j1;) {
        const bool inside = ph + 1 < nph;
        const int nph_i = inside ? ph + 1 : 0;
        Pos np = cur;
        if (!inside && j + 1 < j1) np = pos(j + 1);
        fill(rw, nx, cur, ph);
        fetch(nx, np, nph_i);
        const float4v back = settle(rw, g1 - first_group(ph));
        int tok[4];
        float wt[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 4 * q + i;
          tok[i] = r < cur.n ? sh.tb.token(cur.first + r) : -1;
          wt[i] = r < cur.n ? sh.wt[cur.first + r] * back[i] : 0.0f;
        }
#pragma unroll
        for (int st = 0; st < NS; ++st) {
          if (st + 2 < NS) load(cur, ph, st + 2);
          else load(np, nph_i, st + 2 - NS);
          __builtin_amdgcn_sched_barrier(0);
          dc_wave_sync();
          DcCols<NG> cols;
          cols.take(slot);
          __builtin_amdgcn_sched_barrier(0);
          dc_wave_sync();
          float4v acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < NG; ++i) {
            if (i == NG / 2) {
              __builtin_amdgcn_sched_barrier(0);
              walk.put(w[(st + 1) & 1], slot);
              __builtin_amdgcn_sched_barrier(0);
            }
            dc_mul<PIECES, NG>(acc, rw.fr, cols.code[i], cols.scale[i], i);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (tok[i] >= 0) {
              float* o = mine + tok[i] * (NS * 16) + st * 16 + c;
              *o = __builtin_fmaf(acc[i], wt[i], *o);
            }
        }
        cur = np;
        j = inside ? j : j + 1;
        ph = nph_i;
      }
    }
    __syncthreads();
    // the K shares of each column, in order
    const int cols = SPU * 16, quads = min(cols, p.H - blk * cols) >> 2;
    auto total = [&](int t, int b) -> float4v {  // columns b .. b + 3 of the block
      const int w0 = (b / (NS * 16)) * KS, at = t * (NS * 16) + b % (NS * 16);
      float4v s = {0.0f, 0.0f, 0.0f, 0.0f};
      for (int v = 0; v < KS; ++v) s += *reinterpret_cast<const float4v*>(&sh.acc[w0 + v][at]);
      return s;
    };
    auto put = [&](int t, int col, const float4v& v) {
      if constexpr (BF16) {
        typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
        const bf16x4 o = {(__bf16)v[0], (__bf16)v[1], (__bf16)v[2], (__bf16)v[3]};
        *reinterpret_cast<bf16x4*>(reinterpret_cast<__bf16*>(p.out) + t * p.ldo + col) = o;
      } else {
        *reinterpret_cast<float4v*>(reinterpret_cast<float*>(p.out) + t * p.ldo + col) = v;
      }
    };
    if (parts == 1) {
      for (int i = threadIdx.x; i < p.T * quads; i += kDcThreads) {
        const int t = i / quads, b = (i - t * quads) * 4;
        put(t, blk * cols + b, total(t, b));
      }
    } else {
      // agent-scope stores go past this XCD's cache, so nothing has to be
      // written back: each wave waits for its own to complete before the
      // workgroup counts itself; the last one drops what its cache holds of
      // the parts.  (A release fence writes the whole cache back: one token of
      // the 128-expert layer takes 27.2 us with it, 20.7 us without.)
      for (int i = threadIdx.x; i < p.T * quads; i += kDcThreads) {
        const int t = i / quads, b = (i - t * quads) * 4;
        const float4v v = total(t, b);
        float* at = p.part + ((int64_t)part * p.T + t) * p.H + blk * cols + b;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          __hip_atomic_store(at + e, v[e], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (threadIdx.x == 0)
        sh.last = __hip_atomic_fetch_add(p.count + blk, 1, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT) == parts - 1;
      __syncthreads();
      if (sh.last) {
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        for (int i = threadIdx.x; i < p.T * quads; i += kDcThreads) {
          const int t = i / quads, col = blk * cols + (i - t * quads) * 4;
          float4v v[kDcMaxParts], s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int n = 0; n < kDcMaxParts; ++n)
            v[n] = *reinterpret_cast<const float4v*>(
                p.part + ((int64_t)min(n, parts - 1) * p.T + t) * p.H + col);
#pragma unroll
          for (int n = 0; n < kDcMaxParts; ++n) s += n < parts ? v[n] : float4v{0.0f, 0.0f, 0.0f, 0.0f};
          put(t, col, s);
        }
      }
    }
    __syncthreads();  // the accumulators are free again
  }
}


// How the four waves of a workgroup divide its work: ks of them share K, and
// the 4 / ks groups take ns slabs each; column blocks, and parts of the tiles.
struct DcSplit {
  int ks, ns, blocks, parts;
};
inline int64_t dc_tiles(const nvfp4_moe_decode_args_t* a) {
  const int64_t P = a->T * a->k, few = a->E + P / 16;
  return P < few ? P : few;
}
inline int dc_groups(const nvfp4_moe_decode_args_t* a) {
  return a->x_dtype == NVFP4_IN_F32 ? DcShape<2>::NG : DcShape<1>::NG;
}
// Row tiles that the routing will likely give: an even choice's mean, and a
// tenth more for its spread.
inline double dc_likely_tiles(const nvfp4_moe_decode_args_t* a) {
  const double P = (double)(a->T * a->k), E = (double)a->E;
  if (a->T == 1) return P;
  const double touched = E * (1.0 - std::pow(1.0 - (double)a->k / E, (double)a->T)) + P / 32;
  return 1.1 * (touched < P ? touched : P);
}
// How the gate/up kernel divides a tile's work: KS waves of a workgroup share
// K, and the 4 / KS groups take ns gate slabs (with as many up slabs) of a unit
// each.  A workgroup takes one unit or, of u on average, u + 1/2 (units are
// whole), and a unit costs its K ranges times its slabs and half a slab for the
// rows.  Over 22 layers (7 to 256 experts, H 416 to 7168, I 96 to 14336, 1 to 64
// tokens) the least such cost is within 3% of the fastest of the six choices,
// 0.5% on average; the fewest padded K ranges alone cost up to 1.4 times as
// much (49 tokens, 166 experts, H 5280, I 224: 173 against 127 us).  Larger
// units than ns = 2 would read the rows of a long K in runs too far apart: 344
// against 321 us for 16 tokens of the 256-expert layer.
inline DcSplit dc_split_up(const nvfp4_moe_decode_args_t* a) {
  const int nslab = (int)(a->I >> 4), ng = (int)((a->H + 127) / 128), NG = dc_groups(a);
  DcSplit best{4, 1, 0, 0};
  double least = 0.0;
  for (int ks = kDcWaves; ks >= 1; ks /= 2)
    for (int ns = 1; ns <= 2; ++ns) {
      const int spu = ns * (kDcWaves / ks), ranges = (ng + NG * ks - 1) / (NG * ks);
      const double u = dc_likely_tiles(a) * ((nslab + spu - 1) / spu) / kDcGrid;
      const double cost = (u <= 1.0 ? 1.0 : u + 0.5) * ranges * (2 * ns + 0.5);
      if (least == 0.0 || cost < least) {
        least = cost;
        best = DcSplit{ks, ns, 0, 0};
      }
    }
  return best;
}
// The down kernel: the fewer K ranges are padded the better, and larger blocks
// read the rows of activations less often; but what costs most is workgroups
// without work, so the choice is the first that gives at least 7 of 8
// workgroups some (32 a tile where there are few tiles: one token of the
// 128-expert layer takes 12.1 us for its down product with 64), in that order,
// or the one that keeps most busy: within 3% of the fastest choice over the
// layers above, 10% for the smallest.  It counts on the most tiles there can
// be, since the workspace holds the parts.
inline DcSplit dc_split_down(const nvfp4_moe_decode_args_t* a) {
  const int NG = dc_groups(a), ng = (int)((a->I + 127) / 128), nslab = (int)(a->H >> 4);
  const int64_t tiles = dc_tiles(a);
  int64_t padded[3];
  int order[3] = {0, 1, 2};  // ks = 4, 2, 1
  for (int i = 0; i < 3; ++i) {
    const int ks = kDcWaves >> i;
    padded[i] = (int64_t)((ng + NG * ks - 1) / (NG * ks)) * ks;
    for (int j = i; j > 0 && padded[order[j]] < padded[order[j - 1]]; --j) {
      const int t = order[j];
      order[j] = order[j - 1];
      order[j - 1] = t;
    }
  }
  DcSplit best{1, 2, 1, 1};
  const int64_t enough = tiles * 32 < kDcGrid * 7 / 8 ? tiles * 32 : kDcGrid * 7 / 8;
  int64_t most = -1;
  for (int i = 0; i < 3; ++i)
    for (int ns = a->T <= 32 ? 4 : 2; ns >= 2; ns /= 2) {  // accumulators: T ns <= 128
      DcSplit o{kDcWaves >> order[i], ns, 0, 0};
      const int spu = ns * (kDcWaves / o.ks);
      o.blocks = (nslab + spu - 1) / spu;
      int64_t parts = kDcMaxParts < tiles ? kDcMaxParts : tiles;
      if (parts > kDcGrid / o.blocks) parts = kDcGrid / o.blocks;
      o.parts = (int)(parts < 1 ? 1 : parts);
      const int64_t work = (int64_t)o.blocks * o.parts;
      if (work >= enough) return o;
      if (work > most) {
        most = work;
        best = o;
      }
    }
  return best;
}

struct DcLayout {
  size_t ids, wts, count, rows, h, hexp, part, bytes;
};
inline DcLayout dc_layout(const nvfp4_moe_decode_args_t* a) {
  const size_t P = (size_t)(a->T * a->k);
  const DcSplit d = dc_split_down(a);
  const int64_t nb = d.blocks, parts = d.parts;
  DcLayout l;
  l.ids = 0;
  l.wts = l.ids + nv_round256(P * 4);
  l.count = l.wts + nv_round256(P * 4);
  l.rows = l.count + nv_round256((size_t)nb * 4);
  l.h = l.rows + nv_round256(sizeof(DcRows));
  const size_t Ip = dc_pad((int)a->I);
  l.hexp = l.h + nv_round256(P * Ip * (a->x_dtype == NVFP4_IN_F32 ? 4 : 2));
  l.part = l.hexp + nv_round256(P * (Ip / 16));
  l.bytes = l.part + (parts > 1 ? nv_round256((size_t)parts * a->T * a->H * 4) : 0);
  return l;
}
inline bool dc_shape_ok(const nvfp4_moe_decode_args_t* a) {
  return a->T >= 0 && a->T <= kDcMaxT && a->E >= 1 && a->E <= kDcMaxE && a->k >= 1 &&
         a->k <= a->E && a->k <= kDcMaxK && a->H >= 32 && a->H <= kDcMaxDim && a->H % 32 == 0 &&
         a->I >= 32 && a->I <= kDcMaxDim && a->I % 32 == 0;
}

template <bool F32, bool WHOLE, int NS>
void dc_launch_down(const DecodeParams& p, hipStream_t s) {
  static_assert(kDcMaxT * 2 * 16 <= kDcAcc && 32 * 4 * 16 <= kDcAcc, "sums of a wave");
  hipLaunchKernelGGL((k_dc_down<F32 ? 2 : 1, WHOLE, NS, !F32>), dim3(kDcGrid), dim3(kDcThreads), 0,
                     s, p);
}

template <bool F32, bool WHOLE, int NSH>
void dc_launch_gate_up(const DecodeParams& p, hipStream_t s) {
  const dim3 grid(kDcGrid), wg(kDcThreads);
  if (p.T <= kDcInlineT && p.E <= kDcInlineE) {
    hipLaunchKernelGGL((k_dc_gate_up<F32, F32 ? 2 : 1, WHOLE, true, NSH>), grid, wg, 0, s, p);
    return;
  }
  const dim3 gt((unsigned)p.T);
  if (p.E <= 64) hipLaunchKernelGGL(k_dc_route<1>, gt, dim3(64), 0, s, p);
  else if (p.E <= 128) hipLaunchKernelGGL(k_dc_route<2>, gt, dim3(64), 0, s, p);
  else if (p.E <= 256) hipLaunchKernelGGL(k_dc_route<4>, gt, dim3(64), 0, s, p);
  else hipLaunchKernelGGL(k_dc_route<16>, gt, dim3(64), 0, s, p);
  hipLaunchKernelGGL((k_dc_gate_up<F32, F32 ? 2 : 1, WHOLE, false, NSH>), grid, wg, 0, s, p);
}

template <bool F32>
void dc_launch(const DecodeParams& p, int ns_up, int ns, hipStream_t s) {
  const bool whole_h = p.H % 128 == 0;
  if (ns_up == 2) {
    if (whole_h) dc_launch_gate_up<F32, true, 4>(p, s);
    else dc_launch_gate_up<F32, false, 4>(p, s);
  } else {
    if (whole_h) dc_launch_gate_up<F32, true, 2>(p, s);
    else dc_launch_gate_up<F32, false, 2>(p, s);
  }
  const bool whole = p.I % 128 == 0;
  if (ns == 4) {
    if (whole) dc_launch_down<F32, true, 4>(p, s);
    else dc_launch_down<F32, false, 4>(p, s);
  } else {
    if (whole) dc_launch_down<F32, true, 2>(p, s);
    else dc_launch_down<F32, false, 2>(p, s);
  }
}

}  // namespace

extern "C" {

size_t nvfp4_moe_decode_workspace_size(const nvfp4_moe_decode_args_t* a) {
  return a && dc_shape_ok(a) && a->T > 0 ? dc_layout(a).bytes : 0;
}

int nvfp4_moe_decode(const nvfp4_moe_decode_args_t* a, void* ws, size_t ws_bytes, void* stream) {
  NV_RETURN_IF(!a, NVFP4_ERR_NULL);
  NV_RETURN_IF(a->x_dtype != NVFP4_IN_F32 && a->x_dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(!dc_shape_ok(a) || a->ldx < a->H || a->ldo < a->H || a->ld_logits < a->E,
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
  const DcLayout l = dc_layout(a);
  NV_RETURN_IF(!ws || ws_bytes < l.bytes || !nv_aligned16(ws), NVFP4_ERR_WORKSPACE);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  uint8_t* w = reinterpret_cast<uint8_t*>(ws);
  const DcSplit up = dc_split_up(a), down = dc_split_down(a);
  const DecodeParams p{(int)a->T, (int)a->E, (int)a->k, (int)a->H, (int)a->I, a->x, a->ldx,
                       a->logits, a->ld_logits, a->gu_codes, a->gu_scales, a->gu_tscale,
                       a->d_codes, a->d_scales, a->d_tscale, a->out, a->ldo,
                       a->topk_ids, reinterpret_cast<int32_t*>(w + l.ids),
                       a->topk_weights, reinterpret_cast<float*>(w + l.wts),
                       reinterpret_cast<uint16_t*>(w + l.h), w + l.hexp,
                       reinterpret_cast<float*>(w + l.part),
                       reinterpret_cast<int32_t*>(w + l.count),
                       reinterpret_cast<DcRows*>(w + l.rows),
                       down.blocks, up.ks, down.ks};
  if (a->x_dtype == NVFP4_IN_BF16) dc_launch<false>(p, up.ns, down.ns, s);
  else dc_launch<true>(p, up.ns, down.ns, s);
  return nv_launch_status();
}

}  // extern "C"
