// INT8 W8A8 comparator: per-row quantizer and grouped GEMM.
//
// One FP32 scale per activation row (at run time) and per weight output
// channel: s = RN32(amax / 127), r = RN32(1 / s), code = the nearest integer to
// RN32(x r).  A product is y = s_a s_w sum_k a_k w_k with the sum exact in 32-bit
// integers (K <= 131056), whatever its order, so K may be split over waves freely.
//
// MI355X design:
//  * k_i8_rows: a row stays in the registers of one to eight waves between its
//    maximum and its codes.  HBM-bound when large (8192 x 7168 bf16, 176 MB: 34 us
//    and 5.1 TB/s with inputs beyond the last-level cache in turn, 28 us where one
//    input stays in it), 2 to 5 us when small.
//  * k_i8_few: a few rows against W that streams once, straight into registers;
//    the waves of a workgroup split K.  4.9 us for one row of 4096 x 4096 (3.4 TB/s
//    of codes, which the last-level cache holds), 40 us for the 8 rows of a token
//    at K 7168, N 4096 (5.9 TB/s).
//  * k_i8_gemm: tiles of 64 x 128 to 320 x 256.  Rows of 128 k go into LDS by DMA,
//    two or three chunks deep, at uniform bases and 32-bit offsets; fragments of
//    the next 32 k are read while those in registers are multiplied; the D tiles
//    are W by rows, so that a lane holds four neighbouring columns, and go out
//    through LDS as whole rows of 16-byte pieces (as they come, a store of 2 or 4
//    bytes each, 65536 x 4096 x 1024 took 548 us for 361).  The smallest tile
//    streams W for many experts of few rows: 479 us for 16 tokens of 256 experts
//    (K 7168, N 4096, 102 experts' 2.95 GB: 6.1 TB/s).
//  * What bounds the large products is power: 65536 x 4096 x 8192 (1674 us) runs its
//    matrix cores 79% of the cycles at 1.4 GHz, 256 experts of 256 rows 67% at 1.3
//    GHz, where the 16 tokens' call runs at 2.1 GHz; on zeros the first of them
//    takes 1409 us.  Where the time goes otherwise (parts left out for timing, 1836
//    us then): the copies into LDS 20%, the fragment reads 4%, waits and barriers
//    nothing.  Tried and slower: 16 x 16 x 64 products (1883 for 1836 us); four waves of 128 x 128
//    (K 1024: 373 for 346 us; K 8192: 1729-1766 for 1780-1815); W fetched into
//    the L2 a few chunks ahead (256 experts 2239 for 2102 us); copies of rows
//    behind a group's end left out (2173 for 2137 us).

#include <type_traits>

#include "common.h"

namespace {

typedef int int4v __attribute__((ext_vector_type(4)));
typedef int int16v __attribute__((ext_vector_type(16)));

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

// RW waves per row (RW divides the workgroup's eight).  A lane holds VPL vectors
// of 8 elements between the maximum and the encode; longer rows (K > 512 VPL RW)
// are read again (the second read hits the caches).
template <bool BF16, int RW, int VPL>
__global__ __launch_bounds__(512) void k_i8_rows(const void* x, int64_t rows, int K, int64_t ldx,
                                                 int8_t* codes, float* scales) {
  constexpr int RPW = 8 / RW;  // rows of a workgroup
  __shared__ uint32_t mags[8];
  const int wave = threadIdx.x >> 6, tid = threadIdx.x % (64 * RW);
  const int nv = K >> 3;
  for (int64_t r0 = (int64_t)blockIdx.x * RPW; r0 < rows; r0 += (int64_t)gridDim.x * RPW) {
    const int64_t row = r0 + wave / RW;
    const bool live = row < rows;  // uniform in the row's waves
    const int64_t at = live ? row * ldx : 0;
    float v[VPL][8];
    uint32_t mag = 0;
    if (live) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int c = tid + 64 * RW * i;
        if (c < nv) {
          i8_load8<BF16>(x, at + 8 * c, v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) mag = max(mag, i8_mag(v[i][e]));
      for (int c = tid + 64 * RW * VPL; c < nv; c += 64 * RW) {
        float w[8];
        i8_load8<BF16>(x, at + 8 * c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) mag = max(mag, i8_mag(w[e]));
      }
      mag = i8_wave_max(mag);
    }
    if constexpr (RW > 1) {
      __syncthreads();  // the last row's maxima have been read
      if ((threadIdx.x & 63) == 0) mags[wave] = mag;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < RW; ++i) mag = max(mag, mags[wave / RW * RW + i]);
    }
    if (!live) continue;
    float s, r;
    i8_row_scale(mag, s, r);
    int8_t* out = codes + row * (int64_t)K;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int c = tid + 64 * RW * i;
      if (c < nv) *reinterpret_cast<uint2*>(out + 8 * c) = i8_encode8(v[i], r);
    }
    for (int c = tid + 64 * RW * VPL; c < nv; c += 64 * RW) {
      float w[8];
      i8_load8<BF16>(x, at + 8 * c, w);
      *reinterpret_cast<uint2*>(out + 8 * c) = i8_encode8(w, r);
    }
    if (tid == 0) scales[row] = s;
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
  int vec;  // rows of out start on 16 bytes and hold whole 16-byte pieces
  int32_t* part;  // kPartial: sums over a part of K, [parts][total_rows][pitch]
  int pitch;      // columns, a multiple of four
};

constexpr int kPartial = 3;  // an epilogue of the kernel's own, joined by k_i8_join

// silu(g) * u in FP32 with the hardware exp and reciprocal.
__device__ __forceinline__ float i8_silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Tile of a workgroup, in the order of nv_find_tile<8> (bands of eight m-tiles,
// contiguous ranges of tiles per XCD), found with one scan: a lane counts the
// tiles of consecutive groups.  Without offsets the one group needs none.
__device__ __forceinline__ NvTile i8_find_tile(const I8Params& p, int bm, int n_tiles) {
  constexpr int KEEP = 4;  // groups of a lane kept in registers
  const int lane = threadIdx.x & 63, per = (p.G + 63) >> 6;
  int v[KEEP], sum = 0, inc = 0, m_tiles;
  if (p.offsets) {
    if (per <= KEEP) {
      int o[KEEP + 1];
#pragma unroll
      for (int i = 0; i <= KEEP; ++i) o[i] = p.offsets[min(lane * per + min(i, per), p.G)];
#pragma unroll
      for (int i = 0; i < KEEP; ++i) sum += v[i] = (o[i + 1] - o[i] + bm - 1) / bm;
    } else {
      for (int i = 0; i < per; ++i) sum += nv_group_tiles(p.offsets, p.G, lane * per + i, bm);
    }
    inc = sum;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int n = __shfl_up(inc, o, 64);
      if (lane >= o) inc += n;
    }
    m_tiles = __builtin_amdgcn_readlane(inc, 63);
  } else {
    m_tiles = (p.total_rows + bm - 1) / bm;
  }
  const int n = m_tiles * n_tiles;
  const int bid = blockIdx.x, share = n / 8, rem = n % 8, xcd = bid % 8, li = bid / 8;
  NvTile t{-1, 0, 0};
  if (li >= share + (xcd < rem ? 1 : 0)) return t;
  const int L = xcd * share + (xcd < rem ? xcd : rem) + li;
  int first = 0, tiles = m_tiles;  // of the tile's group
  t.grp = 0;
  if (p.offsets) {
    const int mt = L / n_tiles;
    const int hl = __ffsll((long long)__ballot(inc > mt)) - 1;  // the first lane past it
    first = __builtin_amdgcn_readlane(inc - sum, hl);
    t.grp = hl * per;
    for (int i = 0; i < per; ++i, ++t.grp) {
      if (per <= KEEP) {
        const int w = i == 0 ? v[0] : i == 1 ? v[1] : i == 2 ? v[2] : v[3];
        tiles = __builtin_amdgcn_readlane(w, hl);
      } else {
        tiles = nv_group_tiles(p.offsets, p.G, t.grp, bm);
      }
      if (mt < first + tiles) break;
      first += tiles;
    }
  }
  const int i = L - first * n_tiles, band = i / (8 * n_tiles);
  const int gm = min(8, tiles - band * 8), j = i - band * 8 * n_tiles;
  t.local = band * 8 + j % gm;
  t.nt = j / gm;
  return t;
}

// ----------------------------------------------------------------- few rows

// A workgroup of eight waves computes a tile of up to 16 RT rows of one group: CW =
// 8 / KW blocks of 16 output columns (with SiLU*mul 16 gate and the 16 up
// columns), KW waves to a block, which split K and add up through LDS.  W and the
// rows go from memory to registers in v_mfma_i32_16x16x64_i8's layout (lane l: W
// row or row l % 16, the 16 bytes k = 16 (l / 16) of a 64-k step), a batch of
// steps ahead of its use.  D holds row l % 16 and columns 4 (l / 16) + 0..3 in
// lane l.
constexpr int kFewSteps = 4;

template <int EPI, bool GATHER, int KW, int RT>
__global__ __launch_bounds__(512) void k_i8_few(I8Params p, int n_tiles) {
  constexpr bool SILU = EPI == NVFP4_EPI_SILU_MUL_BF16;
  constexpr int FB = SILU ? 2 : 1, CW = 8 / KW;
  __shared__ int4v red[8][FB * RT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int cols = SILU ? p.N >> 1 : p.N;
  // row tile and column block of the workgroup
  const int mt = (int)(blockIdx.x / (unsigned)n_tiles), nt = (int)(blockIdx.x % (unsigned)n_tiles);
  int grp = 0, beg = mt * 16 * RT, end = p.total_rows;
  if (p.offsets) {
    int run = 0;
    grp = -1;
    for (int g0 = 0; g0 < p.G; g0 += 64) {
      const int tiles = nv_group_tiles(p.offsets, p.G, g0 + lane, 16 * RT);
      int inc = tiles;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int n = __shfl_up(inc, o, 64);
        if (lane >= o) inc += n;
      }
      const unsigned long long hit = __ballot(run + inc > mt);
      if (hit) {
        const int l = __ffsll((long long)hit) - 1;
        grp = __builtin_amdgcn_readfirstlane(g0 + l);
        const int local = mt - run - __builtin_amdgcn_readlane(inc - tiles, l);
        beg = p.offsets[grp] + local * 16 * RT;
        end = p.offsets[grp + 1];
        break;
      }
      run += __builtin_amdgcn_readlane(inc, 63);
    }
    if (grp < 0) return;  // a surplus workgroup
  }
  const int n0 = (nt * CW + wave / KW) * 16;
  const int steps = (p.K + 63) >> 6, part = wave % KW;
  const int s0 = n0 < cols ? (int)((int64_t)steps * part / KW) : 0;
  const int s1 = n0 < cols ? (int)((int64_t)steps * (part + 1) / KW) : 0;
  const int64_t wrow = (int64_t)grp * p.N;
  const int n = n0 + 4 * q;
  const int8_t* w0 = p.w_codes + (wrow + min(n0 + c, cols - 1)) * p.K;
  const int8_t* w1 = w0 + (SILU ? (int64_t)cols * p.K : 0);
  const int8_t* row[RT];
  bool mv[RT];
  float sa[RT], sw[FB][4];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int m = beg + t * 16 + c;
    mv[t] = m < end;
    const int64_t src = mv[t] ? (GATHER ? (int64_t)p.gather[m] : (int64_t)m) : 0;
    row[t] = p.a_codes + src * p.K;
    sa[t] = mv[t] ? p.a_scales[src] : 0.0f;
  }
  const int4v zero = {0, 0, 0, 0};
  int4v wf[2][FB][kFewSteps], af[2][RT][kFewSteps];
  auto load = [&](int s, int h) {
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u) {
      const int k = (s + u) * 64 + q * 16;
      const bool on = s + u < s1 && k < p.K;
      wf[h][0][u] = on ? *reinterpret_cast<const int4v*>(w0 + k) : zero;
      if constexpr (SILU) wf[h][1][u] = on ? *reinterpret_cast<const int4v*>(w1 + k) : zero;
#pragma unroll
      for (int t = 0; t < RT; ++t)
        af[h][t][u] = on && mv[t] ? *reinterpret_cast<const int4v*>(row[t] + k) : zero;
    }
  };
  load(s0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int f = 0; f < FB; ++f) sw[f][i] = p.w_scales[wrow + f * cols + min(n + i, cols - 1)];
  int4v acc[RT][FB];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int f = 0; f < FB; ++f) acc[t][f] = zero;
  auto multiply = [&](int h) {
#pragma unroll
    for (int u = 0; u < kFewSteps; ++u)
#pragma unroll
      for (int t = 0; t < RT; ++t)
#pragma unroll
        for (int f = 0; f < FB; ++f)
          acc[t][f] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[h][f][u], af[h][t][u], acc[t][f], 0, 0, 0);
  };
  for (int s = s0; s < s1; s += 2 * kFewSteps) {
    load(s + kFewSteps, 1);
    multiply(0);
    load(s + 2 * kFewSteps, 0);
    multiply(1);
  }
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int f = 0; f < FB; ++f) red[wave][t * FB + f][lane] = acc[t][f];
  __syncthreads();
  // the KW waves of a block share its row tiles
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    if (t % KW != part || !mv[t] || n >= cols) continue;
    int4v sum[FB];
#pragma unroll
    for (int f = 0; f < FB; ++f) {
      sum[f] = zero;
#pragma unroll
      for (int i = 0; i < KW; ++i) sum[f] += red[wave - part + i][t * FB + f][lane];
    }
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = (sa[t] * sw[0][i]) * (float)sum[0][i];
      if constexpr (SILU) y[i] = i8_silu_mul(y[i], (sa[t] * sw[1][i]) * (float)sum[1][i]);
    }
    using OutT = std::conditional_t<EPI == NVFP4_EPI_F32, float, uint16_t>;
    OutT* out = reinterpret_cast<OutT*>(p.out) + (int64_t)(beg + t * 16 + c) * cols + n;
    if (p.vec) {  // whole pieces of four columns
      if constexpr (EPI == NVFP4_EPI_F32)
        *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
      else
        *reinterpret_cast<uint2*>(out) = make_uint2(i8_bf16(y[0]) | (uint32_t)i8_bf16(y[1]) << 16,
                                                    i8_bf16(y[2]) | (uint32_t)i8_bf16(y[3]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < cols) {
          if constexpr (EPI == NVFP4_EPI_F32) out[i] = y[i];
          else out[i] = i8_bf16(y[i]);
        }
    }
  }
}

// ------------------------------------------------------------ prefill tiles

constexpr int KC = 128;  // k (= bytes) per row per chunk: eight 16-byte pieces

// Position of 16-byte piece lp of a row is lp ^ i8_swz(row): the 8 or 16 rows
// that one phase of a 16-byte LDS read touches lie on distinct banks, and rows 16
// apart share their pattern, so a wave's fragments differ by constant offsets.
__device__ __forceinline__ uint32_t i8_swz(uint32_t row) { return (row ^ ((row >> 3) & 1u)) & 7u; }

template <int WM, int WN, int FM, int FN, int NS, int EPI, bool GATHER>
struct I8Tile {
  static constexpr bool SILU = EPI == NVFP4_EPI_SILU_MUL_BF16;
  static constexpr int NW = WM * WN, NT = 64 * NW;
  static constexpr int BM = WM * FM * 32, BN = WN * FN * 32, ROWS = BM + BN;
  static constexpr int NPI = ROWS * 8 / NT;  // 16-byte pieces per thread per chunk
  static constexpr int NPA = BM * 8 / NT;    // of them in A rows, which come first
  static constexpr int STAGE = ROWS * KC;
  static constexpr int DS = NPI % 2 ? 1 : 2;  // steps over which a chunk's pieces are issued
  static_assert(NW % 2 == 0 && BM * 8 % NT == 0 && BN * 8 % NT == 0, "whole wave-loads");
  static_assert(!SILU || FN % 2 == 0, "SiLU pairs gate and up fragments");
  static_assert(NS >= 2 && (NS - 1) * NPI <= 63, "vmcnt range");

  const I8Params& p;
  uint8_t* lds;
  const uint8_t *abase, *wbase, *ubase;  // the tile's first row of A, of W, of W's up half
  uint32_t at;        // a piece's place in its chunk: the same for all pieces of a lane
  uint32_t off[NPI];  // bytes from there to piece j; in a gather 16-byte units from A's start
  int lane, wave, wm, wn, lr, lh, nt, beg, end, cols, nfull, rem;

  // The chunk behind the last whole one holds `rem` bytes a row; its pieces behind
  // them step back to the chunk's first piece, and the products skip them.
  __device__ __forceinline__ uint32_t step_back(int chunk) const {
    return chunk == nfull && at >= (uint32_t)rem ? at : 0u;
  }
  // Piece j of a chunk into buffer `buf`.
  __device__ __forceinline__ void issue1(int j, int chunk, int buf, uint32_t back) {
    const uint32_t st = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)(lds + buf * STAGE);
    const uint32_t m0 = __builtin_amdgcn_readfirstlane(st + (j * NW + wave) * 1024);
    if (GATHER && j < NPA) {
      const uint8_t* g = abase + (int64_t)chunk * KC - back + (uint64_t)off[j] * 16u;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                   :: "s"(m0), "v"(g) : "memory", "m0");
    } else {
      // wave-loads of gate and of up rows alternate by 32 rows
      const bool up = SILU && ((((j - NPA) * NW + wave) >> 2) & 1);
      const uint8_t* g = (j < NPA ? abase : up ? ubase : wbase) + (int64_t)chunk * KC;
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                   :: "s"(m0), "v"(off[j] - back), "s"(g) : "memory", "m0");
    }
  }

  // Waits until this wave's pieces of the oldest chunk in flight have landed,
  // with `left` chunks issued after it.
  __device__ __forceinline__ void landed(int left) {
    if (NS > 2 && left >= NS - 2)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * NPI) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // Every wave's LDS accesses before it are done, and none after it has begun.
  static __device__ __forceinline__ void barrier() {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  }

  template <int NL>
  __device__ __forceinline__ void run(const float* sw, const float* sa) {
    int16v acc[NL][FN];
#pragma unroll
    for (int a = 0; a < NL; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[a][b][e] = 0;
    const int total = nfull + (rem ? 1 : 0);
    const uint32_t x = (lh ^ i8_swz((uint32_t)lr)) << 4;
    const uint8_t* al = lds + (wm * 32 + lr) * KC;
    const uint8_t* wl = lds + (BM + wn * FN * 32 + lr) * KC;
    int4v af[2][NL], wf[2][FN];
    // fragment i of step s: the W ones first
    auto load = [&](int i, int buf, int s, int4v* av, int4v* wv) {
      const uint32_t o = buf * STAGE + (x ^ (s << 5));
      if (i < FN)
        wv[i] = *reinterpret_cast<const int4v*>(wl + o + i * 32 * KC);
      else
        av[i - FN] = *reinterpret_cast<const int4v*>(al + o + (i - FN) * WM * 32 * KC);
    };
    constexpr int NR = NL + FN, NM = NL * FN;
    // A buffer is free from a chunk's last step on; the pieces of the chunk that
    // takes it are issued over that step and the first DS - 1 of the next chunk.
    constexpr int PART = NPI / DS;
    static_assert(NPI % DS == 0 && DS <= 3, "pieces per step");
    for (int c = 0; c < NS; ++c)
      if (c < total) {
#pragma unroll
        for (int j = 0; j < NPI; ++j)
          if (c < NS - 1 || j < PART) issue1(j, c, c, step_back(c));
      }
    if (total >= NS)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 2) * NPI + PART) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    barrier();
#pragma unroll
    for (int i = 0; i < NR; ++i) load(i, 0, 0, af[0], wf[0]);
    int buf = 0;
    // STEADY: the chunks ahead are there and whole
    auto chunk = [&](auto steady, int ch) {
      constexpr bool STEADY = decltype(steady)::value;
      const int nb = buf + 1 == NS ? 0 : buf + 1, pb = buf == 0 ? NS - 1 : buf - 1;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (s == 3) {
          // every wave has read the chunk and holds its last step; the next one
          // has landed
          if (STEADY)
            landed(NS - 2);
          else if (ch + 1 < total)
            landed(total - ch - 2);
          barrier();
        }
        const bool tail = s == 3 || s < DS - 1;  // a step that issues
        const int nx = s == 3 ? ch + NS : ch + NS - 1, to = s == 3 ? buf : pb;
        const int j0 = s == 3 ? 0 : (s + 1) * PART;
        const bool more = tail && (STEADY || nx < total);
        const uint32_t back = STEADY ? 0u : step_back(nx);
        const int cur = s & 1;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
#pragma unroll
          for (int j = i * 2; j < NR && j < i * 2 + 2; ++j)
            load(j, s == 3 ? nb : buf, (s + 1) & 3, af[cur ^ 1], wf[cur ^ 1]);
          if (more) {
#pragma unroll
            for (int j = i * PART / NM; j < (i + 1) * PART / NM; ++j)
              issue1(j0 + j, nx, to, back);
          }
          // the wave that multiplies goes first (1695 for 1759 us, K 8192)
          if (i == 0) __builtin_amdgcn_s_setprio(1);
          if (i == NM - 1) __builtin_amdgcn_s_setprio(0);
          const int a = i / FN, b = i % FN;
          acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[cur][b], af[cur][a], acc[a][b], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      buf = nb;
    };
    int ch = 0;
    for (; ch + NS < nfull; ++ch) chunk(std::true_type{}, ch);
    for (; ch < nfull; ++ch) chunk(std::false_type{}, ch);
    if (rem) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      barrier();
      for (int s = 0; s * 32 < rem; ++s) {
#pragma unroll
        for (int i = 0; i < NR; ++i) load(i, buf, s, af[0], wf[0]);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const int a = i / FN, b = i % FN;
          int4v av = af[0][a];
          if (s * 32 + lh * 16 >= rem) av = int4v{0, 0, 0, 0};
          acc[a][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[0][b], av, acc[a][b], 0, 0, 0);
        }
      }
    }
    barrier();
    store<NL>(acc, sa, sw);
  }

  // The same products in little code, for tiles of one fragment row a wave
  // (FM == 1): calls of their size are over before a long loop's code is fetched.
  // Waves without rows compute on repeated rows and store nothing; the chunk
  // behind the last whole one is masked like every other.
  __device__ __forceinline__ void run_small(const float* sw, const float* sa) {
    int16v acc[1][FN];
#pragma unroll
    for (int b = 0; b < FN; ++b)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[0][b][e] = 0;
    const int total = nfull + (rem ? 1 : 0);
    // the workgroup's chunks: all, or its part of them
    const int c0 = EPI == kPartial ? total * (int)blockIdx.y / (int)gridDim.y : 0;
    const int c1 = EPI == kPartial ? total * ((int)blockIdx.y + 1) / (int)gridDim.y : total;
#pragma unroll 1
    for (int c = 0; c < NS && c0 + c < c1; ++c) {
      const uint32_t back = step_back(c0 + c);
#pragma unroll
      for (int j = 0; j < NPI; ++j) issue1(j, c0 + c, c, back);
    }
    const uint32_t x = (lh ^ i8_swz((uint32_t)lr)) << 4;
    const uint8_t* al = lds + (wm * 32 + lr) * KC;
    const uint8_t* wl = lds + (BM + wn * FN * 32 + lr) * KC;
    int buf = 0;
#pragma unroll 1
    for (int ch = c0; ch < c1; ++ch) {
      // this wave's pieces of chunk ch have landed, and every wave's behind the barrier
      if (ch + NS <= c1)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NS - 1) * NPI) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      barrier();
      int4v af[4], wf[4][FN];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint32_t o = buf * STAGE + (x ^ (s << 5));
        af[s] = *reinterpret_cast<const int4v*>(al + o);
#pragma unroll
        for (int b = 0; b < FN; ++b) wf[s][b] = *reinterpret_cast<const int4v*>(wl + o + b * 32 * KC);
      }
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (ch * KC + s * 32 + lh * 16 >= p.K) af[s] = int4v{0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[0][b] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wf[s][b], af[s], acc[0][b], 0, 0, 0);
      }
      barrier();  // every wave holds its fragments
      if (ch + NS < c1) {
        const uint32_t back = step_back(ch + NS);
#pragma unroll
        for (int j = 0; j < NPI; ++j) issue1(j, ch + NS, buf, back);
      }
      buf = buf + 1 == NS ? 0 : buf + 1;
    }
    if constexpr (EPI == kPartial) {
      const int m = beg + wm * 32 + lr;
      int32_t* out = p.part + ((int64_t)blockIdx.y * p.total_rows + m) * p.pitch;
#pragma unroll
      for (int b = 0; b < FN; ++b)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int n = nt * BN + (wn * FN + b) * 32 + q * 8 + lh * 4;
          if (m < end && n < p.pitch)
            *reinterpret_cast<int4v*>(out + n) =
                int4v{acc[0][b][4 * q], acc[0][b][4 * q + 1], acc[0][b][4 * q + 2], acc[0][b][4 * q + 3]};
        }
    } else if (beg + wm * 32 < end) {
      store<1>(acc, sa, sw);
    }
  }

  // Element e of fragment (a, b): tile row (a WM + wm) 32 + lr, tile column
  // (wn FN + b) 32 + (e >> 2) 8 + lh 4 + (e & 3).  Each wave turns 32 rows at a
  // time round in its own part of the LDS, so that lanes store whole rows in
  // 16-byte pieces; piece i of row r lies at i ^ (r % pieces).
  template <int NL>
  __device__ __forceinline__ void store(int16v (&acc)[NL][FN], const float* sa, const float* sw) {
    using OutT = std::conditional_t<EPI == NVFP4_EPI_F32, float, uint16_t>;
    constexpr int FB = SILU ? 2 : 1, VEC = 16 / sizeof(OutT);
    constexpr int WC = FN / FB * 32, PPR = WC / VEC;  // columns and pieces of a wave's row
    static_assert(32 * PPR * 16 * NW <= NS * STAGE && (PPR & (PPR - 1)) == 0, "LDS of a wave");
    uint8_t* t = lds + wave * (32 * PPR * 16);
    const int n0 = nt * (BN / FB) + wn * WC;
    const float* swl = sw + wn * FN * 32 + lh * 4;
#pragma unroll
    for (int a = 0; a < NL; ++a) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int b = 0; b < FN; b += FB)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float y[4];
          const float4 s4 = *reinterpret_cast<const float4*>(swl + b * 32 + q * 8);
          const float s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) y[i] = (sa[a] * s[i]) * (float)acc[a][b][4 * q + i];
          if constexpr (SILU) {
            const float4 u4 = *reinterpret_cast<const float4*>(swl + (b + 1) * 32 + q * 8);
            const float u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = i8_silu_mul(y[i], (sa[a] * u[i]) * (float)acc[a][b + 1][4 * q + i]);
          }
          const int c = b / FB * 32 + q * 8 + lh * 4, piece = c / VEC;
          uint8_t* at = t + (lr * PPR + (piece ^ (lr & (PPR - 1)))) * 16;
          if constexpr (sizeof(OutT) == 4)
            *reinterpret_cast<float4*>(at) = make_float4(y[0], y[1], y[2], y[3]);
          else
            *reinterpret_cast<uint2*>(at + lh * 8) =
                make_uint2(i8_bf16(y[0]) | (uint32_t)i8_bf16(y[1]) << 16,
                           i8_bf16(y[2]) | (uint32_t)i8_bf16(y[3]) << 16);
        }
      asm volatile("" ::: "memory");
      const int m0 = beg + (a * WM + wm) * 32;
      OutT* out = reinterpret_cast<OutT*>(p.out) + (int64_t)m0 * cols + n0;
      if (p.vec) {
#pragma unroll
        for (int i = 0; i < 32 * PPR / 64; ++i) {
          const int r = (i * 64 + lane) / PPR, c = lane % PPR;
          const uint4 v = *reinterpret_cast<const uint4*>(t + (r * PPR + (c ^ (r & (PPR - 1)))) * 16);
          if (m0 + r < end && n0 + c * VEC < cols)
            *reinterpret_cast<uint4*>(out + (int64_t)r * cols + c * VEC) = v;
        }
      } else {
        for (int i = lane; i < 32 * WC; i += 64) {
          const int r = i / WC, c = i % WC;
          const OutT v = *reinterpret_cast<const OutT*>(
              t + (r * PPR + (c / VEC ^ (r & (PPR - 1)))) * 16 + c % VEC * sizeof(OutT));
          if (m0 + r < end && n0 + c < cols) out[(int64_t)r * cols + c] = v;
        }
      }
    }
  }
};

template <int WM, int WN, int FM, int FN, int NS, int EPI, bool GATHER>
__global__ __launch_bounds__(64 * WM * WN, 1) void k_i8_gemm(I8Params p, int n_tiles) {
  using Tile = I8Tile<WM, WN, FM, FN, NS, EPI, GATHER>;
  constexpr int BM = Tile::BM, BN = Tile::BN;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NS * Tile::STAGE];
  __shared__ __attribute__((aligned(16))) float sw[BN];  // the columns' scales
  NvTile t = i8_find_tile(p, BM, n_tiles);
  if (t.grp < 0) return;  // identical in every lane of every wave
  t.grp = __builtin_amdgcn_readfirstlane(t.grp);
  t.local = __builtin_amdgcn_readfirstlane(t.local);
  t.nt = __builtin_amdgcn_readfirstlane(t.nt);
  Tile k{p, lds};
  k.lane = threadIdx.x & 63;
  k.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  k.wm = k.wave / WN;
  k.wn = k.wave % WN;
  k.lr = k.lane & 31;
  k.lh = k.lane >> 5;
  k.nt = t.nt;
  k.beg = (p.offsets ? p.offsets[t.grp] : 0) + t.local * BM;
  k.end = p.offsets ? p.offsets[t.grp + 1] : p.total_rows;
  k.cols = Tile::SILU ? p.N >> 1 : p.N;
  k.nfull = p.K / KC;
  k.rem = p.K % KC;
  const int64_t wrow = (int64_t)t.grp * p.N;
  // output column of W row i of the tile; those past the last repeat it
  const int n0 = min(t.nt * (Tile::SILU ? BN / 2 : BN), k.cols - 1);
  auto column = [&](int i) {
    if constexpr (Tile::SILU) {
      const int f = i >> 5, b = f % FN;
      i = (f / FN) * (FN / 2) * 32 + (b >> 1) * 32 + (i & 31);
    }
    return min(n0 + i, k.cols - 1);
  };
  // the loads that the copies' addresses do not need are issued before those that
  // they do, and waited for after them
  static_assert(BN <= Tile::NT, "a scale for a thread");
  const int ci = min((int)threadIdx.x, BN - 1);
  const float my_sw = p.w_scales[wrow + column(ci) + (Tile::SILU && (ci >> 5 & 1) ? k.cols : 0)];
  int src[FM];
#pragma unroll
  for (int a = 0; a < FM; ++a) {
    const int m = min(k.beg + (a * WM + k.wm) * 32 + k.lr, k.end - 1);
    src[a] = GATHER ? p.gather[m] : m;
  }
  k.abase = reinterpret_cast<const uint8_t*>(p.a_codes) + (GATHER ? 0 : (int64_t)k.beg * p.K);
  k.wbase = reinterpret_cast<const uint8_t*>(p.w_codes) + (wrow + n0) * p.K;
  k.ubase = k.wbase + (int64_t)k.cols * p.K;
  // rows 8 NW j apart share their swizzle (NW is even)
  k.at = ((uint32_t)(k.lane & 7) ^ i8_swz((uint32_t)(k.wave * 8 + (k.lane >> 3)))) * 16;
#pragma unroll
  for (int j = 0; j < Tile::NPI; ++j) {
    const int row = (j * Tile::NW + k.wave) * 8 + (k.lane >> 3);
    const uint32_t at = k.at;
    if (j < Tile::NPA) {
      const int r = min(row, k.end - 1 - k.beg);
      if constexpr (GATHER)
        k.off[j] = (uint32_t)p.gather[k.beg + r] * (uint32_t)(p.K >> 4) + (at >> 4);
      else
        k.off[j] = (uint32_t)r * (uint32_t)p.K + at;
    } else {
      k.off[j] = (uint32_t)(column(row - BM) - n0) * (uint32_t)p.K + at;
    }
  }
  float sa[FM];
#pragma unroll
  for (int a = 0; a < FM; ++a) sa[a] = p.a_scales[src[a]];
  if (threadIdx.x < BN) sw[threadIdx.x] = my_sw;
  if constexpr (FM == 1) {
    k.run_small(sw, sa);
  } else {
    // fragments of 32 rows that hold rows: frag a of wave row wm starts at row (a
    // WM + wm) 32.  A wave without rows computes on repeated ones.
    const int frags = (min(k.end - k.beg, BM) + 31) >> 5;
    const int nl = (frags - k.wm + WM - 1) / WM;
    if (nl >= FM) k.template run<FM>(sw, sa);
    else if (FM > 4 && nl == 4) k.template run<(FM > 4 ? 4 : 1)>(sw, sa);
    else if (FM > 3 && nl == 3) k.template run<(FM > 3 ? 3 : 1)>(sw, sa);
    else if (FM > 2 && nl == 2) k.template run<(FM > 2 ? 2 : 1)>(sw, sa);
    else k.template run<1>(sw, sa);
  }
}

// Adds the parts of K (whole numbers: their order does not matter), four columns
// to a thread.
template <int EPI, bool GATHER>
__global__ __launch_bounds__(256) void k_i8_join(I8Params p, int parts) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int per = p.pitch >> 2;
  const int64_t m = i / per;
  if (m >= p.total_rows) return;
  const int n = (int)(i - m * per) * 4;
  const int32_t* at = p.part + m * p.pitch + n;
  int4v sum = *reinterpret_cast<const int4v*>(at);
  for (int z = 1; z < parts; ++z)
    sum += *reinterpret_cast<const int4v*>(at + (int64_t)z * p.total_rows * p.pitch);
  const float sa = p.a_scales[GATHER ? (int64_t)p.gather[m] : m];
  float y[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (sa * p.w_scales[min(n + e, p.N - 1)]) * (float)sum[e];
  using OutT = std::conditional_t<EPI == NVFP4_EPI_F32, float, uint16_t>;
  OutT* out = reinterpret_cast<OutT*>(p.out) + m * p.N + n;
  if (p.vec) {  // whole pieces of four columns
    if constexpr (EPI == NVFP4_EPI_F32)
      *reinterpret_cast<float4*>(out) = make_float4(y[0], y[1], y[2], y[3]);
    else
      *reinterpret_cast<uint2*>(out) = make_uint2(i8_bf16(y[0]) | (uint32_t)i8_bf16(y[1]) << 16,
                                                  i8_bf16(y[2]) | (uint32_t)i8_bf16(y[3]) << 16);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) {
        if constexpr (EPI == NVFP4_EPI_F32) out[e] = y[e];
        else out[e] = i8_bf16(y[e]);
      }
  }
}

// The tile shapes, and the workgroups of a call on one of them (an upper bound:
// every group's last tile may be part of one).
struct I8Shape {
  int bm, bn, threads;
};
constexpr I8Shape kTiles[4] = {{64, 128, 256}, {128, 256, 512}, {256, 256, 512}, {320, 256, 512}};

int64_t i8_workgroups(const I8Shape& t, int64_t rows, int64_t N, int64_t groups) {
  return ((rows + t.bm - 1) / t.bm + groups) * ((N + t.bn - 1) / t.bn);
}

template <int TILE, int WM, int WN, int FM, int FN, int NS, int EPI>
int launch_tiles(const I8Params& p, hipStream_t s) {
  constexpr I8Shape t = kTiles[TILE];
  constexpr int NT = 64 * WM * WN;
  static_assert(t.bm == WM * FM * 32 && t.bn == WN * FN * 32 && t.threads == NT, "tile shape");
  const int n_tiles = (p.N + t.bn - 1) / t.bn;  // SiLU: as many gate as up columns in a tile
  const dim3 grid((unsigned)i8_workgroups(t, p.total_rows, p.N, p.offsets ? p.G : 0));
  if (p.gather)
    hipLaunchKernelGGL((k_i8_gemm<WM, WN, FM, FN, NS, EPI, true>), grid, dim3(NT), 0, s, p, n_tiles);
  else
    hipLaunchKernelGGL((k_i8_gemm<WM, WN, FM, FN, NS, EPI, false>), grid, dim3(NT), 0, s, p, n_tiles);
  return nv_launch_status();
}

// 64 x 128 tiles over `parts` parts of K, and their join.
template <int EPI>
int launch_split(const I8Params& p, int parts, hipStream_t s) {
  const int n_tiles = (p.N + kTiles[0].bn - 1) / kTiles[0].bn;
  const dim3 grid((unsigned)i8_workgroups(kTiles[0], p.total_rows, p.N, 0), (unsigned)parts);
  const dim3 join((unsigned)(((int64_t)p.total_rows * (p.pitch >> 2) + 255) / 256));
  if (p.gather) {
    hipLaunchKernelGGL((k_i8_gemm<2, 2, 1, 2, 2, kPartial, true>), grid, dim3(256), 0, s, p, n_tiles);
    hipLaunchKernelGGL((k_i8_join<EPI, true>), join, dim3(256), 0, s, p, parts);
  } else {
    hipLaunchKernelGGL((k_i8_gemm<2, 2, 1, 2, 2, kPartial, false>), grid, dim3(256), 0, s, p, n_tiles);
    hipLaunchKernelGGL((k_i8_join<EPI, false>), join, dim3(256), 0, s, p, parts);
  }
  return nv_launch_status();
}

template <int EPI, int KW, int RT>
int launch_few(const I8Params& p, int64_t tiles, hipStream_t s) {
  const int cols = EPI == NVFP4_EPI_SILU_MUL_BF16 ? p.N / 2 : p.N;
  const int n_tiles = (cols + 128 / KW - 1) / (128 / KW);
  const dim3 grid((unsigned)(tiles * n_tiles)), block(512);
  if (p.gather)
    hipLaunchKernelGGL((k_i8_few<EPI, true, KW, RT>), grid, block, 0, s, p, n_tiles);
  else
    hipLaunchKernelGGL((k_i8_few<EPI, false, KW, RT>), grid, block, 0, s, p, n_tiles);
  return nv_launch_status();
}

// Which kernel takes a call.
struct I8Plan {
  int few;        // k_i8_few with so many waves to a block of columns, or 0
  int rt;         // its row tiles of 16 to a workgroup
  int64_t tiles;  // workgroups' row tiles at most
  int tile;       // else: which of kTiles
  int parts;      // parts of K that its workgroups share, or 0
};

// Times below are those of the product alone, from quantized rows, in a graph of
// calls back to back.
I8Plan plan_of(const int8_gemm_args_t* a) {
  I8Plan pl{};
  const int64_t rows = a->total_rows, G = a->num_groups;
  const int64_t cols = a->epilogue == NVFP4_EPI_SILU_MUL_BF16 ? a->N / 2 : a->N;
  // Few rows: the tile kernels have one workgroup for 128 columns of a row tile,
  // which leaves CUs idle up to about 1024 units of 16 columns and rows (4096^2: 1
  // row 4.7 us for 11.7, 64 rows 12.1 for 12.4, 128 rows 21 for 12.6; 128
  // experts, K 2048, N 1536, one token's 8 rows 7.9 for 9.7, four tokens' 32 rows
  // 21.6 for 18.0; K 768, N 2048: 4.9 for 6.6).  With the fewest waves to a block
  // of columns that make 1536 in all (1 row of 4096^2: 8, 4, 2 waves 4.7, 6.8, 10.8 us;
  // 8 rows of 128 experts, K 2048: 9.3, 7.8, 12.1; K 768: 6.8, 5.0, 4.9).
  pl.rt = G > 1 || rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  pl.tiles = G == 1 ? (rows + 16 * pl.rt - 1) / (16 * pl.rt) : (rows < G ? rows : G) + rows / 16;
  const int64_t units = pl.tiles * ((cols + 15) / 16);
  if (rows <= (G == 1 ? 64 : 16 * G) && units <= 1024) {
    pl.few = units * 2 >= 1536 ? 2 : units * 4 >= 1536 ? 4 : 8;
    return pl;
  }
  const double mean = (double)rows / (double)G;
  if (G == 1) {
    // rounds over the chip times a tile's time beside the 256 x 256 tile's (N = K =
    // 4096: 512 rows 20, 24, 41 us for tiles 0, 1, 2; 1024 rows 25, 26, 43; 2048
    // rows 54, 36, 48; 4096 rows 98, 70, 60 and 64 for tile 3)
    auto rounds = [&](int i) {
      return (double)((i8_workgroups(kTiles[i], rows, a->N, 0) + 255) / 256);
    };
    const double c[4] = {rounds(0) * 0.19 + 0.1, rounds(1) * 0.62, rounds(2), rounds(3) * 1.25};
    for (int i = 1; i < 4; ++i)
      if (c[i] < c[pl.tile]) pl.tile = i;
    // Where one workgroup a CU does not fill the chip, K is split if that saves
    // more than its sums cost: a chunk of 128 k takes 0.44 us, the join 3 us and
    // 3 bytes a picosecond for the sums' way out and back (N 4096: 128 rows, K 4096
    // 17.9 us whole, 15.2 in four parts; 256 rows 18.4, and 19.7 in two; 200 rows, K
    // 8192 32.8 and 23.9, K 2048 10.6 and 13.9; 100 rows, N 2048, K 7168 28.5 and
    // 13.9).
    const int64_t wgs = i8_workgroups(kTiles[0], rows, a->N, 0);
    double best = 0;
    if (pl.tile == 0 && !a->group_offsets && a->epilogue != NVFP4_EPI_SILU_MUL_BF16)
      for (int parts = 2; parts <= 8 && wgs * parts <= 256 && a->K >= 512 * parts; parts *= 2) {
        const double saved = (double)a->K / 128 * 0.44 * (1 - 1.0 / parts) - 3 -
                             (double)rows * (double)a->N * 8 * parts / 3e6;
        if (saved > best) {
          best = saved;
          pl.parts = parts;
        }
      }
  } else if (mean <= 48) {
    // 128 experts, N 1536, K 2048: 32 rows each 77 us (tile 1: 79), 64 rows 92
    // (87); 256 experts, N 4096, K 7168: 64 rows 1522 (1316)
    pl.tile = 0;
  } else if (mean <= 112) {
    pl.tile = 1;  // 128 rows each: tile 2 104.5 us, tile 1 114.5; 64 rows: 93 and 87
  } else {
    // fewest tiles for rows that vary by twice the square root of their mean: a
    // second tile reads all of W again (256 experts of 256 +- 16 rows, N 4096, K
    // 7168: 2137 us on 320-row tiles, 2476 on 256-row ones)
    const double most = mean + 2 * __builtin_sqrt(mean);
    pl.tile = __builtin_ceil(most / 320) * 1.22 < __builtin_ceil(most / 256) ? 3 : 2;
  }
  return pl;
}

template <int EPI, int RT>
int launch_few_of(const I8Params& p, const I8Plan& pl, hipStream_t s) {
  if (pl.few == 2) return launch_few<EPI, 2, RT>(p, pl.tiles, s);
  if (pl.few == 4) return launch_few<EPI, 4, RT>(p, pl.tiles, s);
  return launch_few<EPI, 8, RT>(p, pl.tiles, s);
}

template <int EPI>
int launch_gemm(const I8Params& p, const I8Plan& pl, hipStream_t s) {
  if (pl.few) {
    if (pl.rt == 1) return launch_few_of<EPI, 1>(p, pl, s);
    if (pl.rt == 2) return launch_few_of<EPI, 2>(p, pl, s);
    return launch_few_of<EPI, 4>(p, pl, s);
  }
  if constexpr (EPI != NVFP4_EPI_SILU_MUL_BF16)
    if (pl.parts) return launch_split<EPI>(p, pl.parts, s);
  if (pl.tile == 0) return launch_tiles<0, 2, 2, 1, 2, 2, EPI>(p, s);  // three to a CU
  if (pl.tile == 1) return launch_tiles<1, 2, 4, 2, 2, 3, EPI>(p, s);
  if (pl.tile == 2) return launch_tiles<2, 4, 2, 2, 4, 2, EPI>(p, s);
  return launch_tiles<3, 2, 4, 5, 2, 2, EPI>(p, s);
}

template <bool BF16, int RW, int VPL>
int launch_rows_of(const void* x, int64_t rows, int K, int64_t ldx, int8_t* codes, float* scales,
                   hipStream_t s) {
  const int64_t wgs = (rows * RW + 7) / 8;
  const dim3 grid((unsigned)(wgs < (1 << 20) ? wgs : (1 << 20)));
  hipLaunchKernelGGL((k_i8_rows<BF16, RW, VPL>), grid, dim3(512), 0, s, x, rows, K, ldx, codes,
                     scales);
  return nv_launch_status();
}

// Times of one input again and again, which the last-level cache holds.  A workgroup
// for a row where rows are few (one wave a row before: 128 x 7168 8.6 us, now 3.9; 512 x 4096 6.2 and 4.0; 1 x 4096 5.1 and 3.9); else waves enough to
// hold it in registers (8192 x 7168 read twice 44 us, four waves of 4 vectors 32,
// eight of 2 29; 65536 x 2048 89, one of 4 76, two of 2 73, four of 1 92; 4096 x
// 4096 two of 4 10.7, four of 2 11.7).
template <bool BF16>
int launch_rows_by_size(const void* x, int64_t rows, int K, int64_t ldx, int8_t* codes, float* scales,
                     hipStream_t s) {
  const int nv = K / 8;
  if (rows <= 512 && nv > 64) {
    if (nv <= 512) return launch_rows_of<BF16, 8, 1>(x, rows, K, ldx, codes, scales, s);
    return launch_rows_of<BF16, 8, 4>(x, rows, K, ldx, codes, scales, s);
  }
  if (nv <= 64) return launch_rows_of<BF16, 1, 1>(x, rows, K, ldx, codes, scales, s);
  if (nv <= 128) return launch_rows_of<BF16, 1, 2>(x, rows, K, ldx, codes, scales, s);
  if (nv <= 256) return launch_rows_of<BF16, 2, 2>(x, rows, K, ldx, codes, scales, s);
  if (nv <= 512) return launch_rows_of<BF16, 2, 4>(x, rows, K, ldx, codes, scales, s);
  if (nv <= 1024) return launch_rows_of<BF16, 8, 2>(x, rows, K, ldx, codes, scales, s);
  return launch_rows_of<BF16, 8, 4>(x, rows, K, ldx, codes, scales, s);
}

int launch_rows(const void* x, int64_t dtype, int64_t rows, int K, int64_t ldx, int8_t* codes,
                float* scales, hipStream_t s) {
  return dtype == NVFP4_IN_BF16 ? launch_rows_by_size<true>(x, rows, K, ldx, codes, scales, s)
                                : launch_rows_by_size<false>(x, rows, K, ldx, codes, scales, s);
}

bool misaligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }

// The checks shared by the workspace size and the call.
int check_gemm(const int8_gemm_args_t* a) {
  NV_RETURN_IF(!a, NVFP4_ERR_NULL);
  NV_RETURN_IF(a->epilogue != NVFP4_EPI_F32 && a->epilogue != NVFP4_EPI_SILU_MUL_BF16 &&
                   a->epilogue != NVFP4_EPI_BF16,
               NVFP4_ERR_DTYPE);
  NV_RETURN_IF(a->num_groups < 1 || a->num_groups > (1 << 20) || a->total_rows < 0 ||
                   a->total_rows > (1 << 30) || a->N < 1 || a->N > (1 << 24) || a->K < 16 ||
                   a->K % 16 || a->K > kMaxK ||
                   (a->epilogue == NVFP4_EPI_SILU_MUL_BF16 && a->N % 2),
               NVFP4_ERR_SHAPE);
  // a gathered row is addressed by 32 bits of 16-byte units, up to seven behind its
  // start before a short chunk's step back
  NV_RETURN_IF(a->src_rows < 0 || a->src_rows > 0x7fffffff || a->src_rows * a->K > (1LL << 36) ||
                   (a->gather_rows && (a->src_rows - 1) * (a->K >> 4) + 7 > 0xffffffffLL) ||
                   (!a->gather_rows && a->src_rows < a->total_rows) ||
                   (a->src_rows == 0 && a->total_rows > 0),
               NVFP4_ERR_SHAPE);
  if (a->x) {
    NV_RETURN_IF(a->x_dtype != NVFP4_IN_F32 && a->x_dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
    NV_RETURN_IF(a->ldx < a->K, NVFP4_ERR_SHAPE);
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
  if (check_gemm(a) != NVFP4_OK || a->total_rows == 0) return 0;
  const I8Plan pl = plan_of(a);
  // quantized rows and their scales, sums over parts of K
  return (a->x ? nv_round256((size_t)a->src_rows * (size_t)a->K) + nv_round256(4 * (size_t)a->src_rows) : 0) +
         4 * (size_t)pl.parts * (size_t)a->total_rows * (size_t)((a->N + 3) & ~3);
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
  const int64_t cols = a->epilogue == NVFP4_EPI_SILU_MUL_BF16 ? a->N / 2 : a->N;
  p.vec = !misaligned(a->out, 16) && cols * esize % 16 == 0;
  const I8Plan pl = plan_of(a);
  // the grid holds fewer than 2^32 threads
  NV_RETURN_IF(!pl.few && i8_workgroups(kTiles[pl.tile], a->total_rows, a->N, a->num_groups) *
                                  kTiles[pl.tile].threads > 0xffffffffLL,
               NVFP4_ERR_SHAPE);
  if (a->x) {
    int8_t* codes = reinterpret_cast<int8_t*>(ws);
    float* scales = reinterpret_cast<float*>(codes + nv_round256((size_t)a->src_rows * p.K));
    p.a_codes = codes;
    p.a_scales = scales;
    ws = scales + nv_round256(4 * (size_t)a->src_rows) / 4;
    const int st = launch_rows(a->x, a->x_dtype, a->src_rows, p.K, a->ldx, codes, scales, s);
    if (st != NVFP4_OK) return st;
  }
  p.part = reinterpret_cast<int32_t*>(ws);
  p.pitch = (p.N + 3) & ~3;
  if (a->epilogue == NVFP4_EPI_SILU_MUL_BF16)
    return launch_gemm<NVFP4_EPI_SILU_MUL_BF16>(p, pl, s);
  if (a->epilogue == NVFP4_EPI_BF16) return launch_gemm<NVFP4_EPI_BF16>(p, pl, s);
  return launch_gemm<NVFP4_EPI_F32>(p, pl, s);
}

}  // extern "C"
