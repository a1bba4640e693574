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
// that is a number) do not overflow, and the row's maximum gives exactly 1.
// Reported log-probabilities are (l_j - m) inv_temperature - ln 2 log2 S.
//
// The forward pass is bound by reading the logits where there are rows enough:
// 4096 x 131072 bf16 with 8 alternatives 174 us (163-185), 6.2 TB/s (a large copy
// reaches 4.9 here); its arithmetic, of which a quarter-rate exponential per
// logit is the largest part, takes about two thirds of that.  A single row is bound by
// the arithmetic of the CU that it is on, and by latency: 1 x 32768 with 5
// alternatives 8 us.  The backward pass reads and writes 2048 x 131072 in 181
// us (177-190), 5.9 TB/s; the forward pass before it takes 88 us (84-96).  These
// are medians and ranges of settled calls: over the first 40 after an idle time
// they are 222, 187 and 96 us.  (The base 2 costs little accuracy: of 4096 x 131072
// the log-probabilities are off by 1.2e-7 of their norm, with natural
// exponentials in FP32 by 6.7e-8.)
#include "common.h"

namespace {

constexpr int kLpMaxTop = 32;
constexpr int64_t kLpMaxV = 1 << 30;        // element indexes with room for a step behind the row
constexpr int64_t kLpMaxT = (1 << 24) - 1;  // a launch has less than 2^32 threads
constexpr int kLpCand = 128;   // candidates that are ranked at a time
constexpr int kLpPieces = 512; // pieces of a row that wait for the ranking
constexpr float kLpLowest = -3.402823466e38f;  // masked tokens (-inf) are below it
constexpr int kLpU = 4;        // 16-byte pieces of a thread in flight, and as many in work
constexpr int kLpBwdU = 4;     // 16-byte pieces of a thread in the backward pass
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kInf = __builtin_inff();

// 16 bytes of logits and what an absent element counts as.
template <typename E>
struct Lanes;
template <>
struct Lanes<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xFF800000u;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    return __uint_as_float(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w);
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};
typedef __bf16 lp_bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t lp_word4 __attribute__((ext_vector_type(4)));
template <>
struct Lanes<uint16_t> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xFF80FF80u;
  static __device__ __forceinline__ float get(const uint4& v, int i) {
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) { return nv_bf16_to_f32(*p); }
  static __device__ __forceinline__ uint32_t pair(float a, float b) {  // nearest even, NaN kept
    const lp_bf16x2 r = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, r);
  }
  static __device__ __forceinline__ void store(uint16_t* p, float v) { *p = (uint16_t)pair(v, v); }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7]));
  }
};

__device__ __forceinline__ bool lp_better(float va, int ia, float vb, int ib) {
  return va > vb || (va == vb && ia < ib);
}

// log p of a logit from the row's maximum m and L = log2 S.
__device__ __forceinline__ float lp_value(float l, float m, float it, float L) {
  return l == -kInf ? l : __builtin_fmaf(-kLn2, L, (l - m) * it);
}

// (m, S, Q) relative to its own maximum, brought to the maximum M.
__device__ __forceinline__ void lp_rebase(float m, float M, float c, float& S, float& Q) {
  const float delta = m == -kInf ? -kInf : (m - M) * c;
  const float f = __builtin_amdgcn_exp2f(delta);
  Q = f > 0.0f ? f * __builtin_fmaf(S, delta, Q) : 0.0f;
  S *= f;  // a NaN stays
}

__device__ __forceinline__ float lp_wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = __builtin_fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
__device__ __forceinline__ float lp_wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// Float order as unsigned order (no NaN).
__device__ __forceinline__ uint32_t lp_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);  // -0 equals +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A bound that at least k of the wave's 64 values reach and that the k-th
// largest is not far above: bisection on the upper 16 bits of the order key.
// Returns the smallest float of the key prefix; -inf if fewer than k values
// are above -inf.
__device__ __forceinline__ float lp_wave_threshold(float v, int k) {
  const uint32_t key = lp_key(v);
  uint32_t lo = 0;
#pragma unroll
  for (int b = 31; b >= 16; --b) {
    const uint32_t t = lo | (1u << b);
    if (__popcll(__ballot(key >= t)) >= k) lo = t;
  }
  const float f = __uint_as_float((lo & 0x80000000u) ? (lo ^ 0x80000000u) : ~lo);
  return f == f ? f : -kInf;  // below the key of -inf
}

// What the lanes of a wave wrote to LDS before it, all of them read after it.
__device__ __forceinline__ void lp_wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct LpShared {
  float val[kLpMaxTop];  // the best so far, ordered
  int idx[kLpMaxTop];
  int n;                 // how many
  float cval[kLpCand];   // candidates of one wave
  int cidx[kLpCand];
};

// Merges the first n candidates into the best list (one wave).  The list and
// up to 64 - k candidates lie on the lanes, and a lane's rank is the number
// of lanes ahead of it: one unsigned comparison of value and inverted index.
__device__ __forceinline__ void lp_rank(LpShared& sh, int n, int k) {
  const int lane = threadIdx.x & 63;
  lp_wave_sync();
  int have = sh.n;
  for (int c0 = 0; c0 < n; c0 += 64 - k) {
    const int live = have + min(64 - k, n - c0);
    float v = -kInf;
    int i = 0x7fffffff;
    if (lane < have) {
      v = sh.val[lane];
      i = sh.idx[lane];
    } else if (lane < live) {
      v = sh.cval[c0 + lane - have];
      i = sh.cidx[c0 + lane - have];
    }
    const uint32_t hi = lp_key(v), lo = ~(uint32_t)i;
    const uint64_t key = ((uint64_t)hi << 32) | lo;
    int rank = 0;
    for (int o = 0; o < live; ++o) {
      const uint64_t other = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)hi, o) << 32) |
                             (uint32_t)__builtin_amdgcn_readlane((int)lo, o);
      rank += other > key ? 1 : 0;
    }
    lp_wave_sync();
    if (lane < live && rank < k) {
      sh.val[rank] = v;
      sh.idx[rank] = i;
    }
    lp_wave_sync();
    have = min(k, live);
  }
  if (lane == 0) sh.n = have;
  lp_wave_sync();
}

// Adds the lanes' kept values to the cnt candidates, ranking those first if
// the list would not hold them (one wave).  Returns the new count.
__device__ __forceinline__ int lp_push(LpShared& sh, int cnt, bool keep, float v, int i, int k) {
  const uint64_t bal = __ballot(keep);
  const int more = __popcll(bal);
  if (cnt + more > kLpCand) {
    lp_rank(sh, cnt, k);
    cnt = 0;
  }
  if (keep) {
    const int at = cnt + __popcll(bal & ((1ull << (threadIdx.x & 63)) - 1));
    sh.cval[at] = v;
    sh.cidx[at] = i;
  }
  return cnt + more;
}

// Pieces in which some logit reaches the bound.
template <int N>
struct LpPieces {
  float v[kLpPieces][N];
  int id[kLpPieces];  // piece, or -1 - element for a single element in v[0]
  int n;              // may exceed the list
};

// Ranks the elements of the first n pieces (one wave).
template <int N>
__device__ __forceinline__ void lp_take(LpShared& sh, const LpPieces<N>& pc, int n, int head,
                                        int k) {
  const int lane = threadIdx.x & 63;
  float g = -kInf;
  for (int c = lane; c < n; c += 64) {
#pragma unroll
    for (int i = 0; i < N; ++i) g = __builtin_fmaxf(g, pc.v[c][i]);
  }
  float tau = __builtin_fmaxf(lp_wave_threshold(g, k), kLpLowest);
  if (sh.n == k) tau = __builtin_fmaxf(tau, sh.val[k - 1]);
  int cnt = 0;
  for (int c0 = 0; c0 < n; c0 += 64) {
    const int c = c0 + lane, id = c < n ? pc.id[c] : 0;
    float v[N], m = -kInf;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = c < n ? pc.v[c][i] : -kInf;
      m = __builtin_fmaxf(m, v[i]);
    }
    if (!__ballot(m >= tau)) continue;
#pragma unroll
    for (int i = 0; i < N; ++i)
      cnt = lp_push(sh, cnt, v[i] >= tau, v[i], id < 0 ? -1 - id : head + id * N + i, k);
  }
  lp_rank(sh, cnt, k);
}

// The best list of a row completed with masked tokens (one wave): fewer than
// top_k logits are above -inf, so the first 2 top_k <= 64 tokens hold enough.
template <typename E>
__device__ __forceinline__ void lp_fill_masked(LpShared& sh, const E* row, int V, int k) {
  const int lane = threadIdx.x & 63;
  const int have = sh.n;
  if (have >= k) return;
  const float l = lane < V ? Lanes<E>::load(row + lane) : kInf;
  const bool none = !(l > -kInf);  // -inf or NaN
  const uint64_t bal = __ballot(none);
  const int at = have + __popcll(bal & ((1ull << lane) - 1));
  if (none && at < k) {
    sh.val[at] = -kInf;
    sh.idx[at] = lane;
  }
  lp_wave_sync();
}

// What one workgroup knows of a row, or of a part of one.
struct LpPart {
  float m, S, Q, pad;
};

__host__ __device__ inline size_t lp_part_bytes(int top_k) {
  return sizeof(LpPart) + 8 * (size_t)top_k;
}

// Writes a row's results (one wave).
template <typename E>
__device__ __forceinline__ void lp_finish(LpShared& sh, const E* row, int V, int64_t t, float gm,
                                          float S, float Q, float it, int64_t y, float ly,
                                          int top_k, float* logprobs,
                                          float* entropy, float* norm, int32_t* top_ids,
                                          float* top_lp) {
  const int lane = threadIdx.x & 63;
  const bool empty = gm == -kInf && S == S;
  const float m = gm == -kInf ? 0.0f : gm;
  const float L = empty ? -kInf : __builtin_log2f(S);
  if (lane == 0) {
    if (logprobs) {
      float lp = 0.0f;
      if (y >= V) lp = __builtin_nanf("");
      else if (y >= 0) lp = S == S ? lp_value(ly, m, it, L) : S;
      logprobs[t] = lp;
    }
    if (entropy) entropy[t] = empty ? 0.0f : (L - Q / S) * kLn2;
    if (norm) {
      norm[2 * t] = m;
      norm[2 * t + 1] = L;
    }
  }
  if (lane < top_k) {
    top_ids[t * top_k + lane] = sh.idx[lane];
    top_lp[t * top_k + lane] = S == S ? lp_value(sh.val[lane], m, it, L) : S;
  }
}

// The target of a row and its logit, fetched before the row is read.
template <typename E>
__device__ __forceinline__ void lp_target(const E* row, int V, const int64_t* targets, int64_t t,
                                          int64_t& y, float& ly) {
  y = targets ? targets[t] : -1;
  ly = y >= 0 && y < V ? Lanes<E>::load(row + y) : 0.0f;
}

// One workgroup of NT threads per (row, part).  A thread takes U 16-byte
// pieces at a time into registers, the next ones in flight behind them: their
// maximum is known before the first exponential, so each element costs one
// exponential and the memory is read once.  The alternatives come from the
// same registers: in the first chunk the 64 maxima over lanes give a bound
// that at least top_k elements reach, later the worst of the best so far is
// one; the few elements at or above it become candidates, which one wave
// ranks when there are many.  Rows start at any element: the pieces are those
// that lie wholly inside the row at 16-byte addresses, and the up to N - 1
// elements before and after them go one to a thread.  STREAM: the logits are
// not kept in the caches.
template <typename E, int NT, bool TOP, bool STREAM>
__global__ __launch_bounds__(NT, 4) void k_logprob(
    const E* __restrict__ logits, int V, int64_t ld, const int64_t* __restrict__ targets,
    const float* __restrict__ inv_t, int top_k, int parts, float* __restrict__ logprobs,
    float* __restrict__ entropy, float* __restrict__ norm, int32_t* __restrict__ top_ids,
    float* __restrict__ top_lp, uint8_t* __restrict__ ws) {
  typedef Lanes<E> LE;
  constexpr int N = LE::N, U = kLpU, NW = NT / 64;
  __shared__ float lane_max[TOP ? NW * 64 : 1];
  __shared__ float red[3 * NW];
  __shared__ LpShared sh;
  __shared__ __attribute__((aligned(16))) LpPieces<N> pc;
  const int64_t t = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const E* row = logits + t * ld;
  const float it = inv_t ? inv_t[t] : 1.0f, c = it * kLog2e;
  const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(E), V);
  const int nv = (V - head) / N, tail = head + nv * N;  // pieces; first element after them
  const uint4* vec = reinterpret_cast<const uint4*>(row + head);
  const int per = (nv + parts - 1) / parts, v0 = min(part * per, nv), v1 = min(v0 + per, nv);

  uint4 x[U];
  auto fetch = [&](int b) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + u * NT + tid;
      x[u] = make_uint4(LE::kNone, LE::kNone, LE::kNone, LE::kNone);
      if constexpr (STREAM) {
        if (i < v1) {
          const lp_word4 w =
              __builtin_nontemporal_load(reinterpret_cast<const lp_word4*>(row + head) + i);
          x[u] = make_uint4(w.x, w.y, w.z, w.w);
        }
      } else {
        if (i < v1) x[u] = vec[i];
      }
    }
  };
  fetch(v0);
  // elements outside the pieces, with the first part's first chunk
  float ev = -kInf;
  int ei = -1;
  if (part == 0) {
    if (tid < head) ei = tid;
    else if (tid >= 32 && tail + tid - 32 < V && tid < 32 + N) ei = tail + tid - 32;
    if (ei >= 0) ev = LE::load(row + ei);
  }
  int64_t y = -1;
  float ly = 0.0f;
  if (wave == 0) lp_target(row, V, targets, t, y, ly);
  if (TOP) {
    if (tid == 0) sh.n = pc.n = 0;
    __syncthreads();
  }
  float m = -kInf, S = 0.0f, Q = 0.0f;
  float tau = -kInf;
  bool masked = false;
  int b = v0, chunk = 0, sync = 8;
  do {
    float f[U * N], pm[U], tm = ev;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float v = -kInf;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        f[u * N + i] = LE::get(x[u], i);
        v = __builtin_fmaxf(v, f[u * N + i]);
      }
      pm[u] = v;
      tm = __builtin_fmaxf(tm, v);
    }
    const int next = b + NT * U;
    if (next < v1) fetch(next);
    const float M = __builtin_fmaxf(m, tm);
    if (M > m) {
      if (m != -kInf) lp_rebase(m, M, c, S, Q);
      m = M;
    }
    const float ref = m == -kInf ? 0.0f : m;
    if (!masked) {
      const float S0 = S, Q0 = Q;
      auto add = [&](float l) {
        const float d = (l - ref) * c, e = __builtin_amdgcn_exp2f(d);
        S += e;
        Q = __builtin_fmaf(d, e, Q);
      };
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b + u * NT + tid < v1) {
#pragma unroll
          for (int i = 0; i < N; ++i) add(f[u * N + i]);
        }
      if (ei >= 0) add(ev);
      masked = __ballot(Q != Q) != 0;
      S = masked ? S0 : S;
      Q = masked ? Q0 : Q;
    }
    if (masked) {
      // masked logits (0 times -inf above) or NaN: again, and from here on,
      // with the factor d bounded below, where 2^d is 0
      auto add = [&](float l) {
        const float d = (l - ref) * c, e = __builtin_amdgcn_exp2f(d);
        S += e;
        Q = __builtin_fmaf(__builtin_fmaxf(d, -1e4f), e, Q);
      };
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (b + u * NT + tid < v1) {
#pragma unroll
          for (int i = 0; i < N; ++i) add(f[u * N + i]);
        }
      if (ei >= 0) add(ev);
    }

    if constexpr (TOP) {
      if (b == v0) {
        lane_max[wave * 64 + lane] = tm;
        __syncthreads();
        float g = -kInf;
#pragma unroll
        for (int w = 0; w < NW; ++w) g = __builtin_fmaxf(g, lane_max[w * 64 + lane]);
        tau = lp_wave_threshold(g, top_k);
      } else if (sh.n == top_k) {
        tau = sh.val[top_k - 1];
      }
      tau = __builtin_fmaxf(tau, kLpLowest);
      auto wait = [&](int id, const float* l) {
        const int at = atomicAdd(&pc.n, 1);
        if (at < kLpPieces) {
          pc.id[at] = id;
#pragma unroll
          for (int i = 0; i < N; ++i) pc.v[at][i] = l[i];
        }
      };
      if (__ballot(tm >= tau)) {
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (pm[u] >= tau) wait(b + u * NT + tid, f + u * N);
        if (ev >= tau) {
          float l[N];
#pragma unroll
          for (int i = 0; i < N; ++i) l[i] = i ? -kInf : ev;
          wait(-1 - ei, l);
        }
      }
    }
    // The waiting pieces are ranked after the last chunk, and in rows of many
    // chunks after 8, 64, ..: a bound that some 1.4 top_k of n tokens reach
    // lets through as many of each further n, and the waves need not wait for
    // each other in between.
    ++chunk;
    if constexpr (TOP) if (chunk == sync || next >= v1) {
      sync *= 8;
      __syncthreads();
      const int n = pc.n;
      if (n > kLpPieces) {
        // more than can wait (ties, rising rows): top_k rounds of an arg-max
        // over everything read so far.  Rows of ties with 20 alternatives: 16 x
        // 131072 177 us for 19; 4096 x 131072 of equal or rising logits, with 8,
        // 10.8 ms for 0.17
        float pv = kInf;
        int pi = -1;
        const int j0 = head + v0 * N, j1 = head + min(next, v1) * N;
        for (int k = 0; k < top_k; ++k) {
          float bv = -kInf;
          int bi = 0x7fffffff;
          auto seen = [&](float l, int j) {
            if (l > -kInf && lp_better(pv, pi, l, j) && lp_better(l, j, bv, bi)) {
              bv = l;
              bi = j;
            }
          };
          for (int j = j0 + tid; j < j1; j += NT) seen(LE::load(row + j), j);
          if (part == 0) {
            if (tid < head) seen(LE::load(row + tid), tid);
            else if (tid >= 32 && tail + tid - 32 < V && tid < 32 + N)
              seen(LE::load(row + tail + tid - 32), tail + tid - 32);
          }
#pragma unroll
          for (int o = 32; o > 0; o >>= 1) {
            const float ov = __shfl_xor(bv, o, 64);
            const int oi = __shfl_xor(bi, o, 64);
            if (lp_better(ov, oi, bv, bi)) {
              bv = ov;
              bi = oi;
            }
          }
          __syncthreads();  // the list may still be read
          if (lane == 0) {
            sh.cval[wave] = bv;
            sh.cidx[wave] = bi;
          }
          __syncthreads();
          for (int w = 0; w < NW; ++w)
            if (lp_better(sh.cval[w], sh.cidx[w], bv, bi)) {
              bv = sh.cval[w];
              bi = sh.cidx[w];
            }
          if (tid == 0) {
            sh.val[k] = bv;
            sh.idx[k] = bi;
          }
          pv = bv;
          pi = bi;
        }
        if (tid == 0) {
          sh.n = top_k;
          pc.n = 0;
        }
      } else if (wave == 0 && n > 0) {
        lp_take<N>(sh, pc, n, head, top_k);
        if (lane == 0) pc.n = 0;
      }
      __syncthreads();
    }
    ev = -kInf;
    ei = -1;
    b = next;
  } while (b < v1);

  // the workgroup's (m, S, Q)
  const float wm = lp_wave_max(m);
  if (wm > -kInf) lp_rebase(m, wm, c, S, Q);
  S = lp_wave_sum(S);
  Q = lp_wave_sum(Q);
  float gm = wm;
  if constexpr (NW > 1) {
    if (lane == 0) {
      red[3 * wave] = wm;
      red[3 * wave + 1] = S;
      red[3 * wave + 2] = Q;
    }
    __syncthreads();
    if (wave > 0) return;
    const float a = lane < NW ? red[3 * lane] : -kInf;
    S = lane < NW ? red[3 * lane + 1] : 0.0f;
    Q = lane < NW ? red[3 * lane + 2] : 0.0f;
    gm = lp_wave_max(a);
    if (gm > -kInf) lp_rebase(a, gm, c, S, Q);
    S = lp_wave_sum(S);
    Q = lp_wave_sum(Q);
  }
  if (parts > 1) {
    uint8_t* out = ws + blockIdx.x * lp_part_bytes(TOP ? top_k : 0);
    if (lane == 0) *reinterpret_cast<LpPart*>(out) = LpPart{gm, S, Q};
    if (TOP && lane < top_k) {
      reinterpret_cast<float*>(out + sizeof(LpPart))[lane] = lane < sh.n ? sh.val[lane] : -kInf;
      reinterpret_cast<int*>(out + sizeof(LpPart))[top_k + lane] = sh.idx[lane];
    }
    return;
  }
  if (TOP) lp_fill_masked(sh, row, V, top_k);
  lp_finish<E>(sh, row, V, t, gm, S, Q, it, y, ly, TOP ? top_k : 0, logprobs, entropy, norm,
               top_ids, top_lp);
}

// Joins the parts of a row: one wave per row.
template <typename E>
__global__ __launch_bounds__(64) void k_logprob_join(
    const E* __restrict__ logits, int V, int64_t ld, const int64_t* __restrict__ targets,
    const float* __restrict__ inv_t, int top_k, int parts, float* __restrict__ logprobs,
    float* __restrict__ entropy, float* __restrict__ norm, int32_t* __restrict__ top_ids,
    float* __restrict__ top_lp, const uint8_t* __restrict__ ws) {
  __shared__ LpShared sh;
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x;
  const E* row = logits + t * ld;
  const float it = inv_t ? inv_t[t] : 1.0f, c = it * kLog2e;
  const size_t step = lp_part_bytes(top_k);
  const uint8_t* in = ws + t * parts * step;
  int64_t y;
  float ly;
  lp_target(row, V, targets, t, y, ly);
  LpPart p{-kInf, 0.0f, 0.0f, 0};  // parts <= 64
  if (lane < parts) p = *reinterpret_cast<const LpPart*>(in + lane * step);
  const float gm = lp_wave_max(p.m);
  if (gm > -kInf) lp_rebase(p.m, gm, c, p.S, p.Q);
  const float S = lp_wave_sum(p.S), Q = lp_wave_sum(p.Q);
  if (top_k) {
    if (lane == 0) sh.n = 0;
    lp_wave_sync();
    const int total = parts * top_k;
    float g = -kInf;
    auto entry = [&](int c, int& i) -> float {
      const int q = c / top_k, e = c - q * top_k;
      const float* val = reinterpret_cast<const float*>(in + q * step + sizeof(LpPart));
      i = reinterpret_cast<const int*>(val)[top_k + e];
      return val[e];
    };
    int i = 0, cnt = 0;
    for (int c = lane; c < total; c += 64) g = __builtin_fmaxf(g, entry(c, i));
    const float tau = __builtin_fmaxf(lp_wave_threshold(g, top_k), kLpLowest);
    for (int c0 = 0; c0 < total; c0 += 64) {
      const float v = c0 + lane < total ? entry(c0 + lane, i) : -kInf;
      cnt = lp_push(sh, cnt, v >= tau, v, i, top_k);
    }
    lp_rank(sh, cnt, top_k);
    lp_fill_masked(sh, row, V, top_k);
  }
  lp_finish<E>(sh, row, V, t, gm, S, Q, it, y, ly, top_k, logprobs, entropy, norm, top_ids,
               top_lp);
}

// The gradient: one pass, each element read and written by the same thread
// (so the gradient may replace the logits).  With k0 = -it (a + b H) and
// k1 = -it b ln 2, grad_j = p_j (k0 + k1 d_j), plus it a at the target.
// STREAM: the gradient is not kept in the caches, and rows go from the last to
// the first, whose end the forward pass left in the last-level cache.
template <typename E, int NT, bool VEC, bool STREAM>
__global__ __launch_bounds__(NT) void k_logprob_bwd(
    const E* logits, int64_t T, int V, int64_t ld, const int64_t* __restrict__ targets,
    const float* __restrict__ inv_t, const float* __restrict__ norm,
    const float* __restrict__ entropy, const float* __restrict__ g_lp,
    const float* __restrict__ g_ent, E* grad, int64_t ldg) {
  typedef Lanes<E> LE;
  constexpr int N = LE::N;
  for (int64_t n = blockIdx.y; n < T; n += gridDim.y) {
    const int64_t t = STREAM ? T - 1 - n : n;
    const E* row = logits + t * ld;
    E* out = grad + t * ldg;
    const float it = inv_t ? inv_t[t] : 1.0f, c = it * kLog2e;
    const float m = norm[2 * t], L = norm[2 * t + 1];
    const bool empty = L == -kInf;
    const int64_t y = targets ? targets[t] : -1;
    float a = (g_lp && y >= 0 && !empty) ? g_lp[t] : 0.0f;
    const float b = (g_ent && !empty) ? g_ent[t] : 0.0f;
    const bool wrong = g_lp && y >= V;
    const bool none = a == 0.0f && b == 0.0f && !wrong;  // zeros; the logits are not read
    if (wrong || (L != L && !none)) a = __builtin_nanf("");
    const float k0 = -it * (a + (g_ent && !empty ? b * entropy[t] : 0.0f)), k1 = -it * kLn2 * b;
    const float Lf = empty ? kInf : L;
    auto value = [&](float l) {
      const float d = __builtin_fmaxf(__builtin_fmaf(l - m, c, -Lf), -1e4f);  // 2^-1e4 is 0
      return __builtin_amdgcn_exp2f(d) * __builtin_fmaf(k1, d, k0);
    };
    auto one = [&](int j) {
      const float g = none ? 0.0f : value(LE::load(row + j));
      LE::store(out + j, j == y ? __builtin_fmaf(it, a, g) : g);
    };
    if constexpr (!VEC) {
      for (int64_t j = (int64_t)blockIdx.x * NT + threadIdx.x; j < V; j += (int64_t)gridDim.x * NT)
        one((int)j);
    } else {
      const int head =
          min((int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / (int)sizeof(E), V);
      const int nv = (V - head) / N, tail = head + nv * N;
      const uint4* vec = reinterpret_cast<const uint4*>(row + head);
      auto put = [&](int i, const uint4& v) {
        if constexpr (STREAM)
          __builtin_nontemporal_store(lp_word4{v.x, v.y, v.z, v.w},
                                      reinterpret_cast<lp_word4*>(out + head) + i);
        else
          reinterpret_cast<uint4*>(out + head)[i] = v;
      };
      for (int i0 = blockIdx.x * (NT * kLpBwdU); i0 < nv; i0 += gridDim.x * (NT * kLpBwdU)) {
        if (none) {
#pragma unroll
          for (int u = 0; u < kLpBwdU; ++u) {
            const int i = i0 + u * NT + threadIdx.x;
            if (i < nv) put(i, make_uint4(0, 0, 0, 0));
          }
          continue;
        }
        uint4 x[kLpBwdU];
#pragma unroll
        for (int u = 0; u < kLpBwdU; ++u) {
          const int i = i0 + u * NT + threadIdx.x;
          if (i < nv) x[u] = vec[i];
        }
#pragma unroll
        for (int u = 0; u < kLpBwdU; ++u) {
          const int i = i0 + u * NT + threadIdx.x;
          if (i < nv) {
            float g[N];
#pragma unroll
            for (int e = 0; e < N; ++e) g[e] = value(LE::get(x[u], e));
            const int64_t rel = y - (head + (int64_t)i * N);
            if (rel >= 0 && rel < N) {
#pragma unroll
              for (int e = 0; e < N; ++e)
                if (e == rel) g[e] = __builtin_fmaf(it, a, g[e]);
            }
            put(i, LE::pack(g));
          }
        }
      }
      if (blockIdx.x == 0) {
        if ((int)threadIdx.x < head) one(threadIdx.x);
        else if (threadIdx.x >= 32 && tail + (int)threadIdx.x - 32 < V) one(tail + threadIdx.x - 32);
      }
    }
  }
}

struct LpCall {
  const void* logits;
  int64_t T;
  int V;
  int64_t ld;
  const int64_t* targets;
  const float* inv_t;
  int top_k, parts;
  float *logprobs, *entropy, *norm;
  int32_t* top_ids;
  float* top_lp;
  uint8_t* ws;
};

// Parts of a row.  One row keeps one CU busy for some 10 us per 131072 logits
// (the exponentials), so few long rows are split over more CUs and joined by a
// second launch.  Measured with 20 alternatives, bf16, in a graph: 16 x 131072
// 14.4 us split by four, 17.6 us whole; 1 x 65536 13.1 against 11.1 us; 128 x
// 131072 20.2 against 17.9 us.
inline int lp_parts(int64_t T, int64_t V) {
  if (T > 64 || V <= 98304) return 1;
  const int64_t n = (V + 32767) / 32768;
  return (int)(n < 64 ? n : 64);
}

template <typename E, int NT, bool TOP, bool STREAM = false>
void lp_launch_nt(const LpCall& a, hipStream_t s) {
  hipLaunchKernelGGL((k_logprob<E, NT, TOP, STREAM>), dim3((unsigned)(a.T * a.parts)), dim3(NT), 0, s,
                     (const E*)a.logits, a.V, a.ld, a.targets, a.inv_t, a.top_k, a.parts,
                     a.logprobs, a.entropy, a.norm, a.top_ids, a.top_lp, a.ws);
}

// Logits of which the caches could keep only a part, with alternatives (a
// rollout's record, which no gradient follows), are read past them: 2048 x
// 131072 bf16 91 against 102 us, 4096 x 131072 177-188 / 199-219; 512 x 131072 the
// same either way.  Where the backward pass follows it would miss the part
// that was kept: 8192 x 32768 265 / 255 for both passes, 4096 x 32000 137 / 121.
constexpr int64_t kLpPastCache = (int64_t)256 << 20;

template <typename E>
int lp_launch(const LpCall& a, hipStream_t s) {
  // One wave where the row is one chunk of it; sixteen where the rows do not
  // outnumber the CUs (1 x 32768 with 8 alternatives: 8.1 us against 9.6 us
  // with four); else four, so that several rows share a CU and one row's
  // loads run behind another's arithmetic.
  const bool small = a.V <= 64 * kLpU * Lanes<E>::N;
  const bool wide = !small && a.T * a.parts <= 256;
  if (a.top_k) {
    if (small) lp_launch_nt<E, 64, true>(a, s);
    else if (wide) lp_launch_nt<E, 1024, true>(a, s);
    else if (a.T * a.V * (int64_t)sizeof(E) >= kLpPastCache)
      lp_launch_nt<E, 256, true, true>(a, s);
    else lp_launch_nt<E, 256, true>(a, s);
  } else {
    if (small) lp_launch_nt<E, 64, false>(a, s);
    else if (wide) lp_launch_nt<E, 1024, false>(a, s);
    else lp_launch_nt<E, 256, false>(a, s);
  }
  if (a.parts > 1)
    hipLaunchKernelGGL(k_logprob_join<E>, dim3((unsigned)a.T), dim3(64), 0, s,
                       (const E*)a.logits, a.V, a.ld, a.targets, a.inv_t, a.top_k, a.parts,
                       a.logprobs, a.entropy, a.norm, a.top_ids, a.top_lp, a.ws);
  return nv_launch_status();
}

// Some array of 32-bit elements is not 4-byte aligned.
template <typename... P>
bool lp_misaligned(P... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ...) & 3) != 0;
}

struct LpGradCall {
  const void* logits;
  int64_t T;
  int V;
  int64_t ld;
  const int64_t* targets;
  const float *inv_t, *norm, *entropy, *g_lp, *g_ent;
  void* grad;
  int64_t ldg;
};

template <typename E, int NT, bool VEC, bool STREAM = false>
void lp_launch_bwd_nt(const LpGradCall& a, hipStream_t s) {
  const int64_t per = VEC ? (int64_t)NT * kLpBwdU * Lanes<E>::N : NT;
  const dim3 grid((unsigned)((a.V + per - 1) / per), (unsigned)(a.T < 65535 ? a.T : 65535));
  hipLaunchKernelGGL((k_logprob_bwd<E, NT, VEC, STREAM>), grid, dim3(NT), 0, s,
                     (const E*)a.logits, a.T, a.V, a.ld, a.targets, a.inv_t, a.norm, a.entropy, a.g_lp, a.g_ent,
                     (E*)a.grad, a.ldg);
}

// 16-byte pieces where every row of the gradient starts at the same place of
// a 16-byte block as its row of logits; single elements otherwise: 2048 x 50257
// bf16 in rows of 50304 with a gradient of the same row stride 65 us, with one
// in rows of 50257 339 us; 300 rows 17 / 51.  From 160 MB
// on logits and gradient are more than the last-level cache of 256 MB holds,
// and the gradient goes past it: forward and backward of 2048 x 131072 bf16 271
// against 292 us, 4096 x 32000 121 / 157, and with a kernel after them that reads
// the gradient 383 / 398 and 197 / 221; smaller ones lose with such a reader (512 x
// 131072 111 / 99).
constexpr int64_t kLpStreamBytes = (int64_t)160 << 20;
template <typename E>
int lp_launch_bwd(const LpGradCall& a, hipStream_t s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(a.logits) ^ reinterpret_cast<uintptr_t>(a.grad)) & 15) == 0 &&
                   (((a.ld - a.ldg) * (int64_t)sizeof(E)) & 15) == 0;
  if (!vec) lp_launch_bwd_nt<E, 256, false>(a, s);
  else if (a.V <= 64 * kLpBwdU * Lanes<E>::N) lp_launch_bwd_nt<E, 64, true>(a, s);
  else if (a.T * a.V * (int64_t)sizeof(E) >= kLpStreamBytes)
    lp_launch_bwd_nt<E, 256, true, true>(a, s);
  else lp_launch_bwd_nt<E, 256, true>(a, s);
  return nv_launch_status();
}

}  // namespace

extern "C" {

size_t token_logprobs_workspace_size(int64_t T, int64_t V, int64_t top_k) {
  if (T < 1 || T > kLpMaxT || V < 1 || V > kLpMaxV || top_k < 0 || top_k > kLpMaxTop) return 0;
  const int parts = lp_parts(T, V);
  return parts > 1 ? nv_round256((size_t)T * parts * lp_part_bytes((int)top_k)) : 0;
}

int token_logprobs(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                   const int64_t* targets, const float* inv_temperature, int64_t top_k,
                   float* logprobs, float* entropy, float* norm, int32_t* top_ids,
                   float* top_logprobs, void* ws, size_t ws_bytes, void* stream) {
  NV_RETURN_IF(dtype != NVFP4_IN_F32 && dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(T < 0 || T > kLpMaxT || V < 1 || V > kLpMaxV || ld < V || top_k < 0 ||
                   top_k > kLpMaxTop || top_k > V,
               NVFP4_ERR_SHAPE);
  if (T == 0) return NVFP4_OK;
  NV_RETURN_IF(!logits || (targets == nullptr) != (logprobs == nullptr) ||
                   (top_k > 0 && (!top_ids || !top_logprobs)),
               NVFP4_ERR_NULL);
  NV_RETURN_IF((reinterpret_cast<uintptr_t>(logits) & (dtype == NVFP4_IN_F32 ? 3 : 1)) ||
                   (reinterpret_cast<uintptr_t>(targets) & 7) ||
                   lp_misaligned(inv_temperature, logprobs, entropy, norm, top_ids, top_logprobs),
               NVFP4_ERR_ALIGN);
  const size_t need = token_logprobs_workspace_size(T, V, top_k);
  NV_RETURN_IF((need && !ws) || ws_bytes < need || (reinterpret_cast<uintptr_t>(ws) & 15),
               NVFP4_ERR_WORKSPACE);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const LpCall a{logits, T, (int)V, ld, targets, inv_temperature, (int)top_k, lp_parts(T, V),
                 logprobs, entropy, norm, top_ids, top_logprobs, reinterpret_cast<uint8_t*>(ws)};
  if (dtype == NVFP4_IN_F32) return lp_launch<float>(a, s);
  return lp_launch<uint16_t>(a, s);
}

int token_logprobs_backward(const void* logits, int dtype, int64_t T, int64_t V, int64_t ld,
                            const int64_t* targets, const float* inv_temperature,
                            const float* norm, const float* entropy, const float* grad_logprobs,
                            const float* grad_entropy, void* grad_logits, int64_t ldg,
                            void* stream) {
  NV_RETURN_IF(dtype != NVFP4_IN_F32 && dtype != NVFP4_IN_BF16, NVFP4_ERR_DTYPE);
  NV_RETURN_IF(T < 0 || T > kLpMaxT || V < 1 || V > kLpMaxV || ld < V || ldg < V ||
                   (logits == grad_logits && ld != ldg),
               NVFP4_ERR_SHAPE);
  if (T == 0) return NVFP4_OK;
  NV_RETURN_IF(!logits || !norm || !grad_logits || (grad_logprobs && !targets) ||
                   (grad_entropy && !entropy),
               NVFP4_ERR_NULL);
  const uintptr_t mask = dtype == NVFP4_IN_F32 ? 3 : 1;
  NV_RETURN_IF((reinterpret_cast<uintptr_t>(logits) & mask) ||
                   (reinterpret_cast<uintptr_t>(grad_logits) & mask) ||
                   (reinterpret_cast<uintptr_t>(targets) & 7) ||
                   lp_misaligned(inv_temperature, norm, entropy, grad_logprobs, grad_entropy),
               NVFP4_ERR_ALIGN);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const LpGradCall a{logits, T, (int)V, ld, targets, inv_temperature, norm, entropy,
                     grad_logprobs, grad_entropy, grad_logits, ldg};
  if (dtype == NVFP4_IN_F32) return lp_launch_bwd<float>(a, s);
  return lp_launch_bwd<uint16_t>(a, s);
}

}  // extern "C"
