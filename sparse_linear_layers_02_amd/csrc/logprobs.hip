// Log probabilities of given tokens, entropies and top alternatives, from what the
// head's product leaves of each group of logits while they are in registers.
//
//   with exponents z = l log2 e, a group's maximum m, s = sum 2^(z - m), q = sum 2^(z - m) (z - m):
//   lse = ln 2 m + ln s;  logp = l_y - lse;  entropy = lse - sum p l = ln s - ln 2 q / s
// Groups join as (m, s, q): relative to the larger maximum M, s 2^(m - M) and
// 2^(m - M) (q + (m - M) s).  Both terms of the entropy are of its own size, so a
// distribution that is nearly certain loses nothing to a difference.
//
// Alternatives: of every 4 mi logits that a lane held, the two largest are kept in
// float32.  The k-th largest of any partition's maxima is no larger than the k-th
// largest logit, so a row's candidates are the firsts above such a bound, and, where
// a second is above it as well, all of that lane's logits.  Candidates' sums are formed
// again, in 64 bits, and ordered by them.
#include "score_internal.h"

namespace sbn {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NONE = -1.0e38f * LOG2E;             // the maximum of no logits

__device__ inline int64_t token_at(const void* tokens, bool is64, int64_t t) {
  return is64 ? ((const int64_t*)tokens)[t] : (int64_t)((const int32_t*)tokens)[t];
}

struct Stat {
  float m, s, q;
};
__device__ inline Stat join(Stat a, Stat b) {
  const float top = fmaxf(a.m, b.m), da = a.m - top, db = b.m - top;
  const float ea = __builtin_amdgcn_exp2f(da), eb = __builtin_amdgcn_exp2f(db);
  return {top, a.s * ea + b.s * eb, ea * (a.q + da * a.s) + eb * (b.q + db * b.s)};
}

struct JoinArgs {
  const float2* stats;
  const float *mean, *target;
  const void* tokens;
  bool tokens64;
  int groups, first, T, V;             // first token of a launch
  float *logp, *entropy, *lse;
};

// 16 tokens a block, 64 threads a token take every 64th group each, then the 64
// triples are joined in a tree.
__global__ __launch_bounds__(1024) void logprob_join_kernel(JoinArgs P) {
  __shared__ float sm[3][64][17];
  const int tl = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int t = P.first + blockIdx.x * 16 + tl;
  Stat a{NONE, 0.0f, 0.0f};
  if (t < P.T) {
    constexpr int AHEAD = 4;
    for (int g = part; g < P.groups; g += 64 * AHEAD) {
      Stat x[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const bool in = g + 64 * k < P.groups;
        const int64_t at = (int64_t)(in ? g + 64 * k : g) * P.T + t;
        const float2 ms = P.stats[at];
        const float q = P.mean[at];
        x[k] = in ? Stat{ms.x, ms.y, q} : Stat{NONE, 0.0f, 0.0f};
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) a = join(a, x[k]);
    }
  }
  auto put = [&](Stat x) { sm[0][part][tl] = x.m, sm[1][part][tl] = x.s, sm[2][part][tl] = x.q; };
  put(a);
  __syncthreads();
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    if (part < d) put(a = join(a, Stat{sm[0][part + d][tl], sm[1][part + d][tl], sm[2][part + d][tl]}));
    __syncthreads();
  }
  if (part == 0 && t < P.T) {
    const float ln = logf(a.s), l = a.m * LN2 + ln;
    P.lse[t] = l;
    if (P.entropy) P.entropy[t] = ln - (a.q / a.s) * LN2;
    if (P.logp) {
      const int64_t y = token_at(P.tokens, P.tokens64, t);
      P.logp[t] = y >= 0 && y < P.V ? P.target[t] - l : 0.0f;
    }
  }
}

// ---------------------------------------------------------------- top alternatives
struct TopArgs {
  const uint16_t *X, *W;
  int64_t ldx, ldw, groups;
  int K, V, mi, T, top;
  const float2* tops;
  const float* lse;
  float scale;
  int64_t* ids;
  float* logp;
};

// sum_k x w in 64 bits and sum_k |x w|, of a wave
__device__ inline double exact_sum(const uint16_t* x, const uint16_t* w, int K, float& size) {
  const int lane = threadIdx.x & 63;
  double s = 0.0;
  float a = 0.0f;
#pragma unroll 2
  for (int c = lane; c < K / 8; c += 64) {
    const uint4 xv = ((const uint4*)x)[c], wv = ((const uint4*)w)[c];
    const uint32_t xs[4] = {xv.x, xv.y, xv.z, xv.w}, ws[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {                    // products of bf16 are exact in float32
      const float lo = __uint_as_float(xs[j] << 16) * __uint_as_float(ws[j] << 16);
      const float hi = __uint_as_float(xs[j] & 0xFFFF0000u) * __uint_as_float(ws[j] & 0xFFFF0000u);
      s += (double)lo;
      s += (double)hi;
      a += fabsf(lo) + fabsf(hi);
    }
  }
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) s += __shfl_xor(s, d);
  size = wave_all(a, Add{});
  return s;
}

// NT threads take a token.  LDS atomics deal out places in a queue, whose order does
// not matter: candidates are ordered by (sum, index) in the end.
template <int NT>
__global__ __launch_bounds__(NT) void logprob_top_kernel(TopArgs P) {
  constexpr int WAVES = NT / 64, SLOTS = 256, QUEUE = 1024, BATCH = 256, MOST = SBN_LOGPROBS_MAX_TOP;
  static_assert(NT % SLOTS == 0 && NT <= QUEUE, "threads");
  __shared__ float slot[NT];
  __shared__ float lower;
  __shared__ uint32_t singles, wholes, largest;      // queued entries, queued groups, bits of the largest sum |x w|
  __shared__ int single[QUEUE], whole[QUEUE];
  __shared__ double value[MOST + BATCH];             // the best so far in order, then a batch
  __shared__ int index[MOST + BATCH];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int per = 4 * P.mi, top = P.top;

  for (int64_t t = blockIdx.x; t < P.T; t += gridDim.x) {
    const float2* row = P.tops + t * P.groups;
    const uint16_t* x = P.X + t * P.ldx;
    // a bound that at least top + 2 firsts reach, if there are as many: the places past
    // the top itself leave room for the margin below, which then rarely asks for more
    float m = -INFINITY;
    for (int64_t g = tid; g < P.groups; g += NT) m = fmaxf(m, row[g].x);
    bool any = false;                                // a row of zeros (padding) makes all logits equal: the first ones win
    for (int c = tid; c < P.K / 8; c += NT) {
      const uint4 v = ((const uint4*)x)[c];
      any |= ((v.x | v.y | v.z | v.w) & 0x7FFF7FFFu) != 0;
    }
    if (!__syncthreads_or(any)) {
      for (int i = tid; i < top; i += NT) P.ids[t * top + i] = i, P.logp[t * top + i] = -P.lse[t];
      continue;
    }
    slot[tid] = m;
    if (tid == 0) lower = -INFINITY;
    __syncthreads();
    if (NT > SLOTS) {
      if (tid < SLOTS)
        for (int i = 1; i < NT / SLOTS; ++i) m = fmaxf(m, slot[tid + i * SLOTS]);
      __syncthreads();
      if (tid < SLOTS) slot[tid] = m;
      __syncthreads();
    }
    if (tid < SLOTS) {
      int better = 0;
#pragma unroll 4
      for (int i = 0; i < SLOTS; i += 4) {
        const v4f o = *(const v4f*)(slot + i);
#pragma unroll
        for (int e = 0; e < 4; ++e) better += o[e] > m || (o[e] == m && i + e < tid);
      }
      if (better == top + 1) lower = m;
    }
    __syncthreads();
    float bound = lower;

    auto entry = [&](int64_t g, int p) { return (int)((g >> 2) * (16 * P.mi) + 16 * (p >> 2) + 4 * (g & 3) + (p & 3)); };
    auto put = [&](int64_t g, int limit) {           // a group's candidates into the queues
      const float2 f = row[g];
      if (f.y >= bound) {
        const uint32_t at = atomicAdd(&wholes, 1u);
        if (at < (uint32_t)limit) whole[at] = (int)g;
      } else if (f.x >= bound) {
        const uint32_t at = atomicAdd(&singles, 1u);
        if (at < (uint32_t)limit) single[at] = entry(g, (int)(__float_as_uint(f.x) & (uint32_t)(per - 1)));
      }
    };
    int have = 0;
    // n entries, the i-th by `name` (or none: < 0), into the best
    auto take = [&](int n, auto name) {
      for (int i = wave; i < n; i += WAVES) {
        const int v = __builtin_amdgcn_readfirstlane(name(i));
        float size = 0.0f;
        double s = -INFINITY;
        if (v >= 0) s = exact_sum(x, P.W + (int64_t)v * P.ldw, P.K, size);
        if (lane == 0) {
          value[have + i] = s, index[have + i] = v >= 0 ? v : 0x7FFFFFFF;
          atomicMax(&largest, __float_as_uint(size));
        }
      }
      __syncthreads();
      constexpr int EACH = (MOST + BATCH + NT - 1) / NT;
      double s[EACH];
      int v[EACH], rank[EACH];
#pragma unroll
      for (int k = 0; k < EACH; ++k) {
        const int i = tid + k * NT;
        rank[k] = MOST;
        if (i < have + n) {
          s[k] = value[i], v[k] = index[i];
          rank[k] = 0;
          for (int j = 0; j < have + n; ++j) rank[k] += value[j] > s[k] || (value[j] == s[k] && index[j] < v[k]);
        }
      }
      __syncthreads();
      have = have + n < top ? have + n : top;
#pragma unroll
      for (int k = 0; k < EACH; ++k)
        if (rank[k] < top) value[rank[k]] = s[k], index[rank[k]] = v[k];
      __syncthreads();
    };
    auto empty_queues = [&](int ns, int nw) {
      for (int b = 0; b < ns; b += BATCH) take(ns - b < BATCH ? ns - b : BATCH, [&](int i) { return single[b + i] < P.V ? single[b + i] : -1; });
      const int groups = BATCH / per;                // of a batch
      for (int b = 0; b < nw; b += groups)
        take((nw - b < groups ? nw - b : groups) * per, [&](int i) {
          const int v = entry(whole[b + i / per], i % per);
          return v < P.V ? v : -1;
        });
    };
    for (int round = 0; round < 4; ++round) {
      have = 0;
      if (tid == 0) singles = wholes = 0, largest = 0;
      __syncthreads();
      for (int64_t g = tid; g < P.groups; g += NT) put(g, QUEUE);
      __syncthreads();
      const uint32_t ns = singles, nw = wholes;
      __syncthreads();
      if (ns <= QUEUE && nw <= QUEUE) {
        empty_queues((int)ns, (int)nw);
      } else {                                       // as many equal logits: by pieces that fit
        for (int64_t b = 0; b < P.groups; b += NT) {
          if (tid == 0) singles = wholes = 0;
          __syncthreads();
          if (b + tid < P.groups) put(b + tid, QUEUE);
          __syncthreads();
          const int n1 = (int)singles, n2 = (int)wholes;
          __syncthreads();
          empty_queues(n1, n2);
        }
      }
      // A logit that was left out is below `bound` in float32, so in 64 bits below it and a margin of
      // both sums' errors and of the last bits that hold its place.
      const double least = value[top - 1];
      const double margin = 2.0 * ((double)(P.K + 64) * 0x1p-24 * (double)__uint_as_float(largest) + 0x1p-17 * fabs(least));
      if (bound == -INFINITY || (double)bound + margin <= least) break;
      bound = __double2float_rd(least - 2.0 * margin);
      __syncthreads();                               // value and largest are read by all
    }
    for (int i = tid; i < top; i += NT) {
      P.ids[t * top + i] = index[i];
      P.logp[t * top + i] = (float)((double)P.scale * value[i] - (double)P.lse[t]);
    }
    __syncthreads();
  }
}

struct Plan {
  size_t target, stats, mean, tops, total;
};
Plan plan(int64_t T, int64_t V, int64_t K, int top) {
  const size_t n = (size_t)logit_groups(T, V, K) * T;
  Plan L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.target = take((size_t)T * sizeof(float));
  L.stats = take(n * sizeof(float2));
  L.mean = take(n * sizeof(float));
  L.tops = take(top ? (size_t)logit_tops(T, V, K).groups * T * sizeof(float2) : 0);
  L.total = o;
  return L;
}

}  // namespace

size_t logprobs_ws_bytes(int64_t T, int64_t V, int64_t K, int top) { return plan(T, V, K, top).total; }

hipError_t launch_logprobs(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens,
                           bool tokens64, int64_t T, int64_t V, int64_t K, float scale, float* logp, float* entropy,
                           float* lse, int top, int64_t* top_ids, float* top_logp, void* ws, hipStream_t st) {
  const Plan L = plan(T, V, K, top);
  uint8_t* w = (uint8_t*)ws;
  float *target = (float*)(w + L.target), *mean = (float*)(w + L.mean);
  float2 *stats = (float2*)(w + L.stats), *tops = top ? (float2*)(w + L.tops) : nullptr;
  hipError_t e = launch_logits(X, ldx, W, ldw, tokens, tokens64, T, V, K, scale, target, stats, mean, tops, st);
  if (e != hipSuccess) return e;
  constexpr int64_t JOIN_TOKENS = 1 << 24;           // of a launch: fewer than 2^32 threads
  for (int64_t t = 0; t < T; t += JOIN_TOKENS) {
    const JoinArgs J{stats, mean, target, tokens, tokens64, (int)logit_groups(T, V, K), (int)t, (int)T, (int)V, logp, entropy,
                     lse};
    SBN_LAUNCH("logprob_join", logprob_join_kernel, dim3((unsigned)cdiv(T - t < JOIN_TOKENS ? T - t : JOIN_TOKENS, 16)),
               dim3(1024), 0, st, J);
  }
  if ((e = hipGetLastError()) != hipSuccess || !top) return e;
  const LogitTops G = logit_tops(T, V, K);
  const TopArgs A{X, W, ldx, ldw, G.groups, (int)K, (int)V, G.mi, (int)T, top, tops, lse, scale, top_ids, top_logp};
  const unsigned blocks = (unsigned)(T < (1 << 20) ? T : (1 << 20));
  if (T <= 256) SBN_LAUNCH("logprob_top", logprob_top_kernel<1024>, dim3(blocks), dim3(1024), 0, st, A);
  else SBN_LAUNCH("logprob_top", logprob_top_kernel<256>, dim3(blocks), dim3(256), 0, st, A);
  return hipGetLastError();
}

}  // namespace sbn
