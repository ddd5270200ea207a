// Log probabilities of given tokens, entropies and top alternatives, from what the
// head's product leaves of each group of logits while they are in registers.
//
//   with a group's largest logit m, exponents z = (l - m) log2 e, r = sum 2^z without that of m
//   itself, q = sum 2^z z:
//   lse = m + ln(1 + r);  logp = l_y - m - ln(1 + r);  entropy = lse - sum p l = ln(1 + r) - ln 2 q / (1 + r)
// Groups join as (m, r, q): to those of the larger m come 2^d (1 + r) and 2^d (q + d (1 + r)), d the
// other's m less the larger one, times log2 e.  No term is larger than what it goes into, so
// distributions that are nearly certain lose nothing to a difference: log probabilities and entropies
// near 0 keep their relative precision, and none is on its wrong side.
// The alternatives' sums are in 64 bits, m in 32: theirs are taken from the 64-bit sum of
// the entry that m is of.
//
// Alternatives: of every 32, 16 or 8 logits, the two largest are kept in float32.  The
// k-th largest of any partition's maxima is no larger than the k-th largest logit, so a
// row's candidates are the firsts above such a bound, and, where a second is above it as
// well, all of its set.  Candidates' sums are formed again, in 64 bits, and ordered by them.
// A sum of K products in float32, in any order, is off by at most K 2^-24 sum |x w| <= K 2^-24
// |x| |w| (twice that if the hardware cuts off instead of rounding), and the product leaves the largest |w|
// of each of its groups of rows.  Sets that hold an entry which with that margin reaches the
// last alternative, and which no one has summed, are candidates of a second round, and then
// none is left.
//
// Bound by dependent reads: of one token (50001 entries, K = 2560, 8 alternatives) 15 to 16 us,
// 2.5 of them the join, 2 the bound, 2 the scan, 4 the sums of K, 1 their order; of 37
// tokens (32001, 4096, 20 alternatives) 25 to 27.  Of 4096 tokens (65536, 2560, 8) 90 to 100 us
// for 67 MB of sets and 300 MB of rows of W, and 9 the join.  Second rounds, which margins by
// norms ask for more often than one from the candidates' sums |x w| would: 20 alternatives of 1024
// tokens (32001, 4096) 59 -> 68 us, of 2051 (26574, 3776) 88 -> 101; 64 of 2000 (8000, 512) 77 -> 70,
// without those sums.  One row of W 50 times as large as the others, 4096 tokens as above: 117 us, with a
// margin for all rows alike 199; 1000 times: 350, 113000.
#include "score_internal.h"

namespace sbn {
namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

__device__ inline int64_t token_at(const void* tokens, bool is64, int64_t t) {
  return is64 ? ((const int64_t*)tokens)[t] : (int64_t)((const int32_t*)tokens)[t];
}

struct Stat {
  float m, r, q;                       // m before the logits' scale
};
__device__ inline Stat join(Stat a, Stat b, float factor) {
  const Stat hi = a.m >= b.m ? a : b, lo = a.m >= b.m ? b : a;
  const float d = (lo.m - hi.m) * factor, e = __builtin_amdgcn_exp2f(d), s = 1.0f + lo.r;
  return {hi.m, hi.r + e * s, hi.q + e * (lo.q + d * s)};
}

struct RowArgs {
  const float2* stats;
  const float *mean, *target;
  const void* tokens;
  bool tokens64;
  int groups, T, V;
  float factor, none;                  // scale log2 e; the maximum of no logits
  float2* rows;                        // [T] m and ln(1 + r), for the alternatives
  float *logp, *entropy, *lse;
  // alternatives
  const uint16_t *X, *W;
  int64_t ldx, ldw;
  int K, top;
  LogitTops sets;
  const float2* tops;
  const float* norms;                  // `each` of a group
  int each;
  float* most;                         // the largest of norms; unused where a block joins its own token's statistics
  float scale;
  int64_t* ids;
  float* top_logp;
};

// a token's outputs from all its logits' statistics; returns m and ln(1 + r)
__device__ inline float2 finish(const RowArgs& P, int64_t t, Stat a) {
  const float ln = log1pf(a.r);
  P.lse[t] = a.m * P.scale + ln;
  if (P.entropy) P.entropy[t] = ln - (a.q / (1.0f + a.r)) * LN2;
  if (P.logp) {
    const int64_t y = token_at(P.tokens, P.tokens64, t);
    P.logp[t] = y >= 0 && y < P.V ? (P.target[t] - a.m) * P.scale - ln : 0.0f;
  }
  return make_float2(a.m, ln);
}
// every `step`-th group from `first` on, AHEAD loads in flight
template <int AHEAD>
__device__ inline Stat join_groups(const RowArgs& P, int64_t t, int first, int step) {
  const Stat none{P.none, -1.0f, 0.0f};
  Stat a = none;
  for (int g = first; g < P.groups; g += step * AHEAD) {
    Stat x[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const bool in = g + step * k < P.groups;
      const int64_t at = (int64_t)(in ? g + step * k : g) * P.T + t;
      const float2 ms = P.stats[at];
      const float q = P.mean[at];
      x[k] = in ? Stat{ms.x, ms.y, q} : none;
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) a = join(a, x[k], P.factor);
  }
  return a;
}

// 16 tokens a block, 64 threads a token take every 64th group each, then the 64
// triples are joined in a tree.
__global__ __launch_bounds__(1024) void logprob_join_kernel(RowArgs P, int first) {
  __shared__ float sm[3][64][17];
  if (P.top && first + blockIdx.x * 16 >= P.T) {     // one block past the tokens, beside the others
    float m = 0.0f;
#pragma unroll 4
    for (int g = threadIdx.x; g < P.groups * P.each; g += 1024) m = fmaxf(m, P.norms[g]);
    m = wave_all(m, Max{});
    if ((threadIdx.x & 63) == 0) sm[0][0][threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x < 16) {
      m = row16_all(sm[0][0][threadIdx.x], Max{});
      if (threadIdx.x == 0) *P.most = m;
    }
    return;
  }
  const int tl = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int t = first + blockIdx.x * 16 + tl;
  Stat a{P.none, -1.0f, 0.0f};
  if (t < P.T) a = join_groups<4>(P, t, part, 64);
  auto put = [&](Stat x) { sm[0][part][tl] = x.m, sm[1][part][tl] = x.r, sm[2][part][tl] = x.q; };
  put(a);
  __syncthreads();
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    if (part < d) put(a = join(a, Stat{sm[0][part + d][tl], sm[1][part + d][tl], sm[2][part + d][tl]}, P.factor));
    __syncthreads();
  }
  if (part == 0 && t < P.T) {
    const float2 row = finish(P, t, a);
    if (P.top) P.rows[t] = row;
  }
}

// ---------------------------------------------------------------- top alternatives
template <int N>
struct Int {
  static constexpr int value = N;
};
template <int CTRL>
__device__ inline double row_moved(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_mov_dpp((int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// the sum of a wave's, as wave_all
__device__ inline double wave_sum(double x) {
  x += row_moved<0xB1>(x);
  x += row_moved<0x4E>(x);
  x += row_moved<0x141>(x);
  x += row_moved<0x140>(x);
  auto halves = [](auto lo, auto hi) {
    return __builtin_bit_cast(double, (uint64_t)hi[0] << 32 | lo[0]) + __builtin_bit_cast(double, (uint64_t)hi[1] << 32 | lo[1]);
  };
  uint64_t b = __builtin_bit_cast(uint64_t, x);
  x = halves(__builtin_amdgcn_permlane16_swap((uint32_t)b, (uint32_t)b, false, false),
             __builtin_amdgcn_permlane16_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false));
  b = __builtin_bit_cast(uint64_t, x);
  return halves(__builtin_amdgcn_permlane32_swap((uint32_t)b, (uint32_t)b, false, false),
                __builtin_amdgcn_permlane32_swap((uint32_t)(b >> 32), (uint32_t)(b >> 32), false, false));
}

// sum_k x w in 64 bits of ROWS rows w, of a wave; loads of 512 AHEAD entries of each at once
template <int AHEAD, int ROWS>
__device__ inline void exact_sums(const uint16_t* x, const uint16_t* const (&w)[ROWS], int K, double (&sum)[ROWS]) {
  const int lane = threadIdx.x & 63, n = K / 8;
  double s0[ROWS], s1[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) s0[r] = s1[r] = 0.0;
#pragma unroll 1
  for (int c0 = lane; c0 < n; c0 += 64 * AHEAD) {
    v4i wv[ROWS][AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int r = 0; r < ROWS; ++r) {
        wv[r][k] = (v4i){0, 0, 0, 0};
        if (c0 + 64 * k < n) wv[r][k] = ((const v4i*)w[r])[c0 + 64 * k];
      }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const v4i xv = ((const v4i*)x)[c0 + 64 * k < n ? c0 + 64 * k : c0];
#pragma unroll
      for (int r = 0; r < ROWS; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {                // products of bf16 are exact in float32 (from 2^-134 up; in 64 bits 3% slower)
          const float lo = __uint_as_float((uint32_t)xv[j] << 16) * __uint_as_float((uint32_t)wv[r][k][j] << 16);
          const float hi = __uint_as_float(xv[j] & 0xFFFF0000u) * __uint_as_float(wv[r][k][j] & 0xFFFF0000u);
          s0[r] += (double)lo;
          s1[r] += (double)hi;
        }
    }
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) sum[r] = wave_sum(s0[r] + s1[r]);
}

// A float that at least k of 256 reach (-Inf if fewer than k are above it), within 2^-11 of
// the k-th largest: the leading bits of the order-preserving integers, one at a time,
// as long as k are no smaller; and the largest.  Each wave for itself.  (Counting for each of the 256
// how many are larger took 12.5 us of one token's 23.)
__device__ inline float reached_by(const float* slot, int k, float& most) {
  constexpr uint32_t LEAST = 0x00800000u;            // the integers of -Inf and below
  const v4f o = *(const v4f*)(slot + 4 * (threadIdx.x & 63));
  uint32_t key[4], found = 0;
  most = wave_all(fmaxf(fmaxf(o[0], o[1]), fmaxf(o[2], o[3])), Max{});
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const uint32_t u = __float_as_uint(o[e]);
    key[e] = u & 0x80000000u ? ~u : u | 0x80000000u;
  }
#pragma unroll 1
  for (uint32_t bit = 0x80000000u; bit >= 1u << 12; bit >>= 1) {
    int n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) n += (int)__popcll(__ballot(key[e] >= (found | bit)));
    if (n >= k) found |= bit;
  }
  return found < LEAST ? -INFINITY : __uint_as_float(found & 0x80000000u ? found ^ 0x80000000u : ~found);
}

// NT threads take a token.  JOIN: they join its statistics as well (few tokens: a
// launch less, and all of a block's threads on one token).  LDS atomics deal out
// places in a queue, whose order does not matter: candidates are ordered by (sum,
// index) in the end.  The code is kept short, without unrolling: one token's block
// fetches each line of it for the first time.
// Many tokens: a wave sums three rows at once, 2 loads of each ahead, 5 blocks a unit:
// 4096 tokens of 65536 entries, K = 2560, 8 alternatives 90 us; 600 of 50000, 4096, 8 40;
// 2051 of 26574, 3776, 20 101; 2641 of 1158, 1024, 5 27 (without second rounds 91, 41, 88, 27,
// and so measured two rows 99, 44, 89, 24; four 104, 41, 100, 30; two with 3 ahead 99, 46, 92, 26;
// one row, 5 ahead, 6 blocks 101, 57, 110, 31; two rows, 7 blocks 111, 48, 106, 27).  Few: one row, 8
// ahead, or, where waves have more than one and 4 ahead are a whole row, two (10 tokens of 2062
// entries, K = 256, 32 alternatives 27 -> 21 us; with two for K = 4096, 20 of 32001, 37 tokens 25 -> 27).
template <int NT, bool JOIN>
__global__ __launch_bounds__(NT, NT == 256 ? 5 : 4) void logprob_top_kernel(RowArgs P) {
  constexpr int WAVES = NT / 64, SLOTS = 256, QUEUE = 1024, BATCH = 256, MOST = SBN_LOGPROBS_MAX_TOP;
  constexpr int HELD = 4;
  static_assert(NT % SLOTS == 0 && NT <= QUEUE, "threads");
  __shared__ __attribute__((aligned(16))) float slot[NT];
  __shared__ float2 largest;                         // m and ln(1 + r)
  __shared__ int leader;                             // the entry that m is of
  __shared__ Stat stat[WAVES];
  __shared__ uint32_t singles, wholes;               // queued entries, queued sets
  __shared__ float x_squares[WAVES], w_norm[WAVES];
  __shared__ int single[QUEUE], whole[QUEUE];
  __shared__ double value[MOST + BATCH];             // the best so far in order, then a batch
  __shared__ int index[MOST + BATCH];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int top = P.top, n = P.sets.groups;
  const LogitTops sets = P.sets;

  for (int t = blockIdx.x; t < P.T; t += gridDim.x) {
    const float2* row = P.tops + (int64_t)t * n;
    const uint16_t* x = P.X + t * P.ldx;
    float firsts[HELD];                              // loaded before the statistics are waited for
#pragma unroll
    for (int k = 0; k < HELD; ++k) firsts[k] = top && tid + k * NT < n ? row[tid + k * NT].x : -INFINITY;
    const int norms = top && JOIN ? P.groups * P.each : 0;
    float w_norms[2];                                // as firsts
#pragma unroll
    for (int k = 0; k < 2; ++k) w_norms[k] = tid + k * NT < norms ? P.norms[tid + k * NT] : 0.0f;
    if (JOIN) {
      Stat a = join_groups<2>(P, t, tid, NT);
      auto over_lanes = [&](int d) {
#pragma unroll 1
        for (; d >= 1; d >>= 1) a = join(a, Stat{__shfl_xor(a.m, d), __shfl_xor(a.r, d), __shfl_xor(a.q, d)}, P.factor);
      };
      over_lanes(32);
      if (lane == 0) stat[wave] = a;
      __syncthreads();
      if (wave == 0) {
        a = stat[lane & (WAVES - 1)];
        over_lanes(WAVES / 2);
        if (tid == 0) largest = finish(P, t, a);
      }
      if (!top) {
        __syncthreads();
        continue;
      }
    } else if (tid == 0) {
      largest = P.rows[t];
    }
    // a bound that at least top + 2 firsts reach, if there are as many: the places past
    // the top itself leave room for the margin below, which then asks for a second round less
    // often (more than two: at best 1 us of 25 less, at worst 30 of 90 more)
    float m = firsts[0];
#pragma unroll
    for (int k = 1; k < HELD; ++k) m = fmaxf(m, firsts[k]);
#pragma unroll 4
    for (int g = tid + HELD * NT; g < n; g += NT) m = fmaxf(m, row[g].x);
    bool any = false;
    float xx = 0.0f;
#pragma unroll 1
    for (int c = tid; c < P.K / 8; c += NT) {
      const v4i v = ((const v4i*)x)[c];
      any |= ((v[0] | v[1] | v[2] | v[3]) & 0x7FFF7FFF) != 0;
      xx = add_squares(__builtin_bit_cast(v8bf, v), xx);
    }
    float w_most = fmaxf(w_norms[0], w_norms[1]);
    for (int g = tid + 2 * NT; g < norms; g += NT) w_most = fmaxf(w_most, P.norms[g]);
    xx = wave_all(xx, Add{});
    if (JOIN) w_most = wave_all(w_most, Max{});
    else w_most = *P.most;
    if (lane == 0) x_squares[wave] = xx, w_norm[wave] = w_most;
    slot[tid] = m;
    if (!__syncthreads_or(any)) {                    // a row of zeros (padding): all logits are equal, the first ones win
      for (int i = tid; i < top; i += NT) P.ids[(int64_t)t * top + i] = i, P.top_logp[(int64_t)t * top + i] = -largest.y;
      __syncthreads();
      continue;
    }
    if (NT > SLOTS) {
      if (tid < SLOTS)
#pragma unroll
        for (int i = 1; i < NT / SLOTS; ++i) m = fmaxf(m, slot[tid + i * SLOTS]);
      __syncthreads();
      if (tid < SLOTS) slot[tid] = m;
      __syncthreads();
    }
    float most_likely;
    const float bound = reached_by(slot, top + 2, most_likely);
    if (tid == 0) leader = 0x7FFFFFFF;
    float reach = 0.0f, least = 0.0f;                // second round: a margin's share of x, and the last alternative
    const float tiny = (float)P.K * 0x1p-124f;       // what products and sums below float32's full precision lose
    int have = 0;
#pragma unroll 1
    for (int round = 0; round < 2; ++round) {
      const float over = round ? bound : INFINITY;   // from here on entries alone, or with their sets, were summed
      bool pieces = false;                           // as many equal logits that the queues do not hold all sets'
      for (int b = 0; b < n;) {
        if (tid == 0) singles = wholes = 0;
        __syncthreads();
        const int stop = pieces ? (n - b < NT ? n : b + NT) : n;
#pragma unroll 1
        for (int g0 = b + tid; g0 < stop; g0 += 4 * NT) {   // a set's candidates into the queues
          float2 fs[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            fs[k] = make_float2(-INFINITY, -INFINITY);
            if (g0 + k * NT < stop) fs[k] = row[g0 + k * NT];
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = fs[k];
            const int g = g0 + k * NT;
            if (g >= stop) continue;
            bool all = f.y >= bound, one = f.x >= bound;
            if (!round && f.x == most_likely) atomicMin(&leader, sets.entry(g, (int)(__float_as_uint(f.x) & (TOPS_MOST - 1))));
            if (round) {                             // 2^-16: the last bits, which hold the place, and roundings here
              const float* norms = P.norms + sets.group(g) * P.each;
              float norm = norms[0];
              for (int k = 1; k < P.each; ++k) norm = fmaxf(norm, norms[k]);
              const float margin = reach * norm + tiny;
              auto may = [&](float key) { return !(key >= over) && !(key + fabsf(key) * 0x1p-16f + margin < least); };
              all = may(f.y), one = may(f.x);
            }
            if (all) {
              const uint32_t at = atomicAdd(&wholes, 1u);
              if (at < QUEUE) whole[at] = g;
            } else if (one) {
              const uint32_t at = atomicAdd(&singles, 1u);
              if (at < QUEUE) single[at] = sets.entry(g, (int)(__float_as_uint(f.x) & (TOPS_MOST - 1)));
            }
          }
        }
        __syncthreads();
        const uint32_t ns = singles, nw = wholes;
        __syncthreads();
        if (!pieces && (ns > QUEUE || nw > QUEUE)) {
          pieces = true;
          continue;
        }
        b = stop;
        const int entries = (int)(ns + (nw << sets.of_log2));
#pragma unroll 1
        for (int e = 0; e < entries; e += BATCH) {   // a batch of entries into the best so far
          const int count = entries - e < BATCH ? entries - e : BATCH;
          // the sums of rows `i0` on, every WAVES-th, of ROWS of them at a time
          auto sums = [&](auto rows, auto ahead) {
            constexpr int ROWS = decltype(rows)::value, AHEAD = decltype(ahead)::value;
#pragma unroll 1
            for (int i0 = wave; i0 < count; i0 += WAVES * ROWS) {
              const uint16_t* w[ROWS];
              int v[ROWS], place[ROWS];
#pragma unroll
              for (int r = 0; r < ROWS; ++r) {
                const int i = i0 + r * WAVES, at = e + i - (int)ns;
                int entry = 0;
                bool none = i >= count;
                if (i < count && at < 0) {
                  entry = single[e + i];
                } else if (i < count) {              // of a set whose first alone came before, without it
                  const int g = whole[at >> sets.of_log2], p = sets.place(g, at & ((1 << sets.of_log2) - 1));
                  const float f = row[g].x;
                  none = f >= over && p == (int)(__float_as_uint(f) & (TOPS_MOST - 1));
                  entry = sets.entry(g, p);
                }
                place[r] = __builtin_amdgcn_readfirstlane(entry);
                none |= (uint32_t)entry >= (uint32_t)P.V;   // past the vocabulary
                v[r] = __builtin_amdgcn_readfirstlane(none ? -1 : entry);
                w[r] = P.W + (int64_t)(v[r] >= 0 ? v[r] : 0) * P.ldw;
              }
              double sum[ROWS];
              exact_sums<AHEAD, ROWS>(x, w, P.K, sum);
#pragma unroll
              for (int r = 0; r < ROWS; ++r) {
                const int i = have + i0 + r * WAVES;
                if (lane == 0 && i < have + count) {
                  value[i] = v[r] >= 0 && sum[r] == sum[r] ? sum[r] : -INFINITY;   // NaN (outside the contract): an order all the same
                  index[i] = place[r];               // of none too: equal ones would leave places of the order empty
                }
              }
            }
          };
          if (!JOIN) sums(Int<3>{}, Int<2>{});
          else if (count > WAVES && P.K <= 4 * 512) sums(Int<2>{}, Int<4>{});
          else sums(Int<1>{}, Int<8>{});
          __syncthreads();
          constexpr int EACH = (MOST + BATCH + NT - 1) / NT;
          double sum[EACH];
          int v[EACH], rank[EACH];
#pragma unroll
          for (int k = 0; k < EACH; ++k) {
            const int i = tid + k * NT;
            rank[k] = MOST, sum[k] = 0.0, v[k] = 0;
            if (i < have + count) {
              sum[k] = value[i], v[k] = index[i];
              rank[k] = 0;
#pragma unroll 4
              for (int j = 0; j < have + count; ++j)
                rank[k] += (int)(value[j] > sum[k]) | ((int)(value[j] == sum[k]) & (int)(index[j] < v[k]));
            }
          }
          __syncthreads();
          have = have + count < top ? have + count : top;
#pragma unroll
          for (int k = 0; k < EACH; ++k)
            if (rank[k] < top) value[rank[k]] = sum[k], index[rank[k]] = v[k];
          __syncthreads();
        }
      }
      if (round || have < top || bound == -INFINITY) break;   // fewer than top: NaN again
      // A logit that was left out is below bound in float32, so in 64 bits below it and its margin
      float squares = 0.0f, most = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) squares += x_squares[w], most = fmaxf(most, w_norm[w]);
      // x squared as the rows of W; 2^-23 and K + 64 leave room for the roundings here
      reach = (float)(P.K + 64) * 0x1p-23f * (1.0f + 0x1p-6f) * sqrtf(squares * (1.0f + 0x1p-6f) + (float)P.K * 0x1p-124f);
      least = __double2float_rd(value[top - 1]);
      if (bound + fabsf(bound) * 0x1p-16f + (reach * most + tiny) < least) break;
      __syncthreads();                               // value is read by all
    }
    static_assert(MOST <= 64, "a wave");
    if (wave == 0) {
      const double sum = lane < have ? value[lane] : 0.0;
      const int id = lane < have ? index[lane] : -1;
      // m's 64-bit sum, if it is an alternative; if not (its 32 bits are as far off), m itself
      const uint64_t its = __ballot(id == leader);
      const double from = its ? __shfl(sum, __builtin_ctzll(its)) : (double)largest.x;
      const bool found = (uint32_t)id < (uint32_t)P.V;   // always, of finite logits
      const float logp = (float)((double)P.scale * (sum - from) - (double)largest.y);
      if (lane < top) {
        P.ids[(int64_t)t * top + lane] = found ? id : 0;
        P.top_logp[(int64_t)t * top + lane] = found ? logp > 0.0f ? 0.0f : logp : NAN;
      }
    }
    __syncthreads();
  }
}

// Tokens are taken in parts whose statistics and sets' pairs stay below so many bytes, of
// 64 tokens at least; pairs of sets of 8, V bytes a token, in parts as were measured.  (What it
// takes: W is read once more for each part, of thousands of tokens.)
constexpr int64_t PART_BYTES = int64_t(1) << 32, PAIRS8_BYTES = int64_t(1) << 29;

struct Plan {
  int64_t part;                                      // tokens of all parts but the last
  size_t target, stats, mean, tops, norms, rows, total;
};
Plan plan(int64_t T, int64_t V, int64_t K, int top) {
  const size_t groups = (size_t)logit_groups(T, V, K);
  const LogitTops sets = logit_tops(T, V, K, top);
  const int64_t pairs = top ? (int64_t)sets.groups * (int64_t)sizeof(float2) : 0;
  int64_t most = PART_BYTES / ((int64_t)groups * 12 + pairs);
  if (top && sets.of_log2 == 3 && most > PAIRS8_BYTES / pairs) most = PAIRS8_BYTES / pairs;
  const int64_t unit = most >= 256 ? 256 : 64;       // tiles' tokens
  most = most < unit ? unit : most / unit * unit;
  Plan L;
  L.part = T <= most ? T : round_up(cdiv(T, cdiv(T, most)), unit);
  const size_t n = groups * L.part;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.target = take((size_t)L.part * sizeof(float));
  L.stats = take(n * sizeof(float2));
  L.mean = take(n * sizeof(float));
  L.tops = take((size_t)L.part * pairs);
  L.norms = take(top ? (groups * logit_norms(T, V, K) + 1) * sizeof(float) : 0);
  L.rows = take(top ? (size_t)L.part * sizeof(float2) : 0);
  L.total = o;
  return L;
}

// Tokens to whose statistics a block each is given: a round of blocks of 1024 threads.
constexpr int64_t FEW_TOKENS = 256;

}  // namespace

size_t logprobs_ws_bytes(int64_t T, int64_t V, int64_t K, int top) { return plan(T, V, K, top).total; }

hipError_t launch_logprobs(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens,
                           bool tokens64, int64_t T, int64_t V, int64_t K, float scale, float* logp, float* entropy,
                           float* lse, int top, int64_t* top_ids, float* top_logp, void* ws, hipStream_t st) {
  const Plan L = plan(T, V, K, top);
  uint8_t* w = (uint8_t*)ws;
  float *target = (float*)(w + L.target), *mean = (float*)(w + L.mean);
  float2 *stats = (float2*)(w + L.stats), *tops = top ? (float2*)(w + L.tops) : nullptr;
  float* norms = top ? (float*)(w + L.norms) : nullptr;        // and after them the largest
  const LogitTops sets = logit_tops(T, V, K, top);
  const int groups = (int)logit_groups(T, V, K), each = logit_norms(T, V, K);
  for (int64_t t0 = 0; t0 < T; t0 += L.part) {
    const int64_t n = T - t0 < L.part ? T - t0 : L.part;
    const uint16_t* x = X + t0 * ldx;
    const void* y = tokens ? (const uint8_t*)tokens + t0 * (tokens64 ? 8 : 4) : nullptr;
    const hipError_t e = launch_logits(x, ldx, W, ldw, y, tokens64, n, T, V, K, scale, target, stats, mean, tops, norms, sets, st);
    if (e != hipSuccess) return e;
    const RowArgs R{stats, mean, target, y, tokens64, groups, (int)n, (int)V,
                    scale * LOG2E, logit_none(scale), (float2*)(w + L.rows), logp ? logp + t0 : nullptr,
                    entropy ? entropy + t0 : nullptr, lse + t0, x, W, ldx, ldw, (int)K, top, sets, tops, norms, each,
                    top ? norms + groups * each : nullptr, scale, top ? top_ids + t0 * top : nullptr,
                    top ? top_logp + t0 * top : nullptr};
    if (T <= FEW_TOKENS) {
      SBN_LAUNCH("logprob_rows", (logprob_top_kernel<1024, true>), dim3((unsigned)n), dim3(1024), 0, st, R);
      continue;
    }
    constexpr int64_t JOIN_TOKENS = 1 << 24;         // of a launch: fewer than 2^32 threads
    for (int64_t t = 0; t < n; t += JOIN_TOKENS) {
      const int64_t rest = n - t, blocks = rest > JOIN_TOKENS ? JOIN_TOKENS / 16 : cdiv(rest, 16) + (top > 0);
      SBN_LAUNCH("logprob_join", logprob_join_kernel, dim3((unsigned)blocks), dim3(1024), 0, st, R, (int)t);
    }
    if (top)
      SBN_LAUNCH("logprob_top", (logprob_top_kernel<256, false>), dim3((unsigned)(n < (1 << 20) ? n : (1 << 20))), dim3(256), 0,
                 st, R);
  }
  return hipGetLastError();
}

}  // namespace sbn
