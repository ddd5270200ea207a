// Launchers of the operators declared in include/sbn_score.h (T >= 1).
#pragma once

#include "sbn_score.h"
#include "train_internal.h"

namespace sbn {

// ----------------------------------------------------------------- the logits' statistics (cross_entropy.hip)
// Statistics come in logit_groups() groups of entries, [group][T]: the maximum of the sums
// x w (logits before their scale) and the sum of exponentials, one of the maximum left out (-1 of
// no entries), and the sum of exponential times exponent, exponents times scale log2 e and
// less the maximum's.  `target` [T]: the token's sum.  tops (or NULL): per token
// logit_tops().groups pairs of the largest and second largest of a set of 32, 16 or 8
// sums (logits before their scale), the first's place in its last 5 bits.  A set is
// what one lane holds of a column; of lanes that hold 8, two.  With tops, norms: per group
// logit_norms() numbers, the largest of which is no less than the norm of any of its rows of W.  (Few tokens: sets of 8
// are 64 KB to read for each at 65536 entries, and of 32 twice as often one with two
// candidates, all of which are then computed.)  Where two in a set are common, sets are of
// 8, parts of a lane's: of about c = top + 3 candidates 512 c^2 / V rows of W are computed for
// their neighbours' sake, with sets of 8 a sixteenth of that, and V bytes a token are written
// and read twice instead of V / 4, which costs least while the caches hold them.  (Logits +
// alternatives, us, with sets of 8 and without: 20 of 32001 entries, 1024 tokens, K = 4096 215 +
// 68, 206 + 92; the same, 8192 tokens 1521 + 365, 1513 + 372; 6 of 20000, 600, 2560 68 + 25, 67
// + 29; 64 of 8000, 2000, 512 27 + 70, 27 + 284; 20 of 32001, 37, 4096 58 + 27, 62 + 28; and
// where they are not taken 32 of 65536, 4096, 2560 1022 + 239, 990 + 207; 8 of 32001, 4096, 2560
// 507 + 97, 500 + 75; 8 of 16000, 8192, 1024 238 + 87, 233 + 84.)
// the sum that stands for no entry: -1e30 as an exponent
inline float logit_none(float scale) { return -1e30f / (scale * 1.4426950408889634f); }
constexpr int TOPS_MOST = 32;
constexpr int tops_of(int mi) { return 4 * mi >= 16 ? 4 * mi : 16; }
struct LogitTops {
  int mi_log2;                         // a lane's 4 mi entries are 4 of each of mi fragments of 16
  int of_log2;                         // entries of a set
  int groups;                          // sets, of V rounded up to whole tiles
  // the logits' group (of those that have statistics) that set g is of
  __host__ __device__ int group(int g) const { return g >> (4 + mi_log2 - of_log2); }
  // the place of set g's q-th entry: among its lane's where that holds several sets, else in the set
  __host__ __device__ int place(int g, int q) const {
    const int sets = 2 + mi_log2 - of_log2;                      // log2 of a lane's sets
    return sets > 0 ? ((g & ((1 << sets) - 1)) << of_log2) + q : q;
  }
  // the vocabulary entry at place p of set g
  __host__ __device__ int entry(int g, int p) const {
    const int per = 2 + mi_log2, lanes = of_log2 - per;          // log2 of a lane's entries and a set's lanes
    const int lane = lanes >= 0 ? (g << lanes) + (p >> per) : g >> -lanes;   // counted through waves, 4 a column
    p &= (1 << per) - 1;
    return ((lane >> 2) << (4 + mi_log2)) + ((p >> 2) << 4) + ((lane & 3) << 2) + (p & 3);
  }
};
static_assert(tops_of(8) == TOPS_MOST && TOPS_MOST == 32, "5 bits");
LogitTops logit_tops(int64_t T, int64_t V, int64_t K, int top);
int64_t logit_groups(int64_t T, int64_t V, int64_t K);
int logit_norms(int64_t T, int64_t V, int64_t K);
// T tokens of `all`, for which logit_tops(), logit_groups() and logit_norms() are asked
hipError_t launch_logits(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens, bool tokens64,
                         int64_t T, int64_t all, int64_t V, int64_t K, float scale, float* target, float2* stats, float* mean,
                         float2* tops, float* norms, const LogitTops& sets, hipStream_t st);

// ----------------------------------------------------------------- logprobs.hip
size_t logprobs_ws_bytes(int64_t T, int64_t V, int64_t K, int top);
// tokens and logp may be NULL (both), entropy may be NULL
hipError_t launch_logprobs(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens,
                           bool tokens64, int64_t T, int64_t V, int64_t K, float scale, float* logp, float* entropy,
                           float* lse, int top, int64_t* top_ids, float* top_logp, void* ws, hipStream_t st);

}  // namespace sbn
