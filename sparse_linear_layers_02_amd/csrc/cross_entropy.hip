// Softmax cross entropy of the output head without keeping the logits, and its
// gradients, on gfx950 bf16 matrix cores.
//
//   l = X W^T;  lse_t = log sum_v exp l[t,v];  loss_t = lse_t - l[t, y_t]
//   D[t,v] = g_t (exp(l[t,v] - lse_t) - [v = y_t]);  dX = D W;  dW = D^T X
// with D held as c (g_t / c) (...), c = max |g|: the factor c stays in float32
// until the products are done.  (With c inside, the mean's g = 1/T for all
// tokens gave every target's entry the same rounding error, up to 2^-8 of the
// gradient: 0.28% at T = 1021 against 0.18% for float32 operands.)
//
// Forward: one product whose epilogue reduces each tile of logits, while it is
// in registers, to the maximum and the sum of exponentials of each token over
// the tile's vocabulary entries, plus the target's logit where it falls in the
// tile; a second launch joins the tiles' pairs (m, s) in a fixed order.
//
// Log probabilities with entropies are the same with logits scaled (l' = scale l):
// the tile's sum of exponential times exponent beside its (m, s), and
//   D[t,v] = g_t ([v = y_t] - p) - h_t p (log p + H_t) = p (c0 + c1 log2 p) + g_t [v = y_t]
// of the entropy H's gradient h, with c = max(|g|, |h|).
//
// Gradients, per piece of the vocabulary: the same product with an epilogue
// that writes D in bf16; dX and dW are then two more products, on D and W and on
// D and X as they lie.  The workspace holds one piece of D, of D_ELEMS elements
// at most (of up to 2^20 tokens).  For a gradient of type SBN_F32_FINE the
// epilogue also writes what the rounding to bf16 left of D, in bf16, and its
// product is added.  (Relative error against 64 bits, 300 tokens of 2500 entries,
// K = 256: 1.4e-3 -> 2.0e-6; both gradients of 8192 tokens of 65536 entries, K =
// 4096: 9.6 -> 16.8 ms.)
//
// All three products are one kernel, C[a][b] = sum_k A[a][k] B[b][k], where an
// operand's rows in memory are either its outputs (X and W of the logits, D of
// dX) or the contraction (W of dX, D and X of dW): those go through the
// transposing LDS reads.  (Transposed copies of D, W and X in memory instead
// took 2% of the largest training step and a quarter of one of 64 tokens.)
#include "once_per_device.h"
#include "score_internal.h"

namespace sbn {
namespace {

constexpr int BK = 64;                              // contraction entries of one stage: 128-byte rows, one cache line
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr float NONE = -1.0e38f * LOG2E;            // the (scaled) maximum of no logits: finite, so that NONE - NONE is 0
// Elements of D in the workspace, 512 MB.  (Half: 1 to 3.5% slower at 4096 to 8192 tokens, dX summed over more pieces; twice: 1% either way.)
// A piece has at least 256 entries: above 2^20 tokens D has 256 elements a token instead.
constexpr int64_t D_ELEMS = int64_t(1) << 28;
constexpr int GMAX_WAVE = 1024;                     // tokens whose largest |dloss| a wave finds in two rounds of loads
constexpr int CUS = 256;
// Log probabilities' gradients take D in two bf16 numbers up to so many tokens: most of
// a row of dW (and of dX) is then of few products, whose rounding of D no others average
// (at worst 2^-8 of the row; of 8 tokens, 32001 entries, K = 2560, in bf16 0.0024 of the
// gradients' norm, with two 0.0016, what rounding them leaves).  It takes 4 to 24% longer
// (8 tokens 112 -> 116 us, 128 138 -> 168), of 256 45%.
constexpr int PAIR_TOKENS = 128;

// PAIR: D in two bf16 numbers; OUT, ADD: C in bf16 or float32, ADD on top of Cin;
// TWIN: the sum of two products, with B and a second B, stage by stage.  (One on top of
// the other, 128 tokens of 50001 entries, K = 4096, with D in two numbers took 939 us, so 542.)
// SCORE, POLICY: the statistics and D of log probabilities with entropies; TOPS: and
// the two largest logits of each tops_of(MI), TOPS8: of each 8.
enum Epi { EPI_STATS, EPI_SCORE, EPI_SCORE_TOPS, EPI_SCORE_TOPS8, EPI_GRAD, EPI_GRAD_PAIR, EPI_POLICY, EPI_POLICY_PAIR, EPI_OUT16, EPI_OUT32,
           EPI_TWIN16, EPI_TWIN32, EPI_ADD32 };

struct GemmArgs {
  const uint16_t *A, *B;               // rows of lda, ldb
  int64_t lda, ldb;
  int nA, nB;                          // outputs
  int mA, mB;                          // outputs in memory: tiles past them read the last ones again
  int kA, kB;                          // contraction rows in memory, where rows are the contraction: past them the last
  int tilesA, tilesB;
  int steps, splits;                   // contraction stages in all, and parts they are split into
  // EPI_STATS, EPI_GRAD: A rows are vocabulary entries, B rows tokens
  const void* labels;
  bool labels64;
  int v0;                              // vocabulary entry of A row 0
  int V;
  float2* stats;                       // [2-wave column groups][nB]: maximum (times log2 e), sum; EPI_SCORE: maximum, sum without it
  float* target;                       // [nB] sum of the label's entry
  const float *lse, *dloss;
  float* gmax;                         // max |dloss|; EPI_GRAD divides by it, EPI_OUT multiplies
  // EPI_SCORE, EPI_POLICY: logits are scale times the sums
  float scale;
  float none;                          // the sum that stands for no entry, -1e30 in scaled exponents
  float* mean;                         // beside stats: sum of exponential times scaled exponent
  float2* tops;                        // [nB][ldt] the two largest sums of each set, the first's place in its last bits
  int64_t ldt;
  float* norms;                        // beside tops: [groups][WB] no less than the largest |row of A| of a group's fragments i, i % WB alike
  const float *entropy, *dentropy;     // dloss: of the log probabilities; either gradient may be NULL
  uint16_t* D;                         // [tpad][ldd], ldd a multiple of 256; 0 past the tokens and past nA
  int64_t ldd;
  int64_t dlow;                        // PAIR: elements from D to what its rounding left
  int64_t twin;                        // EPI_TWIN: bytes from B to the second one; 0 for others
  int tpad;                            // a multiple of 64
  // EPI_OUT: C [nB][ldc], A outputs along the row
  void* C;
  const float* Cin;                    // [nB][ldcin], added first, or NULL (where TRB, EPI_ADD32 only)
  int64_t ldc, ldcin;
  int64_t part_stride;                 // elements of C from one part of the contraction to the next
};

__device__ inline int64_t label_at(const void* labels, bool is64, int t) {
  return is64 ? ((const int64_t*)labels)[t] : (int64_t)((const int32_t*)labels)[t];
}

// max |dloss| over the tokens first, first + step, ... with a target, of a wave
__device__ inline float max_dloss(const float* dloss, const void* labels, bool is64, int V, int T, int first, int step) {
  constexpr int AHEAD = 8;                           // loads in flight
  float m = 0.0f;
  for (int t0 = first; t0 < T; t0 += step * AHEAD) {
    float g[AHEAD];
    int64_t y[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int t = t0 + step * k < T ? t0 + step * k : t0;
      g[k] = dloss[t];
      y[k] = label_at(labels, is64, t);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (y[k] >= 0 && y[k] < V) m = fmaxf(m, fabsf(g[k]));
  }
  return wave_all(m, Max{});
}

// The same of log probabilities and entropies; a token without a target has its entropy alone
__device__ inline float max_policy(const float* dlogp, const float* dentropy, const void* labels, bool is64, int V, int T,
                                   int first, int step) {
  constexpr int AHEAD = 8;                           // loads in flight
  float m = 0.0f;
  for (int t0 = first; t0 < T; t0 += step * AHEAD) {
    float g[AHEAD], h[AHEAD];
    int64_t y[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int t = t0 + step * k < T ? t0 + step * k : t0;
      g[k] = h[k] = 0.0f, y[k] = -1;
      if (dlogp) g[k] = dlogp[t], y[k] = label_at(labels, is64, t);
      if (dentropy) h[k] = dentropy[t];
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (y[k] >= 0 && y[k] < V) m = fmaxf(m, fabsf(g[k]));
      m = fmaxf(m, fabsf(h[k]));
    }
  }
  return wave_all(m, Max{});
}

// Tile order: the hardware deals consecutive blocks to the 8 XCDs in turn, so
// block b belongs to XCD b % 8.  Each XCD takes a contiguous range of a list in
// which 4 B tiles go together and A runs inside: the 32 blocks an XCD has in
// flight then share 4 B and 8 A row panels in its L2.  (T = 8192, V = 65536,
// K = 4096, gradients included: 13.08 ms with 4, 13.23 with 8, 13.4 with 16.)
// (The quotients are made by the vector unit; scalar(), so that what follows from
// them, the addresses and counters of the loops, is not computed there too.)
__device__ inline int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ inline void tile_of(int b, int blocks, int nta, int ntb, int& ta, int& tb) {
  constexpr int XCDS = 8, GROUP = 4;
  const int per = blocks / XCDS, rem = blocks % XCDS;
  const int x = b % XCDS;
  int i = x * per + (x < rem ? x : rem) + b / XCDS;
  const int g = scalar(i / (nta * GROUP));
  i -= g * nta * GROUP;
  const int w = ntb - g * GROUP < GROUP ? ntb - g * GROUP : GROUP;
  ta = scalar(i / w);
  tb = g * GROUP + (i - ta * w);
}

// acc += a b^T, the accumulator held in the accumulation registers.  Written in
// assembly because the builtin's accumulators of a 256 x 256 tile were moved
// between the register files around every matrix instruction (some 500 moves a
// stage against 128 products).  What the compiler then does not see: a result
// may be read by other instructions only some cycles later.  settle() waits for
// that, and fetch() is the only way the accumulators are read after it.  (The
// fragments come from LDS reads, for which the compiler waits; a result is the
// operand of a product again 8 products later at the soonest.)
__device__ inline void mfma_acc(v4f& acc, v8bf a, v8bf b) {
  asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
typedef short v4s __attribute__((ext_vector_type(4)));
__device__ inline v4s read_transposed(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) v4s*)p);
}
// 16 bytes per lane from base + off into LDS at lds + 16 lane, like g2lds16 (no
// register is written).  In assembly where fragments are read by transposing
// reads: before each of those the compiler would wait for every load into LDS,
// as it does not for plain reads.  The waits are stage_barrier()'s.
__device__ inline void load_to_lds(const uint8_t* base, uint32_t off, const uint8_t* lds) {
  const uint32_t at = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)lds;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(at), "v"(off), "s"(base)
               : "memory", "m0");
}
__device__ inline void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
__device__ inline v4f fetch(v4f& acc) {
  asm volatile("" : "+a"(acc));
  return acc;
}
// All waves meet: each has its LDS reads and all but its latest N loads behind it.
// By the builtin, so that the compiler knows the reads done and adds no wait.
template <int N>
__device__ inline void stage_barrier() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// x, in a branch that few waves take: what is computed from it stays in the branch
__device__ inline int rarely(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Two fragments of results, 4 consecutive outputs a lane each, as 8 consecutive
// outputs in bf16: lane group g (of 16) holds outputs 16 (g % 2) + 8 (g / 2) .. + 7
// of the pair's 32.  The 16-byte pieces of four lanes then make 64 bytes of a row:
// 256 MB written so by 256 blocks take 54 us, in 8-byte pieces of one fragment
// (32 bytes of a row) 68, one lane group after the other 51.
__device__ inline uint4 pack_pair(const float* c, const float* d) {
  const auto lo = __builtin_amdgcn_permlane16_swap(pack_bf16x2(c[0], c[1]), pack_bf16x2(d[0], d[1]), false, false);
  const auto hi = __builtin_amdgcn_permlane16_swap(pack_bf16x2(c[2], c[3]), pack_bf16x2(d[2], d[3]), false, false);
  return make_uint4(lo[0], hi[0], lo[1], hi[1]);
}

// The kernel's arguments, read again where they are used: held over the loops,
// those of the epilogue and of the next tile's start pushed the loops' own
// addresses out of the scalar registers.
typedef __attribute__((address_space(4))) const GemmArgs ArgsInMemory;
__device__ inline ArgsInMemory& reread_args() {
  ArgsInMemory* q = (ArgsInMemory*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(q));
  return *q;
}
__device__ inline float uniform(float x) { return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x))); }
__device__ inline void lds_reads_done() { __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4)); }

// One operand's half stage in LDS: HR outputs x 64 contraction entries.
//
// Rows are outputs (TR false): 128 bytes of 8 chunks of 16; chunk c of row r lies
// at position c ^ (r & 7), so that the 16 rows of a fragment read spread over the
// banks.
// Rows are the contraction (TR true): 2 HR bytes, in groups of 32 (16 outputs);
// group f of row c lies at f ^ swizzle(c).  A transposing read takes, for 16
// lanes, 4 rows of one group; the four 16-lane parts of a wave read rows 8 apart.
// The swizzle puts those 16 rows on all 8 groups of banks, two on each.
template <bool TR, int HR>
struct HalfStage {
  static constexpr bool TRANSPOSED = TR;
  static constexpr int OUTPUTS = HR;
  static constexpr int ROW = TR ? 2 * HR : BK * 2, CHUNKS = ROW / 16, ROWS = 64 / CHUNKS;   // rows of a 1 KB load
  static constexpr int BYTES = HR * BK * 2;
  static constexpr int GROUPS = HR / 16, SPAN = 8 / GROUPS;    // SPAN rows lie side by side over the banks
  static __device__ int swizzle(int k4, int g) { return k4 / SPAN + (g & 1) * (4 / SPAN); }   // row 8 g + k4 (+ 4)

  // Of load `l` (of HR / 8) the row and the chunk's byte in its row in memory, for this lane
  static __device__ int row_of(int l, int lane) { return l * ROWS + lane / CHUNKS; }
  static __device__ int chunk_of(int row, int lane) {
    const int at = lane % CHUNKS;
    return TR ? at ^ (2 * swizzle(row & 3, row >> 3)) : at ^ (row & 7);
  }
};

// WA x WB waves, wave tile 16 MI x 16 MJ, RING half stages of LDS; TRA, TRB: the
// operand's rows in memory are the contraction.
//
// A stage is 64 contraction entries of the tile's outputs, so that a row of it is
// at least one 128-byte line (half of that, with twice the stages in flight,
// measured 10% slower).  It is loaded in two halves, the upper outputs of A and
// of B and then the lower ones, each into the next place of a ring of RING
// places: the loads go out evenly over a stage instead of all after its barrier.
//
// Blocks stay and take tiles in turn.  The loads run AHEAD stages before the
// products and go on into the next tile, so only a block's first tile waits for
// its first stages, and the loads of a tile's last stages are not wasted.
// (Against one tile a block: 64 tokens' gradients 137 for 144 us, 1021 tokens 462
// for 474, evaluation of 4096 tokens 975 for 989, 8192 tokens 12.64 for 12.69 ms;
// 512 tokens of 8000 entries, one round of tiles, 54.9 for 53.3.)
//
// Bound by the matrix cores: at T = 8192, V = 65536, K = 4096 they are busy 74% of
// the forward's cycles and 67 to 69% of the gradients', at the 1.67 to 1.83 GHz
// that the part's power allows under them.  The forward takes 3.01 ms (1.46
// PFLOP/s; the library's bare product on the same card 2.88), D, dX and dW of half
// the entries 1.61, 1.53 and 1.64 ms (1.37, 1.44, 1.34; the library's halves of dX
// and dW 1.61 and 1.87); up to 8% more on cards of lower clocks.  No LDS bank
// conflicts; 6.4 GB fetched from beyond L2 in the forward.  At 17 tokens (FLAT) bound by reading W: a head of 50001 x
// 2560, 256 MB, in 50 us, 5.1 TB/s.  Log probabilities: the entropies' sums take 1.5%
// of the statistics' time, the largest logits and the norms 3% more (4096 tokens, 65536 entries, K =
// 2560: 952, 966 and 992 us; the library's bare product 963 on that card), D with entropies 0 to
// 2% of D's.
template <int WA, int WB, int MI, int MJ, int RING, int EPI, bool TRA, bool TRB>
__global__ __launch_bounds__(64 * WA * WB, 1) void ce_gemm_kernel(GemmArgs P) {
  constexpr int TA = WA * MI * 16, TB = WB * MJ * 16, NW = WA * WB;
  using HA = HalfStage<TRA, TA / 2>;
  using HB = HalfStage<TRB, TB / 2>;
  constexpr int HALF = HA::BYTES + HB::BYTES;
  constexpr int LA = TA / (16 * NW), LB = TB / (16 * NW);    // 1 KB loads per wave and half stage
  constexpr int LPH = LA + LB;
  constexpr bool POLICY = EPI == EPI_POLICY || EPI == EPI_POLICY_PAIR, PAIR = EPI == EPI_GRAD_PAIR || EPI == EPI_POLICY_PAIR;
  constexpr bool GRAD = EPI == EPI_GRAD || PAIR || POLICY;
  constexpr bool TOPS8 = EPI == EPI_SCORE_TOPS8, TOPS = EPI == EPI_SCORE_TOPS || TOPS8, SCORE = EPI == EPI_SCORE || TOPS, STATS = EPI == EPI_STATS || SCORE;
  constexpr bool TWIN = EPI == EPI_TWIN16 || EPI == EPI_TWIN32;
  constexpr int AHEAD = RING / 2;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  static_assert(RING >= 5 && RING % 2 == 1 && (RING - 3) * LPH < 64, "a stage, the next one and a half in flight");

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wa = wave % WA, wb = wave / WA;
  const int work = P.tilesA * P.tilesB * P.splits;
  struct Item {                                      // one tile, one part of its contraction
    int a0, b0, part, s_lo, nsteps;
  };
  auto item = [&](int w, auto& P) {
    const int tiles = P.tilesA * P.tilesB;
    Item t;
    t.part = P.splits > 1 ? scalar(w / tiles) : 0;
    int ta, tb;
    tile_of(w - t.part * tiles, tiles, P.tilesA, P.tilesB, ta, tb);
    t.a0 = ta * TA, t.b0 = tb * TB;
    const int each = P.splits > 1 ? scalar(P.steps / P.splits) : P.steps;
    const int more = P.steps - each * P.splits;      // the first `more` parts have one stage more
    t.s_lo = t.part * each + (t.part < more ? t.part : more);
    t.nsteps = each + (t.part < more ? 1 : 0);
    if (TWIN) t.nsteps *= 2;
    return t;
  };

  // ---- the loading side: the stage to load next
  // Byte offsets of this lane's loads.  Outputs past the operand are clamped here;
  // contraction rows, which only a tile's last stage can pass, when they are loaded.
  const uint32_t ldA = (uint32_t)P.lda * 2, ldB = (uint32_t)P.ldb * 2;
  uint32_t offA[2][LA], offB[2][LB];                 // TR: of the chunk alone
  int lw = blockIdx.x, lleft, k0;                    // item, stages of it left, first contraction entry
  const uint8_t *gA, *gB;
  auto offset = [&](auto half, int l, int h, int out0, int n, uint32_t ld) {
    using H = decltype(half);
    const int row = H::row_of(l, lane), chunk = H::chunk_of(row, lane);
    if constexpr (!H::TRANSPOSED) {
      const int r = h * H::OUTPUTS + row;
      return (uint32_t)(out0 + r < n ? r : n - 1 - out0) * ld + chunk * 16;
    } else {
      const int o = h * H::OUTPUTS + chunk * 8;
      return (uint32_t)(out0 + o < n ? o : n - 8 - out0) * 2;
    }
  };
  auto start_item = [&](const Item& t, auto& P) {
    lleft = t.nsteps;
    k0 = t.s_lo * BK;
    gA = (const uint8_t*)P.A + (TRA ? k0 * P.lda + t.a0 : t.a0 * P.lda + k0) * 2;
    gB = (const uint8_t*)P.B + (TRB ? k0 * P.ldb + t.b0 : t.b0 * P.ldb + k0) * 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int q = 0; q < LA; ++q) offA[h][q] = offset(HA{}, wave * LA + q, h, t.a0, P.mA, ldA);
#pragma unroll
      for (int q = 0; q < LB; ++q) offB[h][q] = offset(HB{}, wave * LB + q, h, t.b0, P.mB, ldB);
    }
  };
  auto next_stage = [&]() {                          // past the last item: its last stage again
    if (lleft > 1) {
      --lleft;
      if (TWIN) {                                    // a stage of B, then the same one of the second B
        if (lleft & 1) {
          gB += P.twin;
          return;
        }
        gB -= P.twin;
      }
      k0 += BK;
      gA += TRA ? P.lda * (2 * BK) : 2 * BK;
      gB += TRB ? P.ldb * (2 * BK) : 2 * BK;
    } else if (lw + (int)gridDim.x < work) {
      lw += (int)gridDim.x;
      ArgsInMemory& Q = reread_args();               // (and keeps this a branch, taken once a tile)
      start_item(item(lw, Q), Q);
    }
  };
  auto load_one = [&](int q, int h, int place) {     // load q of LPH of a half stage
    uint8_t* base = smem + place * HALF;
    auto load = [&](const uint8_t* from, uint32_t off, uint8_t* to) {
      if constexpr (TRA || TRB) load_to_lds(from, off, to);
      else g2lds16(from + off, to);
    };
    if (q < LA) {
      uint32_t off = offA[h][q];
      if (TRA) off += (uint32_t)min(HA::row_of(wave * LA + q, lane), P.kA - 1 - k0) * ldA;
      load(gA, off, base + (wave * LA + q) * 1024);
    } else {
      uint32_t off = offB[h][q - LA];
      if (TRB) off += (uint32_t)min(HB::row_of(wave * LB + q - LA, lane), P.kB - 1 - k0) * ldB;
      load(gB, off, base + HA::BYTES + (wave * LB + q - LA) * 1024);
    }
  };

  // ---- the product side
  const int g16 = lane >> 4, l15 = lane & 15, l4 = 4 * g16, l8 = (g16 & 1) * 16 + (g16 >> 1) * 8;
  v4f acc[MI][MJ];

  // acc[i][j]: A outputs a0 + 16 (wa MI + i) + 4 (lane / 16) + 0..3, B output b0 + 16 (wb MJ + j) + lane % 16;
  // a tile's sums start from Cin, loaded at once (added at the end, each load waited for the stores before it)
  auto start_sums = [&](const Item& t, auto& P) {
    const float* from = STATS || GRAD || (TRB && EPI != EPI_ADD32) ? nullptr : P.Cin;
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        if (from) {
          const int a = t.a0 + 16 * (wa * MI + i) + l4, b = t.b0 + 16 * (wb * MJ + j) + l15;
          acc[i][j] = *(const v4f*)(from + (int64_t)(b < P.nB ? b : P.nB - 1) * P.ldcin + (a < P.nA ? a : 0));
        } else {
          acc[i][j] = (v4f){0.f, 0.f, 0.f, 0.f};
        }
      }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < MJ; ++j) asm volatile("" : "+a"(acc[i][j]));
  };

  // fragment of 16 outputs x 32 contraction entries: lane l holds output l % 16, entries 8 (l / 16) .. + 8
  const int frow = l15 * (BK * 2);
  const int fpos0 = (g16 ^ (lane & 7)) * 16, fpos1 = ((4 + g16) ^ (lane & 7)) * 16;
  // Fragment f of a half stage, 32 contraction entries `sub`.  The transposing read
  // gives lane l of 16 the 4 rows' entries of output l, where lane 4 k + q reads
  // outputs 4 q .. + 3 of row k.
  auto fragment = [&](auto half, const uint8_t* p, int f, int sub) {
    using H = decltype(half);
    if constexpr (H::TRANSPOSED) {
      const int k4 = l15 >> 2;
      p += (8 * g16 + k4) * H::ROW + ((f ^ H::swizzle(k4, g16)) * 32) + (l15 & 3) * 8 + sub * (32 * H::ROW);
      union {
        v4s h[2];
        v8bf v;
      } u;
      u.h[0] = read_transposed(p);
      u.h[1] = read_transposed(p + 4 * H::ROW);
      return u.v;
    } else {
      return __builtin_bit_cast(v8bf, *(const v4i*)(p + f * (16 * BK * 2) + frow + (sub ? fpos1 : fpos0)));
    }
  };
  // B's fragments of both halves of a stage, and A's of one: A's fragment i is read
  // again, for the next half, once the products with it are under way; only its
  // last one, which is needed latest, has two places
  v8bf fa[MI - 1], fl[2], fb[2][MJ];
  // fragment i of A (j of B) of the stage whose halves lie at places p0 and p1
  auto read_a = [&](int p0, int p1, int sub, int i) {
    const int f = WA > 1 ? wa % (WA / 2) * MI + i : i % (MI / 2);
    const bool lower = WA > 1 ? wa >= WA / 2 : i >= MI / 2;
    (i < MI - 1 ? fa[i] : fl[sub]) = fragment(HA{}, smem + (lower ? p1 : p0) * HALF, f, sub);
  };
  auto read_b = [&](int p0, int p1, int sub, int j) {
    const int f = WB > 1 ? wb % (WB / 2) * MJ + j : j % (MJ / 2);
    const bool lower = WB > 1 ? wb >= WB / 2 : j >= MJ / 2;
    fb[sub][j] = fragment(HB{}, smem + (lower ? p1 : p0) * HALF + HA::BYTES, f, sub);
  };
  // taken in snake order: each product shares an operand with the one before (0.3% of a training step)
  auto multiply = [&](int i, int j, int sub) { mfma_acc(acc[i][j], i < MI - 1 ? fa[i] : fl[sub], fb[sub][j]); };
  // TOPS: norms of A's rows, the same in all of a token's tiles and in the waves of one `wa`: the first tile's
  // waves take MI / WB of the fragments each, and read them again.  (Taken from the fragments of the products,
  // they cost 100 to 200 spilled registers.)
  float squares[MI / WB] = {};
  bool norms = false;
  auto square = [&](int p0, int p1) {
    const uint8_t* half = smem + (wa >= WA / 2 ? p1 : p0) * HALF;
#pragma unroll
    for (int k = 0; k < 2 * MI / WB; ++k)
      squares[k / 2] = add_squares(fragment(HA{}, half, wa % (WA / 2) * MI + wb * (MI / WB) + k / 2, k % 2), squares[k / 2]);
  };
  auto wrap = [](int p) { return p >= RING ? p - RING : p; };

  // Stages are numbered through all items of the block; half stage u (of stage
  // u / 2) lies at place u % RING.  Stage n: while the matrix instructions of its
  // first 32 entries run, the fragments of the second 32 are read, and the upper
  // half of stage n + AHEAD is loaded into the place of half stage 2 n - 1; then all
  // waves meet (stage n has been read, stage n + 1 has landed), and while the
  // second 32 run, the next stage's first fragments are read, and the lower half of
  // stage n + AHEAD is loaded into the place of half stage 2 n.
  // GRAD: of few tokens every wave finds the largest |dloss| itself, which a
  // launch of its own would take longer for
  float gmax = 1.0f;
  if (GRAD && P.nB <= GMAX_WAVE) {
    gmax = uniform(POLICY ? max_policy(P.dloss, P.dentropy, P.labels, P.labels64, P.V, P.nB, lane, 64)
                          : max_dloss(P.dloss, P.labels, P.labels64, P.V, P.nB, lane, 64));
    if (blockIdx.x == 0 && tid == 0) {
      P.gmax[0] = gmax;
      if (POLICY) P.gmax[1] = gmax * P.scale;        // the products' factor
    }
  } else if (!STATS && P.gmax) {
    gmax = uniform(*P.gmax);
  }
  const float ginv = gmax >= 0x1p-126f ? 1.0f / gmax : 0.0f;   // smaller ones have no quotient: gradients 0
  Item it = item(blockIdx.x, P);
  if (TOPS) norms = it.b0 == 0;
  start_item(it, P);
#pragma unroll
  for (int n = 0; n < AHEAD; ++n) {
#pragma unroll
    for (int q = 0; q < 2 * LPH; ++q) load_one(q % LPH, q / LPH, 2 * n + q / LPH);
    next_stage();
  }
  start_sums(it, P);
  settle();
  stage_barrier<(RING - 3) * LPH>();                 // stage 0 has landed
#pragma unroll
  for (int j = 0; j < MJ; ++j) read_b(0, 1, 0, j);
#pragma unroll
  for (int i = 0; i < MI; ++i) read_a(0, 1, 0, i);

  int p0 = 0;                                        // place of the stage's upper half
  for (int w = blockIdx.x;; w += (int)gridDim.x) {
    for (int left = it.nsteps; left > 0; --left) {
      const int p1 = wrap(p0 + 1), n0 = wrap(p0 + 2), n1 = wrap(p0 + 3), free0 = wrap(p0 + RING - 1);
      if (TOPS && norms) square(p0, p1);
      lds_reads_done();                              // before new reads, which the first products need not wait for
#pragma unroll
      for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < MJ; ++j)
          if (j * MI / MJ == i) read_b(p0, p1, 1, j);
        read_a(p0, p1, 1, i > 0 ? i - 1 : MI - 1);
#pragma unroll
        for (int q = 0; q < LPH; ++q)
          if (q * MI / LPH == i) load_one(q, 0, free0);
#pragma unroll
        for (int j = 0; j < MJ; ++j) multiply(i, i & 1 ? MJ - 1 - j : j, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      stage_barrier<(RING - 4) * LPH>();
#pragma unroll
      for (int i = 0; i < MI; ++i) {
#pragma unroll
        for (int j = 0; j < MJ; ++j)
          if (j * MI / MJ == i) read_b(n0, n1, 0, j);
        read_a(n0, n1, 0, i > 0 ? i - 1 : MI - 1);
#pragma unroll
        for (int q = 0; q < LPH; ++q)
          if (q * MI / LPH == i) load_one(q, 1, p0);
#pragma unroll
        for (int j = 0; j < MJ; ++j) multiply(i, i & 1 ? MJ - 1 - j : j, 1);
        __builtin_amdgcn_sched_barrier(0);
      }
      next_stage();
      p0 = n0;
    }
    settle();

    ArgsInMemory& P = reread_args();
    const int aw = it.a0 + wa * MI * 16, bw = it.b0 + wb * MJ * 16;
    // a label's place from the lane's first entry: is it one of the lane's?  (Few waves hold one of their tokens' labels.)
    auto holds = [](int want) { return want >= 0 && want < MI * 16 && (want & 12) == 0; };
    if (STATS) {
      const float factor = SCORE ? P.scale * LOG2E : LOG2E;
      const bool ragged = aw + MI * 16 > P.nA;
      const int group = it.a0 / (MI * 16) + wa;
      if constexpr (TOPS) {
        if (norms) {
          float most = 0.0f;
#pragma unroll
          for (int i = 0; i < MI / WB; ++i) most = fmaxf(most, rows_all(squares[i], Add{})), squares[i] = 0.0f;
          // a lane's K / 8 sums of two squares, up to three roundings each: under 2^-6 for K <= 2^18; and what was taken for 0
          most = row16_all(most, Max{}) * (1.0f + 0x1p-6f) + (float)(P.steps * BK) * 0x1p-124f;
          if (lane == 0) P.norms[group * WB + wb] = sqrtf(most);
        }
      }
      int wants[MJ];
#pragma unroll
      for (int j = 0; j < MJ; ++j) {                 // all loads before the first store: they would wait for it
        const int t = bw + 16 * j + l15;
        const int64_t y = t < P.nB && (!SCORE || P.labels) ? label_at(P.labels, P.labels64, t) : -1;
        wants[j] = y >= 0 && y < P.V ? (int)y - aw - l4 : -1;
      }
      asm volatile("" ::: "memory");
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        const int t = bw + 16 * j + l15, want = wants[j];
        if (TOPS) {
          // float order is kept but for the last bits, which hold the place; the middle of the
          // two so far and the new one is the second (and, of a tie, the second is as large)
          constexpr int LANES = tops_of(MI) / (MI * 4);   // lanes of a column that join
          static_assert(LANES == 1 || LANES == 2, "a set is of one half of a column");
          const uint32_t lane_bits = MI * 4 * (g16 & (LANES - 1));
          float first = -3.0e38f, second = -3.0e38f;
#pragma unroll
          for (int i = 0; i < MI; ++i) {
            v4f x = fetch(acc[i][j]);                // again below: held for both, 35 registers were spilled
            if (ragged) {
              const int left = rarely(P.nA - aw - l4);
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (16 * i + e >= left) x[e] = P.none;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float key = __uint_as_float((__float_as_uint(x[e]) & ~(uint32_t)(TOPS_MOST - 1)) | (4 * i + e));
              second = __builtin_amdgcn_fmed3f(first, second, key);
              first = fmaxf(first, key);
            }
            if (TOPS8 && i % 2 == 1) {
              if (t < P.nB) P.tops[(int64_t)t * P.ldt + (group * 4 + g16) * (MI / 2) + i / 2] = make_float2(first, second);
              first = second = -3.0e38f;
            }
          }
          if (LANES > 1 && !TOPS8) {                 // in both, so that the first stays the larger
            first = __uint_as_float(__float_as_uint(first) | lane_bits);
            second = __uint_as_float(__float_as_uint(second) | lane_bits);
            const auto f = __builtin_amdgcn_permlane16_swap(__float_as_uint(first), __float_as_uint(first), false, false);
            const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(second), __float_as_uint(second), false, false);
            const float f0 = __uint_as_float(f[0]), f1 = __uint_as_float(f[1]);
            second = fmaxf(fminf(f0, f1), fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1])));
            first = fmaxf(f0, f1);
          }
          if (t < P.nB && (g16 & (LANES - 1)) == 0 && !TOPS8)
            P.tops[(int64_t)t * P.ldt + (group * 4 + g16) / LANES] = make_float2(first, second);
        }
        float m = -INFINITY;
        v4f c[MI];
#pragma unroll
        for (int i = 0; i < MI; ++i) c[i] = fetch(acc[i][j]);
        if (ragged) {
          const int left = rarely(P.nA - aw - l4);
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (16 * i + e >= left) c[i][e] = SCORE ? P.none : -INFINITY;
        }
        const bool has = holds(want);
        if (__any(has)) {
          const int at = rarely(want);
          float hit = 0.0f;
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (at == 16 * i + e) hit = c[i][e];
          if (has) P.target[t] = hit;
        }
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = fmaxf(m, c[i][e]);
        m = rows_all(m, Max{});
        // a group past the vocabulary has no logits
        const float top = SCORE ? fmaxf(m, P.none) : fmaxf(m * factor, NONE);
        float sum = 0.0f, mean = 0.0f;
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float d = SCORE ? (c[i][e] - top) * factor : c[i][e] * factor - top, x = __builtin_amdgcn_exp2f(d);
            sum += x;
            if (SCORE) mean += x * d, c[i][e] = x;
          }
        sum = rows_all(sum, Add{});
        if (SCORE) {
          mean = rows_all(mean, Add{});
          float rest = sum - 1.0f;                   // without the largest itself
          const bool near = sum < 1.25f;             // whose 1 took the last bits of the others
          if (__any(near)) {
            float small = 0.0f;
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) small += __builtin_amdgcn_fractf(c[i][e]);
            small = rows_all(small, Add{});
            if (near) rest = small + (rintf(sum - small) - 1.0f);   // of several that are as large, all but one
          }
          if (aw >= P.nA) rest = -1.0f, mean = 0.0f;
          if (lane < 16 && t < P.nB) P.mean[(int64_t)group * P.nB + t] = mean;
          sum = rest;
        }
        if (lane < 16 && t < P.nB) P.stats[(int64_t)group * P.nB + t] = make_float2(top, sum);
      }
    } else if (GRAD) {
      const float factor = POLICY ? P.scale * LOG2E : LOG2E;
      int want[MJ];
      float g[MJ], ls[MJ], c0[MJ], c1[MJ];           // POLICY: D = p (c0 + c1 log2 p), and g at the token
      uint32_t kept[MJ], used[MJ];                   // all ones, or 0: what a token without a target (POLICY: a gradient) holds gives 0
#pragma unroll
      for (int j = 0; j < MJ; ++j) {                 // all loads before the first store: they would wait for it
        const int t = bw + 16 * j + l15;
        const bool live = t < P.nB;
        const int64_t y = live && (!POLICY || P.labels) ? label_at(P.labels, P.labels64, t) : -1;
        kept[j] = y >= 0 && y < P.V ? ~0u : 0u;
        ls[j] = live ? P.lse[t] * LOG2E : 0.0f;
        if (POLICY) {                                // loads that do not wait for each other
          float dl = 0.0f, h = 0.0f, ent = 0.0f;
          if (live && P.dloss) dl = P.dloss[t];
          if (live && P.dentropy) h = P.dentropy[t] * ginv, ent = P.entropy[t];
          g[j] = kept[j] ? dl * ginv : 0.0f;
          c0[j] = -(g[j] + (h != 0.0f ? h * ent : 0.0f)), c1[j] = -LN2 * h;
          used[j] = g[j] != 0.0f || h != 0.0f ? ~0u : 0u;
        } else {
          g[j] = kept[j] ? P.dloss[t] * ginv : 0.0f;
        }
        want[j] = kept[j] ? (int)y - P.v0 - aw - l4 : -1;
      }
      asm volatile("" ::: "memory");
      const bool ragged = aw + MI * 16 > P.nA;
      if (bw < P.tpad) {                             // a multiple of the wave's 64 tokens
#pragma unroll
        for (int j = 0; j < MJ; ++j) {
          uint16_t* row = P.D + (int64_t)(bw + 16 * j + l15) * P.ldd + aw + l8;
          const bool hits = __any(holds(want[j]));
#pragma unroll
          for (int i = 0; i < MI; i += 2) {
            float d[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const v4f c = fetch(acc[i + h][j]);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float z = c[e] * factor - ls[j];
                d[h][e] = __builtin_amdgcn_exp2f(z);
                if (POLICY) d[h][e] *= fmaf(c1[j], z, c0[j]);
              }
            }
            if (hits) {
              const int at = rarely(want[j]);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (at == 16 * (i + h) + e) d[h][e] += POLICY ? g[j] : -1.0f;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 4; ++e)            // (a select became a branch for each element)
                d[h][e] = __uint_as_float(__float_as_uint(POLICY ? d[h][e] : g[j] * d[h][e]) & (POLICY ? used[j] : kept[j]));
            if (ragged) {
              const int left = rarely(P.nA - aw - l4);
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  if (16 * (i + h) + e >= left) d[h][e] = 0.0f;
            }
            *(uint4*)(row + 16 * i) = pack_pair(d[0], d[1]);
            if (PAIR) {
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 4; ++e) d[h][e] -= (float)(__bf16)d[h][e];
              *(uint4*)(row + P.dlow + 16 * i) = pack_pair(d[0], d[1]);
            }
          }
        }
      }
    } else {
      const int64_t at = it.part * P.part_stride + (int64_t)bw * P.ldc;
#pragma unroll
      for (int j = 0; j < MJ; ++j) {
        if (bw + 16 * j + l15 >= P.nB) continue;     // for all four groups of a column alike
        const int64_t row = at + (int64_t)(16 * j + l15) * P.ldc + aw;
#pragma unroll
        for (int i = 0; i < MI; i += 2) {
          if (aw + 16 * i >= P.nA) break;            // nA is a multiple of 64
          float c[2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4f x = fetch(acc[i + h][j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) c[h][e] = x[e] * gmax;
          }
          if (EPI != EPI_OUT16 && EPI != EPI_TWIN16) {
            float* to = (float*)P.C + row + 16 * i + l4;
            *(v4f*)to = *(const v4f*)c[0], *(v4f*)(to + 16) = *(const v4f*)c[1];
          } else {
            *(uint4*)((uint16_t*)P.C + row + 16 * i + l8) = pack_pair(c[0], c[1]);
          }
        }
      }
    }
    if (w + (int)gridDim.x >= work) break;
    it = item(w + (int)gridDim.x, P);
    if (TOPS) norms = it.b0 == 0;
    start_sums(it, P);
  }
  wait_vmcnt<0>();                                   // no load into LDS outlives the block
}

// lse and loss of a token from its groups' (maximum, sum): 16 tokens a block, 64
// threads a token take every 64th group each, then the 64 pairs are joined in a
// tree.  (64 tokens a block and 16 threads a token took 31 us for 17 tokens of
// 50001 entries: one block, whose loads wait for each other.)  2^26 tokens in one
// launch would be 2^32 threads, more than it runs: `first` is a launch's first token.
__global__ __launch_bounds__(1024) void ce_join_kernel(const float2* __restrict__ stats, int groups, int first, int T,
                                                       const void* __restrict__ labels, bool labels64, int V,
                                                       const float* __restrict__ target, float* __restrict__ loss,
                                                       float* __restrict__ lse) {
  __shared__ float2 sm[64][17];
  const int tl = threadIdx.x & 15, part = threadIdx.x >> 4;
  const int t = first + blockIdx.x * 16 + tl;
  auto join = [](float2 a, float2 b) {
    const float top = fmaxf(a.x, b.x);
    return make_float2(top, a.y * __builtin_amdgcn_exp2f(a.x - top) + b.y * __builtin_amdgcn_exp2f(b.x - top));
  };
  float2 a = make_float2(NONE, 0.0f);
  if (t < T) {
    constexpr int AHEAD = 8;
    for (int g = part; g < groups; g += 64 * AHEAD) {
      float2 x[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k)
        x[k] = g + 64 * k < groups ? stats[(int64_t)(g + 64 * k) * T + t] : make_float2(NONE, 0.0f);
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) a = join(a, x[k]);
    }
  }
  sm[part][tl] = a;
  __syncthreads();
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) {
    if (part < d) sm[part][tl] = join(sm[part][tl], sm[part + d][tl]);
    __syncthreads();
  }
  if (part == 0 && t < T) {
    a = sm[0][tl];
    const float l = a.x * LN2 + logf(a.y);
    const int64_t y = label_at(labels, labels64, t);
    lse[t] = l;
    loss[t] = y >= 0 && y < V ? l - target[t] : 0.0f;
  }
}

// max |dloss| over the tokens with a target (POLICY: of both gradients, and that times
// the logits' scale), for more than GMAX_WAVE tokens
template <bool POLICY>
__global__ __launch_bounds__(1024) void ce_gmax_kernel(const float* __restrict__ dloss, const float* __restrict__ dentropy,
                                                       const void* __restrict__ labels, bool labels64, int V, int T,
                                                       float scale, float* __restrict__ gmax) {
  __shared__ float sm[16];
  float m = POLICY ? max_policy(dloss, dentropy, labels, labels64, V, T, threadIdx.x, 1024)
                   : max_dloss(dloss, labels, labels64, V, T, threadIdx.x, 1024);
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 16; ++w) m = fmaxf(m, sm[w]);
    gmax[0] = m;
    if (POLICY) gmax[1] = m * scale;
  }
}

template <int N>
struct Count {
  static constexpr int value = N;
};
// C[row][a] = Cin[row][a] (if any) + the sum over the parts, 4 columns a thread;
// Cin [rows][ldcin] may be C itself.  FEW: so many parts, or 0 for more than 8: all loads of up
// to 8 parts in flight.  (With a count that only the launch knows 2 to 4 parts took 2 to 9% longer, one
// part after the other 6, 7 and 16 parts 15, 5 and 25 to 48%.  3 parts of 4096 x 2560: 24.6 us, 6 TB/s.)
template <int FEW>
__global__ __launch_bounds__(256) void ce_sum_kernel(const float* __restrict__ part, int splits, int64_t rows, int cols,
                                                     const float* Cin, int64_t ldcin, const float* gmax, void* C,
                                                     bool c_f32, int64_t ldc) {
  const float scale = gmax ? *gmax : 1.0f;
  const int64_t n = rows * (cols / 4);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    v4f c = ((const v4f*)part)[i];
    auto add = [&](auto count, int p, int most) {    // parts p on, `count` or the first `most` of them
      constexpr int N = decltype(count)::value;
      v4f x[N];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < most) x[k] = ((const v4f*)part)[(p + k) * n + i];
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (k < most) c += x[k];
    };
    if constexpr (FEW > 0) {
      add(Count<FEW - 1>{}, 1, FEW - 1);
    } else {
      int p = 1;
      for (; p + 8 <= splits; p += 8) add(Count<8>{}, p, 8);
      if (p < splits) add(Count<7>{}, p, splits - p);
    }
    const int64_t r = i / (cols / 4), a = (i - r * (cols / 4)) * 4;
    if (Cin) c += *(const v4f*)(Cin + r * ldcin + a);
    c *= scale;
    if (c_f32) *(v4f*)((float*)C + r * ldc + a) = c;
    else *(uint2*)((uint16_t*)C + r * ldc + a) = make_uint2(pack_bf16x2(c[0], c[1]), pack_bf16x2(c[2], c[3]));
  }
}

__global__ __launch_bounds__(256) void zero_rows_kernel(uint8_t* p, int64_t rows, int64_t len16, int64_t ld16) {
  const int64_t n = rows * len16;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / len16;
    ((uint4*)p)[r * ld16 + (i - r * len16)] = make_uint4(0u, 0u, 0u, 0u);
  }
}

int grid_for(int64_t items) {
  const int64_t b = cdiv(items, 256);
  return (int)(b < 8192 ? b : 8192);
}

// ---------------------------------------------------------------- tile shapes
// wide: 256 x 256, one block per compute unit; square: 128 x 128; flat: 128 A
// rows x 64 B rows, for few tokens or few tiles; slim: 64 x 64.
enum Tile { WIDE, SQUARE, FLAT, SLIM };
struct TileShape {
  int a, b;
};
constexpr TileShape SHAPE[] = {{256, 256}, {128, 128}, {128, 64}, {64, 64}};

// a product's launches, named by what they compute and their tile shape
using Names = const char* const[4];
#define SBN_TILE_NAMES(what) {what "_wide", what "_square", what "_flat", what "_slim"}
constexpr Names LOGITS = SBN_TILE_NAMES("ce_logits"), DLOGITS = SBN_TILE_NAMES("ce_dlogits"),
                DX = SBN_TILE_NAMES("ce_dx"), DW = SBN_TILE_NAMES("ce_dw"), SCORES = SBN_TILE_NAMES("logprob_logits"),
                DPOLICY = SBN_TILE_NAMES("logprob_dlogits");
#undef SBN_TILE_NAMES

template <int WA, int WB, int MI, int MJ, int RING, int EPI, bool TRA, bool TRB>
hipError_t run_gemm(const char* name, const GemmArgs& P, hipStream_t st) {
  constexpr int TA = WA * MI * 16, TB = WB * MJ * 16;
  constexpr size_t lds = (size_t)RING * (TA + TB) / 2 * BK * 2;
  constexpr int per_cu = (int)((160 << 10) / lds);
  static OncePerDevice once;
  int device = 0;
  hipError_t e = hipGetDevice(&device);
  if (e == hipSuccess)
    e = once(device, [] {
      return hipFuncSetAttribute((const void*)ce_gemm_kernel<WA, WB, MI, MJ, RING, EPI, TRA, TRB>,
                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    });
  if (e != hipSuccess) return e;
  const int64_t work = (int64_t)P.tilesA * P.tilesB * P.splits;
  SBN_LAUNCH(name, (ce_gemm_kernel<WA, WB, MI, MJ, RING, EPI, TRA, TRB>), dim3((unsigned)(work < per_cu * CUS ? work : per_cu * CUS)),
             dim3(64 * WA * WB), lds, st, P);
  return hipGetLastError();
}

template <int EPI, bool TRA = false, bool TRB = false>
hipError_t gemm(Names& names, Tile tile, GemmArgs& P, hipStream_t st) {
  P.tilesA = (int)cdiv(P.nA, SHAPE[tile].a);
  P.tilesB = (int)cdiv(P.nB, SHAPE[tile].b);
  const char* name = names[tile];
  switch (tile) {
    case WIDE: return run_gemm<2, 4, 8, 4, 5, EPI, TRA, TRB>(name, P, st);   // WB as in logit_norms()
    case SQUARE: return run_gemm<2, 2, 4, 4, 5, EPI, TRA, TRB>(name, P, st);
    case SLIM:
      if constexpr (EPI == EPI_SCORE || EPI == EPI_SCORE_TOPS || EPI == EPI_SCORE_TOPS8 || EPI == EPI_POLICY || EPI == EPI_POLICY_PAIR)
        return run_gemm<2, 2, 2, 2, 5, EPI, TRA, TRB>(name, P, st);
    default: return run_gemm<4, 1, 2, 4, 5, EPI, TRA, TRB>(name, P, st);
  }
}

int64_t tiles_of(Tile t, int64_t a, int64_t b) { return cdiv(a, SHAPE[t].a) * cdiv(b, SHAPE[t].b); }

// The tile shape of a product and the parts its contraction is split into
// (splittable: 1 .. `most`), by their estimated time in stages of a wide tile (1.45 us):
//   sum of rounds (stages x stage + start, with parts + 1 or 2), with parts + 2 + (2 parts + 1) a b 6.1e-7
// A compute unit runs one wide block or two of the others.  stage is that of a
// round that fills the machine; where at most one block of two runs on each
// unit, `alone`; of wide tiles it falls to 0.75 as units are idle and the clocks
// higher; flat ones take longer with transposing reads.  The last terms are the
// sum's launch and the parts' way through memory at 4.5 TB/s.
// Both sides measured: dX of 4096 tokens, 65536 entries, K = 2560 (160 wide tiles
// on 256 units) with its D in 1, 2, 3, 4 parts 2.40, 2.48, 2.23, 2.31 ms
// (estimated 2.38, 2.48, 2.19, 2.32).  Loss of 128 tokens, 1000 entries, K = 4096:
// square 34.3 us, flat 27.9; of 200, 32001, 2560: wide 54.5, square 44.4, flat
// 57.3; of 600, 20000, 4096: wide 94, square 109.
struct Choice {
  Tile tile;
  int splits;
};
Choice pick(int64_t a, int64_t b, int64_t steps, bool splittable, int most = 16) {
  const double STAGE[] = {1.0, 0.7, splittable ? 0.54 : 0.44}, ALONE[] = {1.0, 0.33, splittable ? 0.27 : 0.22};
  constexpr double START[] = {6.0, 5.0, 4.0}, PARTS[] = {2.0, 1.0, 1.0};
  Choice best{WIDE, 1};
  double least = 0;
  for (const Tile t : {WIDE, SQUARE, FLAT}) {
    const int slots = t == WIDE ? CUS : 2 * CUS;
    const int64_t n = tiles_of(t, a, b);
    for (int s = 1; s <= (splittable ? most : 1) && (s == 1 || steps / s >= 16); s += s < 16 ? 1 : s / 4) {
      const int64_t full = n * s / slots, rest = n * s % slots;
      double stage = (double)full * STAGE[t];
      if (rest) stage += rest > CUS ? STAGE[t] : ALONE[t] * (t == WIDE ? 0.75 + 0.25 * (double)rest / CUS : 1.0);
      double time = stage * (double)cdiv(steps, s) + (double)(full + (rest > 0)) * (START[t] + (s > 1 ? PARTS[t] : 0.0));
      if (s > 1) time += 2.0 + (2 * s + 1) * (double)a * (double)b * 6.1e-7;
      if (least == 0 || time < least) best = {t, s}, least = time;
    }
  }
  return best;
}

struct CePlan {
  int64_t tpad;                        // tokens along a contraction
  int64_t piece;                       // vocabulary entries of one piece, a multiple of 256
  int64_t pieces;
  Choice x, w;                         // of dX, split over the piece, and dW, split over the tokens
  size_t gmax, d, acc, part, total;
};

// pair: D in two bf16 numbers; twin_x, twin_w: both in one product, of twice the stages
CePlan ce_plan(int64_t T, int64_t V, int64_t K, bool pair, bool twin_x = false, bool twin_w = false) {
  CePlan L;
  L.tpad = round_up(T, 64);
  int64_t most = D_ELEMS / (pair ? 2 : 1) / L.tpad / 256 * 256;
  if (most < 256) most = 256;
  const int64_t vpad = round_up(V, 256);
  L.pieces = cdiv(vpad, most);
  L.piece = round_up(cdiv(vpad, L.pieces), 256);
  L.pieces = cdiv(V, L.piece);
  // few tokens leave few tiles, and two numbers twice the stages: more parts (dX and their sum, 8 tokens
  // of 32001 entries, K = 2560: 42 + 5 -> 32 + 4.5 us; 2 of 47758, K = 320: 41 + 6 -> 14.5 + 5.7)
  L.x = pick(K, T, L.piece / BK * (twin_x ? 2 : 1), true, twin_x && T <= PAIR_TOKENS ? 64 : 16);
  L.w = pick(K, L.piece, L.tpad / BK * (twin_w ? 2 : 1), true);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.gmax = take(2 * sizeof(float));
  L.d = take((size_t)L.tpad * L.piece * 2 * (pair ? 2 : 1));
  L.acc = take(L.pieces > 1 || pair ? (size_t)T * K * 4 : 0);
  const size_t px = L.x.splits > 1 ? (size_t)L.x.splits * T * K * 4 : 0;
  const size_t pw = L.w.splits > 1 ? (size_t)L.w.splits * L.piece * K * 4 : 0;
  L.part = take(px > pw ? px : pw);
  L.total = o;
  return L;
}

// C [nB][ldc] = Cin + A B^T, split as P says and summed
template <bool TRB>
hipError_t product(Names& names, Tile tile, GemmArgs P, bool c_f32, float* part, hipStream_t st) {
  if (P.splits == 1) {
    if (TRB && P.Cin) return gemm<EPI_ADD32, true, TRB>(names, tile, P, st);
    if (P.twin) return c_f32 ? gemm<EPI_TWIN32, true, TRB>(names, tile, P, st) : gemm<EPI_TWIN16, true, TRB>(names, tile, P, st);
    return c_f32 ? gemm<EPI_OUT32, true, TRB>(names, tile, P, st) : gemm<EPI_OUT16, true, TRB>(names, tile, P, st);
  }
  GemmArgs Q = P;                                    // the parts' sums side by side
  Q.C = part, Q.ldc = P.nA, Q.part_stride = (int64_t)P.nB * P.nA;
  Q.Cin = nullptr, Q.gmax = nullptr;
  const hipError_t e = P.twin ? gemm<EPI_TWIN32, true, TRB>(names, tile, Q, st) : gemm<EPI_OUT32, true, TRB>(names, tile, Q, st);
  if (e != hipSuccess) return e;
  constexpr decltype(&ce_sum_kernel<0>) FEW[] = {ce_sum_kernel<2>, ce_sum_kernel<3>, ce_sum_kernel<4>, ce_sum_kernel<5>,
                                                 ce_sum_kernel<6>, ce_sum_kernel<7>, ce_sum_kernel<8>};
  SBN_LAUNCH("ce_sum", (P.splits <= 8 ? FEW[P.splits - 2] : ce_sum_kernel<0>), dim3((unsigned)grid_for((int64_t)P.nB * (P.nA / 4))), dim3(256), 0, st, part,
             P.splits, (int64_t)P.nB, P.nA, P.Cin, P.ldcin, P.gmax, P.C, c_f32, P.ldc);
  return hipGetLastError();
}

Tile stats_tile(int64_t T, int64_t V, int64_t K) { return pick(V, T, K / BK, false).tile; }
int64_t groups_of(Tile t, int64_t V) { return cdiv(V, SHAPE[t].a) * (t == FLAT ? 4 : 2); }
int64_t stats_groups(int64_t T, int64_t V, int64_t K) { return groups_of(stats_tile(T, V, K), V); }

// Of log probabilities' logits and their D: where flat tiles are at most one a unit, twice as
// many of half the entries (us: 37 tokens of 32001 entries, K = 4096, 59.6 -> 57.5, D of K =
// 2560 32.5 -> 29.3; 17 of 3953, 1792 15.6 -> 13.3 and 17.8 -> 13.0; 126 of 1315, 3456 25.7 -> 22.7
// and 27.2 -> 18.8; where there are more than units, 1 of 50001, 2560 49.9 -> 52.3).  The loss
// keeps its tiles, and so its sums' order.
Tile score_tile(int64_t T, int64_t V, int64_t K) {
  const Tile t = stats_tile(T, V, K);
  return t == FLAT && tiles_of(FLAT, V, T) <= CUS ? SLIM : t;
}

}  // namespace

size_t ce_ws_bytes(int64_t T, int64_t V, int64_t K) {
  return align256((size_t)T * sizeof(float)) + align256((size_t)stats_groups(T, V, K) * T * sizeof(float2));
}

hipError_t launch_ce(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* labels,
                     bool labels64, int64_t T, int64_t V, int64_t K, float* loss, float* lse, void* ws,
                     hipStream_t st) {
  GemmArgs P{};
  P.A = W, P.lda = ldw, P.nA = P.mA = (int)V;
  P.B = X, P.ldb = ldx, P.nB = P.mB = (int)T;
  P.steps = (int)(K / BK), P.splits = 1;
  P.labels = labels, P.labels64 = labels64, P.V = (int)V;
  P.target = (float*)ws;
  P.stats = (float2*)((uint8_t*)ws + align256((size_t)T * sizeof(float)));
  const hipError_t e = gemm<EPI_STATS>(LOGITS, stats_tile(T, V, K), P, st);
  if (e != hipSuccess) return e;
  constexpr int64_t JOIN_TOKENS = 1 << 24;           // of a launch
  const int groups = (int)stats_groups(T, V, K);
  for (int64_t t = 0; t < T; t += JOIN_TOKENS)
    SBN_LAUNCH("ce_join", ce_join_kernel, dim3((unsigned)cdiv(T - t < JOIN_TOKENS ? T - t : JOIN_TOKENS, 16)), dim3(1024), 0,
               st, P.stats, groups, (int)t, (int)T, labels, labels64, (int)V, P.target, loss, lse);
  return hipGetLastError();
}

// Of a token's tops: the fragments of 16 entries that a wave holds, and the sets.
LogitTops logit_tops(int64_t T, int64_t V, int64_t K, int top) {
  const Tile t = score_tile(T, V, K);
  const int mi_log2 = t == WIDE ? 3 : t == SQUARE ? 2 : 1;
  const int64_t near = top + 3, rows_spared = near * near * K * (T * V < int64_t(1) << 26 ? 2048 : 1024);
  const int of_log2 = rows_spared > V * V ? 3 : tops_of(1 << mi_log2) == 32 ? 5 : 4;
  return {mi_log2, of_log2, (int)((groups_of(t, V) << (4 + mi_log2)) >> of_log2)};
}

hipError_t launch_logits(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const void* tokens, bool tokens64,
                         int64_t T, int64_t all, int64_t V, int64_t K, float scale, float* target, float2* stats, float* mean,
                         float2* tops, float* norms, const LogitTops& sets, hipStream_t st) {
  GemmArgs P{};
  P.A = W, P.lda = ldw, P.nA = P.mA = (int)V;
  P.B = X, P.ldb = ldx, P.nB = P.mB = (int)T;
  P.steps = (int)(K / BK), P.splits = 1;
  P.labels = tokens, P.labels64 = tokens64, P.V = (int)V;
  P.target = target, P.stats = stats, P.mean = mean, P.tops = tops, P.norms = norms;
  P.ldt = sets.groups;
  P.scale = scale, P.none = logit_none(scale);
  const Tile t = score_tile(all, V, K);
  if (!tops) return gemm<EPI_SCORE>(SCORES, t, P, st);
  return sets.of_log2 == 3 ? gemm<EPI_SCORE_TOPS8>(SCORES, t, P, st) : gemm<EPI_SCORE_TOPS>(SCORES, t, P, st);
}
int logit_norms(int64_t T, int64_t V, int64_t K) {
  const Tile t = score_tile(T, V, K);
  return t == WIDE ? 4 : t == FLAT ? 1 : 2;
}
int64_t logit_groups(int64_t T, int64_t V, int64_t K) { return groups_of(score_tile(T, V, K), V); }

size_t ce_bwd_ws_bytes(int64_t T, int64_t V, int64_t K, bool pair) { return ce_plan(T, V, K, pair).total; }
namespace {
CePlan policy_plan(int64_t T, int64_t V, int64_t K, bool fine_x, bool fine_w) {
  const bool few = T <= PAIR_TOKENS;
  return ce_plan(T, V, K, few || fine_x || fine_w, few || fine_x, few || fine_w);
}
}  // namespace
size_t policy_bwd_ws_bytes(int64_t T, int64_t V, int64_t K, bool fine_x, bool fine_w) {
  return policy_plan(T, V, K, fine_x, fine_w).total;
}

hipError_t launch_ce_backward(const uint16_t* X, int64_t ldx, const uint16_t* W, int64_t ldw, const HeadGrad& H, int64_t T,
                              int64_t V, int64_t K, void* dX, sbn_dtype dxdt, int64_t lddx, void* dW, sbn_dtype dwdt,
                              int64_t lddw, void* ws, hipStream_t st) {
  const bool dx_f32 = dxdt != SBN_BF16, dw_f32 = dwdt != SBN_BF16;
  // a second product, added to the first one's, or one of both numbers
  const bool dx_pair = dX && dxdt == SBN_F32_FINE, dw_pair = dW && dwdt == SBN_F32_FINE, few = H.policy && T <= PAIR_TOKENS,
             pair = dx_pair || dw_pair || few;
  const CePlan L = H.policy ? policy_plan(T, V, K, dx_pair, dw_pair) : ce_plan(T, V, K, pair);
  uint8_t* w = (uint8_t*)ws;
  uint16_t* D = (uint16_t*)(w + L.d);
  float *acc = (float*)(w + L.acc), *part = (float*)(w + L.part), *gmax = (float*)(w + L.gmax);
  float* factor = H.policy ? gmax + 1 : gmax;        // of both products' sums
  const int64_t dlow = L.tpad * L.piece;
  hipError_t e;
  if (T > GMAX_WAVE) {
    if (H.policy)
      SBN_LAUNCH("logprob_gmax", ce_gmax_kernel<true>, dim3(1), dim3(1024), 0, st, H.dloss, H.dentropy, H.labels, H.labels64,
                 (int)V, (int)T, H.scale, gmax);
    else
      SBN_LAUNCH("ce_gmax", ce_gmax_kernel<false>, dim3(1), dim3(1024), 0, st, H.dloss, (const float*)nullptr, H.labels,
                 H.labels64, (int)V, (int)T, 1.0f, gmax);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  for (int64_t i = 0; i < L.pieces; ++i) {
    const int64_t v0 = i * L.piece, nv = V - v0 < L.piece ? V - v0 : L.piece;
    const int64_t vpad = round_up(nv, 64);           // contraction of dX over this piece
    GemmArgs G{};
    G.A = W + v0 * ldw, G.lda = ldw, G.nA = G.mA = (int)nv;
    G.B = X, G.ldb = ldx, G.nB = G.mB = (int)T;
    G.steps = (int)(K / BK), G.splits = 1;
    G.labels = H.labels, G.labels64 = H.labels64, G.v0 = (int)v0, G.V = (int)V;
    G.lse = H.lse, G.dloss = H.dloss, G.gmax = gmax;
    G.scale = H.scale, G.entropy = H.entropy, G.dentropy = H.dentropy;
    G.D = D, G.ldd = L.piece, G.dlow = dlow, G.tpad = (int)L.tpad;
    const Tile tile = H.policy ? score_tile(T, nv, K) : stats_tile(T, nv, K);
    if (H.policy) e = pair ? gemm<EPI_POLICY_PAIR>(DPOLICY, tile, G, st) : gemm<EPI_POLICY>(DPOLICY, tile, G, st);
    else e = pair ? gemm<EPI_GRAD_PAIR>(DLOGITS, tile, G, st) : gemm<EPI_GRAD>(DLOGITS, tile, G, st);
    if (e != hipSuccess) return e;
    for (int low = 0; dX && low <= (int)(dx_pair && !H.policy); ++low) {
      GemmArgs P{};
      P.A = W + v0 * ldw, P.lda = ldw, P.nA = P.mA = (int)K, P.kA = (int)nv;
      P.B = D + low * dlow, P.ldb = L.piece, P.nB = P.mB = (int)T;
      P.steps = (int)(vpad / BK), P.splits = L.x.splits <= P.steps ? L.x.splits : P.steps;
      const bool last = i + 1 == L.pieces && low == (int)(dx_pair && !H.policy);
      P.twin = H.policy && (few || dx_pair) ? 2 * dlow : 0;
      P.Cin = i > 0 || low > 0 ? acc : nullptr, P.ldcin = K;
      P.gmax = last ? factor : nullptr;
      P.C = last ? dX : acc, P.ldc = last ? lddx : K;
      if ((e = product<false>(DX, L.x.tile, P, last ? dx_f32 : true, part, st)) != hipSuccess) return e;
    }
    for (int low = 0; dW && low <= (int)(dw_pair && !H.policy); ++low) {
      GemmArgs P{};
      P.A = X, P.lda = ldx, P.nA = P.mA = (int)K, P.kA = (int)T;
      P.B = D + low * dlow, P.ldb = L.piece, P.nB = (int)nv, P.mB = (int)vpad, P.kB = (int)L.tpad;
      P.steps = (int)(L.tpad / BK), P.splits = L.w.splits;
      P.C = (uint8_t*)dW + v0 * lddw * (dw_f32 ? 4 : 2), P.ldc = lddw;
      P.Cin = low > 0 ? (const float*)P.C : nullptr, P.ldcin = lddw;
      P.twin = H.policy && (few || dw_pair) ? 2 * dlow : 0;
      P.gmax = low == (int)(dw_pair && !H.policy) ? factor : nullptr;
      if ((e = product<true>(DW, L.w.tile, P, dw_f32, part, st)) != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

hipError_t launch_zero_rows(void* p, int64_t rows, int64_t len, int64_t ld, int elem_bytes, hipStream_t st) {
  const int64_t l16 = len * elem_bytes / 16;
  SBN_LAUNCH("zero_rows", zero_rows_kernel, dim3((unsigned)grid_for(rows * l16)), dim3(256), 0, st, (uint8_t*)p, rows,
             l16, ld * elem_bytes / 16);
  return hipGetLastError();
}

}  // namespace sbn
