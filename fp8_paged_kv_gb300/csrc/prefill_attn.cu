// prefill_attn.cu -- attention of several query tokens per request over an e4m3
// cache with block scales, on the fifth-generation tensor cores: chunks of prompts
// and drafted tokens (causal), or an encoder's states (all tokens).
//
// The rows of a request and kv head are its query tokens' heads that read it (token
// by token, the heads of a group one after another): one read of a block of K and V
// serves 256 rows, and a causal border crosses few blocks (32 tokens at 8 heads per
// group).  Two or three launches, each a dependent of the one before:
//   plan    dead requests, the work list (one CTA; of up to 32 requests and some 16384
//           rows a warp of every CTA of the next launch makes its part of the list itself)
//   attn    the list, a CTA per SM
//   merge   rows whose unit was cut between CTAs, by log-sum-exp
//
// * Unit: up to 256 rows of one (request, kv head) over the tokens that its last
//   row sees.  Units are laid end to end in cost (blocks of 128 tokens, dearer for
//   units of more than 128 rows, and a start), the kv heads one after another, and
//   the line is cut into one equal range per CTA.  A unit that lies within a range
//   is answered by its CTA; of the others every piece leaves a partial (m, l, O),
//   merged in a fixed order: repeated calls give the same bits.  Where whole units,
//   as many to each CTA, come out sooner than cut ones and their merge, none is cut.
//
// Piece pipeline (one CTA per SM, 16 warps), per block of 128 tokens:
//   warp 15     finds the pieces and the blocks' scales ahead of the others
//   warp 12     lands K rows (128-byte swizzle) by a tensor map
//   warps 8-11  V codes from the pool to f16 core matrices (exact), a block ahead in
//               registers, zeroes where no token lies; and, some after each block, the
//               next piece's queries: q 2^e as two e4m3 parts
//   warps 13, 14  issue S = Q K^T (e4m3, over both parts against the same K rows) and
//               O += P V (f16) of row tile 0 and 1, tcgen05.mma of M = N = 128
//   warps 0-3, 4-7  softmax of row tile 0 and 1, a thread per row: no shuffles.  P
//               (two f16 parts, in the columns of the scores it came from) is the A operand
// Units of more than 128 rows use both tiles on every block; smaller ones give the
// two tiles alternate blocks of the same rows, joined at the end in tensor memory.
//
// What bounds it: a row tile's chain.  Of 128 tokens its scores take 569 cycles of products, its softmax some 2700
// (powers, 4 cycles each for a warp, the weights' second parts, and one warp's latencies), the products of the second
// half's weights 570, and the next scores overwrite those weights: about 3900, in which both tiles' products are 3420.
// Replayed from a graph, 64/8 heads: a prompt of 8192 tokens 990 us (1110 TFLOP/s, 58 % of a plain library product's
// rate; 965 where calls share their inputs), 8192 rows over all of 8192 tokens 1870 us (1180), the last 1024 of 32768
// 950 us (1140).  Few rows: a start (list, queries, pipeline; 6 us), some 2300 cycles for 128 tokens, an end (3 us):
// 16 requests of 4 tokens over 2048 33 us, 4 tokens over 131072 85 us.  Short prompts: queries in, results out and the
// piece's start and end come on top (16 x 512: 212 us, of which some 40 go when neither queries nor results touch HBM).
//
// Scales.  Of each tile of 16 tokens (16 columns of S) K's scale multiplies the
// scores and V's goes into the weights: with ev its exponent, P = 2^(s + ev - m + 7),
// m the largest s + ev (within 2^8), so that the weights that meet V's codes use f16's
// range (up to 2^15) whatever the order of the scales; the sum takes P 2^(-ev - 7),
// which is 2^(s - m), and O is taken back by 2^-7 on its way out.
//
// Weights are two f16 parts, rounded, and what that left, as in the framework's other
// attention: 2^-22 of a weight is lost, or 2^-32 of the largest where that is more.
// With one part 2^-11 of each was: where values cancel, results were 4 times outside
// what two parts allow, beside a block whose V scale is 2^24 as large 9 times.  It
// cost a prompt of 8192 tokens 763 -> 953 us (three quarters of that the products), 4 tokens
// over 131072 79 -> 87, 16 x 4 over 2048 29 -> 34.
//
// Tokens that a row does not see have no part in it: their scores become -inf before
// anything is taken from them, and where a block holds tokens that only some rows
// see, their V codes that are NaN become 0 (0 NaN = NaN) and the rows that do see
// them are given the NaN afterwards.
#include <atomic>

#include "block_scale.cuh"
#include "tc_attn.cuh"

namespace fpk {
namespace {

constexpr int kChTile = 16;
constexpr int kChDim = 128;
constexpr int kChGroupMax = 8;
constexpr int kChBlk = 128;  // tokens of a block
constexpr int kChBlkTiles = kChBlk / kChTile;
constexpr int kChUnitRows = 256;
constexpr float kChLog2e = 1.4426950408889634f;
constexpr float kChLn2 = 0.6931471805599453f;
constexpr float kChGrow = 8.f;  // log2 growth of a maximum that rescales O
// Blocks of a row tile (a power of two) after which O leaves tensor memory and begins anew: the tensor cores cut the last
// bits of every sum off.  (A row of 131072 tokens: 8.2e-4 of it without, 5.5e-5 now; 32: 2 % more time.  1024 rows of
// 32768 940 -> 964 us.)
constexpr int kChFold = 64;
constexpr int kChLift = 7;      // log2 of a weight with the score m: up to 2^15 with that growth, which f16 holds
constexpr float kChMinMult = 1e-37f;  // of a row's scale times K's: -inf times it is -inf still
__device__ __forceinline__ float at_least_min(float mult) { return mult < kChMinMult ? kChMinMult : mult; }  // (a NaN stays one)
// Costs in the work list, in some 600 cycles: of a block with both tiles at work and with one, of a unit's start.  (8 and 5,
// 7 and 4, or starts of 24 and 20: within 2 % where many units are cut, 3 requests of 300 rows over 1000 55 -> 64 us.)
constexpr int kChCostPair = 6, kChCostSolo = 4;
constexpr int kChStartPair = 20, kChStartSolo = 16;
// What cutting units costs a call: another start, partials, their merge (16 requests of 4 tokens over 2048: 37.2 us cut,
// 33.0 whole; 24 of them, 2 units to a CTA then: 48.5 cut, 54.5 whole; 3 of 300 over 1000: 62.4 and 55.5; cut by this rule
// although whole ones would be sooner: 16 prompts of 512, 212 and 190).
constexpr int kChCut = 48;

constexpr int kChThreads = 512;
constexpr int kChVWarp = 8, kChLoadWarp = 12, kChMmaWarp = 13, kChPlanWarp = 15;
constexpr int kChPieces = 4;  // pieces known ahead
constexpr int kChPlanThreads = 1024;
constexpr int kChTurnSpins = 4096;
// Merge: CTAs per cut unit, few where a call has few rows, or its requests on average.  (4 instead of 16: 16 requests of
// 32 rows over 2048 tokens 35.0 -> 33.1 us, one token over 4096 22.1 -> 20.7, 16 tokens over 16 18.6 -> 16.5; 512 rows over
// 4000 39.6 -> 56.3.)  An average says little of a batch of drafts and a chunk: with 128 for both, 60 drafts of 32 rows and
// a chunk of 4000 rows took 190.8 us instead of 180.5, 20 and one of 1600 98.5 instead of 92.2; 8 of 128 rows lose 33.2 -> 34.9.
constexpr int kChMergeWarps = 8, kChMergeFew = 4, kChMergeMany = 16, kChMergeAll = 128, kChMergeMean = 64;
constexpr int kChNear = 1024, kChNearUnits = 4096;    // requests and units that the plan keeps in shared memory
constexpr int64_t kChSmallRows = 16384, kChSmallPages = 32768;  // of a kv head's rows, and page table entries, without a plan

struct alignas(16) ChUnit {
  int y;       // place in a kv head's line
  int r;
  int row0, rows;  // of the request's rows
  int tokens;  // that its last row sees
  int c0;      // the request's first query token
  int behind;  // query tokens behind the first one, of those that see fewer: token t sees L - max(0, behind - t), or none
  int L;       // 0: dead
};
static_assert(sizeof(ChUnit) == 32, "two 16-byte words");

// A CTA's range [b0, b1), its first unit, and the unit that it begins and others end (cut >= 0: up to CTA cut).
struct alignas(16) ChStart {
  int unit, h, b0, b1;
  ChUnit u;
  int units, T;    // of a kv head
  int cut, cut_h;
  ChUnit cut_u;
};
static_assert(sizeof(ChStart) == 96, "six 16-byte words");

struct ChArgs {
  const uint16_t* q;
  const int32_t* cu_seqlens;
  const uint16_t* kv_scales;
  const uint8_t* kv_pool;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const uint8_t* abort_mask;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  int32_t* base;    // [B + 1] first unit of each request
  int32_t* dead;    // [B]
  ChUnit* unit;
  ChStart* start;   // [ctas]
  float2* part_ml;  // partials: [2 ctas][256 rows]
  float* part_o;
  int small;        // without a plan
  int boxed;        // 32 rows are whole tokens' heads: results go out by tensor map
  int most;         // units of a kv head that there can be
  int n_tokens, causal, B, Hq, Hkv, G, page_size, num_pages, max_pages, ctas, zbox;
  uint32_t by_g, by_tpp;
  float sm_scale_log2;
};

constexpr int kNanRow = -128;  // exponent of a row with a NaN or an infinity

struct ChCfg {
  static constexpr int kQTile = 128 * 256;  // both parts of a tile's queries
  static constexpr int kKStage = kChBlk * kChDim, kV16 = 2 * kKStage;
  static constexpr int kQTiles = 4;         // of this piece and the next
  static constexpr int kKStages = 2, kV16Bufs = 2;
  static constexpr int kScales = 8;         // blocks whose scales are known
  static constexpr int kNan = 16;           // pieces with a flag of NaN values
  static constexpr int kPieceBytes = 64 + 32 * 4;
  static constexpr int kOffK = kQTiles * kQTile;
  static constexpr int kOffV16 = kOffK + kKStages * kKStage;
  static constexpr int kOffPiece = kOffV16 + kV16Bufs * kV16;
  static constexpr int kOffScale = kOffPiece + kChPieces * kPieceBytes;  // float2 [kScales][8]: K's factor, V's exponent
  static constexpr int kOffTile = kOffScale + kScales * kChBlkTiles * 8;  // int [kScales][8]: the pool's tiles (0 behind the last)
  static constexpr int kOffMult = kOffTile + kScales * kChBlkTiles * 4;
  static constexpr int kOffBars = kOffMult + kQTiles * 128;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKFree = kBarKFull + kKStages;
  static constexpr int kBarReady = kBarKFree + kKStages;       // converted V block
  static constexpr int kBarUsed = kBarReady + kV16Bufs;        // .. read by the MMA
  static constexpr int kBarS = kBarUsed + kV16Bufs;            // [tile]
  static constexpr int kBarP = kBarS + 2;                      // [tile][half of the block]
  static constexpr int kBarO = kBarP + 4;                      // [tile] a block's product added to O
  static constexpr int kBarHalf = kBarO + 2;                   // [tile] the first half's product added
  static constexpr int kBarOFree = kBarHalf + 2;               // [tile] O of a piece read
  static constexpr int kBarQ = kBarOFree + 2;                  // [buffer] queries staged
  static constexpr int kBarQFree = kBarQ + kQTiles;            // [buffer] queries of a piece read
  static constexpr int kBarPiece = kBarQFree + kQTiles;        // [kChPieces] piece known
  static constexpr int kBarPieceFree = kBarPiece + kChPieces;  // [kChPieces] piece read by every warp
  static constexpr int kBarScale = kBarPieceFree + kChPieces;  // [kScales] a block's scales known
  static constexpr int kBarScaleFree = kBarScale + kScales;    // [kScales] .. read
  static constexpr int kBarJoin = kBarScaleFree + kScales;     // tile 1's state of a unit of one row tile
  static constexpr int kBarDone = kBarJoin + 1;                // [2] every MMA of a warp completed
  static constexpr int kBars = kBarDone + 2;
  static constexpr int kOffMisc = kOffBars + 8 * kBars;        // tensor memory base, failure flag, turns of the tiles, NaN flags
  static constexpr int kSmem = kOffMisc + 16 + kNan;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// Context length of request r if it is alive by its length and abort flag, else 0.
__device__ __forceinline__ int live_length(const ChArgs& a, int r) {
  const int L = __ldg(a.seq_lens + r);
  if (L <= 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_pages) * a.page_size) return 0;
  if (a.abort_mask != nullptr && __ldg(a.abort_mask + r) != 0) return 0;
  return L;
}
// First query token of request r, and behind its last (r = B: the end).
__device__ __forceinline__ int query_start(const ChArgs& a, int r) {
  return min(max(__ldg(a.cu_seqlens + r), 0), a.n_tokens);
}
// (L may be near 2^31: nothing is added to it)
__device__ __forceinline__ int seen(const ChUnit& u, int token) { return max(0, u.L - max(0, u.behind - token)); }

// ---------------------------------------------------------------------------
// work list
// ---------------------------------------------------------------------------
__device__ __forceinline__ int blocks_of(int tokens) { return (tokens + kChBlk - 1) / kChBlk; }
__device__ __forceinline__ int block_cost(int rows) { return rows > 128 ? kChCostPair : kChCostSolo; }
__device__ __forceinline__ int start_cost(int rows) { return rows > 128 ? kChStartPair : kChStartSolo; }
__device__ __forceinline__ int unit_cost(const ChUnit& u) { return start_cost(u.rows) + block_cost(u.rows) * blocks_of(u.tokens); }
// Blocks [i0, i1) of a unit at place y that a range [b0, b1) owns: those that start in it.
__device__ __forceinline__ void owned_blocks(const ChUnit& u, int y, int b0, int b1, int& i0, int& i1) {
  const int w = block_cost(u.rows), n = blocks_of(u.tokens), at = y + start_cost(u.rows);
  const int lo = max(b0 - at, 0) + w - 1, hi = max(b1 - at, 0) + w - 1;
  i0 = min(n, w == kChCostPair ? lo / kChCostPair : lo / kChCostSolo);
  i1 = min(n, w == kChCostPair ? hi / kChCostPair : hi / kChCostSolo);
}
__device__ __forceinline__ ChUnit load_unit(const ChUnit* at) {
  const int4* p = reinterpret_cast<const int4*>(at);
  const int4 x = __ldcg(p), y = __ldcg(p + 1);
  return {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}

__device__ __forceinline__ ChUnit near_unit(const int4& x, const int4& y) { return {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w}; }

// CTA c owns [begin(c), begin(c + 1)) of the line: its length / n, one more for the first (its length mod n) CTAs.
struct ChRanges {
  int share, more;
  __device__ __forceinline__ int begin(int c) const { return c * share + min(c, more); }
  __device__ __forceinline__ int owner(int y) const {
    const int big = more * (share + 1);
    return y < big ? y / (share + 1) : more + (y - big) / share;
  }
};
__device__ __forceinline__ ChRanges ranges_of(int line, int n) {
  ChRanges r;
  r.share = line / n;
  r.more = line - r.share * n;
  return r;
}

// Whether the units, the dearest of which costs `top`, are dealt out whole, as many to each CTA: the ranges end with
// units then.
__device__ __forceinline__ bool uncut(const ChArgs& a, int units, int T, int top) {
  const int all = units * a.Hkv;
  return (all + a.ctas - 1) / a.ctas * top <= T * a.Hkv / a.ctas + kChCut;
}

// Sums of a CTA's threads: the sum of the threads before, and of all.
__device__ __forceinline__ int block_scan(int mine, int& all, int* s_sum) {
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  __syncthreads();  // (s_sum's last readers)
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int sums = s_sum[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, sums, o);
    if (lane >= o) sums += v;
  }
  const int below = __shfl_sync(kFull, sums, max(warp - 1, 0));
  all = __shfl_sync(kFull, sums, 31);
  return incl - mine + (warp > 0 ? below : 0);
}

// The work list, and the CTAs' ranges, by one CTA.  Few dependent reads: the requests and the units' places stay in
// shared memory (where there are more than fit, in the workspace), and warps without a request of their own share the
// others' page tables.
__global__ void __launch_bounds__(kChPlanThreads, 1) prefill_plan_kernel(const ChArgs a) {
  __shared__ int s_sum[kChPlanThreads / 32];
  __shared__ int s_base[kChNear + 1], s_bad[kChNear], s_y[kChNearUnits], s_top;
  griddep_wait();
  griddep_launch_dependents();
  const unsigned kFull = 0xffffffffu;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  constexpr int kThreads = kChPlanThreads, kWarps = kThreads / 32;
  const bool near = a.B <= kChNear;
  int32_t* const base = near ? s_base : a.base;
  int32_t* const dead = near ? s_bad : a.dead;
  for (int i = t; i < min(a.B, kChNear); i += kThreads) s_bad[i] = 0;
  if (t == 0) s_top = 0;
  __syncthreads();
  // requests that are dead, by a bad page or otherwise
  const int ways = a.B < kWarps ? kWarps / a.B : 1;
#pragma unroll 1
  for (int r = warp / ways; r < a.B; r += kWarps / ways) {
    const int L = live_length(a, r), pages = L > 0 ? (L - 1) / a.page_size + 1 : 0;
    const int32_t* const row = a.page_table + static_cast<int64_t>(r) * a.max_pages;
    bool bad = L == 0;
#pragma unroll 8
    for (int i = warp % ways * 32 + lane; i < pages; i += 32 * ways) bad |= static_cast<unsigned>(__ldg(row + i)) >= static_cast<unsigned>(a.num_pages);
    bad = __any_sync(kFull, bad);
    if (lane == 0 && (bad || !near)) dead[r] = bad;  // (with several ways the flags begin at 0)
  }
  // units of each request
  int units = 0;
  bool down = false;
#pragma unroll 1
  for (int r0 = 0; r0 < a.B; r0 += kThreads) {
    const int r = r0 + t;
    const int n = r < a.B ? query_start(a, r + 1) - query_start(a, r) : 0;
    const int rows = max(0, n) * a.G;
    down |= n < 0;
    int all;
    const int before = block_scan((rows + kChUnitRows - 1) / kChUnitRows, all, s_sum);
    if (r < a.B) base[r] = units + before;
    units = min(units + all, a.most + 1);
  }
  if (__syncthreads_or(down)) {
    // cu_seqlens that decrease: rows of several requests, and more units than the list may have places for; nothing is
    // answered.  (Without, a request's rows are its own and the units no more than a.most.)
    if (t == 0) atomicOr(a.status, kStatusBadStart);
    units = 0;
  }
  if (t == 0) base[a.B] = units;
  __syncthreads();
  // the last request whose first unit is not behind x (of empty ones the last has units)
  auto request_of = [&](int x) -> int {
    int lo = 0, hi = a.B - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (base[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
  };
  auto unit_at = [&](int x, int& r, int y) -> ChUnit {
    while (base[r + 1] <= x) ++r;
    ChUnit u;
    u.y = y;
    u.r = r;
    u.c0 = query_start(a, r);
    const int n = query_start(a, r + 1) - u.c0, rows = n * a.G;
    u.L = dead[r] ? 0 : __ldg(a.seq_lens + r);
    u.behind = a.causal ? n - 1 : 0;
    u.row0 = (x - base[r]) * kChUnitRows;
    u.rows = min(kChUnitRows, rows - u.row0);
    u.tokens = seen(u, quotient(u.row0 + u.rows - 1, a.by_g));
    return u;
  };
  // their places: each thread a run of units
  const int chunk = (units + kThreads - 1) / kThreads;
  const int x0 = min(units, t * chunk), x1 = min(units, x0 + chunk);
  const int lo = x0 < x1 ? request_of(x0) : 0;
  int mine = 0, top = 0, r = lo;
#pragma unroll 1
  for (int x = x0; x < x1; ++x) {
    const int cost = unit_cost(unit_at(x, r, 0));
    mine += cost;
    top = max(top, cost);
  }
  if (top > 0) atomicMax(&s_top, top);
  int T;
  int y = block_scan(mine, T, s_sum);
  r = lo;
#pragma unroll 1
  for (int x = x0; x < x1; ++x) {
    const ChUnit u = unit_at(x, r, y);
    a.unit[x] = u;
    if (x < kChNearUnits) s_y[x] = y;
    y += unit_cost(u);
  }
  __syncthreads();
  // the ranges, with their first unit (the last one that starts at or before it) and the one that they leave to others
  const ChRanges rg = ranges_of(T * a.Hkv, a.ctas);
  const bool whole = uncut(a, units, T, s_top);
  const ChRanges by = ranges_of(units * a.Hkv, a.ctas);
  const bool near_units = units <= kChNearUnits;
  auto unit_of = [&](int place, int& x, int& h) -> ChUnit {
    h = min(place / T, a.Hkv - 1);
    const int at = place - h * T;
    int l = 0, m = units - 1;
#pragma unroll 1
    while (l < m) {
      const int mid = (l + m + 1) >> 1;
      if ((near_units ? s_y[mid] : a.unit[mid].y) <= at) l = mid; else m = mid - 1;
    }
    x = l;
    int q = request_of(l);
    return unit_at(l, q, near_units ? s_y[l] : a.unit[l].y);
  };
  // unit `of` of all heads'
  auto place_of = [&](int of) -> int {
    const int h = of / units, x = of - h * units;
    return h == a.Hkv ? a.Hkv * T : h * T + (near_units ? s_y[x] : a.unit[x].y);
  };
#pragma unroll 1
  for (int c = t; c < a.ctas; c += kThreads) {
    ChStart s = {};
    s.b0 = !whole ? rg.begin(c) : units > 0 ? place_of(by.begin(c)) : 0;
    s.b1 = !whole ? rg.begin(c + 1) : units > 0 ? place_of(by.begin(c + 1)) : 0;
    s.units = units;
    s.T = T;
    s.cut = -1;
    if (s.b0 < s.b1) {
      s.u = unit_of(s.b0, s.unit, s.h);
      if (!whole && s.b1 < T * a.Hkv) {
        int x;
        s.cut_u = unit_of(s.b1, x, s.cut_h);
        const int at = s.cut_h * T + s.cut_u.y, blocks = blocks_of(s.cut_u.tokens);
        int i0, i1;
        owned_blocks(s.cut_u, at, s.b0, s.b1, i0, i1);
        if (i0 == 0 && i1 > 0 && i1 < blocks)
          s.cut = rg.owner(at + start_cost(s.cut_u.rows) + (blocks - 1) * block_cost(s.cut_u.rows));
      }
    }
    a.start[c] = s;
  }
}

// The list of up to 32 requests, a lane each, by a warp that keeps it in its registers.
struct ChSmall {
  int base, n, c0, L, y;  // of this lane's request: first unit, query tokens, the first of them, context (0: dead), place
  int units, T;           // of a kv head
};
// Unit i of request r, at place y.
__device__ __forceinline__ ChUnit small_unit(const ChArgs& a, const ChSmall& s, int r, int i, int y) {
  const unsigned kFull = 0xffffffffu;
  const int n = __shfl_sync(kFull, s.n, r);
  ChUnit u;
  u.r = r;
  u.y = y;
  u.c0 = __shfl_sync(kFull, s.c0, r);
  u.L = __shfl_sync(kFull, s.L, r);
  u.behind = a.causal ? n - 1 : 0;
  u.row0 = i * kChUnitRows;
  u.rows = min(kChUnitRows, n * a.G - u.row0);
  u.tokens = seen(u, quotient(u.row0 + u.rows - 1, a.by_g));
  return u;
}
// The unit behind u, x of all: of the same request, or the first of the next one that has any (of several that begin
// at x the last has units).
__device__ __forceinline__ ChUnit small_next(const ChArgs& a, const ChSmall& s, const ChUnit& u, int x) {
  const int r = 31 - __clz(__ballot_sync(0xffffffffu, s.base <= x));
  return small_unit(a, s, r, r == u.r ? u.row0 / kChUnitRows + 1 : 0, u.y + unit_cost(u));
}
__device__ __forceinline__ ChUnit small_first(const ChArgs& a, const ChSmall& s) {
  return small_unit(a, s, 31 - __clz(__ballot_sync(0xffffffffu, s.base <= 0)), 0, 0);
}
// The unit of request r behind those that end at or before place `at`, or behind the first x - its first.  A lane
// looks at a unit.
__device__ __forceinline__ ChUnit small_find(const ChArgs& a, const ChSmall& s, int r, int at, int& x) {
  const unsigned kFull = 0xffffffffu;
  const int base = __shfl_sync(kFull, s.base, r), n = __shfl_sync(kFull, s.n, r);
  int y = __shfl_sync(kFull, s.y, r), i = 0;
#pragma unroll 1
  for (int i0 = 0;; i0 += 32) {
    const ChUnit mine = small_unit(a, s, r, i0 + (threadIdx.x & 31), 0);
    const int cost = mine.rows > 0 ? unit_cost(mine) : 0;
    int ends = cost;  // of this lane's unit
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int p = __shfl_up_sync(kFull, ends, o);
      if ((threadIdx.x & 31) >= o) ends += p;
    }
    const bool behind = y + ends <= at || base + i0 + static_cast<int>(threadIdx.x & 31) < x;
    const int passed = __popc(__ballot_sync(kFull, mine.rows > 0 && behind));
    i = i0 + passed;
    y += passed > 0 ? __shfl_sync(kFull, ends, passed - 1) : 0;
    if (passed < 32 || (i0 + 32) * kChUnitRows >= n * a.G) break;
  }
  x = base + i;
  return small_unit(a, s, r, i, y);
}
// The unit that a place of the line belongs to: the last one that starts at or before it.
__device__ __forceinline__ ChUnit small_unit_of(const ChArgs& a, const ChSmall& s, int place, int& x, int& h) {
  h = min(place / s.T, a.Hkv - 1);
  x = 0;
  return small_find(a, s, 31 - __clz(__ballot_sync(0xffffffffu, s.n > 0 && s.y <= place - h * s.T)), place - h * s.T, x);
}
// Unit `of` of all heads'.
__device__ __forceinline__ ChUnit small_unit_at(const ChArgs& a, const ChSmall& s, int of, int& x, int& h) {
  h = of / s.units;
  x = of - h * s.units;
  return small_find(a, s, 31 - __clz(__ballot_sync(0xffffffffu, s.base <= x)), -1, x);
}
// (s.n, s.c0 and s.L are given; s.n below 0 where cu_seqlens decrease)
__device__ __forceinline__ void small_plan(const ChArgs& a, unsigned bad, ChSmall& s, ChStart& st) {
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  if (bad >> lane & 1) s.L = 0;
  const bool down = __any_sync(kFull, s.n < 0);  // (as in the plan)
  if (down) {
    if (lane == 0 && blockIdx.x == 0) atomicOr(a.status, kStatusBadStart);
    s.n = 0;
  }
  int mine = (s.n * a.G + kChUnitRows - 1) / kChUnitRows, cost = 0, top = 0;
  ChUnit u;
  u.L = s.L;
  u.behind = a.causal ? s.n - 1 : 0;
#pragma unroll 1
  for (int i = 0; i < mine; ++i) {
    u.rows = min(kChUnitRows, s.n * a.G - i * kChUnitRows);
    u.tokens = seen(u, quotient(i * kChUnitRows + u.rows - 1, a.by_g));
    cost += unit_cost(u);
    top = max(top, unit_cost(u));
  }
  int x = mine, y = cost;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int p = __shfl_up_sync(kFull, x, o), q = __shfl_up_sync(kFull, y, o);
    if (lane >= o) x += p, y += q;
  }
  s.units = __shfl_sync(kFull, x, 31);
  s.T = __shfl_sync(kFull, y, 31);
  s.base = x - mine;
  s.y = y - cost;
  st.b0 = st.b1 = 0;
  st.units = s.units;
  st.T = s.T;
  st.cut = -1;
  st.unit = st.h = st.cut_h = 0;
  if (uncut(a, s.units, s.T, __reduce_max_sync(kFull, top))) {
    const int all = s.units * a.Hkv;
    const ChRanges by = ranges_of(all, a.ctas);
    const int from = by.begin(blockIdx.x), to = by.begin(blockIdx.x + 1);
    if (from == to) return;
    st.u = small_unit_at(a, s, from, st.unit, st.h);
    st.b0 = st.h * s.T + st.u.y;
    st.b1 = s.T * a.Hkv;
    if (to == all) return;
    int h;
    const int y_to = small_unit_at(a, s, to, x, h).y;
    st.b1 = h * s.T + y_to;
    return;
  }
  const ChRanges rg = ranges_of(s.T * a.Hkv, a.ctas);
  st.b0 = rg.begin(blockIdx.x);
  st.b1 = rg.begin(blockIdx.x + 1);
  if (st.b0 >= st.b1) return;
  st.u = small_unit_of(a, s, st.b0, st.unit, st.h);
  if (st.b1 == s.T * a.Hkv) return;
  st.cut_u = small_unit_of(a, s, st.b1, x, st.cut_h);
  const int at = st.cut_h * s.T + st.cut_u.y, blocks = blocks_of(st.cut_u.tokens);
  int i0, i1;
  owned_blocks(st.cut_u, at, st.b0, st.b1, i0, i1);
  if (i0 == 0 && i1 > 0 && i1 < blocks)
    st.cut = rg.owner(at + start_cost(st.cut_u.rows) + (blocks - 1) * block_cost(st.cut_u.rows));
}

struct alignas(16) ChPiece {
  ChUnit u;
  int h, i0, i1, blocks;  // blocks [i0, i1) of the unit's
  int qset;               // pair of query buffers: a tile's each, or the first for a unit of one row tile
  int t0;                 // parity of the blocks before, and tile of the first one of a unit of one row tile
  int last;               // no piece: the end
  int pad;
  __device__ __forceinline__ bool pair() const { return u.rows > 128; }
};
struct alignas(16) ChSlot {
  ChPiece piece;
  int pages[32];  // of the first four blocks' tiles, -1 where the unit has none
};
static_assert(sizeof(ChSlot) == ChCfg::kPieceBytes, "slot of the piece ring");

// The next piece of a CTA's range; units without tokens belong to the range that holds their place.
struct ChCursor {
  int x, h, units, T, b0, b1;
  ChUnit u;
  ChSmall s;
};
__device__ __forceinline__ bool next_piece(const ChArgs& a, ChCursor& c, ChPiece& p) {
  for (;;) {
    if (c.x == c.units) {
      c.x = 0;
      if (++c.h >= a.Hkv) return false;
      c.u = a.small ? small_first(a, c.s) : load_unit(a.unit);
    }
    const int y = c.h * c.T + c.u.y;
    if (y >= c.b1) return false;
    p.u = c.u;
    p.h = c.h;
    p.blocks = blocks_of(c.u.tokens);
    owned_blocks(c.u, y, c.b0, c.b1, p.i0, p.i1);
    if (++c.x < c.units) c.u = a.small ? small_next(a, c.s, c.u, c.x) : load_unit(a.unit + c.x);
    if (p.i0 < p.i1 || (p.blocks == 0 && y >= c.b0)) return true;
  }
}

// tc_wait of the softmax warps and of those that work ahead: the hardware may hold one back for a microsecond, so
// that their looking leaves the issue slots to the others (8192-token prompt 798 -> 776 us, with weights in one part; the
// other warps answer sooner without).
__device__ __forceinline__ void idle_wait(uint32_t bar, uint32_t parity, uint32_t* status, volatile int* failed) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  if (ok == 0) tc_wait_long(bar, parity, status, failed);
}

// ---------------------------------------------------------------------------
// products
// ---------------------------------------------------------------------------
// O += P V over half a block, P from tensor memory: a step is 16 tokens, 8 columns of each part of P and 4 KiB of V.
#define CH_O_STEP(pcol, voff, acc)                                                                  \
  "add.u32 p, %1, " #pcol ";\n\tadd.s64 b, %2, " #voff ";\n\t@e tcgen05.mma.cta_group::1.kind::f16" \
  " [%0], [p], b, %3, " acc ";\n\t"
__device__ __forceinline__ void issue_half_o(uint32_t d, uint32_t p, uint64_t vdesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, first, yes;\n\t.reg .b32 p;\n\t.reg .b64 b;\n\telect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.u32 first, %4, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t" CH_O_STEP(0, 0, "first") CH_O_STEP(8, 256, "yes")
          CH_O_STEP(16, 512, "yes") CH_O_STEP(24, 768, "yes") CH_O_STEP(32, 0, "yes") CH_O_STEP(40, 256, "yes")
              CH_O_STEP(48, 512, "yes") CH_O_STEP(56, 768, "yes") "}" ::"r"(d),
      "r"(p), "l"(vdesc), "r"(kTcOF16), "r"(acc)
      : "memory");
}

// What rounding to the two f16 of hi left of e, as two f16.  (Mixed-precision products: 8192-token prompt 953 us, with
// conversions of hi and a packed subtraction 1021.)
__device__ __forceinline__ uint32_t left_f16x2(float2 e, uint32_t hi) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b, n;\n\t.reg .f32 x, y;\n\tmov.b32 {a, b}, %1;\n\tmov.b16 n, 0xBC00;\n\t"
      "fma.rn.f32.f16 x, a, n, %2;\n\tfma.rn.f32.f16 y, b, n, %3;\n\tcvt.rn.f16x2.f32 %0, y, x;\n\t}"
      : "=r"(r)
      : "r"(hi), "f"(e.x), "f"(e.y));
  return r;
}

// 16 consecutive columns of this thread's tensor memory lane and their largest value (a NaN counts only among
// NaNs), not waited for.
__device__ __forceinline__ void tmem_ld16_max(uint32_t taddr, uint32_t* r, float& top) {
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, %16, [%17];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=f"(top)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16}; "
      ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
// Waits, and keeps the registers' uses behind the wait.
__device__ __forceinline__ void tmem_settle64(uint32_t (&r)[64], float (&top)[4]) {
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 64; ++i) asm volatile("" : "+r"(r[i]));
  asm volatile("" : "+f"(top[0]), "+f"(top[1]), "+f"(top[2]), "+f"(top[3]));
}

// 32 bytes of bf16: a whole sector from one thread.
__device__ __forceinline__ void st_global_u8(uint16_t* dst, const uint32_t (&x)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]), "r"(x[1]), "r"(x[2]),
               "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

__device__ __forceinline__ void prefetch_l2(const void* at, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(at), "r"(bytes) : "memory");
}

// The e4m3 codes of four f16 values.
__device__ __forceinline__ uint32_t f16x4_to_e4m3x4(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tcvt.rn.satfinite.e4m3x2.f16x2 l, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 h, %2;\n\tmov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "r"(x), "r"(y));
  return r;
}
// The larger magnitudes of two pairs of bf16, signs apart; NaN if one is.
__device__ __forceinline__ uint32_t max_abs_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}

// The first n halves (of 2) of a word.
__device__ __forceinline__ uint32_t first_halves(int n) { return n <= 0 ? 0u : n == 1 ? 0xFFFFu : 0xFFFFFFFFu; }
// The halves of x that hold an f16 NaN, as 0xFFFF.
__device__ __forceinline__ uint32_t nan_halves(uint32_t x) {
  const uint32_t hit = ((x & 0x7FFF7FFFu) + 0x03FF03FFu) & 0x80008000u;
  return (hit >> 15) * 65535u;
}

// 16 bytes of the pool, which goes by: no line of L1 for it.
__device__ __forceinline__ uint4 ld_stream(const uint8_t* at) {
  uint4 x;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "l"(at));
  return x;
}

// 32 consecutive columns, waited for.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Adds O of a warp's rows (32 tensor memory lanes) to what the workspace keeps of it, times f, and clears it (first:
// nothing is kept yet); or, at the end of a piece, adds that to O.  What is kept lies where the warp's 32 rows have their
// partial, as [four dims][lane]: whole lines for a warp (a row's 512 bytes by its thread took four times as long).
__device__ __noinline__ void fold_o(uint32_t to, float4* kept, float f, bool first, bool last) {
#pragma unroll 1
  for (int c = 0; c < 8; c += 2) {
    float4 x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = first ? make_float4(0.f, 0.f, 0.f, 0.f) : __ldcg(kept + (4 * c + i) * 32);
    uint32_t r[32];
    tmem_ld32(to + 16 * c, r);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = make_float4(fmaf(x[i].x, f, __uint_as_float(r[4 * i])), fmaf(x[i].y, f, __uint_as_float(r[4 * i + 1])),
                         fmaf(x[i].z, f, __uint_as_float(r[4 * i + 2])), fmaf(x[i].w, f, __uint_as_float(r[4 * i + 3])));
      if (!last) __stcg(kept + (4 * c + i) * 32, x[i]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t y[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[4 * i] = last ? __float_as_uint(x[4 * h + i].x) : 0u;
        y[4 * i + 1] = last ? __float_as_uint(x[4 * h + i].y) : 0u;
        y[4 * i + 2] = last ? __float_as_uint(x[4 * h + i].z) : 0u;
        y[4 * i + 3] = last ? __float_as_uint(x[4 * h + i].w) : 0u;
      }
      tmem_st16(to + 16 * c + 16 * h, y);
    }
  }
  tmem_wait_st();
}

// 32 columns of O of a row tile (`mine`) and of the other one's (`other`, 128 columns on), joined.
__device__ __forceinline__ void join_o32(uint32_t to, bool mine, bool other, float f0, float f1, float (&x)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] = 0.f;
  uint32_t r[32];
  if (mine) {
    tmem_ld32(to, r);
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(r[k]) * f0;
  }
  if (other) {
    tmem_ld32(to + 128, r);
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = fmaf(__uint_as_float(r[k]), f1, x[k]);
  }
}

__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                   reinterpret_cast<uint64_t>(tmap)),
               "r"(x), "r"(y), "r"(z), "r"(src)
               : "memory");
}

// 16 columns of O of a row tile (`mine`) and of the other one's (`other`, 128 columns on), joined.
__device__ __forceinline__ void join_o(uint32_t to, bool mine, bool other, float f0, float f1, float (&x)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) x[k] = 0.f;
  uint32_t r[16];
  if (mine) {
    tmem_ld16(to, r);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = __uint_as_float(r[k]) * f0;
  }
  if (other) {
    tmem_ld16(to + 128, r);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = fmaf(__uint_as_float(r[k]), f1, x[k]);
  }
}

// A row's NaN values: of the tokens [from, to) of its request, those that some rows of its unit do not see.
// bf16 (out) or fp32 (a partial).
__device__ __noinline__ void poison_row(const ChArgs& a, int r, int h, int from, int to, uint16_t* out, float* part) {
  const int tpp = a.page_size >> 4;
#pragma unroll 1
  for (int j = from; j < to; ++j) {
    const int page = __ldg(a.page_table + static_cast<int64_t>(r) * a.max_pages + j / a.page_size);
    if (page < 0 || page >= a.num_pages) continue;
    const int64_t tile = (static_cast<int64_t>(page) * a.Hkv + h) * tpp + j % a.page_size / kChTile;
    const uint8_t* const v = a.kv_pool + tile * 2 * kChTile * kChDim + kChTile * kChDim + j % kChTile;
#pragma unroll 1
    for (int d = 0; d < kChDim; ++d)
      if ((v[d * kChTile] & 0x7F) == 0x7F) {
        if (out != nullptr) out[d] = 0x7FFF;
        if (part != nullptr) part[d] = __int_as_float(0x7fffffff);
      }
  }
}

__global__ void __launch_bounds__(kChThreads, 1)
    prefill_attn_kernel(const ChArgs a, const __grid_constant__ CUtensorMap kmap,
                        const __grid_constant__ CUtensorMap omap) {
  using C = ChCfg;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const sm = smem_raw;
  const uint32_t sbase = smem_addr(sm);
  if (sbase & 1023u) {  // (cannot happen: the array is aligned, and there is no other shared memory)
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadStart);
    return;
  }
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
  volatile int* const s_failed = reinterpret_cast<volatile int*>(sm + C::kOffMisc + 4);
  volatile int* const s_turns = reinterpret_cast<volatile int*>(sm + C::kOffMisc + 8);
  volatile uint8_t* const s_nan = sm + C::kOffMisc + 16;
  ChSlot* const s_piece = reinterpret_cast<ChSlot*>(sm + C::kOffPiece);
  float2* const s_scale = reinterpret_cast<float2*>(sm + C::kOffScale);
  int* const s_tile = reinterpret_cast<int*>(sm + C::kOffTile);
  int8_t* const s_exp = reinterpret_cast<int8_t*>(sm + C::kOffMult);  // [buffer][row] e of the queries; kNanRow
  auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBars + 8 * i; };
  for (int i = threadIdx.x; i < C::kBars; i += kChThreads) {
    int arrivals = 1;
    if (i >= C::kBarKFree && i < C::kBarKFree + C::kKStages) arrivals = 2;           // both tiles' products
    if (i >= C::kBarReady && i < C::kBarReady + C::kV16Bufs) arrivals = 4;           // converting warps
    if (i >= C::kBarUsed && i < C::kBarUsed + C::kV16Bufs) arrivals = 2;
    if (i >= C::kBarP && i < C::kBarP + 4) arrivals = 4;                             // a tile's softmax warps
    if (i >= C::kBarOFree && i < C::kBarOFree + 2) arrivals = 4;
    if (i >= C::kBarQ && i < C::kBarQ + C::kQTiles) arrivals = 4;                             // converting warps
    if (i >= C::kBarQFree && i < C::kBarQFree + C::kQTiles) arrivals = 10;                    // MMA and softmax warps
    if (i >= C::kBarPieceFree && i < C::kBarPieceFree + kChPieces) arrivals = 15;    // every other warp
    if (i >= C::kBarScaleFree && i < C::kBarScaleFree + C::kScales) arrivals = 12;   // softmax and converting warps
    if (i == C::kBarJoin) arrivals = 4;
    mbar_init(bar(i), arrivals);
    fence_barrier_init();
  }
  if (threadIdx.x < C::kNan) s_nan[threadIdx.x] = 0;
  if (threadIdx.x == 0) *s_failed = s_turns[0] = s_turns[1] = 0;
  if (warp == kChMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the plan is there, or what it needs
  griddep_launch_dependents();
  ChCursor cur;
  int4 first;
  if (a.small) {
    // page tables by all warps, the list by one (what it needs of the requests is asked for ahead)
    unsigned bad = 0;
    cur.s.n = cur.s.c0 = cur.s.L = 0;
    if (warp == kChPlanWarp && lane < a.B) {
      cur.s.c0 = query_start(a, lane);
      cur.s.n = query_start(a, lane + 1) - cur.s.c0;
      cur.s.L = __ldg(a.seq_lens + lane);
    }
    const int ways = 16 / min(a.B, 16);
#pragma unroll 1
    for (int r = warp / ways; r < a.B; r += 16 / ways) {
      const int L = live_length(a, r), pages = L > 0 ? (L - 1) / a.page_size + 1 : 0;
      const int32_t* const row = a.page_table + static_cast<int64_t>(r) * a.max_pages;
      bool out = L == 0;
#pragma unroll 4
      for (int i = warp % ways * 32 + lane; i < pages; i += 32 * ways) out |= static_cast<unsigned>(__ldg(row + i)) >= static_cast<unsigned>(a.num_pages);
      if (__any_sync(kFull, out)) bad |= 1u << r;
    }
    int* const s_bad = reinterpret_cast<int*>(sm);  // (the queries' place)
    if (lane == 0) s_bad[warp] = static_cast<int>(bad);
    __syncthreads();
    if (warp == kChPlanWarp) {
      bad = __reduce_or_sync(kFull, lane < 16 ? static_cast<unsigned>(s_bad[lane]) : 0u);
      ChStart st;
      small_plan(a, bad, cur.s, st);
      cur.u = st.u;
      cur.units = st.units;
      cur.T = st.T;
      first = make_int4(st.unit, st.h, st.b0, st.b1);
      if (lane == 0) {
        s_bad[16] = st.b0 < st.b1;
        a.start[blockIdx.x] = st;  // (for the merge)
      }
    }
    __syncthreads();
    if (warp != kChPlanWarp) first = make_int4(0, 0, 0, s_bad[16]);
    __syncthreads();
  } else {
    const int4* const start = reinterpret_cast<const int4*>(a.start + blockIdx.x);
    first = __ldcg(start);
    if (warp == kChPlanWarp) {
      cur.u = near_unit(__ldcg(start + 1), __ldcg(start + 2));
      const int4 more_of = __ldcg(start + 3);
      cur.units = more_of.x;
      cur.T = more_of.y;
    }
  }
  const uint32_t tmem = *s_tmem;
  auto wait = [&](int i, uint32_t parity) { tc_wait(bar(i), parity & 1u, a.status, s_failed); };
  uint32_t pn = 0;
  auto take_piece = [&](ChPiece& p) -> bool {
    wait(C::kBarPiece + pn % kChPieces, pn / kChPieces);
    p = s_piece[pn % kChPieces].piece;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kBarPieceFree + pn % kChPieces));
    ++pn;
    return __all_sync(kFull, p.last == 0 && !*s_failed);
  };
  if (first.z < first.w) {
    ChPiece p;
    const int tpp = a.page_size >> 4;
    if (warp == kChPlanWarp) {
      // ===================== pieces and scales, ahead of the other warps =====================
      auto wait = [&](int i, uint32_t parity) { idle_wait(bar(i), parity & 1u, a.status, s_failed); };
      cur.x = first.x;
      cur.h = first.y;
      cur.b0 = first.z;
      cur.b1 = first.w;
      int qset = 0, t0 = 0;
      uint32_t j = 0;  // blocks whose scales are out
      bool more = true;
#pragma unroll 1
      for (uint32_t n = 0; more; ++n) {
        more = next_piece(a, cur, p);
        if (!more) p.i0 = p.i1 = 0;
        p.last = !more;
        p.qset = qset;
        qset ^= 1;
        p.t0 = t0;
        t0 ^= (p.i1 - p.i0) & 1;
        const int32_t* const row = a.page_table + static_cast<int64_t>(more ? p.u.r : 0) * a.max_pages;
        const int tiles = (p.u.tokens + kChTile - 1) / kChTile;
        // the first blocks' pages: copies need not wait for the table, which may come from far
        auto page_of = [&](int b) -> int {
          const int tile = b * kChBlkTiles + lane;
          return more && tile < min(tiles, p.i1 * kChBlkTiles) ? max(-1, __ldg(row + quotient(tile, a.by_tpp))) : -1;
        };
        int page = page_of(p.i0);
        if (more && p.i0 < p.i1) {
          // its queries, into L2: a group's heads of each token lie together
          const int first = quotient(p.u.row0, a.by_g), last = quotient(p.u.row0 + p.u.rows - 1, a.by_g);
#pragma unroll 1
          for (int i = first + lane; i <= last; i += 32)
            prefetch_l2(a.q + (static_cast<int64_t>(p.u.c0 + i) * a.Hq + p.h * a.G) * kChDim, a.G * kChDim * 2);
        }
        if (n >= kChPieces) wait(C::kBarPieceFree + n % kChPieces, n / kChPieces - 1);
        ChSlot* const at = s_piece + n % kChPieces;
        at->pages[lane] = page;
        if (lane == 0) at->piece = p;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPiece + n % kChPieces));
#pragma unroll 1
        for (int b = p.i0; b < p.i1; b += 4) {
          const int tile = b * kChBlkTiles + lane;
          uint32_t raw = 0;
          int place = -1;
          if (page >= 0 && page < a.num_pages) {
            place = (page * a.Hkv + p.h) * tpp + tile - quotient(tile, a.by_tpp) * tpp;
            raw = __ldg(a.kv_scales + place);
            // K and V of the tile, into L2: the copies of few rows' blocks follow one another faster than HBM answers
            prefetch_l2(a.kv_pool + static_cast<int64_t>(place) * (2 * kChTile * kChDim), 2 * kChTile * kChDim);
          }
          if (b + 4 < p.i1) page = page_of(b + 4);
          const float2 x = make_float2(exp2_int(scale_exponent(raw & 255u)), static_cast<float>(scale_exponent(raw >> 8)));
#pragma unroll 1
          for (int k = 0; k < 4 && b + k < p.i1; ++k, ++j) {
            const uint32_t st = j % C::kScales;
            if (j >= C::kScales) wait(C::kBarScaleFree + st, j / C::kScales - 1);
            if (lane >> 3 == k) {
              s_scale[st * kChBlkTiles + (lane & 7)] = x;
              s_tile[st * kChBlkTiles + (lane & 7)] = max(place, 0);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarScale + st));
          }
        }
        if (*s_failed) more = false;
      }
    } else if (warp == kChLoadWarp) {
      // ===================== K rows into their ring =====================
      auto wait = [&](int i, uint32_t parity) { idle_wait(bar(i), parity & 1u, a.status, s_failed); };
      // Lane c copies box c of a block (zbox tiles, within a page).
      const uint64_t pol = l2_policy_evict_normal();  // (other units and CTAs read the same pages)
      const int box_t = (lane & 7) * a.zbox;  // first tile of the box in a block
      const bool copies = lane < kChBlkTiles / a.zbox;
      uint32_t j = 0;
      for (;;) {
        wait(C::kBarPiece + pn % kChPieces, pn / kChPieces);
        const ChSlot& slot = s_piece[pn % kChPieces];
        p = slot.piece;
        // pages of 16 tiles, one per lane of a half-warp: of this block and the next (an even number of blocks
        // into the piece), and of the two behind them, asked for two blocks before they are needed
        int now = slot.pages[lane & 15], then = slot.pages[16 + (lane & 15)];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPieceFree + pn % kChPieces));
        ++pn;
        if (__any_sync(kFull, p.last != 0 || *s_failed)) break;
        const int32_t* const row = a.page_table + static_cast<int64_t>(p.u.r) * a.max_pages;
        const int tiles = (p.u.tokens + kChTile - 1) / kChTile;
#pragma unroll 1
        for (int i = p.i0; i < p.i1; ++i, ++j) {
          const uint32_t st = j % C::kKStages, f = bar(C::kBarKFull + st);
          const int behind = i - p.i0;
          if (behind > 0 && (behind & 1) == 0) {
            now = then;
            then = -1;
            const int tile = (i + 2) * kChBlkTiles + (lane & 15);
            if (tile < min(tiles, p.i1 * kChBlkTiles)) then = __ldg(row + quotient(tile, a.by_tpp));
          }
          const int tile = i * kChBlkTiles + box_t;
          const int pg = __shfl_sync(kFull, now, (behind & 1) * 8 + box_t, 16);
          const bool good = copies && tile < tiles && pg >= 0 && pg < a.num_pages;
          const uint32_t boxes = __popc(__ballot_sync(kFull, good));
          if (j >= C::kKStages) wait(C::kBarKFree + st, j / C::kKStages - 1);
          if (lane == 0) {
            if (boxes == 0) mbar_arrive(f);
            else mbar_arrive_expect_tx(f, boxes * a.zbox * (kChTile * kChDim));
          }
          __syncwarp();
          if (good)
            tma_load_3d(sbase + C::kOffK + st * C::kKStage + box_t * kChTile * kChDim, &kmap, 0, 0,
                        (pg * a.Hkv + p.h) * tpp + tile - quotient(tile, a.by_tpp) * tpp, f, pol);
        }
      }
      // every copy has landed before the CTA ends
      if (lane == 0) {
#pragma unroll 1
        for (uint32_t b = j > C::kKStages ? j - C::kKStages : 0; b < j; ++b)
          mbar_wait(bar(C::kBarKFull + b % C::kKStages), (b / C::kKStages) & 1, a.status);
      }
    } else if (warp >= kChVWarp && warp < kChVWarp + 4) {
      // ===================== queries, and V blocks made ready for the MMA =====================
      const int d = threadIdx.x - kChVWarp * 32, vw = warp - kChVWarp;  // this thread's dim
      const int c = lane & 7;
      const float sign = a.sm_scale_log2 < 0.f ? -1.f : 1.f;  // a negative scale's sign goes to the query
      uint32_t j = 0, used = 0, phases = 0;  // V blocks; query buffers used before, and the parities of their frees
      // The piece whose blocks are converted (i .. p.i1 to go), and the next one, whose queries are: steps at .. n of
      // 16 rows, four a warp (eight lanes a row, 16 dims each).
      ChPiece next;
      p.i0 = p.i1 = 0;
      int i = 0, at = 0, n = 0, least = 0;
      uint32_t piece = 0;
      bool known = false, ended = false;
      uint4 x[kChBlkTiles];
      const uint8_t* const codes = a.kv_pool + kChTile * kChDim + d * 16;
      int place[kChBlkTiles];  // of a block's tiles
      auto places = [&](uint32_t b) {
        const int4* const at = reinterpret_cast<const int4*>(s_tile + b % C::kScales * kChBlkTiles);
        const int4 lo = at[0], hi = at[1];
        place[0] = lo.x, place[1] = lo.y, place[2] = lo.z, place[3] = lo.w;
        place[4] = hi.x, place[5] = hi.y, place[6] = hi.z, place[7] = hi.w;
      };
      auto fetch = [&](int t) { x[t] = ld_stream(codes + static_cast<int64_t>(place[t]) * (2 * kChTile * kChDim)); };
      uint4 q[2][2];
      auto ask = [&](int s0) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int s = s0 + k, row = next.u.row0 + 16 * s + 4 * vw + (lane >> 3);
          q[k][0] = q[k][1] = make_uint4(0, 0, 0, 0);
          if (s < n && row < next.u.row0 + next.u.rows) {
            // (query token row / G, head row % G of the group)
            const uint4* const at = reinterpret_cast<const uint4*>(
                a.q + (static_cast<int64_t>(next.u.c0) * a.Hq + next.h * a.G + row + static_cast<int64_t>(quotient(row, a.by_g)) * (a.Hq - a.G)) * kChDim +
                16 * c);
            q[k][0] = __ldg(at);
            q[k][1] = __ldg(at + 1);
          }
        }
      };
      auto fetched = [&](uint32_t b) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarScaleFree + b % C::kScales));
      };
      for (;;) {
        // V goes first wherever its buffer is free, a step of the queries else
        const bool queries = known && at < n;
        if (i < p.i1 && (!queries || j < C::kV16Bufs ||
                         __all_sync(kFull, mbar_test(bar(C::kBarUsed + j % C::kV16Bufs), (j / C::kV16Bufs - 1) & 1)))) {
          // ---- V: this thread's dim of a block's tiles, the next block's on their way while one is converted
          const int nv = min(kChBlk, p.u.tokens - i * kChBlk), first_hidden = least - i * kChBlk;
          const uint32_t buf = j % C::kV16Bufs;
          const bool more = i + 1 < p.i1;
          if (more) {
            wait(C::kBarScale + (j + 1) % C::kScales, (j + 1) / C::kScales);
            places(j + 1);
          }
          if (j >= C::kV16Bufs) wait(C::kBarUsed + buf, j / C::kV16Bufs - 1);
          uint8_t* const o = sm + C::kOffV16 + buf * C::kV16 + d * 16;
#pragma unroll
          for (int t = 0; t < kChBlkTiles; ++t) {
            // codes of dim d, tokens 16 t .. 16 t + 15, to two rows of 8 f16
            uint32_t y[8];
            e4m3x4_to_f16x4(x[t].x, y[0], y[1]);
            e4m3x4_to_f16x4(x[t].y, y[2], y[3]);
            e4m3x4_to_f16x4(x[t].z, y[4], y[5]);
            e4m3x4_to_f16x4(x[t].w, y[6], y[7]);
            uint4* const w = reinterpret_cast<uint4*>(o + t * kChTile * kChDim * 2);
            w[0] = make_uint4(y[0], y[1], y[2], y[3]);
            w[128] = make_uint4(y[4], y[5], y[6], y[7]);
            if (more) fetch(t);
          }
          if (nv < kChBlk || first_hidden < kChBlk) {
            // what lies behind the last token: 0; and NaN in tokens that not every row sees (they would reach the others)
            uint32_t hits = 0;
#pragma unroll 1
            for (int tok = max(0, min(nv, first_hidden)) & ~7; tok < kChBlk; tok += 8) {
              uint4* const w = reinterpret_cast<uint4*>(o + (tok >> 4) * (kChTile * kChDim * 2) + (tok & 8) * 256);
              const uint4 v = *w;
              uint32_t y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                y[k] &= first_halves(nv - tok - 2 * k);
                const uint32_t nans = nan_halves(y[k]) & ~first_halves(first_hidden - tok - 2 * k);
                y[k] &= ~nans;
                hits |= nans;
              }
              *w = make_uint4(y[0], y[1], y[2], y[3]);
            }
            if (hits) s_nan[piece % C::kNan] = 1;
          }
          fence_proxy_async_smem();
          if (more) fetched(j + 1);
          else __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kBarReady + buf));
          ++i;
          ++j;
        } else if (queries) {
          // ---- the next piece's queries, two steps at a time (all that are left behind the last block); each operation
          // for all values before the next one: only the warp's own instructions hide their time
          const int end = i == p.i1 ? n : at + 2;
#pragma unroll 1
          for (; at < end; at += 2) {
            const int buf = 2 * next.qset + (at >> 3);
            if ((at & 7) == 0) {
              if (used >> buf & 1) {
                wait(C::kBarQFree + buf, phases >> buf & 1);
                phases ^= 1u << buf;
              }
              used |= 1u << buf;
            }
            uint32_t r[2][8], top[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              r[k][0] = q[k][0].x, r[k][1] = q[k][0].y, r[k][2] = q[k][0].z, r[k][3] = q[k][0].w;
              r[k][4] = q[k][1].x, r[k][5] = q[k][1].y, r[k][6] = q[k][1].z, r[k][7] = q[k][1].w;
            }
            ask(at + 2);
            // largest |q| of the row: bf16 magnitudes order as integers
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = max_abs_bf16x2(r[k][2 * e], r[k][2 * e + 1]);
              x[0] = max_abs_bf16x2(max_abs_bf16x2(x[0], x[1]), max_abs_bf16x2(x[2], x[3]));
              top[k] = max(x[0] & 0x7FFFu, x[0] >> 16 & 0x7FFFu);
            }
#pragma unroll
            for (int o = 1; o < 8; o <<= 1)
#pragma unroll
              for (int k = 0; k < 2; ++k) top[k] = max(top[k], __shfl_xor_sync(kFull, top[k], o));
            // q 2^e has its largest value in [128, 256): e = 134 - that value's exponent
            int ex[2];
            uint32_t w[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              ex[k] = static_cast<int>(top[k] >> 7);
              ex[k] = ex[k] == 255 ? kNanRow : ex[k] == 0 ? (top[k] == 0 ? 0 : 126) : min(max(134 - ex[k], -126), 126);
              const float up = sign * exp2_int(max(ex[k], -126));
#pragma unroll
              for (int e = 0; e < 8; ++e)  // (f16 holds it but for what lies below 2^-24, which neither part would)
                w[k][e] = pack_f16x2(__uint_as_float(r[k][e] << 16) * up, __uint_as_float(r[k][e] & 0xFFFF0000u) * up);
            }
            uint32_t y[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) y[k][e] = f16x4_to_e4m3x4(w[k][2 * e], w[k][2 * e + 1]);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint32_t h0, h1;
                e4m3x4_to_f16x4(y[k][e], h0, h1);
                w[k][2 * e] = sub_f16x2(w[k][2 * e], h0);
                w[k][2 * e + 1] = sub_f16x2(w[k][2 * e + 1], h1);
              }
            uint32_t z[2][4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < 4; ++e) z[k][e] = f16x4_to_e4m3x4(w[k][2 * e], w[k][2 * e + 1]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int row = 16 * ((at + k) & 7) + 4 * vw + (lane >> 3);  // of the tile
              uint8_t* const dst = sm + buf * C::kQTile + row * 128 + ((c ^ (row & 7)) << 4);
              *reinterpret_cast<uint4*>(dst) = make_uint4(y[k][0], y[k][1], y[k][2], y[k][3]);
              *reinterpret_cast<uint4*>(dst + 16384) = make_uint4(z[k][0], z[k][1], z[k][2], z[k][3]);
              if (c == 0) s_exp[buf * 128 + row] = static_cast<int8_t>(ex[k]);
            }
            if ((at & 7) == 6 || at + 2 == n) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::kBarQ + buf));
            }
          }
        }
        // ---- the next piece, once it is known; it is waited for when there is nothing else to do
        if (!known && p.i1 - i <= C::kScales && (i == p.i1 || __all_sync(kFull, mbar_test(bar(C::kBarPiece + pn % kChPieces), pn / kChPieces & 1)))) {
          ended = !take_piece(next);
          known = true;
          at = 0;
          n = ended || next.i0 == next.i1 ? 0 : (next.u.rows + 31) / 32 * 2;  // (what lies behind the last row stays what it was)
          ask(0);
          if (d == 0) s_nan[(pn - 1 + C::kNan / 2) % C::kNan] = 0;
        }
        // ---- on to it
        if (i == p.i1 && known && at >= n) {
          if (ended) break;
          p = next;
          piece = pn - 1;
          known = false;
          i = p.i0;
          least = seen(p.u, quotient(p.u.row0, a.by_g));  // tokens that every row sees
          if (i < p.i1) {
            wait(C::kBarScale + j % C::kScales, j / C::kScales);
            places(j);
#pragma unroll
            for (int t = 0; t < kChBlkTiles; ++t) fetch(t);
            fetched(j);
          }
        }
      }
    } else if (warp == kChMmaWarp || warp == kChMmaWarp + 1) {
      // ===================== MMA issue, a warp per row tile =====================
      // The warp runs as one, an elected lane issues.  A tile's products alternate: S of a block, PV of the
      // same block in halves as the softmax hands P over, S of the next (which overwrites S and P: the
      // products of one thread run in order).  While a tile's softmax runs the other tile has the tensor
      // cores; on a unit of both tiles the warps take turns (PV and the next S), or else the two would run
      // in step.  All waits of a turn come before it, and turns are counted in shared memory, not by a
      // barrier (no result hangs on it, a turn not seen is gone without).
      //
      // On a unit of one row tile block j belongs to tile j mod 2.  A barrier's parity tells neighbouring
      // phases apart, no others, so a warp has to see every phase of a barrier it waits for: slots are even
      // in number, and a tile has its own and sees all of theirs.
      const int t = warp - kChMmaWarp;
      const uint32_t base = __reduce_max_sync(kFull, sbase), tm = __reduce_max_sync(kFull, tmem);  // uniform registers
      const uint32_t bars = base + C::kOffBars;
      const uint64_t qdesc = smem_desc(base, 16, 1024, 2), kdesc = smem_desc(base + C::kOffK, 16, 1024, 2);
      // V, 16 tokens a step: two columns of core matrices (8 dims x 8 tokens, 128 B apart along the dims, 2 KiB along the tokens)
      const uint64_t vdesc = smem_desc(base + C::kOffV16, 2048, 128, 0);
      uint32_t j0 = 0, n0 = 0, n1 = 0, begun = 0, phases = 0;  // (phases: parities of the query buffers)
      int turns = 0;
      const uint32_t turn_of = base + C::kOffMisc + 8 + 4 * (t ^ 1);
      static_assert(C::kKStages % 2 == 0 && C::kV16Bufs == 2 && C::kScales % 2 == 0, "slots that tiles own");
      while (take_piece(p)) {
        const int pair_in = __any_sync(kFull, p.pair());
        const uint32_t nb = __reduce_max_sync(kFull, p.i1 - p.i0), qb = __reduce_max_sync(kFull, 2 * p.qset);
        const uint32_t halves = __reduce_max_sync(kFull, max(0, p.u.tokens - p.i0 * kChBlk + 63) / 64);  // of the piece, and behind it
        if (nb == 0) continue;
        const uint32_t step = pair_in ? 1 : 2;
        // (of a pair its own: tile 0's is filled first, so that who sees tile 1's has that phase behind it too)
        const uint32_t mine = qb + (pair_in ? t : 0);
        wait(C::kBarQ + mine, phases >> mine);
        phases ^= (pair_in ? 3u : 1u) << qb;
        const uint64_t qd = qdesc + mine * (C::kQTile >> 4);
        bool begins = true;
#pragma unroll 1
        for (uint32_t i = pair_in ? 0 : (j0 ^ t) & 1; i < nb + step; i += step) {
          // PV of this tile's block before, S of block i: what they need first, then the turn
          const bool pair = varying(pair_in) != 0;
          const uint32_t ks = (j0 + i) % C::kKStages, m = i - step, jm = j0 + m, vs = jm % C::kV16Bufs;
          if (i < nb) wait(C::kBarKFull + ks, (j0 + i) / C::kKStages);
          if (i >= step) {
            wait(C::kBarReady + vs, jm / C::kV16Bufs);
            if (begins && begun > 0) wait(C::kBarOFree + t, begun - 1);  // O of the piece before has been read
            wait(C::kBarP + 2 * t, n0++);
          }
          tc_fence_after();
          const uint64_t vd = vdesc + vs * (C::kV16 >> 4);
          const uint32_t od = tm + 256 + t * 128, pd = tm + t * 128, acc = !begins;
          const bool both = 2 * m + 1 < halves;
          if (pair) {
#pragma unroll 1
            for (int spins = 0; load_shared(turn_of) - turns < t && spins < kChTurnSpins; ++spins) {
            }
          }
          if (i >= step) {
            issue_half_o(od, pd, vd, acc);
            commit_elected(bars + 8 * (C::kBarHalf + t));
            if (both) {
              wait(C::kBarP + 2 * t + 1, n1++);
              tc_fence_after();
              issue_half_o(od, pd + 64, vd + 1024, 1);
            }
            commit_elected(bars + 8 * (C::kBarO + t));  // (before S: who sees S knows O's phase to be over)
            begun += begins;
            begins = false;
          }
          if (i < nb) issue_s<true>(tm + t * 128, qd, kdesc + ks * (C::kKStage >> 4));
          if (pair) {
            ++turns;
            if (lane == 0) s_turns[t] = turns;
          }
          if (i < nb) {
            commit_elected(bars + 8 * (C::kBarS + t));
            commit_elected(bars + 8 * (C::kBarKFree + ks));
            if (!pair) commit_elected(bars + 8 * (C::kBarKFree + ks));
          }
          if (i >= step) {
            commit_elected(bars + 8 * (C::kBarUsed + vs));
            if (!pair) commit_elected(bars + 8 * (C::kBarUsed + vs));  // for the other tile too
          }
        }
        j0 += nb;
        // the queries: this warp's S are done (of a pair it answers twice, for its own buffer)
        commit_elected(bars + 8 * (C::kBarQFree + mine));
        if (pair_in) commit_elected(bars + 8 * (C::kBarQFree + mine));
      }
      // every product and every arrival it owes is done before the CTA ends
      commit_elected(bars + 8 * (C::kBarDone + t));
      mbar_wait(bar(C::kBarDone + t), 0, a.status);
    } else {
      // ===================== softmax, a thread per row =====================
      auto wait = [&](int i, uint32_t parity) { idle_wait(bar(i), parity & 1u, a.status, s_failed); };
      const int t = warp >> 2;  // row tile
      const int row = threadIdx.x & 127;
      const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * 128 + lanes;
      uint32_t ns = 0;            // S blocks taken of this tile
      uint32_t j0 = 0;            // blocks of the pieces before
      uint32_t phases = 0;        // parities of the query buffers
      uint32_t joins = 0;
      // (a piece's slot is read twice, here and for its results: what those need would take registers from the blocks)
      auto piece_read = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPieceFree + (pn - 1) % kChPieces));
      };
      for (;;) {
        wait(C::kBarPiece + pn % kChPieces, pn / kChPieces);
        p = s_piece[pn++ % kChPieces].piece;
        if (__any_sync(kFull, p.last != 0 || *s_failed)) break;
        const bool pair = p.pair();
        const int nb = p.i1 - p.i0;
        const int lrow = pair ? t * 128 + row : row;  // row of the unit
        const bool busy = lrow - lane < p.u.rows;     // some row of the warp's is
        const int limit = seen(p.u, quotient(p.u.row0 + min(lrow, p.u.rows - 1), a.by_g));
        const int least = __reduce_min_sync(kFull, limit);  // tokens that every row of the warp sees
        const int nan_slot = static_cast<int>((pn - 1) % C::kNan);
        const int buf = 2 * p.qset + (pair ? t : 0);
        // (of a pair each tile's warps answer for their own buffer, twice: they have seen no other filled)
        auto free_queries = [&]() {
          if (nb > 0 && lane <= (pair ? 1 : 0)) mbar_arrive(bar(C::kBarQFree + buf));
        };
        float m = -INFINITY, l = 0.f;
        bool any = false;
        // O of kChFold blocks at a time is added up in the rows' place for a partial, beside the maximum that it goes by
        int folds = 0;
        auto fold = [&](bool last) {
          const int64_t slot = static_cast<int64_t>(2 * blockIdx.x + (p.i0 == 0 ? 0 : 1)) * kChUnitRows + t * 128 + row;
          float2* const kept = a.part_ml + slot;
          const float was = folds == 0 ? -INFINITY : __ldcg(kept).x;
          fold_o(to, reinterpret_cast<float4*>(a.part_o + (slot - lane) * kChDim) + lane, was == -INFINITY ? 0.f : fast_exp2(was - m),
                 folds == 0, last);
          if (!last) __stcg(kept, make_float2(m, 0.f));
          ++folds;
          __syncwarp();  // (the place is written row by row next, if at all)
        };
        if (nb > 0) {
          wait(C::kBarQ + buf, phases >> buf);
          phases ^= (pair ? 3u : 1u) << (2 * p.qset);
          const int e = s_exp[buf * 128 + row];
          // a NaN query: its row is NaN, unless it sees nothing (all its scores are -inf then, and have to stay so)
          const float mult = limit == 0 ? 1.f : e == kNanRow ? __int_as_float(0x7fffffff) : fabsf(a.sm_scale_log2) * exp2_int(-e);
          __syncwarp();
          if (mult != mult) m = mult;
          // ---- blocks
#pragma unroll 1
          for (int i = pair ? 0 : t ^ p.t0; i < nb; i += pair ? 1 : 2) {
            const uint32_t js = j0 + i, st = js % C::kScales;
            const int at = (p.i0 + i) * kChBlk;
            const int halves = p.u.tokens - at > 64 ? 2 : 1;  // (a half without tokens is left out)
            // the scales, before S is there: shared memory answers late while the products read it
            wait(C::kBarScale + st, js / C::kScales);
            const float2* const sc = s_scale + st * kChBlkTiles;
            float f[4], ev[4];
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              const float2 x = sc[g];
              f[g] = at_least_min(mult * x.x);
              ev[g] = x.y;
            }
            wait(C::kBarS + t, ns);
            tc_fence_after();
            if (busy && any && ((pair ? i : i >> 1) & (kChFold - 1)) == 0) fold(false);
            if (busy) {
              if (least - at < 64 * halves) {
                // columns that a row does not see: -inf, by a short loop over tensor memory (selects on
                // registers would be a second copy of the code below, fetched anew each time)
#pragma unroll 1
                for (int k = max(0, least - at) / 16; k < 4 * halves; ++k) {
                  uint32_t x[16];
                  tmem_ld16(ts + 16 * k, x);
                  const int left = limit - at - 16 * k;
#pragma unroll
                  for (int c = 0; c < 16; ++c) x[c] = c < left ? x[c] : 0xFF800000u;
                  tmem_st16(ts + 16 * k, x);
                }
                tmem_wait_st();
              }
              // Half a block at a time, each with a look at its own maximum: the first half's weights are on
              // their way while the second's are made.
#pragma unroll 1
              for (int h = 0; h < halves; ++h) {
                uint32_t s[64];
                float top[4];
                float2 next[4];  // the other half's scales, asked for ahead
#pragma unroll
                for (int g = 0; g < 4; ++g) tmem_ld16_max(ts + 64 * h + 16 * g, s + 16 * g, top[g]);
#pragma unroll
                for (int g = 0; g < 4; ++g) next[g] = sc[4 + g];
                tmem_settle64(s, top);
                const float mb = fmaxf(fmaxf(fmaf(top[0], f[0], ev[0]), fmaf(top[1], f[1], ev[1])),
                                       fmaxf(fmaf(top[2], f[2], ev[2]), fmaf(top[3], f[3], ev[3])));
                const bool grown = mb > m + kChGrow || (m == -INFINITY && mb != -INFINITY);
                if (__any_sync(kFull, grown)) {
                  const float x = !grown ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - mb);
                  if (grown) m = mb;
                  l *= x;
                  if (any || h > 0) {
                    // O so far: of the blocks before, whose product S came behind, and of this one's first half
                    if (h > 0) {
                      wait(C::kBarHalf + t, ns);
                      tc_fence_after();
                    }
#pragma unroll 1
                    for (int c = 0; c < 8; ++c) tmem_scale16(to + 16 * c, x);
                    tmem_wait_st();
                  }
                }
                const float ref = m == -INFINITY ? 0.f : m - kChLift;
                // arguments of the next 16 columns beside the powers of these: the powers' pipe is the slow one
                auto arguments = [&](int g) {
                  const float2 f2 = make_float2(f[g], f[g]), b2 = make_float2(ev[g] - ref, ev[g] - ref);
#pragma unroll
                  for (int k = 16 * g; k < 16 * g + 16; k += 2) {
                    const float2 e = fma2(make_float2(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), f2, b2);
                    s[k] = __float_as_uint(e.x);
                    s[k + 1] = __float_as_uint(e.y);
                  }
                };
                arguments(0);
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  if (g < 3) arguments(g + 1);
                  uint32_t w[8], v[8];
                  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                  for (int k = 0; k < 8; ++k) {
                    const float2 e = make_float2(fast_exp2(__uint_as_float(s[16 * g + 2 * k])), fast_exp2(__uint_as_float(s[16 * g + 2 * k + 1])));
                    sum[k & 1] = add2(sum[k & 1], e);
                    w[k] = pack_f16x2(e.x, e.y);
                    v[k] = left_f16x2(e, w[k]);
                  }
                  tmem_st8(ts + 64 * h + 8 * g, w);  // over columns that have been read
                  tmem_st8(ts + 64 * h + 32 + 8 * g, v);
                  const float2 x = add2(sum[0], sum[1]);
                  // 2^(-ev - lift), from the integer in the last bits of ev + 1.5 2^23
                  l = fmaf(x.x + x.y, __int_as_float((0x4B400000 + 127 - kChLift - __float_as_int(ev[g] + 12582912.f)) << 23), l);
                }
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                  f[g] = at_least_min(mult * next[g].x);
                  ev[g] = next[g].y;
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C::kBarP + 2 * t + h));
              }
            } else {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) {
                mbar_arrive(bar(C::kBarP + 2 * t));
                if (halves == 2) mbar_arrive(bar(C::kBarP + 2 * t + 1));
              }
            }
            if (lane <= (pair ? 0 : 1)) mbar_arrive(bar(C::kBarScaleFree + st));
            any = true;
            ++ns;
          }
          if (any) {
            wait(C::kBarO + t, ns - 1);
            tc_fence_after();
            if (busy && folds > 0) fold(true);
          }
        }
        j0 += nb;
        // ---- results: a row's thread, of a unit of one row tile the one of tile 0
        p = s_piece[(pn - 1) % kChPieces].piece;
        piece_read();
        const int grow = p.u.row0 + min(lrow, p.u.rows - 1), token = quotient(grow, a.by_g);
        const int ends = seen(p.u, token);
        const bool valid = lrow < p.u.rows;
        const bool whole = p.i0 == 0 && p.i1 == p.blocks;
        const int64_t slot = static_cast<int64_t>(2 * blockIdx.x + (p.i0 == 0 ? 0 : 1)) * kChUnitRows + lrow;
        float f0 = 1.f, f1 = 0.f;
        bool other = false;  // tile 1's O counts too
        if (!pair && nb > 0) {
          other = (1 ^ p.t0) < nb;  // tile 1 has had a block
          if (t == 1) {
            if (any) {
              // (to tile 0, by way of the workspace: the slot's places behind the unit's rows.  The next join's
              // are written when O, which tile 0 reads behind these, has been freed.)
              __stcg(a.part_ml + slot + 128, make_float2(m, l));
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::kBarJoin));
            }
            free_queries();
            continue;
          }
          if (other) {
            wait(C::kBarJoin, joins++);
            tc_fence_after();
            const float2 ml = __ldcg(a.part_ml + slot + 128);
            const float M = ml.x > m || m == -INFINITY ? ml.x : m;
            f0 = m == -INFINITY ? 0.f : fast_exp2(m - M);
            f1 = ml.x == -INFINITY ? 0.f : fast_exp2(ml.x - M);
            l = l * f0 + ml.y * f1;
            m = M;
          }
        } else if (!pair && t == 1) {
          continue;
        }
        const int64_t orow = static_cast<int64_t>(p.u.c0 + token) * a.Hq + p.h * a.G + grow - token * a.G;
        const bool none = l == 0.f;
        const float inv = exp2_int(-kChLift) * (whole && !none ? 1.f / l : 1.f);
        if (whole && nb > 0 && a.boxed && lrow - lane + 32 <= p.u.rows) {
          // The warp's 32 rows are whole tokens' heads: by way of its rows' place in the query buffer, which has been
          // read, as two boxes of 64 dims (rows of 128 bytes with the 128-byte swizzle).  Stores from registers touch a
          // line per row, a cycle each, and what is asked of shared memory behind them waits as long.  (A piece without
          // blocks has no buffer: that of its turn may hold a later piece's queries by now.  Its zeroes go from registers.)
          uint8_t* const mine = sm + buf * C::kQTile + (row - lane) * 256 + lane * 128;
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            float x[32];
            join_o32(to + 32 * c, any, other, f0 * inv, f1 * inv, x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(mine + (c >> 1) * 4096 + ((((c & 1) * 4 + i) ^ (lane & 7)) << 4)) =
                  make_uint4(pack_bf16x2(x[8 * i], x[8 * i + 1]), pack_bf16x2(x[8 * i + 2], x[8 * i + 3]),
                                    pack_bf16x2(x[8 * i + 4], x[8 * i + 5]), pack_bf16x2(x[8 * i + 6], x[8 * i + 7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const uint32_t src = smem_addr(mine);
            tma_store_3d(&omap, src, 0, p.h * a.G, p.u.c0 + token);
            tma_store_3d(&omap, src + 4096, 64, p.h * a.G, p.u.c0 + token);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        } else if (busy) {
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            float x[16];
            join_o(to + 16 * c, any, other, f0 * inv, f1 * inv, x);
            const int d = 16 * c;
            if (valid && whole) {
              uint32_t y[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) y[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
              st_global_u8(a.out + orow * kChDim + d, y);
            } else if (valid) {
#pragma unroll
              for (int k = 0; k < 16; k += 8) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = x[k + i];
                st_global8(a.part_o + slot * kChDim + d + k, y);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (any) mbar_arrive(bar(C::kBarOFree + t));
          if (other) mbar_arrive(bar(C::kBarOFree + 1));
        }
        if (s_nan[nan_slot] != 0) {
          if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");  // (the rows are out)
          __syncwarp();
          const int lo = max(seen(p.u, quotient(p.u.row0, a.by_g)), p.i0 * kChBlk), hi = min(ends, p.i1 * kChBlk);
          if (valid) poison_row(a, p.u.r, p.h, lo, hi, whole ? a.out + orow * kChDim : nullptr, whole ? nullptr : a.part_o + slot * kChDim);
        }
        if (valid) {
          if (!whole) a.part_ml[slot] = make_float2(m, l);
          else if (a.lse != nullptr) a.lse[orow] = none ? -INFINITY : (m + __log2f(l)) * kChLn2;
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        free_queries();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kChMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// kParts CTAs for each CTA of the products that begins a unit and leaves its end to others; a warp per row: a
// lane finds one partial (its place, m, l), then all lanes add its O.
template <int kParts>
__global__ void __launch_bounds__(32 * kChMergeWarps) prefill_merge_kernel(const ChArgs a) {
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, c = blockIdx.x / kParts;
  griddep_wait();
  const int4* const start = reinterpret_cast<const int4*>(a.start + c);
  const int4 cut = __ldcg(start + 3), u0 = __ldcg(start + 4), u1 = __ldcg(start + 5);
  if (cut.z < 0) return;
  const ChUnit u = near_unit(u0, u1);
  const int T = cut.y, y = cut.w * T + u.y;
  const ChRanges rg = ranges_of(T * a.Hkv, a.ctas);
#pragma unroll 1
  for (int row = blockIdx.x % kParts * kChMergeWarps + (threadIdx.x >> 5); row < u.rows; row += kParts * kChMergeWarps) {
    float M = -INFINITY, W = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int base = c; base <= cut.z; base += 32) {
      const int k = base + lane;
      const int64_t slot = static_cast<int64_t>(2 * k + (k == c ? 0 : 1)) * kChUnitRows + row;
      float2 ml = make_float2(-INFINITY, 0.f);
      if (k <= cut.z) {
        int b, e;
        owned_blocks(u, y, rg.begin(k), rg.begin(k + 1), b, e);
        if (b < e) ml = __ldcg(a.part_ml + slot);
      }
      float mx = ml.x;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      const float mn = fmaxf(M, mx);
      const bool has = ml.y != 0.f;  // (a NaN sum counts, whatever its maximum)
      const float f = !has ? 0.f : ml.x == -INFINITY ? 1.f : fast_exp2(ml.x - mn);
      float ws = ml.y * f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kFull, ws, o);
      const float old = M == -INFINITY ? 0.f : fast_exp2(M - mn);
      W = W * old + ws;
      acc = make_float4(acc.x * old, acc.y * old, acc.z * old, acc.w * old);
      M = mn;
      unsigned todo = __ballot_sync(kFull, has);
#pragma unroll 1
      while (todo) {
        float fk[4];
        float4 o[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int src = todo ? __ffs(todo) - 1 : 0;
          const float fx = __shfl_sync(kFull, f, src);
          const int64_t sx = __shfl_sync(kFull, slot, src);
          fk[x] = todo ? fx : 0.f;
          o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (todo) o[x] = __ldcg(reinterpret_cast<const float4*>(a.part_o + sx * kChDim) + lane);
          todo &= todo - 1;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x)
          acc = make_float4(fmaf(o[x].x, fk[x], acc.x), fmaf(o[x].y, fk[x], acc.y), fmaf(o[x].z, fk[x], acc.z),
                            fmaf(o[x].w, fk[x], acc.w));
      }
    }
    const bool none = W == 0.f;
    const float inv = none ? 0.f : 1.f / W;
    const int grow = u.row0 + row, token = quotient(grow, a.by_g);
    const int64_t orow = static_cast<int64_t>(u.c0 + token) * a.Hq + cut.w * a.G + grow - token * a.G;
    reinterpret_cast<uint2*>(a.out + orow * kChDim)[lane] =
        none ? make_uint2(0, 0) : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (lane == 0 && a.lse != nullptr) a.lse[orow] = none ? -INFINITY : (M + __log2f(W)) * kChLn2;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int kChMaxDevices = 64;
std::atomic<int> g_ch_ready[kChMaxDevices];

int prepare_prefill(int dev) {
  if (g_ch_ready[dev].load(std::memory_order_relaxed) > 0) return FPK_OK;
  if (cudaFuncSetAttribute(prefill_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, ChCfg::kSmem) != cudaSuccess)
    return FPK_ECUDA;
  g_ch_ready[dev].store(1, std::memory_order_relaxed);
  return FPK_OK;
}

// bf16 results [n_tokens][Hq][128]: boxes of 64 dims, G heads, 32 / G tokens.
int encode_rows_map(CUtensorMap* m, void* out, int Hq, int n_tokens, int G) {
  EncodeTiled enc = tensor_map_encoder();
  if (enc == nullptr) return FPK_ECUDA;
  const cuuint64_t dims[3] = {kChDim, static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(n_tokens)};
  const cuuint64_t strides[2] = {kChDim * 2, static_cast<cuuint64_t>(Hq) * kChDim * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(32 / G)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, out, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FPK_OK : FPK_ECUDA;
}

// Most units of a kv head.
int64_t most_units(int64_t B, int64_t n_tokens, int64_t G) { return n_tokens * G / kChUnitRows + B; }

struct ChLayout {
  size_t base, dead, unit, start, ml, o, total;
};
ChLayout prefill_layout(int64_t B, int64_t n_tokens, int64_t G, int64_t ctas) {
  auto up = [](int64_t x) { return (static_cast<size_t>(x) + 255) & ~static_cast<size_t>(255); };
  ChLayout l;
  l.base = 256;
  l.dead = l.base + up((B + 1) * 4);
  l.unit = l.dead + up(B * 4);
  l.start = l.unit + up(most_units(B, n_tokens, G) * static_cast<int64_t>(sizeof(ChUnit)));
  l.ml = l.start + up(ctas * static_cast<int64_t>(sizeof(ChStart)));
  l.o = l.ml + up(2 * ctas * kChUnitRows * 8);
  l.total = l.o + up(2 * ctas * kChUnitRows * kChDim * 4);
  return l;
}

}  // namespace
}  // namespace fpk

extern "C" size_t fpk_prefill_workspace_bytes(int32_t B, int32_t n_tokens, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || n_tokens < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > fpk::kChGroupMax || D != fpk::kChDim) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= fpk::kChMaxDevices) return 0;
  const int ctas = fpk::device_sm_count(dev);
  return ctas > 0 ? fpk::prefill_layout(B, n_tokens, Hq / Hkv, ctas).total : 0;
}

extern "C" int fpk_paged_prefill_attn_fp8_block(const void* q, const int32_t* cu_seqlens, int32_t n_tokens,
                                                const uint8_t* kv_pool, const uint8_t* kv_scales,
                                                const int32_t* page_table, int32_t max_pages,
                                                const int32_t* seq_lens, const uint8_t* abort_mask, int32_t causal,
                                                void* out, float* lse, void* workspace, size_t workspace_bytes,
                                                float sm_scale, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                                int32_t page_size, int32_t num_pages, void* stream) {
  using namespace fpk;
  if (B < 0 || n_tokens < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0 || max_pages < 0 ||
      Hq % Hkv != 0)
    return FPK_EINVAL;
  const int G = Hq / Hkv;
  if (D != kChDim || G > kChGroupMax || page_size % kChTile != 0 || page_size > 256) return FPK_EUNSUPPORTED;
  const int tpp = page_size / kChTile;
  const int64_t tiles = static_cast<int64_t>(num_pages) * Hkv * tpp;
  // tile numbers are 32-bit tensor-map coordinates; the work list's length is counted in 31 bits, tokens are rounded up
  // to blocks in them (a context of at most 2^31 - 128), rows are divided by reciprocals (2^28)
  const int64_t width = (static_cast<int64_t>(max_pages) * page_size + kChBlk - 1) / kChBlk;
  const int64_t units = most_units(B, n_tokens, G), longest = width * kChCostPair + kChStartPair;
  if (tiles > 0x7fffffff || static_cast<int64_t>(n_tokens) * G >= (int64_t(1) << 28) || width >= (int64_t(1) << 24) ||
      longest > 0x7fffffff / ((units > 0 ? units : 1) * Hkv))
    return FPK_EUNSUPPORTED;
  if (B == 0 || n_tokens == 0) return FPK_OK;
  if (!q || !cu_seqlens || !kv_pool || !kv_scales || !page_table || !seq_lens || !out || !workspace) return FPK_EINVAL;
  if (!aligned16(q) || !aligned16(kv_pool) || (reinterpret_cast<uintptr_t>(kv_scales) & 1u) != 0 ||
      (reinterpret_cast<uintptr_t>(out) & 31u) != 0 || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FPK_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kChMaxDevices) return FPK_ECUDA;
  const int ctas = device_sm_count(dev);
  if (ctas <= 0) return FPK_ECUDA;
  const ChLayout l = prefill_layout(B, n_tokens, G, ctas);
  if (workspace_bytes < l.total) return FPK_ENOSPC;
  const int st = prepare_prefill(dev);
  if (st != FPK_OK) return st;
  int zbox = 1;  // tiles per copy: a power of two that divides a page and a block
  while (zbox < kChBlkTiles && tpp % (2 * zbox) == 0) zbox *= 2;
  CUtensorMap kmap;
  if (encode_pool_map(&kmap, kv_pool, tiles > 0 ? tiles : 1, true, false, zbox) != FPK_OK) return FPK_ECUDA;
  // results: dims, heads, tokens; boxes of a warp's rows, which are whole tokens' heads where G divides 32
  const bool boxed = 32 % G == 0;
  CUtensorMap omap = kmap;
  if (boxed && encode_rows_map(&omap, out, Hq, n_tokens, G) != FPK_OK) return FPK_ECUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ChArgs a;
  a.boxed = boxed;
  a.q = static_cast<const uint16_t*>(q);
  a.cu_seqlens = cu_seqlens;
  a.kv_scales = reinterpret_cast<const uint16_t*>(kv_scales);
  a.kv_pool = kv_pool;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.abort_mask = abort_mask;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.base = reinterpret_cast<int32_t*>(ws + l.base);
  a.dead = reinterpret_cast<int32_t*>(ws + l.dead);
  a.unit = reinterpret_cast<ChUnit*>(ws + l.unit);
  a.start = reinterpret_cast<ChStart*>(ws + l.start);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  a.most = static_cast<int>(units);
  a.n_tokens = n_tokens;
  a.causal = causal != 0;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = G;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.ctas = ctas;
  a.zbox = zbox;
  a.by_g = G == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + G - 1) / G);
  a.by_tpp = tpp == 1 ? 0u : static_cast<uint32_t>(((uint64_t(1) << 32) + tpp - 1) / tpp);
  a.sm_scale_log2 = sm_scale * kChLog2e;
  a.small = B <= 32 && static_cast<int64_t>(n_tokens) * G <= kChSmallRows && static_cast<int64_t>(B) * max_pages <= kChSmallPages;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((!a.small && launch_dependent(prefill_plan_kernel, 1, kChPlanThreads, 0, s, a) != FPK_OK) ||
      launch_dependent(prefill_attn_kernel, ctas, kChThreads, ChCfg::kSmem, s, a, kmap, omap) != FPK_OK)
    return FPK_ECUDA;
  const int64_t rows = static_cast<int64_t>(n_tokens) * G;
  if (rows <= kChMergeAll || rows <= static_cast<int64_t>(kChMergeMean) * B)
    return launch_dependent(prefill_merge_kernel<kChMergeFew>, ctas * kChMergeFew, 32 * kChMergeWarps, 0, s, a);
  return launch_dependent(prefill_merge_kernel<kChMergeMany>, ctas * kChMergeMany, 32 * kChMergeWarps, 0, s, a);
}
