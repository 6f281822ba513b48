// prefix_attn.cu -- decode attention of a batch whose requests share prefixes,
// on the fifth-generation tensor cores.
//
// A group's shared prefix is a matrix product: the rows are the queries of all
// its requests that read one kv head (requests x GQA group), the columns the
// prefix's tokens.  What a request has of its own is decode attention, bound by
// HBM.  Four launches, each a dependent of the one before:
//   plan    the work list of the prefixes (one CTA)
//   own     beside the plan: the own tokens, and the queries as the prefixes'
//           products read them
//   attn    the prefixes, a CTA per SM
//   merge   each row's partials, by log-sum-exp
// (Without groups: paged_decode_split_kernel and the merge, which then only rounds.)
//
// * Unit: (group, kv head, up to 256 query rows) over the group's shared pages.
// * Units are laid end to end in cost (blocks of 128 tokens, dearer for units of
//   more than 128 rows, and a start) and the line is cut into one equal range per
//   CTA; a CTA runs a piece of a unit after another.  Every piece writes its partial
//   (m, l, O); the merge takes a row's partials in a fixed order, so repeated calls
//   give the same bits.
//
// Piece pipeline (one CTA per SM, 16 warps), per block of 128 tokens:
//   warp 15     finds the pieces ahead of the others
//   warp 12     lands K rows (128-byte swizzle) and V tiles by tensor maps
//   warps 8-11  e4m3 cache: V codes to f16 core matrices (exact), so that softmax
//               weights enter the second product in f16; both caches: zeroes
//               where no token lies (stale shared memory may hold NaN, and 0 NaN = NaN)
//   warps 13, 14  issue S = Q K^T and O += P V (tcgen05.mma, M = N = 128) of row
//               tile 0 and 1
//   warps 0-3, 4-7  softmax of row tile 0 and 1, a thread per row: no shuffles,
//               the row's maximum, sum and rescale are the thread's own.  P (both
//               parts of half a block in the columns of its scores) replaces S in
//               tensor memory as the A operand of the second product.
// Units of more than 128 rows use both tiles on every block; smaller ones give
// the two tiles alternate blocks of the same rows, each with its own partial.
//
// What bounds it.  A block of 256 rows is 3070 cycles of products (the two parts
// of an e4m3 query cost what one f16 product does, the two parts of the weights
// what two do): a tile's S, softmax, P V and next S follow one another (S and P
// share the tile's 128 columns of tensor memory, the accumulators have the other
// half), and two tiles in turn do not quite hide the chain: about 3700 cycles.  128
// requests x 32768 shared tokens, 64/8 heads, e4m3: the prefixes' kernel 114 us
// with the tensor cores at 81 %, the call 148 us (108 us are the products at the
// measured bf16 rate); in bf16, 164 us.  Few rows or short prefixes are bound by
// the four launches' chain of dependent reads: 4 requests x 512 tokens 18 us,
// 32 x 8192 34 us (41 where nothing is in L2).
//
// Precision.  bf16 cache: q, K, P and V in bf16 (the product takes one type, and V's
// range does not fit f16).  Weights are two parts, hi + lo, as in the framework's other
// decode attention: one bf16 part errs by up to 2^-8 of a weight, one f16 part by 2^-11,
// which shows where values cancel.  (With one part 128 x 32768 took 121 us.)  e4m3 cache:
// K enters as it lies; q x 2^e (its largest value in [128, 256)) as two e4m3 parts
// c0 + c1: a bf16's eight bits fill exactly two parts of four, but for values below
// 2^-9 of the largest, which lose at most 2^-17 of it; the MMAs' K runs over both parts
// against the same K rows, at the rate of one f16 product; weights are two f16 parts,
// and V is exact in one.  Scores, sums and O stay in fp32.  O is rescaled only when a
// row's maximum has grown by more than 2^8 since the last time: weights are then at most
// 2^8, far inside f16.
#include <atomic>

#include "attn_plan.cuh"
#include "tc_attn.cuh"

namespace fpk {
namespace {

constexpr int kPfTile = 16;
constexpr int kPfDim = 128;
constexpr int kPfGroupMax = 8;
constexpr int kPfBlk = 128;                    // tokens of a block
constexpr int kPfBlkTiles = kPfBlk / kPfTile;
constexpr int kPfUnitRows = 256;               // query rows of a prefix unit: two MMA tiles
constexpr float kPfLog2e = 1.4426950408889634f;
constexpr float kPfLn2 = 0.6931471805599453f;
constexpr float kPfGrow = 8.f;                 // log2 growth of a maximum that rescales O
// A row's scale is not taken below this (a scale of 0 leaves weights of 1 all the same): -inf times
// it is -inf still.  A NaN stays one.
constexpr float kPfMinMult = 1e-37f;
__device__ __forceinline__ float at_least_min(float mult) { return mult < kPfMinMult ? kPfMinMult : mult; }
// Costs in the work list, in some 500 cycles: of a block with both tiles at work and with one, and
// of a unit's start (queries, first products, partials).  (3 for a block with one, or starts of 8 and 3: 61
// ragged requests in five groups 60 -> 63 us, whole batches on one prompt the same.)
constexpr int kPfCostPair = 6, kPfCostSolo = 2;
constexpr int kPfStartPair = 12, kPfStartSolo = 5;

constexpr int kPfThreads = 512;
constexpr int kPfVWarp = 8, kPfLoadWarp = 12, kPfMmaWarp = 13, kPfPlanWarp = 15;  // two MMA warps
constexpr int kPfPieces = 4, kPfPieceBytes = 176;  // pieces known ahead
constexpr int kPfPlanThreads = 1024;
constexpr int kPfTurnSpins = 4096;  // looks at the other tile's turns, some 40 cycles each
constexpr int kPfMergeWarps = 4;

// What the planning kernel finds of each group.
struct alignas(16) PfGroup {
  int32_t y0;      // place of its units in the work list
  int32_t ptiles;  // tiles of the shared prefix
  int32_t first, count, leader;
  int32_t g, b0, b1;  // (of a CTA's first group: its number, the CTA's range)
};
static_assert(sizeof(PfGroup) == 32, "two 16-byte words");

struct PfArgs {
  const uint16_t* q;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const uint8_t* abort_mask;
  const int32_t* group_starts;
  const int32_t* prefix_lens;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  int32_t* gstart;   // [n_groups + 1] group starts, clamped and non-decreasing
  PfGroup* group;    // [n_groups]
  PfGroup* start;    // [ctas] the group in whose units a CTA's range begins: its record, number and the CTA's range
  int32_t* group_of; // [B], -1: none
  int32_t* own_len;  // [B] tokens behind the shared prefix; 0 for a dead request
  int32_t* dead;     // [B]
  const uint8_t* kv_pool;
  uint8_t* q_image;  // [2][Hkv][B][G][128 bytes]: query rows as the products read them (two parts, or two halves)
  float* q_mult;     // [Hkv][B][G]: their score multipliers
  const float* all_out;  // without groups: [B][Hq][D], [B][Hq], attention over all tokens
  const float* all_lse;
  float2* part_ml;   // partials: prefixes' 2 per (request, query head) and 256 rows per CTA, then own parts' osplits
  float* part_o;
  int n_groups, B, Hq, Hkv, G, page_size, num_pages, max_pages, ctas, zbox, osplits;
  uint32_t by_g, by_tpp;  // ceil(2^32 / G), ceil(2^32 / tiles of a page); 0 for 1
  float sm_scale_log2;
};

// Shared-memory map of the main kernel, from a 1024-byte aligned base.
template <bool kFp8>
struct PfCfg {
  static constexpr int kElem = kFp8 ? 1 : 2;
  static constexpr int kQTile = 128 * 256;                     // parts (or halves) of a tile's queries
  static constexpr int kKStage = kPfBlk * kPfDim * kElem;
  static constexpr int kVStage = kKStage;
  static constexpr int kKStages = kFp8 ? 4 : 2;
  static constexpr int kVStages = kFp8 ? 2 : 3;
  static constexpr int kV16 = kPfBlk * kPfDim * 2;             // converted V block
  static constexpr int kV16Bufs = kFp8 ? 2 : 0;
  static constexpr int kOffK = 2 * kQTile;
  static constexpr int kOffV = kOffK + kKStages * kKStage;
  static constexpr int kOffV16 = kOffV + kVStages * kVStage;
  static constexpr int kOffPiece = kOffV16 + kV16Bufs * kV16;
  static constexpr int kOffBars = kOffPiece + kPfPieces * kPfPieceBytes;
  // barriers
  static constexpr int kReady = kFp8 ? kV16Bufs : kVStages;    // V blocks ready for the MMA
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKFree = kBarKFull + kKStages;
  static constexpr int kBarVFull = kBarKFree + kKStages;
  static constexpr int kBarVFree = kBarVFull + kVStages;
  static constexpr int kBarReady = kBarVFree + kVStages;
  static constexpr int kBarUsed = kBarReady + kReady;          // e4m3: converted block read by the MMA
  static constexpr int kBarS = kBarUsed + kV16Bufs;            // [tile]
  static constexpr int kBarP = kBarS + 2;                      // [tile][half of the block]
  static constexpr int kBarO = kBarP + 4;                      // [tile] a product added to O
  static constexpr int kBarOFree = kBarO + 2;                  // [tile] O of a piece read
  static constexpr int kBarQ = kBarOFree + 2;                  // [buffer] queries staged
  static constexpr int kBarQFree = kBarQ + 2;                  // [buffer] queries of a piece read
  static constexpr int kBarPiece = kBarQFree + 2;              // [kPfPieces] piece known
  static constexpr int kBarPieceFree = kBarPiece + kPfPieces;  // [kPfPieces] piece read by every warp
  static constexpr int kBarDone = kBarPieceFree + kPfPieces;   // [2] every MMA of a warp completed
  static constexpr int kBars = kBarDone + 2;
  static constexpr int kOffMisc = kOffBars + 8 * kBars;        // tensor memory base, failure flag, turns taken by each tile
  static constexpr int kSmem = kOffMisc + 16;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// Context length of request r if it is alive by its length and abort flag, else 0.
__device__ __forceinline__ int live_length(const PfArgs& a, int r) {
  const int L = __ldg(a.seq_lens + r);
  if (L <= 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_pages) * a.page_size) return 0;
  if (a.abort_mask != nullptr && __ldg(a.abort_mask + r) != 0) return 0;
  return L;
}

// ---------------------------------------------------------------------------
// work list
// ---------------------------------------------------------------------------
// The part of a unit's place that its start takes; its blocks lie behind.
__device__ __forceinline__ int start_cost(int w) { return w == kPfCostPair ? kPfStartPair : kPfStartSolo; }
// Prefix units of a group, per kv head: `units` of up to 256 rows, all but the
// last of cost kPfCostPair per block (`step` each), the last of cost `wlast`.
struct PfPrefix {
  int blocks, units, wlast, step, head_cost;
};
__device__ __forceinline__ PfPrefix prefix_shape(int ptiles, int gcount, int G) {
  PfPrefix p;
  const int rows = gcount * G;
  p.blocks = (ptiles + kPfBlkTiles - 1) / kPfBlkTiles;
  p.units = (rows + kPfUnitRows - 1) / kPfUnitRows;
  p.wlast = rows - (p.units - 1) * kPfUnitRows > 128 ? kPfCostPair : kPfCostSolo;
  p.step = kPfStartPair + kPfCostPair * p.blocks;
  p.head_cost = p.step * (p.units - 1) + start_cost(p.wlast) + p.wlast * p.blocks;
  return p;
}

// CTA c owns the blocks that start in [begin(c), begin(c + 1)): T / n each, one
// more for the first T mod n CTAs.
struct PfRanges {
  int share, more;
  __device__ __forceinline__ int begin(int c) const { return c * share + min(c, more); }
  __device__ __forceinline__ int owner(int y) const {
    const int big = more * (share + 1);
    return y < big ? y / (share + 1) : more + (y - big) / share;
  }
};
__device__ __forceinline__ PfRanges ranges_of(int T, int n) {
  PfRanges r;
  r.share = T / n;
  r.more = T - r.share * n;
  return r;
}
// Blocks [i0, i1) that a range [b0, b1) owns of the n blocks of cost w of a unit, the first block at y.
__device__ __forceinline__ void owned_blocks(int y, int n, int w, int b0, int b1, int& i0, int& i1) {
  const int lo = max(b0 - y, 0) + w - 1, hi = max(b1 - y, 0) + w - 1;
  i0 = min(n, w == kPfCostPair ? lo / kPfCostPair : lo / kPfCostSolo);
  i1 = min(n, w == kPfCostPair ? hi / kPfCostPair : hi / kPfCostSolo);
}

struct alignas(16) PfPiece {
  int r;           // request whose table is read: the leader
  int h;
  int row0, rows;  // rows of the group
  int gfirst;      // request of row 0
  int i0, i1;      // blocks of the unit; none: the end
  int tokens;      // of the unit
  int qbuf;        // query buffer of a unit of one row tile
  int t0;          // parity of the blocks before, and tile of the first one of a unit of one row tile
  int pad[2];
  __device__ __forceinline__ bool pair() const { return rows > 128; }
};
struct alignas(16) PfSlot {
  PfPiece piece;
  int pages[32];  // of the first four blocks' tiles, -1 where the unit has none
};
static_assert(sizeof(PfSlot) == kPfPieceBytes, "slot of the piece ring");

struct PfCursor {
  PfGroup q;
  int g, h, u;  // u: unit of the head
  int y, b0, b1;
};

__device__ __forceinline__ PfGroup load_group(const PfGroup* at) {
  const int4* p = reinterpret_cast<const int4*>(at);
  const int4 x = __ldcg(p), y = __ldcg(p + 1);
  PfGroup q;
  q.y0 = x.x;
  q.ptiles = x.y;
  q.first = x.z;
  q.count = x.w;
  q.leader = y.x;
  q.g = y.y;
  q.b0 = y.z;
  q.b1 = y.w;
  return q;
}

__device__ __forceinline__ PfCursor begin_range(const PfArgs& a, const PfGroup& q) {
  PfCursor c;
  c.q = q;
  c.g = q.g;
  c.b0 = q.b0;
  c.b1 = q.b1;
  const PfPrefix p = prefix_shape(q.ptiles, q.count, a.G);
  const int at = q.b0 - q.y0;
  c.h = at / p.head_cost;
  c.u = min((at - c.h * p.head_cost) / p.step, p.units - 1);
  c.y = q.y0 + c.h * p.head_cost + c.u * p.step;
  return c;
}

__device__ __forceinline__ bool next_piece(const PfArgs& a, PfCursor& c, PfPiece& p) {
  for (;;) {
    if (c.y >= c.b1) return false;
    if (c.q.ptiles == 0 || c.h == a.Hkv) {
      if (++c.g >= a.n_groups) return false;
      c.q = load_group(a.group + c.g);
      c.h = c.u = 0;
      c.y = c.q.y0;
      continue;
    }
    const PfPrefix s = prefix_shape(c.q.ptiles, c.q.count, a.G);
    const int w = c.u == s.units - 1 ? s.wlast : kPfCostPair;
    p.r = c.q.leader;
    p.h = c.h;
    p.row0 = c.u * kPfUnitRows;
    p.rows = min(kPfUnitRows, c.q.count * a.G - p.row0);
    p.gfirst = c.q.first;
    p.tokens = c.q.ptiles * kPfTile;
    owned_blocks(c.y + start_cost(w), s.blocks, w, c.b0, c.b1, p.i0, p.i1);
    c.y += start_cost(w) + s.blocks * w;
    if (++c.u == s.units) {
      c.u = 0;
      ++c.h;
    }
    if (p.i0 < p.i1) return true;
  }
}

// One CTA: group ranges, shared pages and leaders, what the requests have of their
// own, the work list and every CTA's first group.
__global__ void __launch_bounds__(kPfPlanThreads, 1) prefix_plan_kernel(const PfArgs a) {
  __shared__ int s_sum[kPfPlanThreads / 32];
  __shared__ int s_max[kPfPlanThreads / 32];
  griddep_wait();  // what ran before is over: the own parts, which do not wait, may start behind it
  griddep_launch_dependents();
  const unsigned kFull = 0xffffffffu;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int tpp = a.page_size >> 4;
  // group starts: clamped, then the running maximum
  int carry = 0;
#pragma unroll 1
  for (int base = 0; a.n_groups > 0 && base <= a.n_groups; base += kPfPlanThreads) {
    const int i = base + t;
    int v = i <= a.n_groups ? min(max(__ldg(a.group_starts + i), 0), a.B) : 0;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, v, o);
      if (lane >= o) v = max(v, x);
    }
    if (lane == 31) s_max[warp] = v;
    __syncthreads();
    int w = s_max[lane];  // the warps' maxima, then those of the warps up to each
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(kFull, w, o);
      if (lane >= o) w = max(w, x);
    }
    const int before = __shfl_sync(kFull, w, max(warp - 1, 0));
    if (i <= a.n_groups) a.gstart[i] = max(max(v, carry), warp > 0 ? before : 0);
    carry = max(carry, __shfl_sync(kFull, w, 31));
    __syncthreads();
  }
#pragma unroll 1
  for (int r = t; r < a.B; r += kPfPlanThreads) {
    const int L = live_length(a, r);
    a.own_len[r] = L;
    a.group_of[r] = -1;
    a.dead[r] = L == 0;
  }
  __syncthreads();
  // what each group shares: whole pages of the prefix that every live request holds
#pragma unroll 1
  for (int g = warp; g < a.n_groups; g += kPfPlanThreads / 32) {
    const int lo = a.gstart[g], hi = a.gstart[g + 1];
    int least = 0x7fffffff, leader = 0x7fffffff;
#pragma unroll 1
    for (int r = lo + lane; r < hi; r += 32) {
      const int L = a.own_len[r];
      if (L > 0) {
        least = min(least, L);
        leader = min(leader, r);
      }
    }
    least = __reduce_min_sync(kFull, least);
    leader = __reduce_min_sync(kFull, leader);
    const int pages = hi - lo < 2 || leader == 0x7fffffff ? 0 : max(0, min(__ldg(a.prefix_lens + g), least)) / a.page_size;
    if (lane == 0) {
      PfGroup& q = a.group[g];
      q.ptiles = pages * tpp;
      q.first = lo;
      q.count = hi - lo;
      q.leader = leader;
    }
    if (pages == 0) continue;
#pragma unroll 1
    for (int r = lo + lane; r < hi; r += 32) {
      a.own_len[r] = max(0, a.own_len[r] - pages * a.page_size);
      a.group_of[r] = g;
    }
  }
  __syncthreads();
  // places in the work list
  const int chunk = (a.n_groups + kPfPlanThreads - 1) / kPfPlanThreads;
  const int gb = min(a.n_groups, t * chunk), ge = min(a.n_groups, gb + chunk);
  auto cost_of = [&](int g) -> int {
    const PfGroup& q = a.group[g];
    return q.ptiles > 0 ? prefix_shape(q.ptiles, q.count, a.G).head_cost * a.Hkv : 0;
  };
  int mine = 0;
#pragma unroll 1
  for (int g = gb; g < ge; ++g) mine += cost_of(g);
  int incl = mine;
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[warp] = incl;
  __syncthreads();
  int sums = s_sum[lane];
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(kFull, sums, o);
    if (lane >= o) sums += x;
  }
  const int below = __shfl_sync(kFull, sums, max(warp - 1, 0));
  const int T = __shfl_sync(kFull, sums, 31);
  int y = incl - mine + (warp > 0 ? below : 0);
#pragma unroll 1
  for (int g = gb; g < ge; ++g) {
    a.group[g].y0 = y;
    y += cost_of(g);
  }
  __syncthreads();
  // every CTA's first group: the last one whose units start at or before its range
  const PfRanges rg = ranges_of(T, a.ctas);
#pragma unroll 1
  for (int c = t; c < a.ctas; c += kPfPlanThreads) {
    const int b0 = rg.begin(c);
    int lo = 0, hi = a.n_groups - 1;
#pragma unroll 1
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.group[mid].y0 <= b0) lo = mid; else hi = mid - 1;
    }
    PfGroup q = a.group[lo];
    q.g = lo;
    q.b0 = b0;
    q.b1 = rg.begin(c + 1);
    a.start[c] = q;
  }
}

// ---------------------------------------------------------------------------
// products and weights in two parts
// ---------------------------------------------------------------------------
// O += P V over half a block, P from tensor memory: a step is 16 tokens, 8 columns of each part of P and 4 KiB of V.
#define PF_O_STEP(pcol, voff, acc)                                                                  \
  "add.u32 p, %1, " #pcol ";\n\tadd.s64 b, %2, " #voff ";\n\t@e tcgen05.mma.cta_group::1.kind::f16" \
  " [%0], [p], b, %3, " acc ";\n\t"
__device__ __forceinline__ void issue_o(uint32_t d, uint32_t p, uint64_t vdesc, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred e, first, yes;\n\t.reg .b32 p;\n\t.reg .b64 b;\n\telect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.u32 first, %4, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\t" PF_O_STEP(0, 0, "first") PF_O_STEP(8, 256, "yes")
          PF_O_STEP(16, 512, "yes") PF_O_STEP(24, 768, "yes") PF_O_STEP(32, 0, "yes") PF_O_STEP(40, 256, "yes")
              PF_O_STEP(48, 512, "yes") PF_O_STEP(56, 768, "yes") "}" ::"r"(d),
      "r"(p), "l"(vdesc), "r"(idesc), "r"(acc)
      : "memory");
}

// A pair of softmax weights as two parts, each of two f16 (e4m3 cache) or two bf16: rounded, and what that left.
template <bool kFp8>
__device__ __forceinline__ void weight_parts(float2 e, uint32_t& hi, uint32_t& lo) {
  if (kFp8) {
    hi = pack_f16x2(e.x, e.y);
    const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = pack_f16x2(e.x - h.x, e.y - h.y);
  } else {
    hi = pack_bf16x2(e.x, e.y);
    lo = pack_bf16x2(e.x - __uint_as_float(hi << 16), e.y - __uint_as_float(hi & 0xFFFF0000u));
  }
}

template <bool kFp8>
__global__ void __launch_bounds__(kPfThreads, 1)
    prefix_attn_kernel(const PfArgs a, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  using C = PfCfg<kFp8>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const sm = smem_raw;
  const uint32_t sbase = smem_addr(sm);
  if (sbase & 1023u) {  // (cannot happen: the array is aligned, and there is no other shared memory)
    if (threadIdx.x == 0) atomicOr(a.status, kStatusBadStart);
    return;
  }
  auto bar = [&](int i) -> uint32_t { return sbase + C::kOffBars + 8 * i; };
  PfSlot* const s_piece = reinterpret_cast<PfSlot*>(sm + C::kOffPiece);
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(sm + C::kOffMisc);
  volatile int* const s_failed = reinterpret_cast<volatile int*>(sm + C::kOffMisc + 4);
  const unsigned kFull = 0xffffffffu;
  const int warp = __shfl_sync(kFull, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  griddep_launch_dependents();
  if (threadIdx.x < C::kBars) {
    const int i = threadIdx.x;
    int arrivals = 1;
    if (i < C::kBarVFull && i >= C::kBarKFree) arrivals = 2;                         // MMA warps
    if (i >= (kFp8 ? C::kBarUsed : C::kBarVFree) && i < (kFp8 ? C::kBarS : C::kBarReady)) arrivals = 2;
    if (i >= C::kBarReady && i < C::kBarReady + C::kReady) arrivals = 4;             // V warps
    if (kFp8 && i >= C::kBarVFree && i < C::kBarVFree + C::kVStages) arrivals = 4;   // V warps
    if (i >= C::kBarP && i < C::kBarP + 4) arrivals = 4;                             // a tile's softmax warps
    if (i >= C::kBarOFree && i < C::kBarOFree + 2) arrivals = 4;                     // a tile's softmax warps
    if (i >= C::kBarQFree && i < C::kBarQFree + 2) arrivals = 10;                    // MMA and softmax warps
    if (i >= C::kBarPieceFree && i < C::kBarPieceFree + kPfPieces) arrivals = 16;    // every other warp; K's and V's half of one
    mbar_init(bar(i), arrivals);
    fence_barrier_init();
  }
  volatile int* const s_turns = reinterpret_cast<volatile int*>(sm + C::kOffMisc + 8);
  if (threadIdx.x == 0) *s_failed = s_turns[0] = s_turns[1] = 0;
  if (warp == kPfMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(s_tmem)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_wait();  // the plan is there
  const uint32_t tmem = *s_tmem;
  const PfGroup first = load_group(a.start + blockIdx.x);
  auto wait = [&](int i, uint32_t parity) { tc_wait(bar(i), parity & 1u, a.status, s_failed); };
  // the next piece, from the planning warp; false at the end
  uint32_t pn = 0;
  auto take_piece = [&](PfPiece& p) -> bool {
    wait(C::kBarPiece + pn % kPfPieces, pn / kPfPieces);
    p = s_piece[pn % kPfPieces].piece;
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(C::kBarPieceFree + pn % kPfPieces));
    ++pn;
    return __all_sync(kFull, p.i0 < p.i1 && !*s_failed);
  };
  if (first.b0 < first.b1) {
    PfPiece p;
    const int tpp = a.page_size >> 4;
    if (warp == kPfPlanWarp) {
      // ===================== pieces, ahead of the other warps =====================
      // And the check that a group's tables agree: the units of kv head 0 cover every shared page once per
      // 256 rows, and each request of the unit must name the leader's pages, which must be in the pool.
      PfCursor cur = begin_range(a, first);
      int qbuf = 0, t0 = 0;
      bool more = true;
#pragma unroll 1
      for (uint32_t n = 0; more; ++n) {
        more = next_piece(a, cur, p);
        if (!more) p.i0 = p.i1 = 0;
        p.qbuf = qbuf;
        qbuf ^= 1;
        p.t0 = t0;
        t0 ^= (p.i1 - p.i0) & 1;
        // the first blocks' pages: copies need not wait for the table, which may come from far
        const int tile = p.i0 * kPfBlkTiles + lane;
        const bool some = more && tile * kPfTile < p.tokens;
        const int32_t* lead = a.page_table + static_cast<int64_t>(more ? p.r : 0) * a.max_pages;
        const int page = some ? max(-1, __ldg(lead + quotient(tile, a.by_tpp))) : -1;
        if (n >= kPfPieces) wait(C::kBarPieceFree + n % kPfPieces, n / kPfPieces - 1);
        PfSlot* const at = s_piece + n % kPfPieces;
        at->pages[lane] = page;
        if (lane == 0) at->piece = p;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(C::kBarPiece + n % kPfPieces));
        if (more && p.h == 0) {
          const int p0 = quotient(p.i0 * kPfBlkTiles, a.by_tpp);
          const int p1 = quotient(min(p.i1 * kPfBlkTiles, p.tokens / kPfTile) + tpp - 1, a.by_tpp);
          const int r0 = p.gfirst + quotient(p.row0, a.by_g), r1 = p.gfirst + quotient(p.row0 + p.rows - 1, a.by_g);
#pragma unroll 1
          for (int i = p0 + lane; i < p1; i += 32) {
            const int want = __ldg(lead + i);
            const bool in = want >= 0 && want < a.num_pages;
#pragma unroll 4
            for (int r = r0; r <= r1; ++r)
              if (!in || __ldg(a.page_table + static_cast<int64_t>(r) * a.max_pages + i) != want) a.dead[r] = 1;
          }
        }
      }
    } else if (warp == kPfLoadWarp) {
      // ===================== K rows, V tiles into their rings =====================
      // The lower half-warp copies K, the upper one V, each with its own piece and place (the rings drain
      // at different times), in one loop that looks at both and waits for neither.  Lane c of a half
      // copies box c of a block (zbox tiles, within a page); bf16 K: lanes 8 + c the other 64 dims.
      const bool kw = lane < 16;
      const unsigned group = kw ? 0xffffu : 0xffff0000u;
      const bool leads = (lane & 15) == 0;
      const uint64_t pol = l2_policy_evict_normal();  // (other units and CTAs read the same pages)
      const int c = lane & 7;
      const int box_t = c * a.zbox;                        // first tile of the box in a block
      const bool copies = c < kPfBlkTiles / a.zbox && ((lane & 8) == 0 || (kw && !kFp8));
      const uint32_t stages = kw ? C::kKStages : C::kVStages;
      const uint32_t full = bar(kw ? C::kBarKFull : C::kBarVFull), free = bar(kw ? C::kBarKFree : C::kBarVFree);
      const uint32_t ring = sbase + (kw ? C::kOffK : C::kOffV) +
                            (kw ? (lane & 8) / 8 * kPfBlk * 128 + box_t * kPfTile * 128 : box_t * kPfTile * kPfDim * C::kElem);
      const void* const map = kw ? &kmap : &vmap;
      const int mx = kw ? (lane & 8) * 8 : 0, my = kw ? 0 : kFp8 ? 16 : 128;
      auto all_of_half = [&](bool x) -> bool { return (__ballot_sync(kFull, x) & group) == group; };
      const int32_t* row = nullptr;
      int i = 0, tiles = 0;
      uint32_t j = 0, st = 0, round = 0, idle = 0;
      bool have = false, done = false;
      // pages of 16 tiles, one per lane of the half: of this block and the next (an even number of blocks
      // into the piece), and of the two behind them, asked for two blocks before they are needed
      int now = -1, then = -1;
      while (!__all_sync(kFull, done)) {
        ++idle;
        if (all_of_half(!have && !done && mbar_test(bar(C::kBarPiece + pn % kPfPieces), pn / kPfPieces & 1))) {
          const PfSlot& slot = s_piece[pn % kPfPieces];
          p = slot.piece;
          then = slot.pages[16 + (lane & 15)];
          now = slot.pages[lane & 15];
          __syncwarp(group);
          if (leads) mbar_arrive(bar(C::kBarPieceFree + pn % kPfPieces));
          ++pn;
          have = p.i0 < p.i1;
          done = !have;
          i = p.i0;
          row = a.page_table + static_cast<int64_t>(p.r) * a.max_pages;
          tiles = p.tokens / kPfTile;
          idle = 0;
        }
        const bool goes = all_of_half(have && (round == 0 || mbar_test(free + 8 * st, (round - 1) & 1)));
        if (goes) {
          const int behind = i - p.i0;
          if (behind > 0 && (behind & 1) == 0) {
            now = then;
            then = -1;
            const int tile = (i + 2) * kPfBlkTiles + (lane & 15);
            if (tile < min(tiles, p.i1 * kPfBlkTiles)) then = __ldg(row + quotient(tile, a.by_tpp));
          }
          const int tile = i * kPfBlkTiles + box_t;
          const int pg = __shfl_sync(group, now, (behind & 1) * 8 + box_t, 16);
          // (one outside the pool is not copied: the check has it)
          const bool good = copies && tile < tiles && pg >= 0 && pg < a.num_pages;
          const uint32_t boxes = __popc(__ballot_sync(group, good));
          const uint32_t f = full + 8 * st;
          if (leads) {
            const uint32_t bytes = boxes * a.zbox * (kPfTile * (kw ? 128 : kPfDim * C::kElem));
            if (bytes == 0) mbar_arrive(f);
            else mbar_arrive_expect_tx(f, bytes);
          }
          __syncwarp(group);
          if (good)
            tma_load_3d(ring + st * C::kKStage, map, mx, my,
                        (pg * a.Hkv + p.h) * tpp + tile - quotient(tile, a.by_tpp) * tpp, f, pol);
          if (++st == stages) st = 0, ++round;
          ++j;
          if (++i == p.i1) have = false;
          idle = 0;
        }
        // (whoever waits for a copy gives up in time)
        if (__any_sync(kFull, (idle & 255u) == 255u && *s_failed != 0)) done = true;
      }
      // every copy has landed before the CTA ends
      if (leads) {
#pragma unroll 1
        for (uint32_t b = j > stages ? j - stages : 0; b < j; ++b)
          mbar_wait(full + 8 * (b % stages), (b / stages) & 1, a.status);
      }
    } else if (warp >= kPfVWarp && warp < kPfVWarp + 4) {
      // ===================== V blocks made ready for the MMA =====================
      const int d = threadIdx.x - kPfVWarp * 32;  // this thread's dim
      uint32_t j = 0;
      while (take_piece(p)) {
#pragma unroll 1
        for (int i = p.i0; i < p.i1; ++i, ++j) {
          const int nv = min(kPfBlk, p.tokens - i * kPfBlk);
          const uint32_t vs = j % C::kVStages;
          uint8_t* const v = sm + C::kOffV + vs * C::kVStage;
          wait(C::kBarVFull + vs, j / C::kVStages);
          if (kFp8) {
            const uint32_t buf = j % C::kReady;
            if (j >= static_cast<uint32_t>(C::kReady)) wait(C::kBarUsed + buf, j / C::kReady - 1);
            uint8_t* const o = sm + C::kOffV16 + buf * C::kV16 + d * 16;
            const int tiles = (nv + kPfTile - 1) / kPfTile;
#pragma unroll 2
            for (int t = 0; t < tiles; ++t) {
              // codes of dim d, tokens 16 t .. 16 t + 15, to two rows of 8 f16
              const uint4 x = *reinterpret_cast<const uint4*>(v + t * kPfTile * kPfDim + d * 16);
              uint32_t y[8];
              e4m3x4_to_f16x4(x.x, y[0], y[1]);
              e4m3x4_to_f16x4(x.y, y[2], y[3]);
              e4m3x4_to_f16x4(x.z, y[4], y[5]);
              e4m3x4_to_f16x4(x.w, y[6], y[7]);
              uint4* const w = reinterpret_cast<uint4*>(o + t * kPfTile * kPfDim * 2);
              w[0] = make_uint4(y[0], y[1], y[2], y[3]);
              w[128] = make_uint4(y[4], y[5], y[6], y[7]);
            }
            if (nv < kPfBlk) {  // f16 of token k, dim d: rows of 8 tokens, 2 KiB apart
#pragma unroll 1
              for (int k = nv; k & 63; k = (k | 7) + 1)
                for (uint8_t* e = o + (k >> 3) * 2048 + (k & 7) * 2; e < o + (k >> 3) * 2048 + 16; e += 2)
                  *reinterpret_cast<uint16_t*>(e) = 0;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(C::kBarReady + buf));
              mbar_arrive(bar(C::kBarVFree + vs));
            }
          } else {
            if (nv < kPfBlk) {
              // rows of 16 tokens with the 32-byte swizzle: the two 16-byte halves change places
              // in every other group of four rows
#pragma unroll 1
              for (int k = nv; k & 63; k = (k | 7) + 1) {
                uint8_t* const x = v + (k >> 4) * kPfTile * kPfDim * 2 + d * 32 + (((k >> 3) & 1) ^ ((d >> 2) & 1)) * 16;
                for (uint8_t* e = x + (k & 7) * 2; e < x + 16; e += 2) *reinterpret_cast<uint16_t*>(e) = 0;
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarReady + vs));
          }
        }
      }
    } else if (warp == kPfMmaWarp || warp == kPfMmaWarp + 1) {
      // ===================== MMA issue, a warp per row tile =====================
      // The warp runs as one, an elected lane issues.  A tile's products alternate: S of a block, PV of the
      // same block in halves as the softmax hands P over, S of the next (which overwrites S and P: the
      // products of one thread run in order).  While a tile's softmax runs the other tile has the tensor
      // cores; on a unit of both tiles the warps take turns (PV and the next S), or else the two would run
      // in step, their softmaxes too, and leave the tensor cores idle (with weights in one part 4080 cycles a
      // block of 256 rows, the products' own time being 2050).  An issuing warp stands still until the tensor cores take its product,
      // so all waits of a turn come before it, what follows is straight code (it comes cold from the instruction
      // caches each time), and turns are counted in shared memory, not by a barrier (no result hangs on it, a turn
      // not seen is gone without): 3820 cycles a block without these three, about 2900 with them (in two parts 3700).
      //
      // On a unit of one row tile block j belongs to tile j mod 2.  A barrier's parity tells neighbouring
      // phases apart, no others, so a warp has to see every phase of a barrier it waits for: where the
      // number of slots is even, a tile has its own slots and sees all of theirs; bf16 V has three slots,
      // and both warps see and free every block.  (Turns do not keep the warps in step: the CPU model
      // of these barriers passes without them.)
      const int t = warp - kPfMmaWarp;
      const uint32_t base = __reduce_max_sync(kFull, sbase), tm = __reduce_max_sync(kFull, tmem);  // uniform registers
      const uint32_t bars = base + C::kOffBars;
      const uint64_t qdesc = smem_desc(base, 16, 1024, 2), kdesc = smem_desc(base + C::kOffK, 16, 1024, 2);
      // V, 16 tokens a step: e4m3 as two columns of core matrices (8 dims x 8 tokens, 128 B apart along
      // the dims, 2 KiB along the tokens), bf16 as rows of 32 bytes with the 32-byte swizzle
      const uint64_t vdesc = kFp8 ? smem_desc(base + C::kOffV16, 2048, 128, 0) : smem_desc(base + C::kOffV, 16, 256, 6);
      uint32_t j0 = 0, v3 = 0, v3ph = 0, n0 = 0, n1 = 0, begun = 0, uses0 = 0, uses1 = 0;
      int turns = 0;
      const uint32_t turn_of = base + C::kOffMisc + 8 + 4 * (t ^ 1);
      static_assert(C::kKStages % 2 == 0 && (!kFp8 || C::kReady == 2), "slots that tiles own");
      while (take_piece(p)) {
        const int pair_in = __any_sync(kFull, p.pair());
        const uint32_t nb = __reduce_max_sync(kFull, p.i1 - p.i0), qb = __reduce_max_sync(kFull, p.qbuf);
        const uint32_t halves = __reduce_max_sync(kFull, (p.tokens - p.i0 * kPfBlk + 63) / 64);  // of the piece, and behind it
        const uint32_t step = pair_in ? 1 : 2;
        if (pair_in || qb == 0) wait(C::kBarQ, uses0++);
        if (pair_in || qb == 1) wait(C::kBarQ + 1, uses1++);
        const uint64_t qd = qdesc + (pair_in ? t : qb) * (C::kQTile >> 4);
        bool begins = true;
        uint32_t passed = 0;  // bf16: V blocks seen
        // the other tile's bf16 V blocks up to block m
        auto pass_v = [&](uint32_t m) {
#pragma unroll 1
          while (!kFp8 && passed < m) {
            wait(C::kBarReady + v3, v3ph);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C::kBarVFree + v3));
            if (++v3 == C::kReady) v3 = 0, v3ph ^= 1;
            ++passed;
          }
        };
#pragma unroll 1
        for (uint32_t i = pair_in ? 0 : (j0 ^ t) & 1; i < nb + step; i += step) {
          // PV of this tile's block before, S of block i: what they need first, then the turn
          const bool pair = varying(pair_in) != 0;
          const uint32_t ks = (j0 + i) % C::kKStages, m = i - step, jm = j0 + m;
          if (i < nb) wait(C::kBarKFull + ks, (j0 + i) / C::kKStages);
          uint32_t vs = 0;
          if (i >= step) {
            pass_v(m);
            vs = kFp8 ? jm % C::kReady : v3;
            wait(C::kBarReady + vs, kFp8 ? jm / C::kReady : v3ph);
            if (begins && begun > 0) wait(C::kBarOFree + t, begun - 1);  // O of the piece before has been read
            wait(C::kBarP + 2 * t, n0++);
          }
          tc_fence_after();
          const uint64_t vd = vdesc + vs * ((kFp8 ? C::kV16 : C::kVStage) >> 4);
          const uint32_t od = tm + 256 + t * 128, pd = tm + t * 128, acc = !begins;
          const bool both = 2 * m + 1 < halves;
          if (pair) {
#pragma unroll 1
            for (int spins = 0; load_shared(turn_of) - turns < t && spins < kPfTurnSpins; ++spins) {
            }
          }
          if (i >= step) {
            issue_o(od, pd, vd, kFp8 ? kTcOF16 : kTcOBf16, acc);
            if (both) {
              wait(C::kBarP + 2 * t + 1, n1++);
              tc_fence_after();
              issue_o(od, pd + 64, vd + 1024, kFp8 ? kTcOF16 : kTcOBf16, 1);
            }
            begun += begins;
            begins = false;
          }
          if (i < nb) issue_s<kFp8>(tm + t * 128, qd, kdesc + ks * (C::kKStage >> 4));
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
            commit_elected(bars + 8 * (C::kBarO + t));
            const uint32_t bv = bars + 8 * ((kFp8 ? C::kBarUsed : C::kBarVFree) + vs);
            commit_elected(bv);
            if (kFp8 && !pair) commit_elected(bv);  // for the other tile too
            if (!kFp8) {
              ++passed;
              if (++v3 == C::kReady) v3 = 0, v3ph ^= 1;
            }
          }
        }
        pass_v(nb);
        j0 += nb;
        // the queries: this warp's S are done (of a pair it answers for both buffers: it has seen both filled)
#pragma unroll 1
        for (uint32_t b = pair_in ? 0 : qb; b <= (pair_in ? 1 : qb); ++b) commit_elected(bars + 8 * (C::kBarQFree + b));
      }
      // every product and every arrival it owes is done before the CTA ends
      commit_elected(bars + 8 * (C::kBarDone + t));
      mbar_wait(bar(C::kBarDone + t), 0, a.status);
    } else {
      // ===================== softmax, a thread per row =====================
      const int t = warp >> 2;                       // row tile
      const int row = threadIdx.x & 127;
      const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
      const uint32_t ts = tmem + t * 128 + lanes, to = tmem + 256 + t * 128 + lanes;
      uint32_t ns = 0;                               // S blocks taken of this tile
      uint32_t uses[2] = {0, 0};                     // query buffers taken
      while (take_piece(p)) {
        const bool pair = p.pair();
        const int nb = p.i1 - p.i0;
        const int lrow = pair ? t * 128 + row : row;  // row of the unit
        const bool valid = lrow < p.rows;
        const bool busy = lrow - lane < p.rows;       // some row of the warp's is
        const int buf = pair ? t : p.qbuf;
        // ---- the queries into shared memory
        if (pair || t == 0) {
          const uint32_t u = buf ? uses[1] : uses[0];
          if ((warp & 3) == 0) {
            if (u > 0) wait(C::kBarQFree + buf, u - 1);
            if (lane == 0) {
              const int n = max(0, min(128, p.rows - lrow));
              const int64_t at = (static_cast<int64_t>(p.h) * a.B + p.gfirst) * a.G + p.row0 + lrow;
              const uint8_t* const src = a.q_image + at * 128;
              const uint32_t dst = sbase + buf * C::kQTile;
              if (n > 0) {
                mbar_arrive_expect_tx(bar(C::kBarQ + buf), n * 256);
                bulk_copy(dst, src, n * 128, bar(C::kBarQ + buf));
                bulk_copy(dst + 16384, src + static_cast<int64_t>(a.B) * a.Hq * 128, n * 128, bar(C::kBarQ + buf));
              } else {
                mbar_arrive(bar(C::kBarQ + buf));
              }
            }
          }
        }
        const float mult = valid ? __ldcg(a.q_mult + (static_cast<int64_t>(p.h) * a.B + p.gfirst) * a.G + p.row0 + lrow) : 0.f;
        wait(C::kBarQ + buf, buf ? uses[1] : uses[0]);
        // (whoever asked for the rows has them before the CTA ends, whatever failed elsewhere)
        if ((pair || t == 0) && (warp & 3) == 0) mbar_wait(bar(C::kBarQ + buf), (buf ? uses[1] : uses[0]) & 1, a.status);
        __syncwarp();
        if (pair || p.qbuf == 0) ++uses[0];
        if (pair || p.qbuf == 1) ++uses[1];
        // (of a pair each tile's warps answer for their own buffer, twice: they have seen no other filled)
        if (lane <= (pair ? 1 : 0)) mbar_arrive(bar(C::kBarQFree + buf));
        // ---- blocks
        float m = -INFINITY, l = 0.f;
        bool any = false;
#pragma unroll 1
        for (int i = pair ? 0 : t ^ p.t0; i < nb; i += pair ? 1 : 2) {
          wait(C::kBarS + t, ns);
          if (ns > 0) wait(C::kBarO + t, ns - 1);  // (over already: S came behind that product)
          tc_fence_after();
          const int nv = p.tokens - (p.i0 + i) * kPfBlk, halves = nv > 64 ? 2 : 1;  // (a half without tokens is left out)
          if (busy) {
            if (nv < kPfBlk) {
              // columns behind the last token: -inf, written to tensor memory by a short loop (selects
              // on registers would be a second copy of the code below, fetched anew for every tail)
#pragma unroll 1
              for (int k = nv; k & 63;) {
                if (k & 7) {
                  tmem_fill1(ts + k, -INFINITY);
                  ++k;
                } else if (k & 31) {
                  tmem_fill8(ts + k, -INFINITY);
                  k += 8;
                } else {
                  tmem_fill32(ts + k, -INFINITY);
                  k += 32;
                }
              }
              tmem_wait_st();
            }
            // the second half's maximum, then the first half with its own
            float s[64], mx;
            {
              const float top = halves == 2 ? tmem_ld64_max(ts + 64, s) : -INFINITY;
              mx = fmaxf(tmem_ld64_max(ts, s), top);
            }
            const float mb = mx == -INFINITY ? -INFINITY : mx * mult;
            const bool grown = mb > m + kPfGrow || (m == -INFINITY && mb != -INFINITY);
            if (__any_sync(kFull, grown)) {
              const float f = !grown ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - mb);
              if (grown) m = mb;
              l *= f;
              if (any) {  // O of the blocks before
#pragma unroll 1
                for (int c = 0; c < 8; ++c) tmem_scale16(to + 16 * c, f);
              }
            }
            const float ref = m == -INFINITY ? 0.f : m;
            const float2 mult2 = make_float2(mult, mult), ref2 = make_float2(-ref, -ref);
            float2 sum[2] = {make_float2(l, 0.f), make_float2(0.f, 0.f)};
#pragma unroll 1
            for (int h = 0; h < halves; ++h) {
              if (h == 1) tmem_ld64(ts + 64, s);
              // (stored eight columns at a time: with 16 or 32 the compiler holds more than the registers can)
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint32_t w[8], v[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                  float2 e = fma2(make_float2(s[16 * g + 2 * k], s[16 * g + 2 * k + 1]), mult2, ref2);
                  e.x = fast_exp2(e.x);
                  e.y = fast_exp2(e.y);
                  sum[k & 1] = add2(sum[k & 1], e);
                  weight_parts<kFp8>(e, w[k], v[k]);
                }
                tmem_st8(ts + 64 * h + 8 * g, w);  // over columns that have been read
                tmem_st8(ts + 64 * h + 32 + 8 * g, v);
              }
              tmem_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(bar(C::kBarP + 2 * t + h));
            }
            l = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          } else {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(bar(C::kBarP + 2 * t));
              if (halves == 2) mbar_arrive(bar(C::kBarP + 2 * t + 1));
            }
          }
          any = true;
          ++ns;
        }
        // ---- the row's partial: pieces at a unit's start by row, others by CTA
        const int grow = p.row0 + lrow, rq = quotient(grow, a.by_g);
        int64_t slot = static_cast<int64_t>(2) * a.B * a.Hq + static_cast<int64_t>(blockIdx.x) * kPfUnitRows + t * 128 + row;
        if (p.i0 == 0 && valid)
          slot = static_cast<int64_t>(pair ? 0 : t) * a.B * a.Hq +
                 static_cast<int64_t>(p.gfirst + rq) * a.Hq + p.h * a.G + grow - rq * a.G;
        if (any) {
          wait(C::kBarO + t, ns - 1);
          tc_fence_after();
          if (busy) {
            const float vscale = kFp8 ? __ldg(a.v_scale) : 1.f;
            float* const dst = a.part_o + slot * kPfDim;
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              float o[64];
              tmem_ld64(to + 64 * c, o);
              if (valid) {
#pragma unroll
                for (int k = 0; k < 64; k += 8) {
                  const float x[8] = {o[k] * vscale,     o[k + 1] * vscale, o[k + 2] * vscale, o[k + 3] * vscale,
                                      o[k + 4] * vscale, o[k + 5] * vscale, o[k + 6] * vscale, o[k + 7] * vscale};
                  st_global8(dst + 64 * c + k, x);
                }
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(C::kBarOFree + t));
        }
        if (valid) a.part_ml[slot] = make_float2(m, l);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kPfMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

// ---------------------------------------------------------------------------
// own parts
// ---------------------------------------------------------------------------
// A request's own tokens, kv head by kv head, in up to osplits splits of at
// least 256 tokens: a CTA of four warps per split, a warp taking every fourth
// tile of 16 tokens, by bulk copies into a ring of its own (mma.sync: the rows
// are the at most eight heads of a GQA group, which is too few for a tcgen05
// tile, and the work is reading: 192 KiB per SM on their way).  The layout of
// the pool suits the fragments with the dims of K and the tokens of V permuted:
// lane (g, c) = (lane / 4, lane % 4) holds 16-byte chunks c, c + 4, .. of its K
// tokens -- S takes them as they come, of q and K alike -- and tokens 4 c ..
// 4 c + 3 of its V dims, which are the very tokens of the scores that the lane
// holds for head g: P enters the second product from the registers where S
// left it.  70 MB of own tokens of 128 requests: 27 us from a cold L2, 100 MB of
// 61 ragged requests in bf16 24 us (registers as the only buffer: 33 and 29).
constexpr int kOwnWarps = 4;
constexpr int kOwnMinTiles = 16;  // of a split
constexpr float kOwnFails = -1.f;  // sum of a split with a page outside the pool
__device__ __forceinline__ int own_splits(int tiles, int most) {
  return min(most, (tiles + kOwnMinTiles - 1) / kOwnMinTiles);
}
// First slot of the own parts' partials: split z of row i is at own_slot0 + z rows + i.
__device__ __forceinline__ int64_t own_slot0(const PfArgs& a) {
  return static_cast<int64_t>(2) * a.B * a.Hq + static_cast<int64_t>(a.ctas) * kPfUnitRows;
}

// The ring of a warp, and the CTA's shared memory: rings (later the warps' O), barriers, maxima and sums.
constexpr int kOwnRing = 16384;
template <bool kFp8>
struct OwnCfg {
  static constexpr int kTileBytes = 2 * kPfTile * kPfDim * (kFp8 ? 1 : 2);
  static constexpr int kStages = kOwnRing / kTileBytes;
};
constexpr int kOwnSmem = kOwnWarps * (kOwnRing + 4 * 8 + kPfGroupMax * 8);
constexpr int kOwnRow = kPfDim + 4;
static_assert(kPfGroupMax * kOwnRow * 4 <= kOwnRing, "a warp's O fits its ring");

template <bool kFp8>
__device__ __forceinline__ void own_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if (kFp8) mma_f16(d, a, b0, b1);
  else mma_bf16(d, a, b0, b1);
}

// The pages that request r shares and its group's first request, found by one warp on its own (as the planning
// kernel finds them for all): the group ends at the first start above r.
struct OwnShare {
  int skip, lo;
};
__device__ __forceinline__ OwnShare share_of(const PfArgs& a, int r, int lane) {
  const unsigned kFull = 0xffffffffu;
  auto start = [&](int i) -> int { return min(max(__ldg(a.group_starts + i), 0), a.B); };
  int live[4];  // the first 128 lengths, asked for with the starts
#pragma unroll
  for (int k = 0; k < 4; ++k) live[k] = lane + 32 * k < a.B ? live_length(a, lane + 32 * k) : 0;
  int first = 0x7fffffff;
#pragma unroll 4
  for (int i = lane; i <= a.n_groups; i += 32)
    if (start(i) > r) first = min(first, i);
  first = __reduce_min_sync(kFull, first);
  OwnShare s = {0, 0};
  if (first == 0 || first > a.n_groups) return s;
  const int prefix = __ldg(a.prefix_lens + first - 1), hi = start(first);
#pragma unroll 4
  for (int i = lane; i < first; i += 32) s.lo = max(s.lo, start(i));
  s.lo = __reduce_max_sync(kFull, s.lo);
  if (hi - s.lo < 2) return s;
  int least = 0x7fffffff;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (lane + 32 * k >= s.lo && lane + 32 * k < hi && live[k] > 0) least = min(least, live[k]);
#pragma unroll 4
  for (int i = max(s.lo, 128) + lane; i < hi; i += 32) {
    const int L = live_length(a, i);
    if (L > 0) least = min(least, L);
  }
  least = __reduce_min_sync(kFull, least);
  s.skip = least == 0x7fffffff ? 0 : max(0, min(prefix, least)) / a.page_size;
  return s;
}

// The query rows of request r, kv head h, as the products of a prefix read them: 128-byte rows with the 128-byte
// swizzle of their place in the group's units.  e4m3 scores take a query as two parts, q 2^e = p0 + p1, e such
// that the row's largest value lies in [128, 256): p0 is the value rounded to e4m3, p1 what that left, so that
// the pair holds eight bits of mantissa (bf16 has eight) down to 2^-6 and steps of 2^-9 below.
template <bool kFp8>
__device__ __forceinline__ void put_query(const PfArgs& a, int r, int h, int lo, int lane) {
  const unsigned kFull = 0xffffffffu;
  const int g = lane >> 2, c = lane & 3;  // head of the group, dims 32 c .. 32 c + 31
  const int64_t at = (static_cast<int64_t>(h) * a.B + r) * a.G + g;
  const int swizzle = ((r - lo) * a.G + g) & 7;
  uint8_t* const p0 = a.q_image + at * 128;
  uint8_t* const p1 = p0 + static_cast<int64_t>(a.B) * a.Hq * 128;
  const uint4* const src = reinterpret_cast<const uint4*>(
      a.q + (static_cast<int64_t>(r) * a.Hq + h * a.G + (g < a.G ? g : 0)) * kPfDim + 32 * c);
  // a negative scale's sign goes to the query: maxima of raw scores are then those of scaled ones
  const uint32_t flip = a.sm_scale_log2 < 0.f ? 0x80008000u : 0u;
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 x = __ldg(src + i);
    w[4 * i] = x.x ^ flip;
    w[4 * i + 1] = x.y ^ flip;
    w[4 * i + 2] = x.z ^ flip;
    w[4 * i + 3] = x.w ^ flip;
  }
  float mult = fabsf(a.sm_scale_log2) * (kFp8 ? __ldg(a.k_scale) : 1.f);
  if (kFp8) {
    uint32_t top = 0;  // largest |q|: bf16 magnitudes order as integers
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, max(w[i] & 0x7FFFu, (w[i] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    // e = 134 - the largest value's exponent
    const int ex = static_cast<int>(top >> 7);
    const int e = ex == 0 ? (top == 0 ? 0 : 126) : min(max(134 - ex, -126), 126);
    const float up = __int_as_float((127 + e) << 23);
    mult = ex == 255 ? __int_as_float(0x7fffffff) : mult * __int_as_float((127 - e) << 23);
    mult = at_least_min(mult);
    if (g < a.G) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t u[4], v[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const uint32_t x = w[8 * i + k];
          const float x0 = __uint_as_float(x << 16) * up, x1 = __uint_as_float(x & 0xFFFF0000u) * up;
          const uint32_t y = f32x2_to_e4m3x2(x0, x1);
          const float2 f = e4m3x2_to_float2(y);
          const uint32_t z = f32x2_to_e4m3x2(x0 - f.x, x1 - f.y);
          if (k & 1) {
            u[k >> 1] |= y << 16;
            v[k >> 1] |= z << 16;
          } else {
            u[k >> 1] = y;
            v[k >> 1] = z;
          }
        }
        const int to = ((2 * c + i) ^ swizzle) * 16;
        *reinterpret_cast<uint4*>(p0 + to) = make_uint4(u[0], u[1], u[2], u[3]);
        *reinterpret_cast<uint4*>(p1 + to) = make_uint4(v[0], v[1], v[2], v[3]);
      }
    }
  } else if (g < a.G) {
    uint8_t* const half = c < 2 ? p0 : p1;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(half + ((((c & 1) * 4 + i) ^ swizzle) << 4)) =
          make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    mult = at_least_min(mult);
  }
  if (g < a.G && c == 0) a.q_mult[at] = mult;
}

template <bool kFp8>
__device__ __forceinline__ void own_part(const PfArgs& a) {
  using C = OwnCfg<kFp8>;
  extern __shared__ __align__(128) uint8_t s_own[];
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int z = static_cast<int>(blockIdx.x) % a.osplits, seg = static_cast<int>(blockIdx.x) / a.osplits;
  const int r = seg / a.Hkv, h = seg - r * a.Hkv;
  const int live = live_length(a, r);
  const OwnShare share = share_of(a, r, lane);
  const int skip = share.skip, L = max(0, live - skip * a.page_size);
  if (z == 0 && skip > 0 && warp == kOwnWarps - 1) put_query<kFp8>(a, r, h, share.lo, lane);
  const int tiles = (L + kPfTile - 1) / kPfTile, n = own_splits(tiles, a.osplits);
  if (z >= n) return;
  const int t0 = static_cast<int>(static_cast<int64_t>(tiles) * z / n);
  const int t1 = static_cast<int>(static_cast<int64_t>(tiles) * (z + 1) / n);
  uint8_t* const ring = s_own + warp * kOwnRing;
  const uint32_t bars = smem_addr(s_own + kOwnWarps * kOwnRing) + warp * 32;
  float2* const s_ml = reinterpret_cast<float2*>(s_own + kOwnWarps * (kOwnRing + 32));
  const int tpp = a.page_size >> 4;
  const int32_t* row = a.page_table + static_cast<int64_t>(r) * a.max_pages + skip;
  const int count = (t1 - t0 - warp + kOwnWarps - 1) / kOwnWarps;  // this warp's tiles: t0 + warp + 4 k
  // pages of 32 tiles, a lane each, and of the 32 behind them
  auto pages_of = [&](int k) -> int {
    return k + lane < count ? __ldg(row + quotient(t0 + warp + kOwnWarps * (k + lane), a.by_tpp)) : -1;
  };
  int pages = pages_of(0), behind = pages_of(32);
  if (lane < C::kStages) {
    mbar_init(bars + 8 * lane, 1);
    fence_barrier_init();
  }
  __syncwarp();
  uint32_t there = 0, phase = 0;  // stages with a tile on its way or landed; parities
  auto ask = [&](int k) {
    if (k >= count) return;
    if (k > 0 && (k & 31) == 0) {
      pages = behind;
      behind = pages_of(k + 32);
    }
    const int page = __shfl_sync(kFull, pages, k & 31), st = k % C::kStages;
    there &= ~(1u << st);
    if (page < 0 || page >= a.num_pages) return;
    there |= 1u << st;
    const int t = t0 + warp + kOwnWarps * k;
    if (lane == 0) {
      const int64_t tile = (static_cast<int64_t>(page) * a.Hkv + h) * tpp + t - quotient(t, a.by_tpp) * tpp;
      mbar_arrive_expect_tx(bars + 8 * st, C::kTileBytes);
      bulk_copy(smem_addr(ring) + st * C::kTileBytes, a.kv_pool + tile * C::kTileBytes, C::kTileBytes, bars + 8 * st);
    }
  };
#pragma unroll 1
  for (int k = 0; k < C::kStages; ++k) ask(k);
  // ---- queries of the GQA group (head g): A fragments, rows 8 .. 15 zero; e4m3: f16 of q 2^e
  uint32_t qa[8][2];
  float mult = fabsf(a.sm_scale_log2) * (kFp8 ? __ldg(a.k_scale) : 1.f);
  {
    uint4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = g < a.G ? __ldg(reinterpret_cast<const uint4*>(
                                 a.q + (static_cast<int64_t>(r) * a.Hq + h * a.G + g) * kPfDim +
                                 (kFp8 ? 16 * (c + 4 * (i >> 1)) + 8 * (i & 1) : 8 * (c + 4 * i))))
                     : make_uint4(0, 0, 0, 0);
    const uint32_t flip = a.sm_scale_log2 < 0.f ? 0x80008000u : 0u;
    uint32_t q[16] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w,
                      w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w};
    if (kFp8) {
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = max(top, max(q[i] & 0x7FFFu, (q[i] >> 16) & 0x7FFFu));
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      const int ex = static_cast<int>(top >> 7);
      const int e = ex == 0 ? (top == 0 ? 0 : 126) : min(max(134 - ex, -126), 126);
      const float up = __int_as_float((127 + e) << 23);
      mult = ex == 255 ? __int_as_float(0x7fffffff) : mult * __int_as_float((127 - e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        q[i] = pack_f16x2(__uint_as_float(q[i] << 16) * up, __uint_as_float(q[i] & 0xFFFF0000u) * up);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      qa[i][0] = q[2 * i] ^ flip;
      qa[i][1] = q[2 * i + 1] ^ flip;
    }
  }
  mult = at_least_min(mult);
  float m = -INFINITY, l = 0.f, o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i][k] = 0.f;
  bool bad = false;
#pragma unroll 1
  for (int k = 0; k < count; ++k) {
    const int st = k % C::kStages, t = t0 + warp + kOwnWarps * k;
    if ((there >> st & 1) == 0) {
      bad = true;  // a page outside the pool
      ask(k + C::kStages);
      continue;
    }
    mbar_wait(bars + 8 * st, phase >> st & 1, a.status);
    __syncwarp();
    phase ^= 1u << st;
    const uint8_t* const tile = ring + st * C::kTileBytes;
    // ---- scores of head g, tokens 4 c .. 4 c + 3: columns g of the halves are tokens tok, tok + 2
    float s[2][4] = {};
    constexpr int el = kFp8 ? 1 : 2;
    const uint8_t* const krow = tile + (4 * (g >> 1) + (g & 1)) * kPfDim * el + c * 16;
#pragma unroll
    for (int n2 = 0; n2 < 2; ++n2) {
#pragma unroll
      for (int i = 0; i < 2 * el; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(krow + 2 * n2 * kPfDim * el + 64 * i);
        const uint32_t kw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int y = 0; y < 4 / el; ++y) {
          uint32_t b0, b1;
          if (kFp8) {
            e4m3x4_to_f16x4(kw[y], b0, b1);
          } else {
            b0 = kw[2 * y];
            b1 = kw[2 * y + 1];
          }
          const int step = i * (4 / el) + y;
          const uint32_t af[4] = {qa[step][0], 0u, qa[step][1], 0u};
          own_mma<kFp8>(s[n2], af, b0, b1);
        }
      }
    }
    uint32_t v[16][2];
    const uint8_t* const vrow = tile + kPfTile * kPfDim * el + (g * kPfTile + 4 * c) * el;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      if (kFp8) {
        e4m3x4_to_f16x4(*reinterpret_cast<const uint32_t*>(vrow + i * 8 * kPfTile), v[i][0], v[i][1]);
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(vrow + i * 8 * kPfTile * 2);
        v[i][0] = x.x;
        v[i][1] = x.y;
      }
    }
    __syncwarp();  // the stage has been read
    ask(k + C::kStages);
    float e[4] = {s[0][0], s[0][1], s[1][0], s[1][1]};
    const int left = L - t * kPfTile - 4 * c;  // tokens of this lane's four that exist
    if (L - t * kPfTile < kPfTile) {
      // an unwritten slot may hold NaN: no score, and no value
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (k >= left) e[k] = -INFINITY;
      const uint32_t m01 = left >= 2 ? 0xFFFFFFFFu : left == 1 ? 0xFFFFu : 0u;
      const uint32_t m23 = left >= 4 ? 0xFFFFFFFFu : left == 3 ? 0xFFFFu : 0u;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        v[i][0] &= m01;
        v[i][1] &= m23;
      }
    }
    float mx = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
    const float mb = mx == -INFINITY ? -INFINITY : mx * mult;
    const bool grown = mb > m || (m == -INFINITY && mb != -INFINITY);
    if (__any_sync(kFull, grown)) {
      const float f = !grown ? 1.f : m == -INFINITY ? 0.f : fast_exp2(m - mb);
      if (grown) m = mb;
      l *= f;
      // O's columns are heads 2 c, 2 c + 1
      const float f0 = __shfl_sync(kFull, f, 8 * c), f1 = __shfl_sync(kFull, f, 8 * c + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i][0] *= f0;
        o[i][1] *= f1;
        o[i][2] *= f0;
        o[i][3] *= f1;
      }
    }
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      e[k] = fast_exp2(fmaf(e[k], mult, -ref));
      l += e[k];
    }
    uint32_t p0, p1, r0, r1;
    weight_parts<kFp8>(make_float2(e[0], e[1]), p0, r0);
    weight_parts<kFp8>(make_float2(e[2], e[3]), p1, r1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t af[4] = {v[2 * i][0], v[2 * i + 1][0], v[2 * i][1], v[2 * i + 1][1]};
      own_mma<kFp8>(o[i], af, p0, p1);
      own_mma<kFp8>(o[i], af, r0, r1);
    }
  }
  // ---- the four warps' states
  l += __shfl_xor_sync(kFull, l, 1);
  l += __shfl_xor_sync(kFull, l, 2);
  if (c == 0) s_ml[warp * kPfGroupMax + g] = make_float2(m, l);
  float* const mine = reinterpret_cast<float*>(ring);  // (its last tile has been read)
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mine[2 * c * kOwnRow + 16 * i + g] = o[i][0];
    mine[(2 * c + 1) * kOwnRow + 16 * i + g] = o[i][1];
    mine[2 * c * kOwnRow + 16 * i + 8 + g] = o[i][2];
    mine[(2 * c + 1) * kOwnRow + 16 * i + 8 + g] = o[i][3];
  }
  const bool fails = __syncthreads_or(bad);
  const float vscale = kFp8 ? __ldg(a.v_scale) : 1.f;
  const int64_t slot = own_slot0(a) + static_cast<int64_t>(z) * a.B * a.Hq + static_cast<int64_t>(r) * a.Hq + h * a.G;
  for (int hd = warp; hd < a.G; hd += kOwnWarps) {
    float M = -INFINITY, W = 0.f;
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) M = fmaxf(M, s_ml[w * kPfGroupMax + hd].x);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kOwnWarps; ++w) {
      const float2 ml = s_ml[w * kPfGroupMax + hd];
      if (ml.x == -INFINITY && ml.y == 0.f) continue;  // (no score but NaN ones: the sum is NaN, and so is the part's)
      const float f = fast_exp2(ml.x - M);
      const float4 y = *reinterpret_cast<const float4*>(s_own + w * kOwnRing + (hd * kOwnRow + 4 * lane) * 4);
      W = fmaf(ml.y, f, W);
      acc.x = fmaf(y.x, f, acc.x);
      acc.y = fmaf(y.y, f, acc.y);
      acc.z = fmaf(y.z, f, acc.z);
      acc.w = fmaf(y.w, f, acc.w);
    }
    *reinterpret_cast<float4*>(a.part_o + (slot + hd) * kPfDim + 4 * lane) =
        make_float4(acc.x * vscale, acc.y * vscale, acc.z * vscale, acc.w * vscale);
    if (lane == 0) a.part_ml[slot + hd] = fails ? make_float2(0.f, kOwnFails) : make_float2(M, W);
  }
}

// Runs beside the planning kernel: it needs nothing of it.  Its end implies that kernel's, though: one CTA waits.
template <bool kFp8>
__global__ void __launch_bounds__(32 * kOwnWarps, 3) prefix_own_kernel(const PfArgs a) {
  griddep_launch_dependents();
  own_part<kFp8>(a);
  if (blockIdx.x == 0) griddep_wait();
}

// ---------------------------------------------------------------------------
// merge
// ---------------------------------------------------------------------------
// Bound by reading the partials (256 rows x 512 bytes per CTA and piece, some 22 MB in all): 9 us from L2, and
// 5 us for next to nothing, four dependent reads.  One warp per (request, query head): the partials of its own splits and those
// of the pieces of its unit, in that order.  A lane finds one partial (its row in
// the partial arrays, m, l), then all lanes add its O.
__global__ void __launch_bounds__(32 * kPfMergeWarps) prefix_merge_kernel(const PfArgs a) {
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kPfMergeWarps + (threadIdx.x >> 5);
  const int64_t rows = static_cast<int64_t>(a.B) * a.Hq;
  griddep_wait();
  if (row >= rows) return;
  uint2* const out = reinterpret_cast<uint2*>(a.out + row * kPfDim) + lane;
  if (a.n_groups == 0) {
    const float4 y = __ldcg(reinterpret_cast<const float4*>(a.all_out + row * kPfDim) + lane);
    *out = make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
    if (lane == 0 && a.lse != nullptr) a.lse[row] = __ldcg(a.all_lse + row);
    return;
  }
  const int r = static_cast<int>(row / a.Hq), hq = static_cast<int>(row - static_cast<int64_t>(r) * a.Hq);
  const int L = __ldcg(a.own_len + r), gi = __ldcg(a.group_of + r);
  bool dead = __ldcg(a.dead + r) != 0;
  float M = -INFINITY, W = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!dead) {
    const int own = own_splits((L + kPfTile - 1) / kPfTile, a.osplits);
    int cands = own, y = 0, blocks = 0, w = kPfCostSolo, subs = 0, c0 = 0, lrow = 0;
    PfRanges rg = {0, 0};
    if (gi >= 0) {
      const PfGroup q = load_group(a.group + gi);
      rg = ranges_of(load_group(a.start + a.ctas - 1).b1, a.ctas);  // (the last range ends where the list does)
      const PfPrefix s = prefix_shape(q.ptiles, q.count, a.G);
      const int h = quotient(hq, a.by_g);
      const int i = (r - q.first) * a.G + hq - h * a.G, u = i / kPfUnitRows;
      lrow = i % kPfUnitRows;
      blocks = s.blocks;
      w = u == s.units - 1 ? s.wlast : kPfCostPair;
      y = q.y0 + h * s.head_cost + u * s.step + start_cost(w);
      subs = w == kPfCostPair ? 0 : 1;  // log2 of the row tiles with a partial each
      c0 = rg.owner(y);
      cands += (rg.owner(y + (blocks - 1) * w) - c0 + 1) << subs;
    }
#pragma unroll 1
    for (int base = 0; base < cands; base += 32) {
      const int k = base + lane;
      float2 ml = make_float2(-INFINITY, 0.f);
      int64_t slot = own_slot0(a) + k * rows + row;
      bool there = k < own;
      if (k >= own && k < cands) {
        const int c = c0 + ((k - own) >> subs), sub = (k - own) & subs;
        int i0, i1;
        owned_blocks(y, blocks, w, rg.begin(c), rg.begin(c + 1), i0, i1);
        slot = i0 == 0 ? sub * rows + row : 2 * rows + static_cast<int64_t>(c) * kPfUnitRows + sub * 128 + lrow;
        there = i0 < i1;
      }
      if (there) ml = __ldcg(a.part_ml + slot);
      dead = __any_sync(kFull, ml.y < 0.f) || dead;
      float mx = ml.x;
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, o));
      const float mn = fmaxf(M, mx);
      const bool has = ml.x != -INFINITY;  // a NaN maximum counts
      const float f = has ? fast_exp2(ml.x - mn) : 0.f;
      float ws = ml.y * f;
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kFull, ws, o);
      const float old = M == -INFINITY ? 0.f : fast_exp2(M - mn);
      W = W * old + ws;
      acc.x *= old;
      acc.y *= old;
      acc.z *= old;
      acc.w *= old;
      M = mn;
      unsigned todo = __ballot_sync(kFull, has);
#pragma unroll 1
      while (todo) {
        float fk[8];
        float4 o[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          const int src = todo ? __ffs(todo) - 1 : 0;
          const float fx = __shfl_sync(kFull, f, src);
          const int64_t sx = __shfl_sync(kFull, slot, src);
          fk[x] = todo ? fx : 0.f;
          o[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (todo) o[x] = __ldcg(reinterpret_cast<const float4*>(a.part_o + sx * kPfDim) + lane);
          todo &= todo - 1;
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          acc.x = fmaf(o[x].x, fk[x], acc.x);
          acc.y = fmaf(o[x].y, fk[x], acc.y);
          acc.z = fmaf(o[x].z, fk[x], acc.z);
          acc.w = fmaf(o[x].w, fk[x], acc.w);
        }
      }
    }
  }
  dead = dead || W == 0.f;
  const float inv = dead ? 0.f : 1.f / W;
  *out = dead ? make_uint2(0, 0)
              : make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0 && a.lse != nullptr) a.lse[row] = dead ? -INFINITY : (M + __log2f(W)) * kPfLn2;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
constexpr int kPfMaxDevices = 64;
std::atomic<int> g_pf_ready[2][kPfMaxDevices];

template <bool kFp8>
int prepare_prefix(int dev) {
  std::atomic<int>& slot = g_pf_ready[kFp8][dev];
  if (slot.load(std::memory_order_relaxed) > 0) return FPK_OK;
  if (cudaFuncSetAttribute(prefix_attn_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           PfCfg<kFp8>::kSmem) != cudaSuccess ||
      cudaFuncSetAttribute(prefix_own_kernel<kFp8>, cudaFuncAttributeMaxDynamicSharedMemorySize, kOwnSmem) != cudaSuccess)
    return FPK_ECUDA;
  slot.store(1, std::memory_order_relaxed);
  return FPK_OK;
}

// Most splits of a request's own tokens per kv head, from the batch's size alone: four CTAs per SM in all, of which
// three are resident (twice as many: 2 us more for 4 to 32 requests).  Large batches have one split whatever a
// request's length: 63 requests with 8192 shared tokens and one of 131072 tokens of its own, 8 kv heads, take
// 1200 us (paged_decode_split_kernel, without sharing, 170).
int own_splits_most(int64_t B, int64_t Hkv, int64_t ctas) {
  const int64_t n = 4 * ctas / (B * Hkv > 0 ? B * Hkv : 1);
  return static_cast<int>(n < 1 ? 1 : n > 32 ? 32 : n);
}

struct PfLayout {
  size_t gstart, group, start, per_request, ml, o, image, mult, total;
};
// Behind the workspace of decode attention (batches without groups; its first word is the status word).
PfLayout prefix_layout(int64_t B, int64_t Hq, int64_t Hkv, int64_t ctas, size_t decode_bytes) {
  auto up = [](int64_t x) { return (static_cast<size_t>(x) + 255) & ~static_cast<size_t>(255); };
  const int64_t slots = 2 * B * Hq + ctas * kPfUnitRows + own_splits_most(B, Hkv, ctas) * B * Hq;
  PfLayout l;
  l.gstart = up(static_cast<int64_t>(decode_bytes));
  l.group = l.gstart + up((B + 1) * 4);
  l.start = l.group + up(B * static_cast<int64_t>(sizeof(PfGroup)));
  l.per_request = l.start + up(ctas * static_cast<int64_t>(sizeof(PfGroup)));
  l.ml = l.per_request + up(3 * B * 4);
  l.o = l.ml + up(slots * 8);
  l.image = l.o + up(slots * kPfDim * 4);
  l.mult = l.image + up(B * Hq * 256);
  l.total = l.mult + up(B * Hq * 4);
  return l;
}

// Bytes behind the first 256 of a decode attention workspace that hold its arrival counters, for any split count
// up to 32 resident CTAs per SM (which is more than there can be; what lies behind is written later in the call).
size_t decode_counter_bytes(int64_t B, int64_t Hq, int64_t Hkv) {
  int dev = 0;
  const int W = cudaGetDevice(&dev) == cudaSuccess ? 32 * device_sm_count(dev) : 0;
  const WsLayout l = layout(B, Hkv, Hq / Hkv, W);
  return l.part_ml - l.seg_count;
}

template <bool kFp8>
int prefix_entry(const void* q, const void* kv_pool, const float* k_scale, const float* v_scale,
                 const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                 const uint8_t* abort_mask, const int32_t* group_starts, const int32_t* prefix_lens,
                 int32_t n_groups, void* out, float* lse, void* workspace, size_t workspace_bytes,
                 float sm_scale, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                 int32_t num_pages, void* stream) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0 || max_pages < 0 ||
      n_groups < 0 || Hq % Hkv != 0)
    return FPK_EINVAL;
  const int G = Hq / Hkv;
  if (D != kPfDim || G > kPfGroupMax || page_size % kPfTile != 0 || page_size > 256) return FPK_EUNSUPPORTED;
  const int tpp = page_size / kPfTile;
  const int64_t tiles = static_cast<int64_t>(num_pages) * Hkv * tpp;
  // tile numbers are 32-bit tensor-map coordinates; rows and the work list's length (at most a unit
  // of the table's width per request and kv head) are counted in 31 bits, rows divided by reciprocals (2^28)
  const int64_t width = (static_cast<int64_t>(max_pages) * page_size + kPfBlk - 1) / kPfBlk;
  const int64_t longest = width * kPfCostPair + kPfStartPair;
  if (tiles > 0x7fffffff || static_cast<int64_t>(B) * Hq >= (int64_t(1) << 28) || width > (int64_t(1) << 24) ||
      longest > 0x7fffffff / (static_cast<int64_t>(B > 0 ? B : 1) * Hkv))
    return FPK_EUNSUPPORTED;
  if (B == 0) return FPK_OK;
  if (!q || !kv_pool || !page_table || !seq_lens || !out || !workspace) return FPK_EINVAL;
  if (kFp8 && (!k_scale || !v_scale)) return FPK_EINVAL;
  if (n_groups > B || (n_groups > 0 && (!group_starts || !prefix_lens))) return FPK_EINVAL;
  if (!aligned16(q) || !aligned16(kv_pool) || (reinterpret_cast<uintptr_t>(out) & 31u) != 0 ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FPK_EINVAL;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kPfMaxDevices) return FPK_ECUDA;
  const int ctas = device_sm_count(dev);
  if (ctas <= 0) return FPK_ECUDA;
  const size_t decode_bytes = fpk_decode_workspace_bytes(B, Hq, Hkv, D, 0);
  if (decode_bytes == 0) return FPK_ECUDA;
  const PfLayout l = prefix_layout(B, Hq, Hkv, ctas, decode_bytes);
  if (workspace_bytes < l.total) return FPK_ENOSPC;
  const int st = prepare_prefix<kFp8>(dev);
  if (st != FPK_OK) return st;
  int zbox = 1;  // tiles per copy: a power of two that divides a page and a block
  while (zbox < kPfBlkTiles && tpp % (2 * zbox) == 0) zbox *= 2;
  CUtensorMap kmap, vmap;
  if (encode_pool_map(&kmap, kv_pool, tiles > 0 ? tiles : 1, kFp8, false, zbox) != FPK_OK ||
      encode_pool_map(&vmap, kv_pool, tiles > 0 ? tiles : 1, kFp8, true, zbox) != FPK_OK)
    return FPK_ECUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  PfArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.abort_mask = abort_mask;
  a.group_starts = group_starts;
  a.prefix_lens = prefix_lens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.status = reinterpret_cast<uint32_t*>(ws);
  a.gstart = reinterpret_cast<int32_t*>(ws + l.gstart);
  a.group = reinterpret_cast<PfGroup*>(ws + l.group);
  a.start = reinterpret_cast<PfGroup*>(ws + l.start);
  a.group_of = reinterpret_cast<int32_t*>(ws + l.per_request);
  a.own_len = a.group_of + B;
  a.dead = a.own_len + B;
  a.all_out = reinterpret_cast<float*>(ws + l.o);
  a.all_lse = reinterpret_cast<float*>(ws + l.ml);
  a.kv_pool = static_cast<const uint8_t*>(kv_pool);
  a.q_image = ws + l.image;
  a.q_mult = reinterpret_cast<float*>(ws + l.mult);
  a.osplits = own_splits_most(B, Hkv, ctas);
  a.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  a.part_o = reinterpret_cast<float*>(ws + l.o);
  a.n_groups = n_groups;
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
  a.sm_scale_log2 = sm_scale * kPfLog2e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int merge = static_cast<int>((static_cast<int64_t>(B) * Hq + kPfMergeWarps - 1) / kPfMergeWarps);
  if (n_groups == 0) {
    // the arrival counters of decode attention, which lie elsewhere for other shapes, begin at zero
    if (cudaMemsetAsync(ws + 256, 0, decode_counter_bytes(B, Hq, Hkv), s) != cudaSuccess) return FPK_ECUDA;
    float* all_out = reinterpret_cast<float*>(ws + l.o);
    float* all_lse = reinterpret_cast<float*>(ws + l.ml);
    const int done =
        kFp8 ? fpk_paged_decode_attn_fp8(q, static_cast<const uint8_t*>(kv_pool), k_scale, v_scale, page_table, max_pages,
                                         seq_lens, abort_mask, all_out, all_lse, ws, decode_bytes, 0, sm_scale, B, Hq,
                                         Hkv, D, page_size, num_pages, stream)
             : fpk_paged_decode_attn_bf16(q, kv_pool, page_table, max_pages, seq_lens, abort_mask, all_out, all_lse, ws,
                                          decode_bytes, 0, sm_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
    if (done != FPK_OK) return done;
    return launch_dependent(prefix_merge_kernel, merge, 32 * kPfMergeWarps, 0, s, a);
  }
  const int64_t own = static_cast<int64_t>(B) * Hkv * a.osplits;
  if (own > 0x7fffffff) return FPK_EUNSUPPORTED;
  if (launch_dependent(prefix_plan_kernel, 1, kPfPlanThreads, 0, s, a) != FPK_OK ||
      launch_dependent(prefix_own_kernel<kFp8>, static_cast<int>(own), 32 * kOwnWarps, kOwnSmem, s, a) != FPK_OK ||
      launch_dependent(prefix_attn_kernel<kFp8>, ctas, kPfThreads, PfCfg<kFp8>::kSmem, s, a, kmap, vmap) != FPK_OK)
    return FPK_ECUDA;
  return launch_dependent(prefix_merge_kernel, merge, 32 * kPfMergeWarps, 0, s, a);
}

}  // namespace
}  // namespace fpk

extern "C" size_t fpk_prefix_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > fpk::kPfGroupMax || D != fpk::kPfDim) return 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= fpk::kPfMaxDevices) return 0;
  const int ctas = fpk::device_sm_count(dev);
  const size_t decode = fpk_decode_workspace_bytes(B, Hq, Hkv, D, 0);
  return ctas > 0 && decode > 0 ? fpk::prefix_layout(B, Hq, Hkv, ctas, decode).total : 0;
}

extern "C" int fpk_paged_decode_attn_fp8_prefix(const void* q, const uint8_t* kv_pool, const float* k_scale,
                                                const float* v_scale, const int32_t* page_table,
                                                int32_t max_pages, const int32_t* seq_lens,
                                                const uint8_t* abort_mask, const int32_t* group_starts,
                                                const int32_t* prefix_lens, int32_t n_groups, void* out,
                                                float* lse, void* workspace, size_t workspace_bytes,
                                                float sm_scale, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                                int32_t page_size, int32_t num_pages, void* stream) {
  return fpk::prefix_entry<true>(q, kv_pool, k_scale, v_scale, page_table, max_pages, seq_lens, abort_mask,
                                 group_starts, prefix_lens, n_groups, out, lse, workspace, workspace_bytes,
                                 sm_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
}

extern "C" int fpk_paged_decode_attn_bf16_prefix(const void* q, const void* kv_pool, const int32_t* page_table,
                                                 int32_t max_pages, const int32_t* seq_lens,
                                                 const uint8_t* abort_mask, const int32_t* group_starts,
                                                 const int32_t* prefix_lens, int32_t n_groups, void* out,
                                                 float* lse, void* workspace, size_t workspace_bytes,
                                                 float sm_scale, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                                 int32_t page_size, int32_t num_pages, void* stream) {
  return fpk::prefix_entry<false>(q, kv_pool, nullptr, nullptr, page_table, max_pages, seq_lens, abort_mask,
                                  group_starts, prefix_lens, n_groups, out, lse, workspace, workspace_bytes,
                                  sm_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
}
