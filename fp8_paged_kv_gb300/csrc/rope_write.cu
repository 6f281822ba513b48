// rope_write.cu -- rotary positions for queries and keys, fused with the cache
// write of the rotated keys and the values.
//
// Pair i of a head at position p turns by the angle p f_i:
//   (x, y) -> s (x cos a - y sin a, y cos a + x sin a),  a = p f_i.
// The angle is reduced in turns: f / (2 pi) is held as a fraction of 2^64, and the
// low 64 bits of its product with p are the fraction of a turn, whatever p: far
// positions keep the accuracy of near ones (2^-32 turns at 2^31).
//
// A unit is 16 values of a head, 8 pairs, and belongs to one thread: in the half
// layout its two 16-byte chunks lie rot_dim/2 apart, interleaved or unrotated
// ones are adjacent, and no pair ever crosses two threads.  The same unit of
// every head of a token turns by the same angles, so a thread keeps a unit's
// eight cosines and sines in registers over the heads that it walks.
//
// Both kernels move bytes and are bound by HBM (or, for few tokens, by a
// launch and three dependent loads).  Appends have a thread per (token, unit,
// slice of the heads).  Prompts go by 16-token tiles of the cache: what a CTA
// does is cut out of one list of (tile, eight heads) steps, as many for each
// CTA, and values are written as whole rows of a tile's dim-major block.
// 16384 tokens, 64/8 heads, e4m3 cache: 105 us, 6.0 TB/s of 638 MB (89 % of what a
// copy reaches); a thread per (token, unit) over all heads with element stores of V
// took 171 us.  2011 tokens in 7 chunks, bf16: 19 us, a launch, three dependent
// reads and three steps per CTA.  Appends: 4 us for one token, 5 us for 64.
//
// Block scales (kBlock): a block's scale follows its largest value, so a key is
// rotated before its scale is known.  An append's head is eight neighbouring
// lanes: they find the token's largest value by shuffles.  Of a prompt's tile the
// keys' largest values go through shared memory (a head is four warps), those of
// values stay within the warp that writes them.  Where a scale grows, the codes of
// the block's earlier tokens are brought under it, all their loads in flight at
// once; tokens that are written together have one scale from the start.  16384 tokens
// (64 query, 8 kv heads): 105.6 us, 6.0 TB/s, as with one scale for all; 2011 tokens in
// 7 chunks: 22 us; appends: 4 us for one token, 6 us for 64.
//
// Rounding: fp32 throughout, a rotated value rounded once to what it is stored as.
#include <algorithm>

#include "block_scale.cuh"
#include "step_ops.cuh"

namespace fpk {
namespace {

constexpr int kRopeDim = 128;
constexpr int kRopeUnits = kRopeDim / 16;  // units of 16 values per head
constexpr int kRopeThreads = 256;
constexpr int kRopeBatch = 4;                // heads in flight per thread
constexpr int kRopeStep = 2 * kRopeBatch;    // heads per step of a prompt's tile
constexpr int kRopeStage = 16 * kRopeStep * kRopeDim * 2, kRopeStages = 3;
constexpr int kRopeWarpStage = kRopeStage / (kRopeThreads / 32);

struct RopeArgs {
  WriteArgs w;               // k_src, v_src, pool, table, tags; seq_lens or cu_seqlens
  const uint16_t* q;
  uint16_t* q_out;
  const float* inv_freq;
  const int32_t* start_pos;  // nullable
  uint8_t* scales;           // kBlock: E8M0 bytes [num_pages][Hkv][tiles][2]
  float rot_scale;
  int Hq, rot, interleaved, hsplit;
};

// 2 / pi, its first 64 bits (2^64 (2 / pi), rounded down, from pi to 40 digits).
constexpr uint32_t kTwoOverPiHi = 0xA2F9836Eu, kTwoOverPiLo = 0x4E441529u;

struct Turn {
  float c[8], s[8];
};

// Turns per position of pair i, f / (2 pi) modulo 1, in steps of 2^-64: the 24 bits of f times the 64 of
// 2 / pi, the upper 64 of these shifted to their place.  Within 2 steps for |f| < 2, twice as many for each
// doubling behind.
__device__ __forceinline__ uint64_t turn_rate(const RopeArgs& a, int i) {
  const uint32_t f = __float_as_uint(__ldg(a.inv_freq + i));
  const uint32_t m = (f & 0x7FFFFFu) << 8 | 0x80000000u;
  const uint64_t x = static_cast<uint64_t>(m) * kTwoOverPiHi + __umulhi(m, kTwoOverPiLo);
  const int down = 128 - static_cast<int>(f >> 23 & 255u);
  const uint64_t r = down >= 64 || down <= -64 ? 0 : down >= 0 ? x >> down : x << -down;
  return f >> 31 ? 0 - r : r;
}

// Half turns (within 1) of a pair at a position: what lies behind the product's upper 32 bits is below 2^-32 turns.
__device__ __forceinline__ float half_turns(int pos, uint64_t rate) {
  const uint64_t turns = static_cast<uint64_t>(static_cast<int64_t>(pos)) * rate;
  return static_cast<float>(static_cast<int32_t>(turns >> 32)) * 0x1p-31f;
}

// The eight cosines and sines of a unit at a position, to out[0], [stride], .. [3 stride]: a short loop (the
// unrolled one is 8 KiB of code, fetched anew each time).  rate(i): the turns of its pair i.
template <class Rate>
__device__ __forceinline__ void unit_angles(const RopeArgs& a, int pos, const Rate& rate, float4* out, int stride) {
#pragma unroll 1
  for (int i = 0; i < 4; ++i) {
    float c[2], s[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) sincospif(half_turns(pos, rate(2 * i + k)), &s[k], &c[k]);
    out[i * stride] = make_float4(c[0] * a.rot_scale, c[1] * a.rot_scale, s[0] * a.rot_scale, s[1] * a.rot_scale);
  }
}
__device__ __forceinline__ void load_turn(Turn& t, const float4* in, int stride) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 x = in[i * stride];
    t.c[2 * i] = x.x;
    t.c[2 * i + 1] = x.y;
    t.s[2 * i] = x.z;
    t.s[2 * i + 1] = x.w;
  }
}

// 16 values: the unit's chunks x0 (8 bf16) and x1 (8 bf16), rotated, as fp32.
__device__ __forceinline__ void rotate_unit(const uint4& r0, const uint4& r1, const Turn& t, bool turns,
                                            bool interleaved, float (&y)[16]) {
  const uint32_t w[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[2 * i] = __uint_as_float(w[i] << 16);
    y[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  if (!turns) return;
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = y[2 * i], z = y[2 * i + 1];
      y[2 * i] = x * t.c[i] - z * t.s[i];
      y[2 * i + 1] = z * t.c[i] + x * t.s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = y[i], z = y[8 + i];
      y[i] = x * t.c[i] - z * t.s[i];
      y[8 + i] = z * t.c[i] + x * t.s[i];
    }
  }
}

__device__ __forceinline__ uint32_t codes(float x, float y) {
  return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// e4m3 codes of eight values; a divisor without a normal reciprocal is divided by out of line.
__device__ __noinline__ uint2 quant8_slow(float4 x, float4 y, float s) {
  return make_uint2(codes(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s)) | codes(__fdiv_rn(x.z, s), __fdiv_rn(x.w, s)) << 16,
                    codes(__fdiv_rn(y.x, s), __fdiv_rn(y.y, s)) | codes(__fdiv_rn(y.z, s), __fdiv_rn(y.w, s)) << 16);
}
template <bool kBlock>
__device__ __forceinline__ uint2 quant8(const float* y, const Divisor& s) {
  if (kBlock)  // a power of two: the product is the quotient
    return make_uint2(codes(y[0] * s.r, y[1] * s.r) | codes(y[2] * s.r, y[3] * s.r) << 16,
                      codes(y[4] * s.r, y[5] * s.r) | codes(y[6] * s.r, y[7] * s.r) << 16);
  if (!s.recip_ok) return quant8_slow(make_float4(y[0], y[1], y[2], y[3]), make_float4(y[4], y[5], y[6], y[7]), s.s);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    w[i] = codes(div_fast(y[4 * i], s), div_fast(y[4 * i + 1], s)) |
           codes(div_fast(y[4 * i + 2], s), div_fast(y[4 * i + 3], s)) << 16;
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint4 pack8(const float* y) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// A unit's chunks: first values of the two.
struct Unit {
  int d0, d1;
  bool turns;
};
__device__ __forceinline__ Unit unit_of(const RopeArgs& a, int u) {
  Unit x;
  x.turns = 16 * u < a.rot;
  const bool half = x.turns && !a.interleaved;
  x.d0 = half ? 8 * u : 16 * u;
  x.d1 = half ? 8 * u + (a.rot >> 1) : 16 * u + 8;
  return x;
}

// Division by the scale 2^e.
__device__ __forceinline__ Divisor block_divisor(int e) { return {exp2_int(e), exp2_int(-e), true}; }

// The largest finite magnitude of a unit.
__device__ __forceinline__ float unit_top(const float (&y)[16]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) top = fmaxf(top, finite_magnitude(y[i]));
  return top;
}

// A unit of a rotated key into its row of the K block.
template <bool kFp8, bool kBlock>
__device__ __forceinline__ void put_key(const WriteArgs& w, int64_t row, const Unit& x, const float (&y)[16],
                                        const Divisor& ks) {
  if (kFp8) {
    *reinterpret_cast<uint2*>(w.kv_pool + row + x.d0) = quant8<kBlock>(y, ks);
    *reinterpret_cast<uint2*>(w.kv_pool + row + x.d1) = quant8<kBlock>(y + 8, ks);
  } else {
    uint16_t* pool = reinterpret_cast<uint16_t*>(w.kv_pool);
    *reinterpret_cast<uint4*>(pool + row + x.d0) = pack8(y);
    *reinterpret_cast<uint4*>(pool + row + x.d1) = pack8(y + 8);
  }
}

// The page of position pos of request r, -1 if its token may not be written.
__device__ __forceinline__ int page_for(const WriteArgs& w, int r, int64_t pos) {
  if (pos < 0) return -1;
  const int64_t pi = pos / w.page_size;
  if (pi >= w.max_pages) return -1;
  const int64_t e = static_cast<int64_t>(r) * w.max_pages + pi;
  const bool guarded = w.live_tags != nullptr && w.expected_tags != nullptr;
  const int page = __ldg(w.page_table + e);
  const uint32_t want = guarded ? __ldg(w.expected_tags + e) : 0u;
  if (page < 0 || page >= w.num_pages || (guarded && __ldg(w.live_tags + page) != want)) return -1;
  return page;
}

__device__ __forceinline__ float key_top(const RopeArgs& a, const Unit& x, const Turn& t, const uint4& x0, const uint4& x1) {
  float y[16];
  rotate_unit(x0, x1, t, x.turns, a.interleaved, y);
  return unit_top(y);
}
__device__ __forceinline__ float values_top(const uint4& x0, const uint4& x1) {
  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    top = fmaxf(top, fmaxf(finite_magnitude(__uint_as_float(w[i] << 16)), finite_magnitude(__uint_as_float(w[i] & 0xFFFF0000u))));
  return top;
}

// The block of an append's key or value, by the head's eight lanes, one per unit: its scale for a token of
// largest value `top` (this lane's) at `slot`, the earlier tokens brought under it.  tile: the tile's first byte.
__device__ __forceinline__ Divisor grow_block(const RopeArgs& a, int64_t tile, int slot, bool value, const Unit& x,
                                              int u, float top) {
  const unsigned head = 0xFFu << (threadIdx.x & 24);
  uint8_t* const at = a.scales + tile / (16 * kRopeDim) + (value ? 1 : 0);  // (two bytes per tile of 4096)
  int old = slot > 0 ? scale_exponent(*at) : kExpLow;
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = fmaxf(top, __shfl_xor_sync(head, top, o));
  old = __shfl_sync(head, old, 0, 8);  // (every lane has read the byte before one writes it)
  const int e = max(old, block_exponent(top));
  if (u == 0) *at = static_cast<uint8_t>(e + 127);
  if (slot > 0 && e > old) {
    const float f = exp2_int(old - e);
    uint8_t* const block = a.w.kv_pool + tile + (value ? 16 * kRopeDim + 16 * u * 16 : 0);
    if (value) {
      uint4 r[16];
#pragma unroll
      for (int d = 0; d < 16; ++d) r[d] = *reinterpret_cast<const uint4*>(block + 16 * d);
#pragma unroll
      for (int d = 0; d < 16; ++d) *reinterpret_cast<uint4*>(block + 16 * d) = rescale_first(r[d], slot, f);
    } else {
      uint2 r[15][2];
#pragma unroll
      for (int i = 0; i < 15; ++i)
        if (i < slot) {
          r[i][0] = *reinterpret_cast<const uint2*>(block + i * kRopeDim + x.d0);
          r[i][1] = *reinterpret_cast<const uint2*>(block + i * kRopeDim + x.d1);
        }
#pragma unroll
      for (int i = 0; i < 15; ++i)
        if (i < slot) {
          *reinterpret_cast<uint2*>(block + i * kRopeDim + x.d0) = make_uint2(rescale4(r[i][0].x, f), rescale4(r[i][0].y, f));
          *reinterpret_cast<uint2*>(block + i * kRopeDim + x.d1) = make_uint2(rescale4(r[i][1].x, f), rescale4(r[i][1].y, f));
        }
    }
  }
  return block_divisor(e);
}

// One token per request.  Thread = (token, slice, unit); the slice's heads are
// slice, slice + hsplit, ... of the Hq queries, Hkv keys and Hkv values.  A
// token's V column is strided by a tile's 16 tokens: element stores.
template <bool kFp8, bool kBlock>
__global__ void __launch_bounds__(kRopeThreads) rope_append_kernel(const RopeArgs a) {
  const WriteArgs& w = a.w;
  const int64_t i = blockIdx.x * static_cast<int64_t>(kRopeThreads) + threadIdx.x;
  const int u = static_cast<int>(i % kRopeUnits);
  const int slice = static_cast<int>(i / kRopeUnits % a.hsplit);
  const int64_t row = i / kRopeUnits / a.hsplit;
  if (row >= w.rows) return;
  const Unit x = unit_of(a, u);
  const int length = __ldg(w.seq_lens + row), pos = max(length, 1) - 1;
  // a source row of the head list; queries may be rotated in place: plain loads
  auto source = [&](int h) -> const uint16_t* {
    if (h < a.Hq) return a.q + (row * a.Hq + h) * kRopeDim;
    return h < a.Hq + w.Hkv ? w.k_src + (row * w.Hkv + h - a.Hq) * kRopeDim
                            : w.v_src + (row * w.Hkv + h - a.Hq - w.Hkv) * kRopeDim;
  };
  const int heads = a.Hq + 2 * w.Hkv;
  int h = slice;
  const uint16_t* src = source(h);
  bool value = h >= a.Hq + w.Hkv;
  uint4 x0 = *reinterpret_cast<const uint4*>(src + (value ? 16 * u : x.d0));
  uint4 x1 = *reinterpret_cast<const uint4*>(src + (value ? 16 * u + 8 : x.d1));
  if (length <= 0) return;
  const int page = h + (heads - 1 - h) / a.hsplit * a.hsplit >= a.Hq ? page_for(w, static_cast<int>(row), pos) : -1;
  const int tpp = w.page_size >> 4, off = pos % w.page_size;
  __shared__ float4 s_turn[4][kRopeThreads];  // a thread's own
  if (x.turns && !value)
    unit_angles(a, pos, [&](int i) { return turn_rate(a, 8 * u + i); }, &s_turn[0][threadIdx.x], kRopeThreads);
  Turn t;
  load_turn(t, &s_turn[0][threadIdx.x], kRopeThreads);
  for (;;) {
    if (h < a.Hq) {
      float y[16];
      rotate_unit(x0, x1, t, x.turns, a.interleaved, y);
      uint16_t* const out = a.q_out + (row * a.Hq + h) * kRopeDim;
      *reinterpret_cast<uint4*>(out + x.d0) = pack8(y);
      *reinterpret_cast<uint4*>(out + x.d1) = pack8(y + 8);
    } else if (page < 0) {
      if (w.abort_mask != nullptr) w.abort_mask[row] = 1;
      return;
    } else {
      const int hk = h - a.Hq - (value ? w.Hkv : 0);
      const int64_t tile = ((static_cast<int64_t>(page) * w.Hkv + hk) * tpp + (off >> 4)) * 2 * 16 * kRopeDim;
      Divisor bs = {};
      if (kBlock) bs = grow_block(a, tile, off & 15, value, x, u, value ? values_top(x0, x1) : key_top(a, x, t, x0, x1));
      if (!value) {
        float y[16];
        rotate_unit(x0, x1, t, x.turns, a.interleaved, y);
        put_key<kFp8, kBlock>(w, tile + (off & 15) * kRopeDim, x, y,
                              kBlock ? bs : make_divisor(kFp8 ? __ldg(w.k_scale) : 1.f));
      } else {
        const int64_t at = tile + 16 * kRopeDim + 16 * u * 16 + (off & 15);
        const uint32_t vw[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
        if (kFp8) {
          const Divisor vs = kBlock ? bs : make_divisor(__ldg(w.v_scale));
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float y[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              y[2 * k] = __uint_as_float(vw[4 * j + k] << 16);
              y[2 * k + 1] = __uint_as_float(vw[4 * j + k] & 0xFFFF0000u);
            }
            const uint2 c = quant8<kBlock>(y, vs);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              w.kv_pool[at + 16 * (8 * j + k)] = static_cast<uint8_t>((k < 4 ? c.x : c.y) >> (8 * (k & 3)));
          }
        } else {
          uint16_t* pool = reinterpret_cast<uint16_t*>(w.kv_pool);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            pool[at + 32 * j] = static_cast<uint16_t>(vw[j] & 0xFFFFu);
            pool[at + 32 * j + 16] = static_cast<uint16_t>(vw[j] >> 16);
          }
        }
      }
    }
    h += a.hsplit;
    if (h >= heads) return;
    src = source(h);
    value = h >= a.Hq + w.Hkv;
    x0 = *reinterpret_cast<const uint4*>(src + (value ? 16 * u : x.d0));
    x1 = *reinterpret_cast<const uint4*>(src + (value ? 16 * u + 8 : x.d1));
  }
}

// Bytes [b0, b1) of a row of 4 kWords bytes, in the widest aligned pieces: a store costs an L1 cycle per line it
// touches whatever its width (element stores of a 15-token tile: 16 us instead of 1).
template <int kWords, int kElem>
__device__ __forceinline__ void put_row(uint8_t* row, const uint32_t (&c)[kWords], int b0, int b1) {
  auto inside = [&](int b, int n) -> bool { return b0 <= b && b + n <= b1; };
#pragma unroll
  for (int p = 0; p < kWords; p += 4) {
    if (inside(4 * p, 16)) {
      *reinterpret_cast<uint4*>(row + 4 * p) = make_uint4(c[p], c[p + 1], c[p + 2], c[p + 3]);
      continue;
    }
#pragma unroll
    for (int h = p; h < p + 4; h += 2) {
      if (inside(4 * h, 8)) {
        *reinterpret_cast<uint2*>(row + 4 * h) = make_uint2(c[h], c[h + 1]);
        continue;
      }
#pragma unroll
      for (int w = h; w < h + 2; ++w) {
        if (inside(4 * w, 4)) {
          *reinterpret_cast<uint32_t*>(row + 4 * w) = c[w];
          continue;
        }
#pragma unroll
        for (int e = 0; e < 4; e += kElem)
          if (inside(4 * w + e, kElem)) {
            if (kElem == 1) row[4 * w + e] = static_cast<uint8_t>(c[w] >> (8 * e));
            else *reinterpret_cast<uint16_t*>(row + 4 * w + e) = static_cast<uint16_t>(c[w] >> (8 * e));
          }
      }
    }
  }
}

// Values of one tile and head, by a warp: src is the tile's 16 token rows (those that are not new: whatever the
// stage held); lane l writes the rows of dims l, l + 32, l + 64, l + 96, consecutive lanes consecutive rows.
template <bool kFp8, bool kBlock>
__device__ __forceinline__ void put_values(const WriteArgs& w, int64_t vblock, const uint16_t* src, int t0, int n,
                                           const Divisor& vs, int lane, float older = 1.f) {
#pragma unroll 1
  for (int d = lane; d < kRopeDim; d += 32) {
    uint32_t e[8];  // tokens 2 q, 2 q + 1
#pragma unroll
    for (int q = 0; q < 8; ++q)
      e[q] = src[2 * q * kRopeDim + d] | static_cast<uint32_t>(src[(2 * q + 1) * kRopeDim + d]) << 16;
    const int64_t at = vblock + d * 16;
    if (kFp8) {
      uint32_t c[4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float y[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          y[2 * k] = __uint_as_float(e[4 * j + k] << 16);
          y[2 * k + 1] = __uint_as_float(e[4 * j + k] & 0xFFFF0000u);
        }
        const uint2 x = quant8<kBlock>(y, vs);
        c[2 * j] = x.x;
        c[2 * j + 1] = x.y;
      }
      if (kBlock && older != 1.f) {
        // the tokens before: their codes times `older`
        const uint4 was = rescale_first(*reinterpret_cast<const uint4*>(w.kv_pool + at), t0, older);
        const uint32_t o[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int k = min(max(t0 - 4 * i, 0), 4);
          const uint32_t mine = k == 4 ? 0xFFFFFFFFu : (1u << (8 * k)) - 1u;
          c[i] = (o[i] & mine) | (c[i] & ~mine);
        }
        put_row<4, 1>(w.kv_pool + at, c, 0, t0 + n);
        continue;
      }
      put_row<4, 1>(w.kv_pool + at, c, t0, t0 + n);
    } else {
      put_row<8, 2>(w.kv_pool + 2 * at, e, 2 * t0, 2 * (t0 + n));
    }
  }
}

// Tiles of request r have the places cu[r] / 16 + 2 r and on: a request of n
// tokens touches at most n / 16 + 2 tiles wherever its first position lies, so
// that the places need no scan over the requests, and a few stay empty.
__host__ __device__ __forceinline__ int64_t tile_places(int64_t rows, int64_t B) { return rows / 16 + 2 * B; }

// A step of a prompt: eight heads of a tile (queries, then keys: the threads of
// the lower and the upper half take four each; then values, a warp each).
struct Step {
  int request, row0, t0, n;  // n new tokens from source row row0 at rows t0 .. of the tile; 0: nothing to do
  int tile, step, page;      // tile of the request; page: -1 if refused (steps behind the queries')
};

__device__ __forceinline__ void rope_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void rope_copy8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// kBlock: four heads' keys of a tile by the 128 threads of a side (a thread a unit of a token, staged at in[64 k],
// in[64 k + 32] for head k): the blocks' largest values meet in `tops`, then the keys go out, and the tile's earlier
// tokens where their scale has grown.  The heads behind the last one are other threads' stage: not looked at.
__device__ __forceinline__ void put_key_blocks(const RopeArgs& a, int64_t block, int h0, int tpp, int tok, int t0, int n,
                                               const Unit& x, const Turn& t, const uint4* in, float (*tops)[4], int side) {
  const int heads = a.w.Hkv, lane = threadIdx.x & 31, warp = threadIdx.x >> 5 & 3;
  const bool fresh = tok >= t0 && tok < t0 + n;
  int old[kRopeBatch];
#pragma unroll
  for (int k = 0; k < kRopeBatch; ++k) {
    const bool there = h0 + k < heads;
    old[k] = there && t0 > 0 ? scale_exponent(a.scales[2 * (block + static_cast<int64_t>(h0 + k) * tpp)]) : kExpLow;
    float top = 0.f;
    if (there && fresh) top = key_top(a, x, t, in[64 * k], in[64 * k + 32]);
    top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)));
    if (lane == 0) tops[k][warp] = top;
  }
  asm volatile("bar.sync %0, 128;" ::"r"(1 + side) : "memory");
#pragma unroll
  for (int k = 0; k < kRopeBatch; ++k) {
    if (h0 + k >= heads) break;
    const int64_t tile = block + static_cast<int64_t>(h0 + k) * tpp, row = tile * 2 * 16 * kRopeDim + tok * kRopeDim;
    const int e = max(old[k], block_exponent(fmaxf(fmaxf(tops[k][0], tops[k][1]), fmaxf(tops[k][2], tops[k][3]))));
    if (fresh) {
      float y[16];
      rotate_unit(in[64 * k], in[64 * k + 32], t, x.turns, a.interleaved, y);
      put_key<true, true>(a.w, row, x, y, block_divisor(e));
    } else if (tok < t0 && e > old[k]) {
      const float f = exp2_int(old[k] - e);
      uint2* const c0 = reinterpret_cast<uint2*>(a.w.kv_pool + row + x.d0);
      uint2* const c1 = reinterpret_cast<uint2*>(a.w.kv_pool + row + x.d1);
      const uint2 r0 = *c0, r1 = *c1;
      *c0 = make_uint2(rescale4(r0.x, f), rescale4(r0.y, f));
      *c1 = make_uint2(rescale4(r1.x, f), rescale4(r1.y, f));
    }
    if (lane == 0 && warp == 0) a.scales[2 * tile] = static_cast<uint8_t>(e + 127);
  }
}

// The sources of the next two steps are on their way while a step is worked
// on: 128 KiB per SM in flight, each warp's into its own part of a stage, so
// that no warp waits for another.
template <bool kFp8, bool kBlock>
__global__ void __launch_bounds__(kRopeThreads, 2) rope_prefill_kernel(const RopeArgs a) {
  extern __shared__ __align__(16) uint8_t s_stage[];
  __shared__ uint64_t s_rate[kRopeDim / 2];
  __shared__ float s_top[2][2][kRopeBatch][4];  // kBlock: [turn][side][head][warp]
  const WriteArgs& w = a.w;
  const int u = threadIdx.x % kRopeUnits, tok = threadIdx.x / kRopeUnits % 16, lane = threadIdx.x & 31;
  const int side = threadIdx.x / (16 * kRopeUnits), warp = threadIdx.x >> 5;
  const int qsteps = (a.Hq + kRopeStep - 1) / kRopeStep, ksteps = (w.Hkv + kRopeStep - 1) / kRopeStep;
  const int steps = qsteps + 2 * ksteps;
  const int64_t total = tile_places(w.rows, w.B) * steps;
  const int64_t begin = total * blockIdx.x / gridDim.x;
  const int count = static_cast<int>(total * (blockIdx.x + 1) / gridDim.x - begin);
  const Divisor ks = kBlock ? Divisor{} : make_divisor(kFp8 ? __ldg(w.k_scale) : 1.f);
  const Divisor vs = kBlock ? Divisor{} : make_divisor(kFp8 ? __ldg(w.v_scale) : 1.f);
  const Unit x = unit_of(a, u);
  const int tpp = w.page_size >> 4;
  int64_t place = begin / steps - 1;
  int at = static_cast<int>(begin - (place + 1) * steps), left = count;  // the next step's place in its tile; steps not yet asked for
  Step next = {};
  // a warp's part of a stage: [chunk][lane] of 16 bytes, or [token][lane] of 8
  const uint32_t stages = smem_addr(s_stage) + warp * kRopeWarpStage + lane * 16;

  if (2 * static_cast<int>(threadIdx.x) < a.rot) s_rate[threadIdx.x] = turn_rate(a, threadIdx.x);
  __syncthreads();

  // the next step, and its sources asked for
  auto ask = [&](uint32_t stage) {
    if (left > 0) {
      bool entered = false;
      --left;
      if (at == steps) at = 0;
      if (at == 0 || left == count - 1) {
        // a new place: its request is the largest r with cu[r] / 16 + 2 r at or below it
        ++place;
        int lo = 0, hi = w.B - 1;
#pragma unroll 1
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if ((__ldg(w.cu_seqlens + mid) >> 4) + 2 * static_cast<int64_t>(mid) <= place) lo = mid; else hi = mid - 1;
        }
        const int64_t c0 = max(__ldg(w.cu_seqlens + lo), 0);
        const int64_t c1 = min(static_cast<int64_t>(__ldg(w.cu_seqlens + lo + 1)), w.rows);
        const int64_t start = a.start_pos != nullptr ? __ldg(a.start_pos + lo) : 0;
        const int64_t tile = (start >> 4) + place - ((c0 >> 4) + 2 * lo);  // of the request's positions
        const int64_t p0 = max(start, 16 * tile), p1 = min(start + c1 - c0, 16 * tile + 16);
        next.request = lo;
        next.tile = static_cast<int>(tile);
        next.n = static_cast<int>(max(p1 - p0, static_cast<int64_t>(0)));
        next.t0 = static_cast<int>(p0 - 16 * tile);
        next.row0 = static_cast<int>(c0 + p0 - start);
        entered = true;
      }
      next.step = at++;
      const bool key = next.step >= qsteps;
      if (next.n > 0 && next.step < qsteps + ksteps) {
        const int heads = key ? w.Hkv : a.Hq;
        const int h0 = (key ? next.step - qsteps : next.step) * kRopeStep + side * kRopeBatch;
        const uint16_t* const src =
            (key ? w.k_src : a.q) + (static_cast<int64_t>(next.row0 + tok - next.t0) * heads + h0) * kRopeDim;
        if (tok >= next.t0 && tok < next.t0 + next.n)
#pragma unroll
          for (int k = 0; k < kRopeBatch; ++k)
            if (h0 + k < heads) {
              rope_copy16(stage + 2 * k * 512, src + k * kRopeDim + x.d0);
              rope_copy16(stage + (2 * k + 1) * 512, src + k * kRopeDim + x.d1);
            }
      } else if (next.n > 0) {
        const int h = (next.step - qsteps - ksteps) * kRopeStep + warp;
        const uint16_t* src = w.v_src + (static_cast<int64_t>(next.row0) * w.Hkv + h) * kRopeDim + 4 * lane;
        const uint32_t dst = stage - lane * 8;
        if (h < w.Hkv)
#pragma unroll 1
          for (int q = next.t0; q < next.t0 + next.n; ++q, src += static_cast<int64_t>(w.Hkv) * kRopeDim)
            rope_copy8(dst + q * 256, src);
      }
      // (the page is looked up behind the copies: nothing waits for it before the step is worked on)
      if (entered) next.page = next.n > 0 ? page_for(w, next.request, 16 * static_cast<int64_t>(next.tile) + next.t0) : -1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };

  uint32_t st = 0;  // stage asked for; the one worked on is two steps behind it, the next in the ring
  Step s0 = {}, s1 = {};
  Turn t;
  int turned = 0;  // t belongs to the tile
  int tops = 0;    // kBlock: turn of s_top
#pragma unroll 1
  for (int done = -2; done < count; ++done) {
    __syncwarp();  // the stage's last readers
    ask(stages + st * kRopeStage);
    const Step c = s0;
    s0 = s1;
    s1 = next;
    st = st == 2 ? 0 : st + 1;
    if (done < 0) continue;
    asm volatile("cp.async.wait_group 2;" ::: "memory");
    __syncwarp();
    const uint8_t* const mine = s_stage + st * kRopeStage + warp * kRopeWarpStage;
    if (done == 0 || c.step == 0) turned = 0;
    // kBlock: the two sides of a keys' step meet in it, whatever the tile is
    const bool meets = kBlock && c.step >= qsteps && c.step < qsteps + ksteps;
    if (meets && (c.n == 0 || c.page < 0)) {
      asm volatile("bar.sync %0, 128;" ::"r"(1 + side) : "memory");
      tops ^= 1;
    }
    if (c.n == 0) continue;
    if (c.step >= qsteps && c.page < 0) {
      if (threadIdx.x == 0 && w.abort_mask != nullptr) w.abort_mask[c.request] = 1;
      continue;
    }
    const int64_t block = static_cast<int64_t>(c.page) * w.Hkv * tpp + c.tile % tpp;
    if (c.step < qsteps + ksteps) {
      if (x.turns && turned == 0) {
        float4* const turn = reinterpret_cast<float4*>(s_stage + kRopeStages * kRopeStage) + threadIdx.x;
        unit_angles(a, 16 * c.tile + tok, [&](int i) { return s_rate[8 * u + i]; }, turn, kRopeThreads);
        load_turn(t, turn, kRopeThreads);
      }
      turned = 1;
      const bool key = c.step >= qsteps;
      const int heads = key ? w.Hkv : a.Hq;
      const int h0 = (key ? c.step - qsteps : c.step) * kRopeStep + side * kRopeBatch;
      const int64_t row = c.row0 + tok - c.t0;
      if (kBlock && key) {
        put_key_blocks(a, block, h0, tpp, tok, c.t0, c.n, x, t, reinterpret_cast<const uint4*>(mine) + lane, s_top[tops][side],
                       side);
        tops ^= 1;
      } else if (tok >= c.t0 && tok < c.t0 + c.n)
#pragma unroll 2
        for (int k = 0; k < kRopeBatch; ++k)
          if (h0 + k < heads) {
            const uint4* const in = reinterpret_cast<const uint4*>(mine) + lane + 2 * k * 32;
            float y[16];
            rotate_unit(in[0], in[32], t, x.turns, a.interleaved, y);
            if (key) {
              put_key<kFp8, kBlock>(w, (block + static_cast<int64_t>(h0 + k) * tpp) * 2 * 16 * kRopeDim + tok * kRopeDim, x, y, ks);
            } else {
              uint16_t* const out = a.q_out + (row * heads + h0 + k) * kRopeDim;
              *reinterpret_cast<uint4*>(out + x.d0) = pack8(y);
              *reinterpret_cast<uint4*>(out + x.d1) = pack8(y + 8);
            }
          }
    } else {
      const int h = (c.step - qsteps - ksteps) * kRopeStep + warp;
      const int64_t tile = block + static_cast<int64_t>(h) * tpp;
      if (h < w.Hkv && kBlock) {
        uint8_t* const at = a.scales + 2 * tile + 1;
        const int old = c.t0 > 0 ? scale_exponent(*at) : kExpLow;
        float top = 0.f;
#pragma unroll 4
        for (int q = c.t0; q < c.t0 + c.n; ++q) {
          const uint2 v = *reinterpret_cast<const uint2*>(mine + q * 256 + lane * 8);
          top = fmaxf(top, fmaxf(fmaxf(finite_magnitude(__uint_as_float(v.x << 16)), finite_magnitude(__uint_as_float(v.x & 0xFFFF0000u))),
                                 fmaxf(finite_magnitude(__uint_as_float(v.y << 16)), finite_magnitude(__uint_as_float(v.y & 0xFFFF0000u)))));
        }
        // (magnitudes order as their bits; every lane has read the byte before one writes it)
        const int e = max(old, block_exponent(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top)))));
        const float older = exp2_int(__shfl_sync(0xffffffffu, old, 0) - e);
        if (lane == 0) *at = static_cast<uint8_t>(e + 127);
        put_values<kFp8, true>(w, tile * 2 * 16 * kRopeDim + 16 * kRopeDim, reinterpret_cast<const uint16_t*>(mine), c.t0, c.n,
                               block_divisor(e), lane, c.t0 > 0 ? older : 1.f);
      } else if (h < w.Hkv) {
        put_values<kFp8, kBlock>(w, tile * 2 * 16 * kRopeDim + 16 * kRopeDim, reinterpret_cast<const uint16_t*>(mine), c.t0,
                                 c.n, vs, lane);
      }
    }
  }
}

// scales != nullptr: the e4m3 cache with block scales.
int rope_entry(bool fp8, bool prefill, const void* q, const void* k, const void* v, const int32_t* seq_lens,
               const int32_t* cu, int64_t rows, const int32_t* start_pos, const float* inv_freq, void* q_out,
               void* kv_pool, const float* k_scale, const float* v_scale, const int32_t* page_table,
               int32_t max_pages, const uint32_t* live_tags, const uint32_t* expected_tags,
               uint8_t* abort_mask, int32_t rot_dim, int32_t interleaved, float rot_scale, int32_t B,
               int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages, void* stream,
               bool block = false, uint8_t* scales = nullptr) {
  if (B < 0 || Hq < 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0 || max_pages < 0 || rows < 0 ||
      rot_dim < (block ? 0 : 1))
    return FPK_EINVAL;
  if (D != kRopeDim || page_size % 16 != 0 || page_size > 256) return FPK_EUNSUPPORTED;
  if (rot_dim % 16 != 0 || rot_dim > D) return FPK_EUNSUPPORTED;
  if (rows == 0 || B == 0) return FPK_OK;
  if (!k || !v || (rot_dim > 0 && !inv_freq) || !kv_pool || !page_table || (prefill ? !cu : !seq_lens)) return FPK_EINVAL;
  if (Hq > 0 && (!q || !q_out)) return FPK_EINVAL;
  if (block ? !scales : fp8 && (!k_scale || !v_scale)) return FPK_EINVAL;
  if (!aligned16(k) || !aligned16(v) || !aligned16(kv_pool) || !aligned16(q) || !aligned16(q_out)) return FPK_EINVAL;
  RopeArgs a;
  a.w.k_src = static_cast<const uint16_t*>(k);
  a.w.v_src = static_cast<const uint16_t*>(v);
  a.w.seq_lens = seq_lens;
  a.w.cu_seqlens = cu;
  a.w.kv_pool = static_cast<uint8_t*>(kv_pool);
  a.w.k_scale = k_scale;
  a.w.v_scale = v_scale;
  a.w.page_table = page_table;
  a.w.live_tags = live_tags;
  a.w.expected_tags = expected_tags;
  a.w.abort_mask = abort_mask;
  a.w.rows = rows;
  a.w.B = B;
  a.w.Hkv = Hkv;
  a.w.D = D;
  a.w.page_size = page_size;
  a.w.num_pages = num_pages;
  a.w.max_pages = max_pages;
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.inv_freq = inv_freq;
  a.start_pos = start_pos;
  a.scales = scales;
  a.rot_scale = rot_scale;
  a.Hq = Hq;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.hsplit = 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (prefill) {
    auto kern = block ? rope_prefill_kernel<true, true> : fp8 ? rope_prefill_kernel<true, false> : rope_prefill_kernel<false, false>;
    const int64_t steps = (Hq + kRopeStep - 1) / kRopeStep + 2 * static_cast<int64_t>((Hkv + kRopeStep - 1) / kRopeStep);
    constexpr int smem = kRopeStages * kRopeStage + kRopeThreads * 64;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return FPK_ECUDA;
    // As many CTAs as are resident at once, or up to four times as many where each still has eight steps: the SMs
    // run at different speeds (and requests end in empty places), which only CTAs that come later can even out.
    // 16384 tokens: one wave 117 us, four 106; 2011 tokens: one wave (three steps a CTA) 19 us, four 23.
    const int64_t all = tile_places(rows, B) * steps;
    const int64_t wave = resident_grid(reinterpret_cast<const void*>(kern), kRopeThreads, smem, all);
    const int64_t ctas = std::min(std::max(wave, all / 8), 4 * wave);
    kern<<<static_cast<int>(ctas), kRopeThreads, smem, st>>>(a);
  } else {
    // a head per thread while that is no more than two full waves of threads; then as few slices as fill those
    const int64_t heads = Hq + 2 * static_cast<int64_t>(Hkv), full = 2 * 152 * 1024 / kRopeUnits;
    a.hsplit = static_cast<int>(rows * heads <= full ? heads : (full + rows - 1) / rows);
    const int64_t ctas = (rows * a.hsplit * kRopeUnits + kRopeThreads - 1) / kRopeThreads;
    if (ctas > 0x7fffffff) return FPK_EUNSUPPORTED;
    auto kern = block ? rope_append_kernel<true, true> : fp8 ? rope_append_kernel<true, false> : rope_append_kernel<false, false>;
    kern<<<static_cast<int>(ctas), kRopeThreads, 0, st>>>(a);
  }
  return checked_launch_status();
}

}  // namespace
}  // namespace fpk

extern "C" int fpk_rope_append_fp8(const void* q, const void* k_new, const void* v_new, const float* inv_freq,
                                   void* q_out, uint8_t* kv_pool, const float* k_scale, const float* v_scale,
                                   const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                   const uint32_t* live_tags, const uint32_t* expected_tags,
                                   uint8_t* abort_mask, int32_t rot_dim, int32_t interleaved, float rot_scale,
                                   int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                   int32_t num_pages, void* stream) {
  return fpk::rope_entry(true, false, q, k_new, v_new, seq_lens, nullptr, B, nullptr, inv_freq, q_out, kv_pool,
                         k_scale, v_scale, page_table, max_pages, live_tags, expected_tags, abort_mask, rot_dim,
                         interleaved, rot_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
}

extern "C" int fpk_rope_append_bf16(const void* q, const void* k_new, const void* v_new, const float* inv_freq,
                                    void* q_out, void* kv_pool, const int32_t* page_table, int32_t max_pages,
                                    const int32_t* seq_lens, const uint32_t* live_tags,
                                    const uint32_t* expected_tags, uint8_t* abort_mask, int32_t rot_dim,
                                    int32_t interleaved, float rot_scale, int32_t B, int32_t Hq, int32_t Hkv,
                                    int32_t D, int32_t page_size, int32_t num_pages, void* stream) {
  return fpk::rope_entry(false, false, q, k_new, v_new, seq_lens, nullptr, B, nullptr, inv_freq, q_out, kv_pool,
                         nullptr, nullptr, page_table, max_pages, live_tags, expected_tags, abort_mask, rot_dim,
                         interleaved, rot_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
}

extern "C" int fpk_rope_prefill_fp8(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                    int32_t n_tokens, const int32_t* start_pos, const float* inv_freq,
                                    void* q_out, uint8_t* kv_pool, const float* k_scale, const float* v_scale,
                                    const int32_t* page_table, int32_t max_pages, const uint32_t* live_tags,
                                    const uint32_t* expected_tags, uint8_t* abort_mask, int32_t rot_dim,
                                    int32_t interleaved, float rot_scale, int32_t B, int32_t Hq, int32_t Hkv,
                                    int32_t D, int32_t page_size, int32_t num_pages, void* stream) {
  return fpk::rope_entry(true, true, q, k, v, nullptr, cu_seqlens, n_tokens, start_pos, inv_freq, q_out, kv_pool,
                         k_scale, v_scale, page_table, max_pages, live_tags, expected_tags, abort_mask, rot_dim,
                         interleaved, rot_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
}

extern "C" int fpk_rope_prefill_bf16(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                     int32_t n_tokens, const int32_t* start_pos, const float* inv_freq,
                                     void* q_out, void* kv_pool, const int32_t* page_table, int32_t max_pages,
                                     const uint32_t* live_tags, const uint32_t* expected_tags,
                                     uint8_t* abort_mask, int32_t rot_dim, int32_t interleaved,
                                     float rot_scale, int32_t B, int32_t Hq, int32_t Hkv, int32_t D,
                                     int32_t page_size, int32_t num_pages, void* stream) {
  return fpk::rope_entry(false, true, q, k, v, nullptr, cu_seqlens, n_tokens, start_pos, inv_freq, q_out, kv_pool,
                         nullptr, nullptr, page_table, max_pages, live_tags, expected_tags, abort_mask, rot_dim,
                         interleaved, rot_scale, B, Hq, Hkv, D, page_size, num_pages, stream);
}

extern "C" int fpk_rope_append_fp8_block(const void* q, const void* k_new, const void* v_new, const float* inv_freq,
                                         void* q_out, uint8_t* kv_pool, uint8_t* kv_scales, const int32_t* page_table,
                                         int32_t max_pages, const int32_t* seq_lens, const uint32_t* live_tags,
                                         const uint32_t* expected_tags, uint8_t* abort_mask, int32_t rot_dim,
                                         int32_t interleaved, float rot_scale, int32_t B, int32_t Hq, int32_t Hkv,
                                         int32_t D, int32_t page_size, int32_t num_pages, void* stream) {
  return fpk::rope_entry(true, false, q, k_new, v_new, seq_lens, nullptr, B, nullptr, inv_freq, q_out, kv_pool,
                         nullptr, nullptr, page_table, max_pages, live_tags, expected_tags, abort_mask, rot_dim,
                         interleaved, rot_scale, B, Hq, Hkv, D, page_size, num_pages, stream, true, kv_scales);
}

extern "C" int fpk_rope_prefill_fp8_block(const void* q, const void* k, const void* v, const int32_t* cu_seqlens,
                                          int32_t n_tokens, const int32_t* start_pos, const float* inv_freq,
                                          void* q_out, uint8_t* kv_pool, uint8_t* kv_scales, const int32_t* page_table,
                                          int32_t max_pages, const uint32_t* live_tags, const uint32_t* expected_tags,
                                          uint8_t* abort_mask, int32_t rot_dim, int32_t interleaved, float rot_scale,
                                          int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                                          int32_t num_pages, void* stream) {
  return fpk::rope_entry(true, true, q, k, v, nullptr, cu_seqlens, n_tokens, start_pos, inv_freq, q_out, kv_pool,
                         nullptr, nullptr, page_table, max_pages, live_tags, expected_tags, abort_mask, rot_dim,
                         interleaved, rot_scale, B, Hq, Hkv, D, page_size, num_pages, stream, true, kv_scales);
}

extern "C" int fpk_kv_append_fp8_block(const void* k_new, const void* v_new, uint8_t* kv_pool, uint8_t* kv_scales,
                                       const int32_t* page_table, int32_t max_pages, const int32_t* seq_lens,
                                       const uint32_t* live_tags, const uint32_t* expected_tags, uint8_t* abort_mask,
                                       int32_t B, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                                       void* stream) {
  return fpk_rope_append_fp8_block(nullptr, k_new, v_new, nullptr, nullptr, kv_pool, kv_scales, page_table, max_pages,
                                   seq_lens, live_tags, expected_tags, abort_mask, 0, 0, 1.f, B, 0, Hkv, D, page_size,
                                   num_pages, stream);
}

extern "C" int fpk_kv_prefill_fp8_block(const void* k, const void* v, const int32_t* cu_seqlens, int32_t n_tokens,
                                        const int32_t* start_pos, uint8_t* kv_pool, uint8_t* kv_scales,
                                        const int32_t* page_table, int32_t max_pages, const uint32_t* live_tags,
                                        const uint32_t* expected_tags, uint8_t* abort_mask, int32_t B, int32_t Hkv,
                                        int32_t D, int32_t page_size, int32_t num_pages, void* stream) {
  return fpk_rope_prefill_fp8_block(nullptr, k, v, cu_seqlens, n_tokens, start_pos, nullptr, nullptr, kv_pool, kv_scales,
                                    page_table, max_pages, live_tags, expected_tags, abort_mask, 0, 0, 1.f, B, 0, Hkv, D,
                                    page_size, num_pages, stream);
}
