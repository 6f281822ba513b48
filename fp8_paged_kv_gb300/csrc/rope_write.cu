// rope_write.cu -- rotary positions for queries and keys, fused with the cache
// write of the rotated keys and the values.
//
// Pair i of a head at position p turns by the angle p f_i:
//   (x, y) -> s (x cos a - y sin a, y cos a + x sin a),  a = p f_i.
// The angle is reduced in turns: f / (2 pi) is held as a two-float sum and the
// fraction of p f / (2 pi) is taken with the product's rounding error (one FMA)
// added back, so that far positions keep the accuracy of near ones.
//
// One thread owns one unit of a token -- 16 values of a head, 8 pairs -- and
// walks over heads with the unit's eight cosines and sines in registers: the
// same unit of every head turns by the same angles.  In the half layout the
// unit's two 16-byte chunks lie rot_dim/2 apart, interleaved or unrotated ones
// are adjacent, and no pair ever crosses two threads.
#include "step_ops.cuh"

namespace fpk {
namespace {

constexpr int kRopeDim = 128;
constexpr int kRopeUnits = kRopeDim / 16;  // units of 16 values per head
constexpr int kRopeThreads = 256;

struct RopeArgs {
  WriteArgs w;               // k_src, v_src, pool, table, tags; seq_lens or cu_seqlens
  const uint16_t* q;
  uint16_t* q_out;
  const float* inv_freq;
  const int32_t* start_pos;  // nullable
  float rot_scale;
  int Hq, rot, interleaved, hsplit;
};

// 1 / (2 pi) as the sum of two floats: the value rounded to 24 bits and the
// rounded remainder (from pi to 40 digits).
constexpr double kInvTwoPi = 0.15915494309189533576888376337251436203;
constexpr float kInvTwoPiHi = static_cast<float>(kInvTwoPi);
constexpr float kInvTwoPiLo = static_cast<float>(kInvTwoPi - static_cast<double>(kInvTwoPiHi));

// Fraction of a turn (within about one half) of p * (th + tl), p an integer of
// at most 24 significant bits: the product with th is split into its rounded
// value, whose fraction is exact, and its rounding error.
__device__ __forceinline__ float turn_fraction(float p, float th, float tl) {
  const float a = __fmul_rn(p, th);
  const float e = __fmaf_rn(p, th, -a);
  return __fadd_rn(a - rintf(a), __fmaf_rn(p, tl, e));
}

struct Turn {
  float c[8], s[8];
};

__device__ __forceinline__ void unit_angles(const RopeArgs& a, int pos, int u, Turn& t) {
  // positions of more than 24 bits enter as two parts
  const float plo = static_cast<float>(pos & 0xFFFF), phi = static_cast<float>(pos - (pos & 0xFFFF));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = __ldg(a.inv_freq + 8 * u + i);
    const float th = __fmul_rn(f, kInvTwoPiHi);
    const float tl = __fmaf_rn(f, kInvTwoPiLo, __fmaf_rn(f, kInvTwoPiHi, -th));
    float r = turn_fraction(plo, th, tl) + turn_fraction(phi, th, tl);
    sincospif(2.f * r, &t.s[i], &t.c[i]);
    t.s[i] *= a.rot_scale;
    t.c[i] *= a.rot_scale;
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

__device__ __forceinline__ uint2 quant8(const float* y, const Divisor& s) {
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(div_by(y[4 * i], s), div_by(y[4 * i + 1], s)),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(div_by(y[4 * i + 2], s), div_by(y[4 * i + 3], s)),
                                                 __NV_SATFINITE, __NV_E4M3);
    w[i] = lo | (hi << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint4 pack8(const float* y) {
  return make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                    pack_bf16x2(y[6], y[7]));
}

// Thread = (token, head slice, unit): the unit of heads slice, slice + hsplit,
// ...; heads 0 .. Hq-1 are the queries', the following Hkv the cache's.
template <bool kFp8, bool kPrefill>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kernel(const RopeArgs a) {
  const WriteArgs& w = a.w;
  const int64_t total = w.rows * a.hsplit * kRopeUnits;
  const Divisor ks = make_divisor(kFp8 ? __ldg(w.k_scale) : 1.f);
  const Divisor vs = make_divisor(kFp8 ? __ldg(w.v_scale) : 1.f);
  const int tpp = w.page_size >> 4;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(kRopeThreads) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kRopeThreads) {
    const int u = static_cast<int>(i % kRopeUnits);
    const int64_t row = (i / kRopeUnits) % w.rows;
    const int slice = static_cast<int>(i / kRopeUnits / w.rows);
    int r, pos;
    if (kPrefill) {
      r = request_of_row(w.cu_seqlens, w.B, row);
      pos = static_cast<int>(row - __ldg(w.cu_seqlens + r)) + (a.start_pos != nullptr ? __ldg(a.start_pos + r) : 0);
    } else {
      r = static_cast<int>(row);
      pos = __ldg(w.seq_lens + r) - 1;
      if (pos < 0) continue;
    }
    const bool turns = 16 * u < a.rot;
    Turn t;
    if (turns) unit_angles(a, pos, u, t);
    const bool half = turns && !a.interleaved;
    const int d0 = half ? 8 * u : 16 * u;              // first value of the two chunks
    const int d1 = half ? 8 * u + (a.rot >> 1) : 16 * u + 8;
    int h = slice;
#pragma unroll 4
    for (; h < a.Hq; h += a.hsplit) {
      const int64_t at = (row * a.Hq + h) * kRopeDim;
      const uint4 x0 = *reinterpret_cast<const uint4*>(a.q + at + d0);
      const uint4 x1 = *reinterpret_cast<const uint4*>(a.q + at + d1);
      float y[16];
      rotate_unit(x0, x1, t, turns, a.interleaved, y);
      *reinterpret_cast<uint4*>(a.q_out + at + d0) = pack8(y);
      *reinterpret_cast<uint4*>(a.q_out + at + d1) = pack8(y + 8);
    }
    if (h - a.Hq >= w.Hkv) continue;
    // the slot of this token and its guard
    const int pi = pos >= 0 ? pos / w.page_size : -1;
    const int off = pos - pi * w.page_size;
    bool ok = pi >= 0 && pi < w.max_pages;
    int page = -1;
    if (ok) {
      const int64_t e = static_cast<int64_t>(r) * w.max_pages + pi;
      page = __ldg(w.page_table + e);
      ok = page >= 0 && page < w.num_pages;
      if (ok && w.live_tags != nullptr && w.expected_tags != nullptr)
        ok = __ldg(w.live_tags + page) == __ldg(w.expected_tags + e);
    }
    if (!ok) {
      if (w.abort_mask != nullptr) w.abort_mask[r] = 1;
      continue;
    }
    for (int hk = h - a.Hq; hk < w.Hkv; hk += a.hsplit) {
      const int64_t at = (row * w.Hkv + hk) * kRopeDim;
      const uint4 x0 = __ldg(reinterpret_cast<const uint4*>(w.k_src + at + d0));
      const uint4 x1 = __ldg(reinterpret_cast<const uint4*>(w.k_src + at + d1));
      const uint4 v0 = __ldg(reinterpret_cast<const uint4*>(w.v_src + at + 16 * u));
      const uint4 v1 = __ldg(reinterpret_cast<const uint4*>(w.v_src + at + 16 * u + 8));
      const int64_t tile = ((static_cast<int64_t>(page) * w.Hkv + hk) * tpp + (off >> 4)) * 2 * 16 * kRopeDim;
      const int64_t krow = tile + (off & 15) * kRopeDim;
      const int64_t vcol = tile + 16 * kRopeDim + 16 * u * 16 + (off & 15);
      float y[16];
      rotate_unit(x0, x1, t, turns, a.interleaved, y);
      const uint32_t vw[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
      if (kFp8) {
        *reinterpret_cast<uint2*>(w.kv_pool + krow + d0) = quant8(y, ks);
        *reinterpret_cast<uint2*>(w.kv_pool + krow + d1) = quant8(y + 8, ks);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float lo = div_by(__uint_as_float(vw[j] << 16), vs);
          const float hi = div_by(__uint_as_float(vw[j] & 0xFFFF0000u), vs);
          const uint32_t c = __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
          w.kv_pool[vcol + 32 * j] = static_cast<uint8_t>(c & 0xFFu);
          w.kv_pool[vcol + 32 * j + 16] = static_cast<uint8_t>(c >> 8);
        }
      } else {
        uint16_t* pool = reinterpret_cast<uint16_t*>(w.kv_pool);
        *reinterpret_cast<uint4*>(pool + krow + d0) = pack8(y);
        *reinterpret_cast<uint4*>(pool + krow + d1) = pack8(y + 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          pool[vcol + 32 * j] = static_cast<uint16_t>(vw[j] & 0xFFFFu);
          pool[vcol + 32 * j + 16] = static_cast<uint16_t>(vw[j] >> 16);
        }
      }
    }
  }
}

int rope_entry(bool fp8, bool prefill, const void* q, const void* k, const void* v, const int32_t* seq_lens,
               const int32_t* cu, int64_t rows, const int32_t* start_pos, const float* inv_freq, void* q_out,
               void* kv_pool, const float* k_scale, const float* v_scale, const int32_t* page_table,
               int32_t max_pages, const uint32_t* live_tags, const uint32_t* expected_tags,
               uint8_t* abort_mask, int32_t rot_dim, int32_t interleaved, float rot_scale, int32_t B,
               int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages, void* stream) {
  if (B < 0 || Hq < 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0 || max_pages < 0 || rows < 0 ||
      rot_dim <= 0)
    return FPK_EINVAL;
  if (D != kRopeDim || page_size % 16 != 0 || page_size > 256) return FPK_EUNSUPPORTED;
  if (rot_dim % 16 != 0 || rot_dim > D) return FPK_EUNSUPPORTED;
  if (rows == 0 || B == 0) return FPK_OK;
  if (!k || !v || !inv_freq || !kv_pool || !page_table || (prefill ? !cu : !seq_lens)) return FPK_EINVAL;
  if (Hq > 0 && (!q || !q_out)) return FPK_EINVAL;
  if (fp8 && (!k_scale || !v_scale)) return FPK_EINVAL;
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
  a.rot_scale = rot_scale;
  a.Hq = Hq;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.hsplit = 1;
  const int64_t want = (rows * a.hsplit * kRopeUnits + kRopeThreads - 1) / kRopeThreads;
  auto kern = fp8 ? (prefill ? rope_write_kernel<true, true> : rope_write_kernel<true, false>)
                  : (prefill ? rope_write_kernel<false, true> : rope_write_kernel<false, false>);
  const int grid = resident_grid(reinterpret_cast<const void*>(kern), kRopeThreads, 0, want);
  kern<<<grid, kRopeThreads, 0, static_cast<cudaStream_t>(stream)>>>(a);
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
