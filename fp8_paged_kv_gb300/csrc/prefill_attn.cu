// prefill_attn.cu -- attention of several query tokens per request over an e4m3
// cache with block scales: chunks of prompts and drafted tokens (causal), or an
// encoder's states (all tokens).
//
// A warp takes 16 rows (a row is one query head of one token; the heads that
// share a kv head follow one another) over all tokens they see, 16 at a time,
// with its operands straight from the pool: lane (g, c) = (lane / 4, lane % 4)
// holds 16-byte chunks c and c + 4 of its K tokens, and tokens 4 c .. 4 c + 3 of its
// V dims, which are the tokens of the scores that it holds, so that the weights
// enter the second product from the registers where the first left them.
#include "block_scale.cuh"

namespace fpk {
namespace {

constexpr int kChTile = 16;
constexpr int kChDim = 128;
constexpr int kChGroupMax = 8;
constexpr int kChWarps = 4;
constexpr int kChRows = 16 * kChWarps;
constexpr float kChLog2e = 1.4426950408889634f;
constexpr float kChLn2 = 0.6931471805599453f;

struct ChArgs {
  const uint16_t* q;
  const int32_t* cu_seqlens;
  const uint8_t* kv_pool;
  const uint16_t* kv_scales;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const uint8_t* abort_mask;
  uint16_t* out;
  float* lse;
  int n_tokens, causal, B, Hq, Hkv, G, page_size, num_pages, max_pages;
  float sm_scale_log2;
};

__global__ void __launch_bounds__(32 * kChWarps) prefill_attn_kernel(const ChArgs a) {
  const unsigned kFull = 0xffffffffu;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const int h = blockIdx.y;
  int lo = 0, hi = a.B - 1;
  auto place_of = [&](int r) -> int64_t { return static_cast<int64_t>(__ldg(a.cu_seqlens + r)) * a.G / kChRows + r; };
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (place_of(mid) <= blockIdx.x) lo = mid; else hi = mid - 1;
  }
  const int r = lo, c0 = max(__ldg(a.cu_seqlens + r), 0), n = min(__ldg(a.cu_seqlens + r + 1), a.n_tokens) - c0;
  const int64_t rows = static_cast<int64_t>(n) * a.G, row0 = (blockIdx.x - place_of(r)) * kChRows;
  if (row0 >= rows) return;
  const int L = __ldg(a.seq_lens + r), tpp = a.page_size >> 4;
  bool dead = L <= 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_pages) * a.page_size ||
              (a.abort_mask != nullptr && __ldg(a.abort_mask + r) != 0);
  const int32_t* table = a.page_table + static_cast<int64_t>(r) * a.max_pages;
  for (int i = threadIdx.x; !dead && i <= (L - 1) / a.page_size; i += 32 * kChWarps) {
    const int p = __ldg(table + i);
    dead = p < 0 || p >= a.num_pages;
  }
  dead = __syncthreads_or(dead);
  // this lane's rows: g and g + 8 of the warp's 16
  int64_t at[2];
  int limit[2];
  bool valid[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t row = row0 + 16 * warp + g + 8 * i;
    const int t = static_cast<int>(row / a.G);
    valid[i] = row < rows;
    at[i] = static_cast<int64_t>(c0 + (valid[i] ? t : 0)) * a.Hq + h * a.G + (valid[i] ? row - static_cast<int64_t>(t) * a.G : 0);
    limit[i] = dead || !valid[i] ? 0 : a.causal ? max(0, min(L, L - n + t + 1)) : L;
  }
  uint32_t qa[8][4];
  float mult[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint4 x = __ldg(reinterpret_cast<const uint4*>(a.q + at[i] * kChDim + 16 * (c + 4 * (k >> 1)) + 8 * (k & 1)));
      w[4 * k] = x.x;
      w[4 * k + 1] = x.y;
      w[4 * k + 2] = x.z;
      w[4 * k + 3] = x.w;
    }
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = max(top, max(w[k] & 0x7FFFu, (w[k] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(kFull, top, 1));
    top = max(top, __shfl_xor_sync(kFull, top, 2));
    const int ex = static_cast<int>(top >> 7);
    const int e = ex == 0 ? (top == 0 ? 0 : 126) : min(max(134 - ex, -126), 126);
    const float up = exp2_int(e);
    mult[i] = ex == 255 ? __int_as_float(0x7fffffff) : a.sm_scale_log2 * exp2_int(-e);
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        qa[k][i + 2 * j] = pack_f16x2(__uint_as_float(w[2 * k + j] << 16) * up, __uint_as_float(w[2 * k + j] & 0xFFFF0000u) * up);
  }
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
  int most = max(limit[0], limit[1]);
  most = __reduce_max_sync(kFull, most);
#pragma unroll 1
  for (int t = 0; t * kChTile < most; ++t) {
    const int64_t tile = (static_cast<int64_t>(__ldg(table + t / tpp)) * a.Hkv + h) * tpp + t % tpp;
    const uint32_t sb = __ldg(a.kv_scales + tile);
    const float km = exp2_int(scale_exponent(sb & 255u));
    const int ev = scale_exponent(sb >> 8);
    const uint8_t* const block = a.kv_pool + tile * 2 * kChTile * kChDim;
    float s[2][4] = {};
#pragma unroll
    for (int nb = 0; nb < 2; ++nb) {
      const uint8_t* const krow = block + (4 * (g >> 1) + (g & 1) + 2 * nb) * kChDim + c * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(krow + 64 * i));
        const uint32_t kw[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t b0, b1;
          e4m3x4_to_f16x4(kw[y], b0, b1);
          mma_f16(s[nb], qa[4 * i + y], b0, b1);
        }
      }
    }
    uint32_t p[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float e[4] = {s[0][2 * i], s[0][2 * i + 1], s[1][2 * i], s[1][2 * i + 1]};
      float mx = -INFINITY;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        e[k] = t * kChTile + 4 * c + k < limit[i] ? fmaf(e[k], mult[i] * km, static_cast<float>(ev)) : -INFINITY;
        mx = fmaxf(mx, e[k]);
      }
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 2));
      const float mn = fmaxf(m[i], mx), f = m[i] == -INFINITY ? 0.f : fast_exp2(m[i] - mn), ref = mn == -INFINITY ? 0.f : mn;
      m[i] = mn;
      l[i] *= f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        o[j][2 * i] *= f;
        o[j][2 * i + 1] *= f;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = fast_exp2(e[k] - ref);
      l[i] = fmaf((e[0] + e[1]) + (e[2] + e[3]), exp2_int(-ev), l[i]);
      p[0][i] = pack_f16x2(e[0], e[1]);
      p[1][i] = pack_f16x2(e[2], e[3]);
    }
    const uint32_t pa[4] = {p[0][0], p[0][1], p[1][0], p[1][1]};
    const int left = min(4, max(0, L - t * kChTile - 4 * c));
    const uint32_t keep = left == 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      uint32_t b0, b1;
      e4m3x4_to_f16x4(__ldg(reinterpret_cast<const uint32_t*>(block + kChTile * kChDim + (8 * j + g) * kChTile + 4 * c)) & keep,
                      b0, b1);
      mma_f16(o[j], pa, b0, b1);
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    l[i] += __shfl_xor_sync(kFull, l[i], 1);
    l[i] += __shfl_xor_sync(kFull, l[i], 2);
    if (!valid[i]) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
    for (int j = 0; j < 16; ++j)
      *reinterpret_cast<uint32_t*>(a.out + at[i] * kChDim + 8 * j + 2 * c) = pack_bf16x2(o[j][2 * i] * inv, o[j][2 * i + 1] * inv);
    if (c == 0 && a.lse != nullptr) a.lse[at[i]] = l[i] == 0.f ? -INFINITY : (m[i] + __log2f(l[i])) * kChLn2;
  }
}

}  // namespace
}  // namespace fpk

extern "C" size_t fpk_prefill_workspace_bytes(int32_t B, int32_t n_tokens, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || n_tokens < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > fpk::kChGroupMax || D != fpk::kChDim) return 0;
  return 256;
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
  if (B == 0 || n_tokens == 0) return FPK_OK;
  if (!q || !cu_seqlens || !kv_pool || !kv_scales || !page_table || !seq_lens || !out || !workspace) return FPK_EINVAL;
  if (!aligned16(q) || !aligned16(kv_pool) || (reinterpret_cast<uintptr_t>(kv_scales) & 1u) != 0 ||
      (reinterpret_cast<uintptr_t>(out) & 31u) != 0 || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FPK_EINVAL;
  if (workspace_bytes < 256) return FPK_ENOSPC;
  ChArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.cu_seqlens = cu_seqlens;
  a.kv_pool = kv_pool;
  a.kv_scales = reinterpret_cast<const uint16_t*>(kv_scales);
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.abort_mask = abort_mask;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.n_tokens = n_tokens;
  a.causal = causal != 0;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = G;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.sm_scale_log2 = sm_scale * kChLog2e;
  const int64_t places = static_cast<int64_t>(n_tokens) * G / kChRows + B;
  if (places > 0x7fffffff || Hkv > 65535) return FPK_EUNSUPPORTED;
  prefill_attn_kernel<<<dim3(static_cast<unsigned>(places), Hkv), 32 * kChWarps, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return checked_launch_status();
}
