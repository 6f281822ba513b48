// prefix_attn.cu -- decode attention of a batch whose requests share prefixes.
#include "common.cuh"

namespace fpk {
namespace {

constexpr int kPfTile = 16;
constexpr int kPfDim = 128;
constexpr int kPfGroupMax = 8;
constexpr float kPfLog2e = 1.4426950408889634f;
constexpr float kPfLn2 = 0.6931471805599453f;

struct PrefixArgs {
  const uint16_t* q;
  const uint8_t* kv_pool;
  const float* k_scale;
  const float* v_scale;
  const int32_t* page_table;
  const int32_t* seq_lens;
  const uint8_t* abort_mask;
  const int32_t* group_starts;
  const int32_t* prefix_lens;
  uint16_t* out;
  float* lse;
  int n_groups, B, Hq, Hkv, G, page_size, num_pages, max_pages;
  float sm_scale_log2;
};

// Context length of request r if it is alive by its length and abort flag, else 0.
__device__ __forceinline__ int live_length(const PrefixArgs& a, int r) {
  const int L = __ldg(a.seq_lens + r);
  if (L <= 0 || static_cast<int64_t>(L) > static_cast<int64_t>(a.max_pages) * a.page_size) return 0;
  if (a.abort_mask != nullptr && __ldg(a.abort_mask + r) != 0) return 0;
  return L;
}

template <bool kFp8>
__device__ __forceinline__ float pool_value(const uint8_t* pool, int64_t i) {
  if (kFp8) {
    const uint32_t h = e4m3x2_to_f16x2(pool[i]);
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
  }
  return bf16_bits_to_float(reinterpret_cast<const uint16_t*>(pool)[i]);
}

// One CTA per (request, kv head), one thread per dim.
template <bool kFp8>
__global__ void __launch_bounds__(kPfDim) prefix_simple_kernel(const PrefixArgs a) {
  __shared__ float s_q[kPfGroupMax][kPfDim];
  __shared__ float s_s[kPfGroupMax][kPfTile];
  const int r = blockIdx.x / a.Hkv, h = blockIdx.x % a.Hkv, t = threadIdx.x;
  const int64_t row0 = static_cast<int64_t>(r) * a.Hq + h * a.G;
  const int L = live_length(a, r);
  // the request's group, what it shares, and the row that stands for it
  int shared_pages = 0, leader = r;
  for (int g = 0; g < a.n_groups; ++g) {
    const int lo = min(max(__ldg(a.group_starts + g), 0), a.B), hi = min(max(__ldg(a.group_starts + g + 1), 0), a.B);
    if (r < lo || r >= hi || hi - lo < 2) continue;
    int least = max(__ldg(a.prefix_lens + g), 0);
    leader = -1;
    for (int i = lo; i < hi; ++i) {
      const int Li = live_length(a, i);
      if (Li == 0) continue;
      if (leader < 0) leader = i;
      least = min(least, Li);
    }
    shared_pages = leader < 0 ? 0 : least / a.page_size;
  }
  int bad = L == 0;
  if (!bad) {
    const int32_t* row = a.page_table + static_cast<int64_t>(r) * a.max_pages;
    const int32_t* lead = a.page_table + static_cast<int64_t>(max(leader, 0)) * a.max_pages;
    for (int i = t; i < (L + a.page_size - 1) / a.page_size; i += kPfDim) {
      const int p = __ldg(row + i);
      if (p < 0 || p >= a.num_pages || (i < shared_pages && p != __ldg(lead + i))) bad = 1;
    }
  }
  bad = __syncthreads_or(bad);
  if (bad) {
    for (int g = 0; g < a.G; ++g) {
      a.out[(row0 + g) * kPfDim + t] = 0;
      if (t == 0 && a.lse != nullptr) a.lse[row0 + g] = -INFINITY;
    }
    return;
  }
  for (int g = 0; g < kPfGroupMax; ++g)
    s_q[g][t] = g < a.G ? bf16_bits_to_float(a.q[(row0 + g) * kPfDim + t]) : 0.f;
  __syncthreads();
  const float kmul = (kFp8 ? __ldg(a.k_scale) : 1.f) * a.sm_scale_log2;
  const int tpp = a.page_size >> 4;
  float m[kPfGroupMax], l[kPfGroupMax], o[kPfGroupMax];
  for (int g = 0; g < kPfGroupMax; ++g) {
    m[g] = -INFINITY;
    l[g] = o[g] = 0.f;
  }
  for (int tile = 0; tile * kPfTile < L; ++tile) {
    const int page = __ldg(a.page_table + static_cast<int64_t>(r) * a.max_pages + tile / tpp);
    const int64_t kb = ((static_cast<int64_t>(page) * a.Hkv + h) * tpp + tile % tpp) * 2 * kPfTile * kPfDim;
    const int n = min(kPfTile, L - tile * kPfTile);
    const int sg = t >> 4, st = t & 15;
    float s = -INFINITY;
    if (st < n) {
      s = 0.f;
      for (int d = 0; d < kPfDim; ++d) s = fmaf(s_q[sg][d], pool_value<kFp8>(a.kv_pool, kb + st * kPfDim + d), s);
      s *= kmul;
    }
    s_s[sg][st] = s;
    __syncthreads();
    float v[kPfTile];
    for (int j = 0; j < n; ++j) v[j] = pool_value<kFp8>(a.kv_pool, kb + kPfTile * kPfDim + t * kPfTile + j);
    for (int g = 0; g < a.G; ++g) {
      float mn = m[g];
      for (int j = 0; j < n; ++j) mn = fmaxf(mn, s_s[g][j]);
      const float f = m[g] == -INFINITY ? 0.f : exp2f(m[g] - mn);
      o[g] *= f;
      l[g] *= f;
      m[g] = mn;
      for (int j = 0; j < n; ++j) {
        const float p = mn == -INFINITY ? 0.f : exp2f(s_s[g][j] - mn);
        l[g] += p;
        o[g] = fmaf(p, v[j], o[g]);
      }
    }
    __syncthreads();
  }
  const float vmul = kFp8 ? __ldg(a.v_scale) : 1.f;
  for (int g = 0; g < a.G; ++g) {
    const bool none = l[g] == 0.f;
    const __nv_bfloat16 y = __float2bfloat16_rn(none ? 0.f : o[g] * vmul / l[g]);
    a.out[(row0 + g) * kPfDim + t] = __bfloat16_as_ushort(y);
    if (t == 0 && a.lse != nullptr) a.lse[row0 + g] = none ? -INFINITY : (m[g] + log2f(l[g])) * kPfLn2;
  }
}

size_t prefix_workspace(int32_t B, int32_t Hq) {
  (void)B;
  (void)Hq;
  return 256;
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
  if (static_cast<int64_t>(B) * Hq > 0x7fffffff / 4) return FPK_EUNSUPPORTED;
  if (B == 0) return FPK_OK;
  if (!q || !kv_pool || !page_table || !seq_lens || !out || !workspace) return FPK_EINVAL;
  if (kFp8 && (!k_scale || !v_scale)) return FPK_EINVAL;
  if (n_groups > 0 && (!group_starts || !prefix_lens)) return FPK_EINVAL;
  if (!aligned16(q) || !aligned16(kv_pool) || (reinterpret_cast<uintptr_t>(out) & 31u) != 0 ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FPK_EINVAL;
  if (workspace_bytes < prefix_workspace(B, Hq)) return FPK_ENOSPC;
  PrefixArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.kv_pool = static_cast<const uint8_t*>(kv_pool);
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.page_table = page_table;
  a.seq_lens = seq_lens;
  a.abort_mask = abort_mask;
  a.group_starts = group_starts;
  a.prefix_lens = prefix_lens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.n_groups = n_groups;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = G;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.sm_scale_log2 = sm_scale * kPfLog2e;
  prefix_simple_kernel<kFp8><<<B * Hkv, kPfDim, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return checked_launch_status();
}

}  // namespace
}  // namespace fpk

extern "C" size_t fpk_prefix_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D) {
  if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Hq / Hkv > fpk::kPfGroupMax || D != fpk::kPfDim) return 0;
  return fpk::prefix_workspace(B, Hq);
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
