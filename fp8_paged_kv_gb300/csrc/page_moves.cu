// page_moves.cu -- forking requests (shared full pages, a copy of the page in
// use) and compacting a pool (whole pages moved, tables and tags following).
//
// A page's tag changes on every reallocation and a request expects the tag of
// each page it maps ("Cosa ha cambiato Cloudflare per Kimi e GLM" and "La
// sicurezza della cache KV condivisa diventa una questione di produzione",
// remio.ai).  A fork's fresh page and a compaction's target are reallocated
// pages: their tags advance, and the rows that map them from here on expect
// the new tag.  The host's page ledger decides which pages; these kernels move
// the bytes and the entries.  Both are copies, bound by HBM.  64 forks of one
// request, 128 KiB of its last page in each of 32 layers: 48 us (5.7 TB/s, nearly
// all of it writes; the source stays in L2); 4001 pages of 32 KiB in 8 layers moved:
// 328 us, 6.4 TB/s (94 % of what a copy reaches); 3.3 us for a few pages, a launch
// and its chain of reads.
#include "step_ops.cuh"

namespace fpk {
namespace {

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;  // 16-byte loads in flight per thread

struct MoveArgs {
  uint8_t* pool;
  int64_t layer_stride;  // bytes
  int64_t page_bytes;    // bytes of a page in one layer
  int32_t* page_table;
  uint32_t* expected_tags;
  int32_t* seq_lens;
  uint32_t* live_tags;
  uint8_t* abort_mask;
  int n, B, Hkv, page_size, num_pages, max_pages, layers, tile_bytes;
};

// `runs` runs of `units` 16-byte units, `stride` units apart, from src to dst by the CTA's threads: eight loads of
// a thread on their way before its first store, across the runs.
__device__ __forceinline__ void copy_runs(uint8_t* dst, const uint8_t* src, int runs, int units, int stride) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int total = runs * units;  // (a page of one layer: some 2^20 units at most)
#pragma unroll 1
  for (int i = threadIdx.x; i < total; i += kMoveThreads * kMoveUnroll) {
    uint4 x[kMoveUnroll];
    int at[kMoveUnroll];
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k) {
      const int e = i + k * kMoveThreads, run = e / units;
      at[k] = run * stride + e - run * units;
      if (e < total) x[k] = __ldg(s + at[k]);
    }
#pragma unroll
    for (int k = 0; k < kMoveUnroll; ++k)
      if (i + k * kMoveThreads < total) d[at[k]] = x[k];
  }
}

// CTAs [0, n): the row of fork i.  The rest copy, one (fork, layer) each: the
// page in use, its tiles that hold tokens (a run of them per kv head).
__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const MoveArgs a, const int32_t* __restrict__ parent,
                                                            const int32_t* __restrict__ child,
                                                            const int32_t* __restrict__ fresh) {
  const bool row_cta = static_cast<int>(blockIdx.x) < a.n;
  const int64_t job = row_cta ? blockIdx.x : static_cast<int64_t>(blockIdx.x) - a.n;
  const int i = static_cast<int>(row_cta ? job : job % a.n);
  const int pr = __ldg(parent + i), ch = __ldg(child + i), fr = __ldg(fresh + i);
  if (ch < 0 || ch >= a.B) return;
  bool ok = pr >= 0 && pr < a.B && pr != ch;
  const int L = ok ? max(a.seq_lens[pr], 0) : 0;
  const int pages = L / a.page_size + (L % a.page_size != 0);  // L may be near 2^31
  const int rem = L % a.page_size;
  ok = ok && pages <= a.max_pages && (rem == 0 || (fr >= 0 && fr < a.num_pages));
  const int32_t* prow = a.page_table + static_cast<int64_t>(ok ? pr : 0) * a.max_pages;
  const uint32_t* ptag = a.expected_tags + static_cast<int64_t>(ok ? pr : 0) * a.max_pages;
  if (!row_cta) {
    if (!ok || rem == 0) return;
    const int src = prow[pages - 1];
    if (src < 0 || src >= a.num_pages || src == fr) return;
    const int layer = static_cast<int>(job / a.n);
    const int head = (a.page_size >> 4) * (a.tile_bytes >> 4), used = ((rem + 15) >> 4) * (a.tile_bytes >> 4);
    uint8_t* base = a.pool + layer * a.layer_stride;
    copy_runs(base + fr * a.page_bytes, base + src * a.page_bytes, a.Hkv, used, head);
    return;
  }
  int bad = !ok;
  if (ok)
    for (int j = threadIdx.x; j < pages && !bad; j += kMoveThreads) {
      const int p = prow[j];
      bad = p < 0 || p >= a.num_pages || a.live_tags[p] != ptag[j];
    }
  bad = __syncthreads_or(bad);
  const uint32_t tag = !bad && rem != 0 ? a.live_tags[fr] + 1u : 0u;
  __syncthreads();
  int32_t* crow = a.page_table + static_cast<int64_t>(ch) * a.max_pages;
  uint32_t* ctag = a.expected_tags + static_cast<int64_t>(ch) * a.max_pages;
  for (int j = threadIdx.x; j < a.max_pages; j += kMoveThreads) {
    int p = -1;
    uint32_t t = 0;
    if (!bad && j < pages) {
      const bool own = rem != 0 && j == pages - 1;
      p = own ? fr : prow[j];
      t = own ? tag : ptag[j];
    }
    crow[j] = p;
    ctag[j] = t;
  }
  if (threadIdx.x == 0) {
    a.seq_lens[ch] = bad ? 0 : L;
    if (bad && a.abort_mask != nullptr) a.abort_mask[ch] = 1;
    if (!bad && rem != 0) a.live_tags[fr] = tag;
  }
}

// The first remaps CTAs go over the tables, the others copy: CTA = (move, layer), one page.  An entry (r, j) of a
// moved page looks its page up in the ascending list src.  Tags are as they were before the moves.
__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const MoveArgs a, const int32_t* __restrict__ src,
                                                               const int32_t* __restrict__ dst, int remaps) {
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= remaps) {
    const int copies = static_cast<int>(gridDim.x) - remaps;
    for (int64_t job = static_cast<int>(blockIdx.x) - remaps; job < static_cast<int64_t>(a.n) * a.layers; job += copies) {
      const int i = static_cast<int>(job % a.n);
      const int s = __ldg(src + i), d = __ldg(dst + i);
      if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages) continue;
      uint8_t* base = a.pool + job / a.n * a.layer_stride;
      const int units = static_cast<int>(a.page_bytes >> 4);
      copy_runs(base + d * a.page_bytes, base + s * a.page_bytes, 1, units, units);
    }
    return;
  }
  const int64_t total = static_cast<int64_t>(a.B) * a.max_pages;
  for (int64_t e = blockIdx.x * static_cast<int64_t>(kMoveThreads) + threadIdx.x; e < total;
       e += static_cast<int64_t>(remaps) * kMoveThreads) {
    const int r = static_cast<int>(e / a.max_pages);
    const int j = static_cast<int>(e - static_cast<int64_t>(r) * a.max_pages);
    const int p = a.page_table[e];
    const uint32_t expected = a.expected_tags[e];
    const int L = __ldg(a.seq_lens + r);
    if (L <= 0 || j > (L - 1) / a.page_size) continue;
    if (p < 0 || p >= a.num_pages) continue;
    int lo = 0, hi = a.n;  // first index whose source is not below p
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(src + mid) < p) lo = mid + 1; else hi = mid;
    }
    if (lo >= a.n || __ldg(src + lo) != p || a.live_tags[p] != expected) continue;
    const int d = __ldg(dst + lo);
    if (d < 0 || d >= a.num_pages) continue;
    a.page_table[e] = d;
    a.expected_tags[e] = a.live_tags[d] + 1u;
  }
}

// Behind the compaction (every table entry has read the tags by then).
__global__ void __launch_bounds__(kMoveThreads) moved_tags_kernel(const MoveArgs a, const int32_t* __restrict__ src,
                                                                  const int32_t* __restrict__ dst) {
  const int i = blockIdx.x * kMoveThreads + threadIdx.x;
  const int s = i < a.n ? __ldg(src + i) : -1, d = i < a.n ? __ldg(dst + i) : -1;
  griddep_wait();
  if (s < 0 || s >= a.num_pages || d < 0 || d >= a.num_pages) return;
  a.live_tags[d] += 1u;
}

int move_args(MoveArgs& a, void* kv_pool, int32_t elem_bytes, int32_t layers, int64_t layer_stride,
              int32_t* page_table, int32_t max_pages, uint32_t* expected_tags, int32_t* seq_lens,
              uint32_t* live_tags, int32_t n, int32_t B, int32_t Hkv, int32_t D, int32_t page_size,
              int32_t num_pages) {
  if (n < 0 || B < 0 || Hkv <= 0 || D <= 0 || page_size <= 0 || num_pages < 0 || max_pages < 0 || layers < 0 ||
      layer_stride < 0)
    return FPK_EINVAL;
  if (D != 128 || page_size % 16 != 0 || page_size > 256) return FPK_EUNSUPPORTED;
  if (elem_bytes != 1 && elem_bytes != 2) return FPK_EUNSUPPORTED;
  if (n == 0 || B == 0) return FPK_OK;
  if (!kv_pool || !page_table || !expected_tags || !seq_lens || !live_tags) return FPK_EINVAL;
  if (!aligned16(kv_pool) || (layer_stride & 15) != 0) return FPK_EINVAL;
  a.pool = static_cast<uint8_t*>(kv_pool);
  a.layer_stride = layer_stride;
  a.tile_bytes = 2 * 16 * D * elem_bytes;
  a.page_bytes = static_cast<int64_t>(Hkv) * (page_size >> 4) * a.tile_bytes;
  if (layers > 1 && layer_stride < a.page_bytes * num_pages) return FPK_EINVAL;
  a.page_table = page_table;
  a.expected_tags = expected_tags;
  a.seq_lens = seq_lens;
  a.live_tags = live_tags;
  a.abort_mask = nullptr;
  a.n = n;
  a.B = B;
  a.Hkv = Hkv;
  a.page_size = page_size;
  a.num_pages = num_pages;
  a.max_pages = max_pages;
  a.layers = layers;
  return FPK_OK;
}

}  // namespace
}  // namespace fpk

extern "C" int fpk_kv_fork(void* kv_pool, int32_t elem_bytes, int32_t layers, int64_t layer_stride,
                           int32_t* page_table, int32_t max_pages, uint32_t* expected_tags,
                           int32_t* seq_lens, uint32_t* live_tags, uint8_t* abort_mask,
                           const int32_t* parent, const int32_t* child, const int32_t* fresh, int32_t n,
                           int32_t B, int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                           void* stream) {
  using namespace fpk;
  MoveArgs a;
  const int st = move_args(a, kv_pool, elem_bytes, layers, layer_stride, page_table, max_pages, expected_tags,
                           seq_lens, live_tags, n, B, Hkv, D, page_size, num_pages);
  if (st != FPK_OK || n == 0 || B == 0) return st;
  if (!parent || !child || !fresh) return FPK_EINVAL;
  const int64_t ctas = static_cast<int64_t>(n) * (1 + static_cast<int64_t>(layers));
  if (ctas > 0x7fffffff) return FPK_EINVAL;
  a.abort_mask = abort_mask;
  fork_kernel<<<static_cast<int>(ctas), kMoveThreads, 0, static_cast<cudaStream_t>(stream)>>>(a, parent, child,
                                                                                           fresh);
  return checked_launch_status();
}

extern "C" int fpk_kv_compact(void* kv_pool, int32_t elem_bytes, int32_t layers, int64_t layer_stride,
                              int32_t* page_table, int32_t max_pages, uint32_t* expected_tags,
                              const int32_t* seq_lens, uint32_t* live_tags, const int32_t* src,
                              const int32_t* dst, int32_t n, int32_t B, int32_t Hkv, int32_t D,
                              int32_t page_size, int32_t num_pages, void* stream) {
  using namespace fpk;
  MoveArgs a;
  const int st = move_args(a, kv_pool, elem_bytes, layers, layer_stride, page_table, max_pages, expected_tags,
                           const_cast<int32_t*>(seq_lens), live_tags, n, B, Hkv, D, page_size, num_pages);
  if (st != FPK_OK || n == 0 || B == 0) return st;
  if (!src || !dst) return FPK_EINVAL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // pages: as many CTAs as are resident at once; tables: one per 256 entries, up to as many again
  const int64_t jobs = static_cast<int64_t>(n) * layers;
  const int64_t entries = (static_cast<int64_t>(B) * max_pages + kMoveThreads - 1) / kMoveThreads;
  const int full = resident_grid(reinterpret_cast<const void*>(compact_kernel), kMoveThreads, 0, jobs > entries ? jobs : entries);
  const int copies = static_cast<int>(jobs < full ? jobs : full), remaps = static_cast<int>(entries < full ? entries : full);
  if (copies + remaps > 0) {
    compact_kernel<<<copies + remaps, kMoveThreads, 0, s>>>(a, src, dst, remaps);
    if (checked_launch_status() != FPK_OK) return FPK_ECUDA;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((n + kMoveThreads - 1) / kMoveThreads);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = copies + remaps > 0 ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, moved_tags_kernel, a, src, dst) != cudaSuccess) return FPK_ECUDA;
  return checked_launch_status();
}
