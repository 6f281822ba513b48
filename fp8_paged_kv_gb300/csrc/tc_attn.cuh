// tc_attn.cuh -- what the attention kernels on the fifth-generation tensor cores
// share (prefix_attn.cu, prefill_attn.cu): products S = Q K^T with the row tile's
// queries in shared memory, loads and stores of tensor memory, packed fp32 pairs,
// waits that give up together, the pool's tensor maps and dependent launches.
#pragma once

#include "tcgen05.cuh"

namespace fpk {
namespace {

// x / d for d <= 16 by its reciprocal `by`: exact while x (by d - 2^32) < 2^32, that is for x < 2^28.
__device__ __forceinline__ int quotient(int x, uint32_t by) {
  return by == 0 ? x : static_cast<int>(__umulhi(static_cast<uint32_t>(x), by));
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void* tmap, int x, int y, int z, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ uint64_t l2_policy_evict_normal() {
  uint64_t pol;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(pol));
  return pol;
}

// Instruction descriptors: M = N = 128, both operands K-major, D in fp32.
constexpr uint32_t tc_idesc(int n, uint32_t type) {
  return (1u << 4) | (type << 7) | (type << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(128 >> 4) << 24);
}
constexpr uint32_t kTcSE4m3 = tc_idesc(128, 0), kTcSBf16 = tc_idesc(128, 1);  // kind::f8f6f4, kind::f16
constexpr uint32_t kTcOF16 = tc_idesc(128, 0), kTcOBf16 = tc_idesc(128, 1);   // kind::f16

// One elected lane of the (converged) warp issues; everything is predicated, not branched, so that the
// operands stay in uniform registers.
#define TC_COMMIT "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 "
// Arrives on `bar` once every product that this warp's elected lane has issued is done.
__device__ __forceinline__ void commit_elected(uint32_t bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t@e " TC_COMMIT "[%0];\n\t}" ::"r"(bar) : "memory");
}

// S = Q K^T, both operands from shared memory: eight steps of 32 bytes of K, four per atom of 128
// bytes (e4m3: two query parts against the same K rows; bf16: two halves of the dims, K's %4 apart).
#define TC_S_STEP(kind, x, first)                                                             \
  "add.s64 a, %1, " #x ";\n\tadd.s64 b, k, " #x ";\n\t@e tcgen05.mma.cta_group::1.kind::" kind \
  " [%0], a, b, %3, " first ";\n\t"
#define TC_S(kind)                                                                                             \
  "{\n\t.reg .pred e, no, yes;\n\t.reg .b64 a, b, k;\n\telect.sync _|e, 0xffffffff;\n\t"                       \
  "setp.ne.u32 no, 0, 0;\n\tsetp.eq.u32 yes, 0, 0;\n\tmov.b64 k, %2;\n\t" TC_S_STEP(kind, 0, "no")             \
      TC_S_STEP(kind, 2, "yes") TC_S_STEP(kind, 4, "yes") TC_S_STEP(kind, 6, "yes")                            \
  "add.s64 k, %2, %4;\n\tsub.s64 k, k, 1024;\n\t" TC_S_STEP(kind, 1024, "yes") TC_S_STEP(kind, 1026, "yes")    \
      TC_S_STEP(kind, 1028, "yes") TC_S_STEP(kind, 1030, "yes") "}"
template <bool kFp8>
__device__ __forceinline__ void issue_s(uint32_t d, uint64_t qdesc, uint64_t kdesc) {
  if (kFp8)
    asm volatile(TC_S("f8f6f4")::"r"(d), "l"(qdesc), "l"(kdesc), "r"(kTcSE4m3), "n"(0) : "memory");
  else
    asm volatile(TC_S("f16")::"r"(d), "l"(qdesc), "l"(kdesc), "r"(kTcSBf16), "n"(128 * 128 >> 4) : "memory");
}

// 64 consecutive columns of this thread's tensor memory lane, waited for.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
      "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
      "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
      "%62, %63}, [%64]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
}

// The same with their largest value (a NaN counts only among NaNs), found on the way.
__device__ __forceinline__ float tmem_ld64_max(uint32_t taddr, float (&v)[64]) {
  uint32_t r[64];
  float top;
  asm volatile(
      "tcgen05.ld.red.sync.aligned.32x32b.x64.max.f32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, "
      "%22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, "
      "%42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, "
      "%62, %63}, %64, [%65]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63]), "=f"(top)
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 64; ++i) v[i] = __uint_as_float(r[i]);
  return top;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// 16 columns times f.
__device__ __forceinline__ void tmem_scale16(uint32_t taddr, float f) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16]; "
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16}; "
      ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void bulk_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

// 32 bytes: a whole sector from one thread.
__device__ __forceinline__ void st_global8(float* dst, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(x[0]), "f"(x[1]), "f"(x[2]),
               "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}

// Packed fp32 pairs: one instruction each on sm_103a.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
  return r;
}
__device__ __forceinline__ void tmem_fill1(uint32_t taddr, float x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(x)) : "memory");
}
__device__ __forceinline__ void tmem_fill8(uint32_t taddr, float x) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(taddr),
               "r"(__float_as_uint(x))
               : "memory");
}
__device__ __forceinline__ void tmem_fill32(uint32_t taddr, float x) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, "
      "%1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(taddr),
      "r"(__float_as_uint(x))
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A wait that gives up once any wait of the CTA has: control flow then runs on
// to the end without waiting (every address stays in range; the results are
// void and the status word says so), so that no barrier is left waiting.
__device__ __noinline__ void tc_wait_long(uint32_t bar, uint32_t parity, uint32_t* status, volatile int* failed) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return;
    if ((it & 255u) == 0u) {
      if (*failed) return;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *failed = 1;
        atomicOr(status, kStatusWaitTimeout);
        return;
      }
    }
  }
}
// A word that another warp writes.
__device__ __forceinline__ int load_shared(uint32_t at) {
  int x;
  asm volatile("ld.volatile.shared.s32 %0, [%1];" : "=r"(x) : "r"(at) : "memory");
  return x;
}
__device__ __forceinline__ void tc_wait(uint32_t bar, uint32_t parity, uint32_t* status, volatile int* failed) {
  if (!mbar_try_wait(bar, parity)) tc_wait_long(bar, parity, status, failed);
}

// A value the compiler does not know to be a loop's invariant: a loop is not copied for each of its
// cases.  Code is kept small all over: 16 warps run six programs, and what the instruction caches do not
// hold is fetched anew at some ten cycles an instruction.
__device__ __forceinline__ int varying(int x) {
  asm volatile("" : "+r"(x));
  return x;
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// The pool as tiles of rows: K rows come first, V behind them; boxes of zbox tiles.
inline int encode_pool_map(CUtensorMap* m, const void* pool, int64_t tiles, bool fp8, bool v, int zbox) {
  EncodeTiled enc = tensor_map_encoder();
  if (enc == nullptr) return FPK_ECUDA;
  const bool narrow = v && !fp8;  // bf16 V: rows of 16 tokens
  const cuuint64_t inner = narrow ? 16 : 128, rows = narrow ? 256 : 32, el = fp8 ? 1 : 2;
  const cuuint64_t dims[3] = {inner, rows, static_cast<cuuint64_t>(tiles)};
  const cuuint64_t strides[2] = {inner * el, inner * el * rows};
  const cuuint32_t box[3] = {narrow ? 16u : fp8 ? 128u : 64u, narrow ? 128u : 16u, static_cast<cuuint32_t>(zbox)};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapSwizzle sw = !v ? CU_TENSOR_MAP_SWIZZLE_128B : fp8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_32B;
  const CUresult r = enc(m, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                         const_cast<void*>(pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? FPK_OK : FPK_ECUDA;
}

// Launches `kernel` as a programmatic dependent of the kernel before it.
template <typename... Exp, typename... Act>
int launch_dependent(void (*kernel)(Exp...), int grid, int threads, size_t smem, cudaStream_t s, Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<Act&&>(args)...) != cudaSuccess) return FPK_ECUDA;
  return checked_launch_status();
}

}  // namespace
}  // namespace fpk
