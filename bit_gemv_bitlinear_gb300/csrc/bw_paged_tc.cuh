// bw_paged_tc.cuh -- tiled copies out of paged pools, shared by the decode
// and the prefill attention.
#pragma once

#include "bw_paged.cuh"
#include "bw_tc.cuh"

namespace bw {
namespace {

// 4-D tiled bulk copy of one box of `map` at coordinates (dim, row of the
// page, key-value head, page); completes the box's bytes on `bar` (a page out
// of range reads as zeros and is counted all the same).
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map,
                                            int c0, int c1, int c2, int c3,
                                            uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3), "r"(smem_addr(bar))
      : "memory");
}

// The same with an L2 policy.
__device__ __forceinline__ void tma_load_4d_once(void *dst,
                                                 const CUtensorMap *map, int c0,
                                                 int c1, int c2, int c3,
                                                 uint64_t *bar,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_"
      "tx::bytes.L2::cache_hint [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2),
      "r"(c3), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map))
               : "memory");
}

// A pool as a 4-D tensor (D, page rows, heads, pages), boxes of `rows` rows x
// 64 dims in the 128-byte swizzle.
bool encode_pool(CUtensorMap *map, const void *base, const PagedView &v, int D,
                 int rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (!fn) return false;
  const int page = 1 << v.page_shift;
  const cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(page),
                              cuuint64_t(v.hkv), cuuint64_t(v.n_pages)};
  const cuuint64_t strides[3] = {cuuint64_t(D) * 2, cuuint64_t(page) * D * 2,
                                 cuuint64_t(v.page_stride) * 2};
  const cuuint32_t box[4] = {64, cuuint32_t(rows), 1, 1};
  const cuuint32_t elem[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
            const_cast<void *>(base), dims, strides, box, elem,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The page of a box of `rows` positions from `pos` of sequence b; a box that
// nobody sees (seen: [0, s1) and [lo, hi)) and a bad page give a page past the
// pool, which reads as zeros.  Only an entry that is used is looked at.
__device__ __forceinline__ int box_page(const PagedView &v, int b, int pos,
                                        int rows, int s1, int lo, int hi) {
  const bool used = pos < s1 || (pos < hi && pos + rows > lo);
  const int page = used ? seq_page(v, b, pos) : -1;
  return page < 0 ? v.n_pages : page;
}

// CTAs of a kernel that fit on the device at once with `smem` bytes of dynamic
// shared memory (asked once per device and kernel).
template <typename Kernel>
cudaError_t paged_resident(Kernel kernel, std::atomic<int> *cached,
                           int threads, uint32_t smem, int *resident) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    e = cudaFuncSetAttribute(
        kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    int per_sm = 0;
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads,
                                                      smem);
    if (e != cudaSuccess) return e;
    const int sms = device_sm_count();
    if (per_sm < 1 || sms < 1) return cudaErrorInvalidConfiguration;
    n = per_sm * sms;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  *resident = n;
  return cudaSuccess;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2e = 1.44269504088896340736f;

}  // namespace
}  // namespace bw
