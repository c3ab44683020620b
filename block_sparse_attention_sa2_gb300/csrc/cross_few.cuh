// Device helpers that the attention kernels for few query rows share: copies into a warp's ring, the warp's products,
// and the layout of a step's keys in the ring.
#pragma once

#include "sa2_device.cuh"

namespace sa2 {

constexpr int kFewTileBytes = 4096;  // of K, and of V, per step of a warp

// 16 bytes from global to shared memory; zeros where !live (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, bool KV8>
struct FewTile {
  static constexpr int kRow = D * (KV8 ? 1 : 2);     // bytes of a key
  static constexpr int kChunks = kRow / 16;          // 16-byte chunks of a key
  static constexpr int kPer = KV8 ? 16 : 8;          // values per chunk
  static constexpr int kKeys = kFewTileBytes / kRow;  // keys per step: 16, 32 or 64
  // chunk c of key r, swizzled so that the fragments' reads (see the kernel) use all banks
  static __device__ __forceinline__ uint32_t at(int r, int c) {
    if constexpr (kChunks >= 8) return r * kRow + ((c ^ (r & 7)) << 4);
    const int line = r >> 1;  // 64-byte rows: two to a line
    return line * 128 + (((((r & 1) << 2) | c) ^ (line & 7)) << 4);
  }
};

}  // namespace sa2
