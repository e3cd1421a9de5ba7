// The 4-bit formats: the paged Q4 cache and the tiled Q4_0 weights (contracts
// in tqd.h), and the tensor-core pieces the kernels over them share.
//
// Both keep the nibbles of one group of 32 where one mma.sync operand lane
// needs them: a 32-bit word holds eight codes of a group, and
//   word & 0x000F000F         codes 0 and 4 in the low bits of two f16
//   word & 0x00F000F0         codes 1 and 5, times 16
//   (word >> 8) & ...         codes 2, 6 and 3, 7
// V's and the weights become pairs of code - 8 by one packed operation more
// (Unpack).  K's are operands as they are: f16 subnormals, code * 2^-24 and code *
// 2^-20 exactly, the factors undone exactly (the 16 on the other operand, 2^24
// on the sums) and 8 sum q taken off.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "tqd_device.cuh"

namespace tqd {

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = A B + c.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                        float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The two f16 of a word as f32.
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// x rounded to f16.
__device__ __forceinline__ float round_f16(float x) { return __half2float(__float2half_rn(x)); }

// 2^e as f32, e in -126 .. 127.
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }

// The constants of unpacking codes to signed f16, kept in registers (as immediates
// they cost an instruction each: a logic operation takes one).
struct Unpack {
  uint32_t lo, hi, magic, off, sixteenth, off_hi;
  __device__ Unpack() {
    asm volatile("mov.b32 %0, 0x000F000F;" : "=r"(lo));
    asm volatile("mov.b32 %0, 0x00F000F0;" : "=r"(hi));
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(magic));
    off = 0xE408E408u;        // -1032
    sixteenth = 0x2C002C00u;
    off_hi = 0xD480D480u;     // -72
  }
  // The codes in bits 0-3 (low) or 4-7 (high) of each half of x as f16 pairs of
  // code - 8: 1024 + code and 1024 + 16 code are exact f16, so is the result.  (Whole
  // numbers under an f16 exponent: Kim, Henry, Fahim and Awadalla, "Who Says Elephants
  // Can't Run: Bringing Large Scale MoE Models into Cloud Scale Production", 2022.)
  __device__ __forceinline__ uint32_t low(uint32_t x) const {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(x), "r"(lo), "r"(magic));
    asm("add.rn.f16x2 %0, %0, %1;" : "+r"(v) : "r"(off));
    return v;
  }
  __device__ __forceinline__ uint32_t high(uint32_t x) const {
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(x), "r"(hi), "r"(magic));
    asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(v) : "r"(sixteenth), "r"(off_hi));
    return v;
  }
};

// A float of another CTA of the cluster, at the address that it has in this one.
__device__ __forceinline__ float ld_cluster(const float* p, uint32_t rank) {
  float v;
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

constexpr int kQ4Block = 16;  // positions per cache block

// Bytes of one cache block (16 positions of one head): K codes, K scales, V codes, V scales.
__host__ __device__ constexpr int q4_block_bytes(int hd) { return 18 * hd; }
__host__ __device__ constexpr int q4_ks_off(int hd) { return 8 * hd; }
__host__ __device__ constexpr int q4_v_off(int hd) { return 9 * hd; }
__host__ __device__ constexpr int q4_vs_off(int hd) { return 17 * hd; }

// Byte offset inside the block of the K row of position b (0..15): rows are
// stored in the order the score's tensor-core operand takes them.
__host__ __device__ constexpr int q4_k_row(int b, int hd) {
  return (((b >> 1) & 1) * 8 + (b >> 2) * 2 + (b & 1)) * (hd / 2);
}
// Byte offset (from the block's start) of the 2 * hd / 32 bytes that hold, for
// position b, the codes of elements n, n + 8, n + 16, ... (nibble i: element n + 8 i).
__host__ __device__ constexpr int q4_v_piece(int b, int n, int hd) {
  return q4_v_off(hd) + (hd == 128 ? ((b >> 1) & 1) * 512 + (b >> 2) * 128 + n * 16 + (b & 1) * 8
                                   : (b >> 2) * 128 + n * 16 + (b & 3) * 4);
}

struct Q4Cache {
  uint8_t* pages;
  const int32_t* table;
  int n_pages, page_size, n_kv, n_seq, table_stride;
  size_t page_bytes;
};

struct Q4AttnArgs {
  Q4Cache c;
  const float* q;
  float* out;
  const int32_t* lens;
  const int32_t* q_start;  // [n_seq + 1], or null: one query per sequence
  void* scratch;
  int64_t q_stride, out_stride;
  int n_tokens, n_heads;
  float scale;             // 1 / sqrt(head_dim)
};

// Tiles of Q4_0 weights: 16 rows x 128 columns.
constexpr int kQ4TileRows = 16;
constexpr int kQ4TileCols = 128;
constexpr int kQ4TileBytes = 1152;
constexpr int kQ4TileScales = 1024;  // offset of the scales, f16 [16][4]

}  // namespace tqd
