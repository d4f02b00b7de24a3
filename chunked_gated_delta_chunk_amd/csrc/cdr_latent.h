// What the latent attention kernels share (gfx950).
#pragma once
#include "cdr_common.h"

namespace cdr {

constexpr int LC = 512;             // latent dimensions of a cached key, also the values' of the absorbed form
constexpr int LR = 64;              // rope dimensions
constexpr int LROW = LC + LR;       // a cached key
constexpr float LOG2E = 1.44269504088896341f;
constexpr float LN2 = 0.69314718055994531f;

typedef __attribute__((address_space(3))) char lds_char;

// One 16-byte global-to-LDS copy a lane: lane l's 16 bytes at `src` go to LDS offset lds + 16 l; lds is
// the same for the whole wave, which is whole.  Written as one block without register outputs, so
// that the compiler neither waits for it before later LDS reads nor reuses a register of it; the
// caller waits with dma_wait() before the barrier behind which the data is read.  m0 is written: no
// kernel that uses it keeps anything there (gfx9 LDS instructions do not need it).
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory");
}
// the same from a base shared by the wave and each lane's byte offset
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}
// Waits for this wave's copies and loads.  The builtin, not asm: the compiler then knows that its own
// earlier loads have arrived and does not wait for them again behind copies that are still under way.
__device__ __forceinline__ void dma_wait() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    asm volatile("" ::: "memory");
}

// Nothing is moved across this.  Between a batch of LDS reads and the products of the batch before
// it: left alone, the compiler reads one operand, waits and multiplies, one LDS latency a product.
__device__ __forceinline__ void keep_order() { __builtin_amdgcn_sched_barrier(0); }

// Byte offset of an LDS pointer, as m0 and the asm above take it.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
    return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}

// Transposing LDS read: each lane gives the address of four bf16; in each group of 16 lanes these are
// a 4 x 16 tile (lanes 4 k .. 4 k + 3 hold row k), and lane i receives its column i, rows 0 to 3.
typedef short s16x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ s16x4 lds_tr(const void* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(__attribute__((address_space(3))) void*)const_cast<void*>(p));
}
__device__ __forceinline__ bf16x8 join8(const s16x4& a, const s16x4& b) {
    const bf16x8 r = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    return r;
}
__device__ __forceinline__ bf16x8 lds16(const void* p) { return *static_cast<const bf16x8*>(p); }

// Packed rows that no sequence holds, in front of the first offset and behind the last one: each row's `units`
// values of type T at base + row * units set to v.  The workgroups of a launch (`wg` of `wgs`) take rows in turn.
template <typename T>
__device__ __forceinline__ void fill_unheld(T* base, int64_t units, const T& v, const int32_t* cu, int N, int total, int wg,
                                            int wgs) {
    const int first = min(max(cu[0], 0), total), end = min(max(cu[N], first), total);
    const int64_t count = first + total - end;
    for (int64_t i = wg; i < count; i += wgs) {
        T* p = base + (i < first ? i : i - first + end) * units;
        for (int64_t u = threadIdx.x; u < units; u += blockDim.x) p[u] = v;
    }
}

// base-2 exponential and logarithm of the hardware (one unit in the last place)
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

// Where a tile's 16-byte pieces are stored: row `row` keeps piece p at p ^ f(row).  The 64 banks serve a
// 16-byte read in four cycles of 16 lanes (lanes 0-3, 12-15, 20-27 together, and so on) and a transposing
// read in two cycles of 32.  f16, for rows of a multiple of 256 bytes, is one to one on 16 rows and puts
// four neighbouring rows four pieces apart; f8 does the same for rows of 128 bytes, two of which share
// 256.  Counted: no conflicts in either read; with neighbours two pieces apart each transposing read took
// four cycles.  f16w is for the 16-row operands of the decode kernel, where a transposing read takes eight
// rows of two pieces: one to one, rows 0-7 and 8-15 each two pieces apart, and rows 0-3 and 12-15 in
// whole pairs of pieces, so that the four pieces of the other lanes' rows stay clear of theirs.
__device__ __forceinline__ int f16(int row) { return ((row & 3) << 2) | ((row >> 2) & 3); }
__device__ __forceinline__ int f8(int row) { return (((row >> 1) & 1) << 2) | ((row >> 2) & 3); }
__device__ __forceinline__ int f16w(int row) { return (((row & 7) ^ ((row >> 1) & 4)) << 1) | ((row >> 3) & 1); }

// 32x32x16 products: A[m = lane & 31][k = 8 (lane >> 5) + i], B likewise, and the result's register i
// holds row 8 (i / 4) + 4 (lane >> 5) + i % 4 of column lane & 31.
typedef __attribute__((__vector_size__(16 * sizeof(float)))) float f32x16;
__device__ __forceinline__ f32x16 mma(const bf16x8& a, const bf16x8& b, const f32x16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x16 zero16() {
    f32x16 z;
#pragma unroll
    for (int i = 0; i < 16; ++i) z[i] = 0.f;
    return z;
}
// registers 8 t .. 8 t + 7 of a result as the right operand of the next product
__device__ __forceinline__ bf16x8 operand(const f32x16& p, int t) {
    const uint4 v = make_uint4(pack_bf2(p[8 * t], p[8 * t + 1]), pack_bf2(p[8 * t + 2], p[8 * t + 3]),
                               pack_bf2(p[8 * t + 4], p[8 * t + 5]), pack_bf2(p[8 * t + 6], p[8 * t + 7]));
    return __builtin_bit_cast(bf16x8, v);
}

// A value that the compiler computes where it is used: copies of a loop's fixed offsets for every
// unrolled step, kept in registers over the loop, cost more than the one addition that makes them.
__device__ __forceinline__ int fresh(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

}  // namespace cdr
