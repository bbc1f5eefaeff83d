// What the products of 8-bit rows share, whatever the codes: the wavefronts'
// order of weight rows, the tiles' order over the chip, loads straight to LDS
// and their waits, silu, and the stores of a lane's run of columns.
#pragma once

#include "q4_common.h"
#include "q4i8.h"

namespace q4 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kCUs = 256;

// Tiles of 256 x 256 come in rounds of one for each CU.  Where the last round
// would have up to 128, they go to a launch of their own (kHalves, 128 rows
// each, where there are more than 64; kQuarters, 128 x 128, else), which takes
// one round of two thirds or a third of the time.  What it measured stands at
// each kernel's choice.
enum Part { kAll, kWhole, kHalves, kQuarters };
constexpr int kRestMost = 128, kQuartersMost = 64;

// The fragment of 16 weight rows j (of F that share a run of 16 F rows) takes
// row frag_row<F>(j, i) of the run as its row i: lane group i / 4 then holds,
// over the F fragments, the 4 F consecutive rows from 4 F (i / 4) on.
template <int F>
__device__ __forceinline__ int frag_row(int j, int i) { return (i >> 2) * (4 * F) + 4 * j + (i & 3); }

// silu(v) = v / (1 + e^-v) for v >= kFar, where 1 + e^-v is below the 2^126 that
// the reciprocal takes.
constexpr float kFar = -87.f;
__device__ __forceinline__ float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

// silu(v) u below that, where silu(v) is v e^v to the last bit: e^v comes to be no
// normal number, and the product may still be any, so that it takes the two
// halves of e^v one before u and one after (each is normal down to v = -174.6,
// and zero below).
__device__ __forceinline__ float far_silu(float v, float u) {
    const float half = __builtin_amdgcn_exp2f(0.72134752044f * v);
    return v * half * u * half;
}

__device__ __forceinline__ uint32_t bits16(float v, int type) {
    if (type == I8_F16) return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// Stores of 16 and 8 bytes that need no more than their elements' alignment
// (the hardware takes any address; rows of odd N start anywhere).
typedef u32x4_t u32x4_at4_t __attribute__((aligned(4)));
typedef u32x4_t u32x4_at2_t __attribute__((aligned(2)));
typedef u32x2_t u32x2_at2_t __attribute__((aligned(2)));

// Writes the run v[0 .. C) of columns n .. of a row, those past N left out, to
// `base` (of i8_type `type`) from element `at` on.
template <int C>
__device__ __forceinline__ void store_run(void *base, int type, size_t at, int n, int N, const float (&v)[C]) {
    if (n >= N) return;
    const bool whole = n + C <= N;
    if (type == I8_F32) {
        float *y = static_cast<float *>(base) + at;
        if (whole) {
#pragma unroll
            for (int c = 0; c < C; c += 4)
                *reinterpret_cast<u32x4_at4_t *>(y + c) =
                    u32x4_t{__builtin_bit_cast(uint32_t, v[c]), __builtin_bit_cast(uint32_t, v[c + 1]),
                            __builtin_bit_cast(uint32_t, v[c + 2]), __builtin_bit_cast(uint32_t, v[c + 3])};
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (n + c < N) y[c] = v[c];
        }
        return;
    }
    uint16_t *y = static_cast<uint16_t *>(base) + at;
    uint32_t b[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) b[c] = bits16(v[2 * c], type) | bits16(v[2 * c + 1], type) << 16;
    if (whole) {
        if constexpr (C % 8 == 0) {
#pragma unroll
            for (int c = 0; c < C / 2; c += 4)
                *reinterpret_cast<u32x4_at2_t *>(y + 2 * c) = u32x4_t{b[c], b[c + 1], b[c + 2], b[c + 3]};
        } else {
#pragma unroll
            for (int c = 0; c < C / 2; c += 2) *reinterpret_cast<u32x2_at2_t *>(y + 2 * c) = u32x2_t{b[c], b[c + 1]};
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n + c < N) y[c] = (uint16_t)(b[c / 2] >> (16 * (c & 1)));
    }
}

// Workgroups are dealt to the eight XCDs in turn, each with its own L2: XCD x
// takes the x-th eighth of the tiles (of those that the groups have, not of
// those that they might have needed).  -1: workgroup b has none.
__device__ __forceinline__ int eighth_of(int b, int all) {
    const int x = b & 7, per = all >> 3, more = all & 7;
    return (b >> 3) < per + (x < more ? 1 : 0) ? x * per + min(x, more) + (b >> 3) : -1;
}

// The tile (tm, tn) that a workgroup takes, of tiles_m rows of them; false:
// none.  Tiles are ordered in bands of eight tile rows, column by column, so
// that the tiles an XCD runs at one time share rows of a and of w.
__device__ __forceinline__ bool tile_of(int b, int tiles_m, int tiles_n, int &tm, int &tn) {
    const int t = eighth_of(b, tiles_m * tiles_n);
    if (t < 0) return false;
    const int band = t / (8 * tiles_n), first = band * 8, rows = min(8, tiles_m - first);
    const int in = t - band * 8 * tiles_n;
    tm = first + in % rows;
    tn = in / rows;
    return true;
}

// Of `all` tiles, those that kWhole takes.
__device__ __host__ __forceinline__ int whole_rounds(int all) {
    const int left = all % kCUs;
    return left <= kRestMost ? all - left : all;
}

// LDS tiles: rows of 128 bytes in eight 16-byte chunks; chunk c of row r
// sits at slot c ^ (r & 7), so that the 16 lanes of a fragment that read one
// chunk of 16 rows touch every bank alike.
constexpr int BK = 128;

typedef __attribute__((address_space(3))) void *lds_ptr_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const void *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), 0, (int)bytes, 0x00020000);
}

// 16 bytes a lane from memory to LDS, lane l's at `to` + 16 l.  ONCE: read
// once, so that the caches need not keep it (non-temporal).
template <bool ONCE = false>
__device__ __forceinline__ void load16(__amdgpu_buffer_rsrc_t r, char *to, uint32_t voff, int soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)to, 16, voff, soff, 0, ONCE ? 2 : 0);
}

// 4 bytes a lane from an address of its own, lane l's at `to` + l.
__device__ __forceinline__ void load4(const float *from, float *to) {
    __builtin_amdgcn_global_load_lds((__attribute__((address_space(1))) void *)const_cast<float *>(from), (lds_ptr_t)to,
                                     4, 0, 0);
}

template <int N>
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory"); }

// Waits until at most `n` (0 .. MOST) batches of L loads are on their way.
template <int L, int MOST>
__device__ __forceinline__ void wait_batches(int n) {
    if constexpr (MOST == 0) wait_loads<0>();
    else if (n >= MOST) wait_loads<L * MOST>();
    else wait_batches<L, MOST - 1>(n);
}

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;      // of one launch

inline int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

}  // namespace q4
