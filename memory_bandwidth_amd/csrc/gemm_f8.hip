// gemm_f8.hip -- products of e4m3 activations and weights with a scale for each
// block of 128, for gfx950 (see q4f8.h):
//
//     P[m, n] = sum_b sa[m, b] sw[n / 128, b] sum_{k in block b} a[m, k] w[n, k]
//
// plain, as a gated block of two matrices, and that block's backward pass.
//
// A block's sum is what a step of 128 bytes makes: one matrix instruction of
// 16 x 16 x 128 (or four of 16 x 16 x 32) from zero, then a fused multiply-add
// by the scales into the sums, 4 values a lane.  The weights are the first
// operand, so that a lane holds one row m, and one factor sa sw serves
// all its values of a step: a wavefront's columns lie in one block of 128.
//
// Two ways to multiply:
//   fp8   v_mfma_f32_16x16x128_f8f6f4.  It brings the products of eight
//         consecutive k to the exponent of the largest and drops what is below
//         2^-13 of that: 1.5 * 2^-16 of the result (normal codes; measured
//         against float64).  For outputs of 16 bits.  From registers, with the
//         multiply-adds, 3670 TFLOP/s (4420 without them).
//   f16   v_cvt_scalef32_pk_f16_fp8, which is exact, and
//         v_mfma_f32_16x16x32_f16, whose sums are within 2^-26 (same codes).
//         For float32 outputs.  1860 TFLOP/s, conversions and all: one takes eight
//         cycles of a SIMD, two values a lane, and each operand of 16 rows is
//         sixteen of them beside the four products of 16 cycles it enters.
#include "q4_common.h"
#include "q4f8.h"
#include "q4_tiles.h"

#include <algorithm>

namespace {

using namespace q4;

typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));

enum Mode { kPlain, kGated, kBackward };

struct Args {
    const uint8_t *a;
    const float *sa;
    int64_t sa_m, sa_k;
    int sa_shift;              // 0: a row of scales for each row, 7: for each block of 128
    const uint8_t *w[2];       // one matrix, or gate and up
    const float *sw[2];
    const float *bias;
    const void *dh;
    void *y;
    int dh_type, y_type, M, N, K;
    int tiles_m, tiles_n;      // kHalves, kQuarters: of the tiles that are divided
    Part part;
    int whole;                 // kWhole: tiles that are taken; else: tiles before those that are divided
    bool once;                 // the weights are read past the caches
    bool share;                // several row tiles read the same weights
};

// A lane's 32 bytes of a fragment (16 rows of 128): chunks lane / 16 and lane /
// 16 + 4 of row lane % 16.  Which k they are is the same for both operands.
struct Raw { i32x4_t lo, hi; };

template <bool F16> struct Operand;
template <> struct Operand<false> {
    i32x8_t v;
    __device__ __forceinline__ void set(const Raw &r) {
        v = i32x8_t{r.lo[0], r.lo[1], r.lo[2], r.lo[3], r.hi[0], r.hi[1], r.hi[2], r.hi[3]};
    }
};
template <> struct Operand<true> {
    f16x8_t v[4];
    __device__ __forceinline__ static f16x8_t wide(int a, int b) {
        const f16x2_t p = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, false);
        const f16x2_t q = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.f, true);
        const f16x2_t r = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, false);
        const f16x2_t s = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.f, true);
        return f16x8_t{p[0], p[1], q[0], q[1], r[0], r[1], s[0], s[1]};
    }
    __device__ __forceinline__ void set(const Raw &r) {
        v[0] = wide(r.lo[0], r.lo[1]);
        v[1] = wide(r.lo[2], r.lo[3]);
        v[2] = wide(r.hi[0], r.hi[1]);
        v[3] = wide(r.hi[2], r.hi[3]);
    }
};

// Sums of one block: 16 weight rows by 16 rows, from zero.
__device__ __forceinline__ f32x4_t block_sum(const Operand<false> &w, const Operand<false> &x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, f32x4_t{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4_t block_sum(const Operand<true> &w, const Operand<true> &x) {
    f32x4_t t = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) t = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[q], x.v[q], t, 0, 0, 0);
    return t;
}

// Adds a block's sums times their scales.
__device__ __forceinline__ void add_scaled(f32x4_t &acc, const f32x4_t &t, float s) {
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(t[r], s, acc[r]);
}

// A scale that all lanes read alike, through the scalar cache.  A vector load
// would wait behind the ring's.
typedef const float __attribute__((address_space(4))) uniform_float;
__device__ __forceinline__ float uniform_load(const float *p) {
    return *reinterpret_cast<uniform_float *>(reinterpret_cast<uintptr_t>(p));
}

// A run of C columns from n on of a row of dh as it lies there, zero past N: a
// word a value (WIDE) or two values of 16 bits.
template <int C, bool WIDE>
__device__ __forceinline__ void load_run(const void *base, size_t at, int n, int N, uint32_t (&raw)[WIDE ? C : C / 2]) {
    const bool whole = n + C <= N;
    if constexpr (WIDE) {
        const uint32_t *p = static_cast<const uint32_t *>(base) + at;
        if (whole) {
#pragma unroll
            for (int c = 0; c < C; c += 4) {
                const u32x4_t r = *reinterpret_cast<const u32x4_at4_t *>(p + c);
                raw[c] = r[0], raw[c + 1] = r[1], raw[c + 2] = r[2], raw[c + 3] = r[3];
            }
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c) raw[c] = n + c < N ? p[c] : 0u;
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + at;
        if (whole) {
#pragma unroll
            for (int c = 0; c < C / 2; c += 2) {
                const u32x2_t r = *reinterpret_cast<const u32x2_at2_t *>(p + 2 * c);
                raw[c] = r[0], raw[c + 1] = r[1];
            }
        } else {
#pragma unroll
            for (int c = 0; c < C / 2; ++c)
                raw[c] = (n + 2 * c < N ? (uint32_t)p[2 * c] : 0u) |
                         (n + 2 * c + 1 < N ? (uint32_t)p[2 * c + 1] << 16 : 0u);
        }
    }
}
template <bool WIDE>
__device__ __forceinline__ float value_of(const uint32_t *raw, int type, int c) {
    if constexpr (WIDE) {
        const uint32_t b = raw[c];
        return __builtin_bit_cast(float, b);
    } else {
        const uint32_t h = raw[c / 2] >> (16 * (c & 1)) & 0xFFFFu;
        return type == I8_F16 ? (float)__builtin_bit_cast(_Float16, (uint16_t)h) : __builtin_bit_cast(float, h << 16);
    }
}

// The gradients of h = silu(g) u for g and u, with s = 1 / (1 + e^-g):
//     dg = dh u s (1 + g (1 - s)),   du = dh g s
// From e = e^-|g|, which never overflows: of s and 1 - s one is 1 / (1 + e) and
// the other e / (1 + e).  Below kFar, where e is no normal number, s = e^g to the
// last bit, taken in two halves around the other factors as far_silu does.
__device__ __forceinline__ void gated_gradient(float dh, float g, float u, float &dg, float &du) {
    const float e = __expf(-__builtin_fabsf(g)), big = __builtin_amdgcn_rcpf(1.f + e), small = e * big;
    const float s = g < 0.f ? small : big, r = g < 0.f ? big : small;
    dg = dh * (u * (s * __builtin_fmaf(g, r, 1.f)));
    du = dh * (g * s);
}
__device__ __forceinline__ void far_gated_gradient(float dh, float g, float u, float &dg, float &du) {
    const float half = __builtin_amdgcn_exp2f(0.72134752044f * g);
    dg = (1.f + g) * half * u * (half * dh);
    du = g * half * (half * dh);
}

// Writes a wavefront's sums.  acc[i][..]: rows row0 + 16 i + lane % 16 of the
// tile; over its fragments a lane holds the C columns from n on (of two
// matrices, C of gate in the first half of the fragments, C of up in the second).
template <int FM, int C, Mode MODE>
__device__ __forceinline__ void finish(const Args &p, const f32x4_t (&acc)[FM][MODE == kPlain ? C / 4 : C / 2], int m0,
                                       int rows, const float *bias, int row0, int n, int lane) {
    constexpr int UP = C / 4;                            // fragments of gate
    float add[C];
    if constexpr (MODE == kPlain) {
#pragma unroll
        for (int c = 0; c < C; ++c) add[c] = bias ? bias[c] : 0.f;
    }
    if (n >= p.N) return;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = row0 + i * 16 + (lane & 15);
        if (r >= rows) continue;
        const size_t at = (size_t)(m0 + r) * p.N + n;
        float v[C];
        if constexpr (MODE == kPlain) {
#pragma unroll
            for (int c = 0; c < C; ++c) v[c] = acc[i][c >> 2][c & 3] + add[c];
        } else {
            float least = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                v[c] = silu(acc[i][c >> 2][c & 3]) * acc[i][UP + (c >> 2)][c & 3];
                least = __builtin_fminf(least, acc[i][c >> 2][c & 3]);
            }
            if (__builtin_expect(least < kFar, 0)) {             // rare, and then of no account
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float g = acc[i][c >> 2][c & 3];
                    if (g < kFar) v[c] = far_silu(g, acc[i][UP + (c >> 2)][c & 3]);
                }
            }
        }
        store_run<C>(p.y, p.y_type, at, n, p.N, v);
    }
}

// The same for the backward pass.  All rows of dh are on their way before the
// first is used.
template <int FM, int C, bool WIDE>
__device__ __forceinline__ void finish_backward(const Args &p, const f32x4_t (&acc)[FM][C / 2], int m0, int rows,
                                                int row0, int n, int lane) {
    constexpr int UP = C / 4;
    if (n >= p.N) return;
    uint32_t raw[FM][WIDE ? C : C / 2];
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = min(row0 + i * 16 + (lane & 15), rows - 1);
        load_run<C, WIDE>(p.dh, (size_t)(m0 + r) * p.N + n, n, p.N, raw[i]);
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = row0 + i * 16 + (lane & 15);
        if (r >= rows) continue;
        float dg[C], du[C], least = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const float dh = value_of<WIDE>(raw[i], p.dh_type, c), g = acc[i][c >> 2][c & 3];
            gated_gradient(dh, g, acc[i][UP + (c >> 2)][c & 3], dg[c], du[c]);
            least = __builtin_fminf(least, g);
        }
        if (__builtin_expect(least < kFar, 0)) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float dh = value_of<WIDE>(raw[i], p.dh_type, c), g = acc[i][c >> 2][c & 3];
                if (g < kFar) far_gated_gradient(dh, g, acc[i][UP + (c >> 2)][c & 3], dg[c], du[c]);
            }
        }
        const size_t at = (size_t)(m0 + r) * 2 * p.N + n;
        store_run<C>(p.y, p.y_type, at, n, p.N, dg);
        store_run<C>(p.y, p.y_type, at + p.N, n, p.N, du);
    }
}

template <int FM, int C, Mode MODE>
__device__ __forceinline__ void write_out(const Args &p, const f32x4_t (&acc)[FM][MODE == kPlain ? C / 4 : C / 2],
                                          int m0, int rows, const float *bias, int row0, int n, int lane) {
    if constexpr (MODE != kBackward) finish<FM, C, MODE>(p, acc, m0, rows, bias, row0, n, lane);
    else if (p.dh_type == I8_F32) finish_backward<FM, C, true>(p, acc, m0, rows, row0, n, lane);
    else finish_backward<FM, C, false>(p, acc, m0, rows, row0, n, lane);
}

// Loads of the scales of 64 rows for a block: from row `row` on of the tile at
// m0, at `voff` = scale_offset, to LDS.
__device__ __forceinline__ uint32_t scale_offset(const Args &p, int m0, int row) {
    return (uint32_t)(((m0 + row) >> p.sa_shift) - (m0 >> p.sa_shift)) * (uint32_t)p.sa_m * 4u;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rsrc(const Args &p, int m0, int rows, int kb) {
    return rsrc_of(p.sa + (int64_t)(m0 >> p.sa_shift) * p.sa_m + kb * p.sa_k, scale_offset(p, m0, rows - 1) + 4u);
}
__device__ __forceinline__ void load_scale(__amdgpu_buffer_rsrc_t r, char *to, uint32_t voff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)to, 4, voff, 0, 0, 0);
}

// ---------------------------------------------------------------- tiles
//
// A tile of BM rows and BW weight rows (of two matrices: BW / 2 of each) by WM x
// WN wavefronts, or by G groups of as many that share out K: group g takes
// every G-th block of 128, and the groups' sums meet in LDS at the end.  Steps
// of G blocks pass through a ring of D stages in LDS, loaded straight from
// memory (buffer loads to LDS, 1 KiB an instruction: eight rows of 128 bytes,
// the lanes' chunk order making the swizzle), with the rows' scales behind
// them.
//
// Of a wavefront's two sets of fragments the smaller one is held for the
// step, and the larger one streams past it:
//
//     fragments 0 .. S - T - 1:  its products with all held ones, behind them
//                  reads of fragments to come
//     barrier:     step t + 1 has come to LDS and this step's reads are done;
//                  step t + D is loaded over step t
//     the last T:  for each held fragment its products with them, then the
//                  read of the next step's
//
// so there is one barrier a step, with products on either side of it.  The
// last D steps of a tile load the first D of the workgroup's next tile (one
// gridDim.x further), which arrive while this one is stored.  A last step
// that K does not fill is taken as the last 128 bytes of the rows, with the
// activations already used set to zero; every address stays inside the rows.
// Rows past the tile's end repeat its last row, and their results are not stored.
//
// Scales: wavefront v < BM / 64 brings those of 64 rows, the next one (two, with
// two matrices) those of the columns, a lane 16 of them.  They pass through LDS
// as well: read through the scalar cache they would make every wait for an LDS
// read a wait for all.

// Orders what stands between two scheduling barriers: behind each of the
// products an LDS read and five vector instructions.
template <int PRODUCTS>
__device__ __forceinline__ void spread() {
    if constexpr (PRODUCTS > 0) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
        spread<PRODUCTS - 1>();
    }
}

template <int BM, int BW, bool TWO>
constexpr int slice_bytes() { return (BM + BW) * BK + BM * 4 + (TWO ? 512 : 256); }

template <int BM, int BW, int WM, int WN, int G, int D, Mode MODE, bool F16>
__global__ __launch_bounds__(WM * WN * G * 64, 2) void gemm_f8_block(Args p) {
    constexpr bool TWO = MODE != kPlain;
    constexpr int FM = BM / WM / 16, FW = BW / WN / 16, BN = TWO ? BW / 2 : BW, MATS = TWO ? 2 : 1;
    constexpr int W = WM * WN;                                           // wavefronts of a group
    constexpr int LX = BM / 8 / W, LW = BW / 8 / W, LOADS = LX + LW + 1; // load instructions of one of them and step
    constexpr int SLICE = slice_bytes<BM, BW, TWO>(), STAGE = G * SLICE;
    constexpr bool SX = FM >= FW;                                        // the rows' fragments stream
    constexpr int S = SX ? FM : FW, H = SX ? FW : FM;
    // Of the stream: the last ones, and places.  Three at the end against one, 4 x 4
    // fragments of one matrix: 72 against 78 us (4096 x 4096 x 4096, 128 x 256), 74
    // against 79 (128 x 128, four wavefronts); of two matrices 104 against 100
    // (600 x 14336 x 4096, 128 x 128).  Eight by four: 420 against 443.
    constexpr int T = S == 8 || (H == 4 && !TWO) ? 3 : 1, R = T + 1;
    static_assert(S % R == 0, "the next step's first fragment takes a place that is free");
    static_assert(S >= 2 && BM % 64 == 0 && BM / 64 + MATS <= W, "one instruction a wavefront brings all scales");
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, all_waves = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = all_waves % W, group = all_waves / W;
    const int wm = wave / WN, wn = wave % WN;
    const int KB = (p.K + BK - 1) / BK, steps = (KB + G - 1) / G;
    const int tiles = p.part == kWhole ? p.whole : p.tiles_m * p.tiles_n;
    struct Place { int m0, rows, n0; };
    auto place = [&](int id, Place &at) {
        const int b = p.part >= kHalves ? p.whole + (id >> (p.part - kHalves + 1)) : id;
        int tm, tn;
        if (b >= tiles || !tile_of(b, p.tiles_m, p.tiles_n, tm, tn)) return false;
        const int bm = p.part >= kHalves ? 2 * BM : BM;
        at.m0 = tm * bm;
        at.n0 = tn * BN;
        if (p.part >= kHalves) {
            at.m0 += (id & 1) * BM;
            if (p.part == kQuarters) at.n0 = (2 * tn + (id >> 1 & 1)) * BN;
        }
        at.rows = min(BM, p.M - at.m0);
        return at.rows > 0 && at.n0 < p.N;
    };
    int id = blockIdx.x;
    Place cur;
    if (!place(id, cur)) return;

    // In the largest tiles, what a tile's start and end compute from the lane is
    // computed anew each time: kept, it takes registers that the fragments need.
    auto lane_anew = [&]() {
        int l = tid & 63;
        if constexpr (FM * FW >= 32) asm volatile("" : "+v"(l));
        return l;
    };

    // Loads: this wavefront brings 1 / W of the rows of a and of w, and 64 rows' scales.
    // Of two matrices, its weight rows are all gate or all up.
    const uint8_t *w_matrix = TWO && wave * LW / 2 % FW >= FW / 2 ? p.w[1] : p.w[0];
    const uint8_t *a_base, *w_base;
    uint32_t a_bytes, w_bytes;
    uint32_t va[LX], vw[LW], vs;
    // This wavefront's scales: those of a matrix's columns, or of 64 rows.
    const int mat = wave - BM / 64;
    const bool of_columns = mat >= 0 && mat < MATS;
    const int scales_at = (BM + BW) * BK + (of_columns ? BM * 4 + mat * 256 : wave * 64 % BM * 4);
    const int64_t scale_step = of_columns ? 1 : p.sa_k;
    const float *scale_base;
    auto aim = [&](const Place &at) {
        const int lane = lane_anew();
        const int rows = at.rows, cols = min(BN, p.N - at.n0), chunk = ((lane & 7) ^ (lane >> 3)) << 4;
        a_base = p.a + (size_t)at.m0 * p.K, a_bytes = (uint32_t)rows * p.K;
        w_base = w_matrix + (size_t)at.n0 * p.K, w_bytes = (uint32_t)cols * p.K;
        if (of_columns) {
            const int nb = at.n0 >> 7;
            scale_base = (mat == 0 ? p.sw[0] : p.sw[1]) + (size_t)nb * KB;
            vs = (uint32_t)((min(at.n0 + lane * 16, p.N - 1) >> 7) - nb) * (uint32_t)KB * 4u;
        } else {
            scale_base = p.sa + (int64_t)(at.m0 >> p.sa_shift) * p.sa_m;
            vs = scale_offset(p, at.m0, min(wave * 64 % BM + lane, rows - 1));
        }
#pragma unroll
        for (int i = 0; i < LX; ++i)
            va[i] = __umul24(min((wave * LX + i) * 8 + (lane >> 3), rows - 1), p.K) + chunk;
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            // Row r belongs to wavefront column c, its fragment j, row q of it.
            const int r = (wave * LW + i) * 8 + (lane >> 3), c = r / (16 * FW), j = r / 16 % FW, q = r & 15;
            const int n = TWO ? c * (8 * FW) + frag_row<FW / 2>(j % (FW / 2), q) : c * (16 * FW) + frag_row<FW>(j, q);
            vw[i] = __umul24(min(n, cols - 1), p.K) + chunk;
        }
    };
    // Load k of a step: `wanted` false makes it one past the end of an empty
    // array, which no memory is asked for, so that every step has as many.
    struct Source { __amdgpu_buffer_rsrc_t a, w, scale; char *to; int koff; };
    auto source = [&](int slot, int t, bool wanted) {
        const int kb = min(t * G + group, KB - 1);
        return Source{rsrc_of(a_base, wanted ? a_bytes : 0u), rsrc_of(w_base, wanted ? w_bytes : 0u),
                      rsrc_of(scale_base + kb * scale_step, wanted ? 0xFFFFFFFFu : 0u),
                      lds + slot * STAGE + group * SLICE,
                      min((t * G + group) * BK, p.K - BK)};
    };
    auto load = [&](const Source &from, int k) {
        char *at = from.to + (wave * (k < LX ? LX : LW) + (k < LX ? k : BM / 8 + k - LX)) * 1024;
        if (k < LX) load16(from.a, at, va[k < LX ? k : 0], from.koff);
        else if (k < LX + LW) load16(from.w, at, vw[k < LX + LW ? k - LX : 0], from.koff);
        else load_scale(from.scale, from.to + scales_at, vs);
    };

    // Fragment reads: lane l takes row l % 16, chunks l / 16 and l / 16 + 4
    // (which flips bit 6 of the swizzled address).
    const int fr = (lane & 15) * BK + (((lane >> 4) ^ (lane & 7)) << 4);
    const int xat = wm * (16 * FM) * BK, wat = (BM + wn * (16 * FW)) * BK;
    const int sat = (BM + BW) * BK + (wm * (16 * FM) + (lane & 15)) * 4;
    // Chunks of this group's last block that others have used; all eight: it has none.
    const int used = max(0, ((steps - 1) * G + group + 1) * 8 - (p.K >> 4));
    f32x4_t acc[FM][FW];
    Raw held[H], ring[R];
    float scale_x[SX ? R : H];                         // of the rows of ring[] or held[]
    auto read = [&](int at) {
        const char *from = lds + group * SLICE + at;
        Raw r;
        r.lo = *reinterpret_cast<const i32x4_t *>(from + fr);
        r.hi = *reinterpret_cast<const i32x4_t *>(from + (fr ^ 64));
        return r;
    };
    auto read_x = [&](int slot, int i, Raw &r, float &s) {
        r = read(slot * STAGE + xat + i * 16 * BK);
        s = *reinterpret_cast<const float *>(lds + group * SLICE + slot * STAGE + sat + i * 64);
    };
    auto read_stream = [&](int slot, int q) {
        if constexpr (SX) read_x(slot, q, ring[q % R], scale_x[q % R]);
        else ring[q % R] = read(slot * STAGE + wat + q * 16 * BK);
    };
    auto read_held = [&](int slot, int h) {
        if constexpr (SX) held[h] = read(slot * STAGE + wat + h * 16 * BK);
        else read_x(slot, h, held[h], scale_x[h]);
    };
    // The last step's activations that other steps have used are cleared by the
    // wavefront that has loaded them, once they have come.
    auto clear_used = [&](int slot) {
        const int lane = lane_anew();
        char *to = lds + slot * STAGE + group * SLICE;
        if (((lane & 7) ^ (lane >> 3)) < used) {
#pragma unroll
            for (int i = 0; i < LX; ++i)
                *reinterpret_cast<i32x4_t *>(to + (wave * LX + i) * 1024 + lane * 16) = i32x4_t{0, 0, 0, 0};
        }
        // A block that the group has not: no scale of it may be infinite either.
        if (used >= 8) *reinterpret_cast<float *>(to + scales_at + lane * 4) = 0.f;
    };
    auto barrier = [&]() {       // and this wavefront's LDS reads are done
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // The weights' scales of a step, for this wavefront's columns.
    float sw[MATS];
    const int swat = (BM + BW) * BK + BM * 4 + wn * (TWO ? FW / 2 : FW) * 4;
    auto read_sw = [&](int slot) {
#pragma unroll
        for (int s = 0; s < MATS; ++s)
            sw[s] = *reinterpret_cast<const float *>(lds + slot * STAGE + group * SLICE + swat + s * 256);
    };
    // The bias of a tile's columns goes behind the ring, 64 of them a wavefront:
    // fetched at the end, it would cost a trip to memory there.
    float *biases = reinterpret_cast<float *>(lds + D * STAGE);
    auto load_bias = [&](const Place &at, float *to) {
        if (TWO || !p.bias) return;
        const int q = all_waves * 64, col = at.n0 + q + lane_anew();
        if (q < BN) load4(p.bias + min(col, p.N - 1), to + q);
    };
    auto after = [](int slot) { return slot + 1 == D ? 0 : slot + 1; };

    // One step: its products, and the first reads of the next (past a tile's last
    // step they are not used).  The products of the last T fragments of the stream
    // come by held fragment, so that each of those is read anew behind T of
    // them: all at once, behind the last, would have the matrix cores wait for
    // LDS.  A sum is added two products late, so that it has left the matrix cores
    // by then; a step's last two behind the next one's first.
    constexpr int ALL = S * H, MAIN = (S - T) * H;
    static_assert(ALL % 4 == 0 && H >= 2, "places of sums repeat with the steps");
    f32x4_t sum[4];
    float factor[4];
    auto q_of = [](int n) { return n < MAIN ? n / H : S - T + (n - MAIN) % T; };
    auto h_of = [](int n) { return n < MAIN ? n % H : (n - MAIN) / T; };
    auto add = [&](int n) {                            // sum n of a step; -2, -1: of the one before
        if (n < 0) n += ALL;
        add_scaled(acc[SX ? q_of(n) : h_of(n)][SX ? h_of(n) : q_of(n)], sum[n % 4], factor[n % 4]);
    };
    auto step = [&](int t, int slot, const Source &from) {
        const int next = after(slot);
        Operand<F16> kept[H], passing[T];
        float by[SX ? T : H][MATS];                    // scales of the rows in hand, times those of the columns
        auto scale = [&](int at, float x) {
#pragma unroll
            for (int s = 0; s < MATS; ++s) by[at][s] = x * sw[s];
        };
#pragma unroll
        for (int h = 0; h < H; ++h) {
            kept[h].set(held[h]);
            if constexpr (!SX) scale(h, scale_x[h]);
        }
        auto product = [&](int n, const Operand<F16> &x, int at) {
            const int q = q_of(n), h = h_of(n), j = SX ? h : q;
            sum[n % 4] = SX ? block_sum(kept[h], x) : block_sum(x, kept[h]);
            factor[n % 4] = by[SX ? at : h][TWO && j >= FW / 2 ? 1 : 0];
            add(n - 2);
        };
        // Reads of the stream's fragments run up to R - 1 ahead.
        constexpr int EACH = T == 1 ? H : S - T > 1 ? H / 2 : 1;
        static_assert(S - T > 1 || T <= H, "all are read");
        int ahead = 1;
#pragma unroll
        for (int q = 0; q < S - T; ++q) {
            passing[0].set(ring[q % R]);
            if constexpr (SX) scale(0, scale_x[q % R]);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                product(q * H + h, passing[0], 0);
                if (h % EACH == 0 && ahead < min(q + R, S)) read_stream(slot, ahead++);
            }
            if constexpr (!F16) spread<H>();
            __builtin_amdgcn_sched_barrier(0);
        }
        // Additions stay on this side of the branches: moved behind them, all
        // their sums would have to be kept.
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FW; ++j) asm volatile("" : "+v"(acc[i][j]));
        wait_loads<(D - 2) * LOADS>();
        if (t + 2 == steps && used) clear_used(next);
        barrier();
#pragma unroll
        for (int q = S - T; q < S; ++q) {
            passing[q - S + T].set(ring[q % R]);
            if constexpr (SX) scale(q - S + T, scale_x[q % R]);
        }
        read_stream(next, 0);
        if constexpr (!F16) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int h = 0; h < H; ++h) {
#pragma unroll
            for (int q = 0; q < T; ++q) {
                const int n = h * T + q;
                product(MAIN + n, passing[q], q);
                // The step's loads, spread over these products: a wavefront that
                // issues many in a row waits for the memory path to take them.
#pragma unroll
                for (int k = n * LOADS / (H * T); k < (n + 1) * LOADS / (H * T); ++k) load(from, k);
                if constexpr (!F16) __builtin_amdgcn_sched_barrier(0);
            }
            read_held(next, h);
            if (h == H - 1) read_sw(next);
            if constexpr (!F16) __builtin_amdgcn_sched_barrier(0);
        }
    };

    aim(cur);
    int side = 0;                // of the two places for the bias
    load_bias(cur, biases);
#pragma unroll
    for (int d = 0; d < D; ++d) {
        const Source from = source(d, d, d < steps);
#pragma unroll
        for (int k = 0; k < LOADS; ++k) load(from, k);
    }
    wait_loads<(D - 1) * LOADS>();
    if (steps == 1 && used) clear_used(0);
    barrier();
    for (int slot = 0;;) {
        read_stream(slot, 0);
#pragma unroll
        for (int h = 0; h < H; ++h) read_held(slot, h);
        read_sw(slot);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FW; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
        sum[2] = sum[3] = f32x4_t{0, 0, 0, 0};
        factor[2] = factor[3] = 0.f;
        // The last D steps load the next tile's first.
        Place nxt = cur;
        bool more = steps > D;
        for (int t = 0, end = more ? steps - D : 0;;) {
            for (; t < end; ++t) {
                step(t, slot, source(slot, t + D < steps ? t + D : t + D - steps, more));
                slot = after(slot);
            }
            if (end == steps) break;
            end = steps;
            more = G == 1 && steps >= D && place(id + (int)gridDim.x, nxt);
            if (more) {
                aim(nxt);
                // The place is that of the tile before this one: a barrier since then says that
                // every wavefront has read it.  With D steps there has been none.  (Fetched
                // behind the next step's barrier instead, it has the largest tiles spill;
                // bf16 8192 x 4096 x 256 takes 25.2 us so, 26.0 without a bias.)
                if (!TWO && p.bias && steps == D) barrier();
                load_bias(nxt, biases + (side ^ 1) * BN);
            }
        }
        add(-2);
        add(-1);
        constexpr int C = TWO ? 2 * FW : 4 * FW;      // consecutive columns of a lane
        const int lane = lane_anew();
        const int col = wn * (4 * C) + (lane >> 4) * C;
        const float *bias = !TWO && p.bias ? biases + side * BN + col : nullptr;
        if constexpr (G == 1) {
            write_out<FM, C, MODE>(p, acc, cur.m0, cur.rows, bias, wm * (16 * FM), cur.n0 + col, lane);
        } else {
            // The groups' sums meet in the ring's place, and group g finishes
            // rows g, g + G, .. of the fragments.
            static_assert(G * W * FM * FW * 1024 <= D * STAGE, "the sums fit the ring");
            wait_loads<0>();
            __syncthreads();
            f32x4_t *part = reinterpret_cast<f32x4_t *>(lds) + wave * (FM * FW * 64) + lane;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FW; ++j) part[(group * W * FM * FW + i * FW + j) * 64] = acc[i][j];
            __syncthreads();
            for (int i = group; i < FM; i += G) {
                f32x4_t sum[1][FW] = {};
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int j = 0; j < FW; ++j) sum[0][j] += part[(g * W * FM * FW + i * FW + j) * 64];
                write_out<1, C, MODE>(p, sum, cur.m0, cur.rows, bias, wm * (16 * FM) + i * 16, cur.n0 + col, lane);
            }
            return;
        }
        if (!more) return wait_loads<0>();     // LDS is theirs until they have ended
        id += gridDim.x;
        cur = nxt;
        side ^= 1;
    }
}

// ---------------------------------------------------------------- few rows
//
// Tiles of 8 NX rows: what counts is the bytes in flight, and that every CU
// has its share of them.  A wavefront takes FN strips of 16 weight rows (of
// each matrix) and every KS-th block of 128; KS wavefronts of a workgroup
// meet in LDS at the end.  Its blocks pass through a ring of D slots of its own
// in LDS, loaded straight from memory eight rows of 128 bytes an instruction,
// the rows' scales behind them, the next block issued as soon as a slot has
// been read: no barrier, and D - 1 blocks in flight while one is multiplied.
// Blocks past K repeat the row's last 16 bytes against activations of zero.
//
// Up to eight rows take as many slots as fit, up to four: 1 x 28672 x 8192 in 41.3 us
// (44.7 with two), 4 x 14336 x 4096 gated to bf16 21.4 (22.6), to float32 22.2 (23.1).
// With more rows the operands come from the L2, and workgroups side by side on a CU
// count for more, whatever the tile: 333 x 896 x 4864 in 32 x 16 10.7 with two, 17.3
// with four; to float32 in 8 x 16 329 x 933 x 288 gated 5.5 and 9.2, 200 x 333 x 2064
// 5.3 and 7.1, and 12 x 4864 x 896 3.9 both.
constexpr int few_slot(int FM, int FW) { return (2 * FW + 2 * FM) * 1024 + 256; }  // whole fragments, and the scales
constexpr int few_most(int W, int FW) { return std::min(4, 160 * 1024 / (W * few_slot(1, FW))); }

template <int NX, int FN, Mode MODE, bool F16, int W, int D>
__global__ __launch_bounds__(W * 64) void gemm_f8_few(Args p, int ks_log2) {
    constexpr int FM = (NX + 1) / 2, BM = 8 * NX, MATS = MODE == kPlain ? 1 : 2, FW = FN * MATS;
    constexpr int LOADS = 2 * FW + NX + 1;                              // load instructions of a block
    constexpr int SLOT = few_slot(FM, FW);                              // the last fragment may be half loaded
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KS = 1 << ks_log2, ks = wave & (KS - 1);
    // Row tiles that read the same weights lie side by side on one XCD, so that
    // its L2 brings them once; others take the XCDs in turn.
    int tm = (int)blockIdx.x / p.tiles_n, tn = (int)blockIdx.x - tm * p.tiles_n;
    if (p.share) {
        const int id = eighth_of(blockIdx.x, p.tiles_m * p.tiles_n);
        if (id < 0) return;
        tn = id / p.tiles_m;
        tm = id - tn * p.tiles_m;
    }
    const int m0 = tm * BM, rows = min(BM, p.M - m0);
    const int n0 = (tn * (W >> ks_log2) + (wave >> ks_log2)) * (16 * FN);
    const int kc = p.K >> 4, KB = (kc + 7) >> 3;
    const int g = lane >> 4, r = lane & 15;
    f32x4_t acc[FM][FW] = {};
    // The bias of the lane's columns, fetched before the ring's loads: at the end
    // it would cost a trip to memory.
    constexpr int C = 4 * FN;
    const int n = n0 + g * C;
    float bias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) bias[c] = MODE == kPlain && p.bias ? p.bias[min(n + c, p.N - 1)] : 0.f;

    if (n0 < p.N) {
        char *ring = lds + wave * (D * SLOT);
        const int cols = min(16 * FN, p.N - n0);
        const __amdgpu_buffer_rsrc_t rx = rsrc_of(p.a + (size_t)m0 * p.K, (uint32_t)rows * p.K);
        __amdgpu_buffer_rsrc_t rw[MATS];
        const float *swp[MATS];
#pragma unroll
        for (int s = 0; s < MATS; ++s) {
            rw[s] = rsrc_of(p.w[s] + (size_t)n0 * p.K, (uint32_t)cols * p.K);
            swp[s] = p.sw[s] + (size_t)(n0 >> 7) * KB;
        }
        uint32_t vx[NX], vw[2 * FN];
#pragma unroll
        for (int i = 0; i < NX; ++i) vx[i] = (uint32_t)min(i * 8 + (lane >> 3), rows - 1) * p.K;
#pragma unroll
        for (int i = 0; i < 2 * FN; ++i) {
            const int q = (i & 1) * 8 + (lane >> 3);               // row of fragment i / 2
            vw[i] = (uint32_t)min(frag_row<FN>(i >> 1, q), cols - 1) * p.K;
        }
        const uint32_t vs = scale_offset(p, m0, min(lane, rows - 1));
        const int chunk = (lane & 7) ^ (lane >> 3);
        auto load = [&](int slot, int u) {
            char *at = ring + slot * SLOT;
            const uint32_t k = (uint32_t)min(u * 8 + chunk, kc - 1) << 4;
#pragma unroll
            for (int s = 0; s < MATS; ++s)
#pragma unroll
                for (int i = 0; i < 2 * FN; ++i) {
                    char *to = at + (s * 2 * FN + i) * 1024;
                    if (p.once) load16<true>(rw[s], to, vw[i] + k, 0);
                    else load16(rw[s], to, vw[i] + k, 0);
                }
#pragma unroll
            for (int i = 0; i < NX; ++i)
                load16(rx, at + (2 * FW + i) * 1024, vx[i] + k, 0);
            load_scale(scale_rsrc(p, m0, BM, u), at + SLOT - 256, vs);
        };
        const int fr = r * BK + ((g ^ (r & 7)) << 4);
        auto products = [&](int slot, int u, const float (&sw)[MATS]) {
            const char *at = ring + slot * SLOT;
            auto read = [&](int f) {
                Raw v;
                v.lo = *reinterpret_cast<const i32x4_t *>(at + f * 2048 + fr);
                v.hi = *reinterpret_cast<const i32x4_t *>(at + f * 2048 + (fr ^ 64));
                return v;
            };
            Operand<F16> w[FW];
#pragma unroll
            for (int j = 0; j < FW; ++j) w[j].set(read(j));
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                Raw v = read(FW + i);
                const float s = *reinterpret_cast<const float *>(at + SLOT - 256 + (i * 16 + r) * 4);
                if (u * 8 + 8 > kc) {
                    if (u * 8 + g >= kc) v.lo = i32x4_t{0, 0, 0, 0};
                    if (u * 8 + 4 + g >= kc) v.hi = i32x4_t{0, 0, 0, 0};
                }
                Operand<F16> x;
                x.set(v);
#pragma unroll
                for (int j = 0; j < FW; ++j) add_scaled(acc[i][j], block_sum(w[j], x), s * sw[j / FN]);
            }
        };
        int left = (KB - ks + KS - 1) >> ks_log2, u = ks, slot = 0;      // this wavefront's blocks
        float sw[MATS], sw_next[MATS];
        auto load_sw = [&](float (&to)[MATS], int u) {
#pragma unroll
            for (int s = 0; s < MATS; ++s) to[s] = uniform_load(swp[s] + min(u, KB - 1));
        };
        load_sw(sw, u);
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < left) load(d, ks + d * KS);
        for (; left > 0; --left, u += KS) {
            load_sw(sw_next, u + KS);
            wait_batches<LOADS, D - 1>(min(left, D) - 1);
            products(slot, u, sw);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the slot has been read
            if (left > D) load(slot, u + D * KS);
            if (++slot == D) slot = 0;
#pragma unroll
            for (int s = 0; s < MATS; ++s) sw[s] = sw_next[s];
        }
    }
    if (KS > 1) {
        // Every wavefront has read its ring: the partial sums take its place.
        __syncthreads();
        f32x4_t *part = reinterpret_cast<f32x4_t *>(lds) + lane;
        if (ks > 0) {
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FW; ++j) part[(wave * FM * FW + i * FW + j) * 64] = acc[i][j];
        }
        __syncthreads();
        if (ks > 0) return;
        for (int k = 1; k < KS; ++k)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FW; ++j) acc[i][j] += part[((wave + k) * FM * FW + i * FW + j) * 64];
    }
    write_out<FM, C, MODE>(p, acc, m0, rows, bias, 0, n, lane);
}

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxK = 131056;

bool elem_aligned(const void *y, int type) { return q4::aligned(y, type == I8_F32 ? 4 : 2); }

// Where a call's launches go: to the stream, or into a report of their plan,
// with the first one's tile and all workgroups.
struct Report { int rows, cols; int64_t grid; int block; };
struct Target { hipStream_t stream; Report *report; };

int planned(const Target &to, int rows, int cols, int64_t grid, int block) {
    Report &r = *to.report;
    if (!r.grid) r = {rows, cols, 0, block};
    r.grid += grid;
    return Q4_OK;
}

// Wavefronts on one strip's K (log2) and in a workgroup of a few-rows kernel
// of bm rows: as many share K as it takes for 1536 wavefronts, 6 for each CU,
// while each has a block.  16 x 4096 x 14336 takes 13.9 us so and 21.3 with 1024,
// 32 x 14336 x 4096 15.5 and, with 2048, 18.7.  Workgroups of four wavefronts
// rather than eight where those would leave CUs idle or fill them unevenly:
// 1 x 896 x 896 2.57 against 2.82 us, 8 x 28672 x 8192 45.5 against 47.1.
struct Split { int64_t tiles, strips; int log2, waves; };
Split split_of(const Args &p, int bm, int cols, int most) {
    Split s = {tiles_of(p.M, bm), tiles_of(p.N, cols), 0, most};
    const int64_t units = tiles_of(p.K, BK);
    while ((2 << s.log2) <= most && (units >> s.log2) > 1 && (s.tiles * s.strips) << s.log2 < 1536) ++s.log2;
    const int64_t eights = most == 8 ? s.tiles * tiles_of(s.strips, 8 >> s.log2) : 0;
    if (s.log2 < 3 && (eights < kCUs / 2 || eights > kCUs)) s.waves = 4;
    return s;
}

template <int NX, int FN, Mode MODE, bool F16, int W, int D>
int launch_few(Args p, const Split &s, const Target &to) {
    constexpr int FM = (NX + 1) / 2, FW = MODE == kPlain ? FN : 2 * FN;
    constexpr int kLds = W * D * few_slot(FM, FW);
    static_assert(kLds <= 160 * 1024 && D >= 2, "the rings fit, with a block on its way");
    // 128 x 8192 x 8192, tiles of 64 x 32: 32.6 us with, 36.9 without.
    p.share = s.tiles > 1;
    // Weights that one row tile reads pass the caches by: the next layers'
    // would put them out.  With 20 sets of operands in turn a row of 14336 x
    // 4096 takes 12.1 us so and 13.7 through the caches, 4096 x 4096 5.7 and 6.4; with
    // three sets, which the last cache holds, 11.2 and 10.5, 4.8 and 5.3.  Rows that
    // begin within a line share it with the one before, which a cache has to
    // keep: 14336 x 4112 takes 15.0 and 14.4.
    p.once = p.K % 64 == 0 && !p.share;
    p.tiles_m = (int)s.tiles;
    p.tiles_n = (int)tiles_of(s.strips, W >> s.log2);
    const int64_t grid = s.tiles * p.tiles_n;
    if (grid * (W * 64) > kMaxThreads) return Q4_EINVAL;
    if (to.report) return planned(to, 8 * NX, (W >> s.log2) * 16 * FN, grid, W * 64);
    gemm_f8_few<NX, FN, MODE, F16, W, D><<<(unsigned)grid, W * 64, kLds, to.stream>>>(p, s.log2);
    return q4::launch_status();
}

template <int NX, int FN, Mode MODE, bool F16, int W>
int launch_few(const Args &p, const Split &s, const Target &to) {
    if constexpr (NX == 1)
        if (s.tiles == 1)
            return launch_few<NX, FN, MODE, F16, W, few_most(W, MODE == kPlain ? FN : 2 * FN)>(p, s, to);
    return launch_few<NX, FN, MODE, F16, W, 2>(p, s, to);
}

template <int NX, int FN, Mode MODE, bool F16, int MOST = 8>
int launch_few(const Args &p, const Target &to) {
    const Split s = split_of(p, 8 * NX, 16 * FN, MOST);
    if constexpr (MOST == 8)
        if (s.waves == 8) return launch_few<NX, FN, MODE, F16, 8>(p, s, to);
    return launch_few<NX, FN, MODE, F16, 4>(p, s, to);
}

template <int BM, int BW, int WM, int WN, int G, int D, Mode MODE, bool F16>
int launch_block(Args p, const Target &to) {
    constexpr int kBN = MODE == kPlain ? BW : BW / 2;
    constexpr int kLds = D * G * slice_bytes<BM, BW, MODE != kPlain>() + 2 * kBN * 4;
    constexpr int kThreads = WM * WN * G * 64;
    static_assert(kLds <= 160 * 1024, "the ring fits");
    p.tiles_m = (int)tiles_of(p.M, (p.part >= kHalves ? 2 : 1) * BM);
    p.tiles_n = (int)tiles_of(p.N, (p.part == kQuarters ? 2 : 1) * kBN);
    int64_t grid = (int64_t)p.tiles_m * p.tiles_n;
    if (grid > 1 << 30) return Q4_EINVAL;
    if (p.part == kWhole) grid = p.whole;
    if (p.part >= kHalves) grid = (grid - p.whole) << (p.part - kHalves + 1);
    // Workgroups that stay and go through the tiles, each loading its next one
    // while it finishes the last: 8192 x 14336 x 4096 in 256 x 256 takes 422 us so
    // and 431 with a workgroup a tile, 4096 x 8192 x 512 gated 51.8 and 56.7.
    const int64_t steps = tiles_of(p.K, BK);
    if (G == 1 && p.part < kHalves && steps >= D)
        grid = std::min<int64_t>(grid, kCUs * (160 * 1024 / kLds));
    else if (grid * kThreads > kMaxThreads) return Q4_EINVAL;
    if (to.report) return planned(to, BM, kBN, grid, kThreads);
    gemm_f8_block<BM, BW, WM, WN, G, D, MODE, F16><<<(unsigned)grid, kThreads, kLds, to.stream>>>(p);
    return q4::launch_status();
}

enum Kernel { kFew8, kFew16, kFew32, kFew32x32, kFew64, kTile64, kTile128, kTileWide, kTile256, kTileDeep, kKernels };

// Estimates that order the kernels by their times, in us.  Tiles: for one, and for
// a step of it (`many`: where a CU has several, each of them); tiles that have a CU
// to themselves come in whole rounds.  Few rows: the start, a block of a wavefront
// alone and for each of the CU's (of two matrices), the blocks that the ring's first
// wait stands for; and, as the weights are read past the L2 again for every row
// tile, a MB of them, what each more row tile adds of that, and what is taken off.
// 64 x 64 tiles are for where there is one for each CU at most; 32 x 32 and 64 x 32
// for one matrix.  The constants are the fit's: one by itself is no time that was
// measured (starts below zero are none), and all are of the kernels as they were then.
struct Linear { double start, step; double at(int64_t steps) const { return start + step * (double)steps; } };
struct FewCost { double start, block, shared, shared_two, first; };
struct Costs {
    FewCost few8, few16, few32, few32x32, few64;
    double mb, again, off;
    Linear deep;
    double stretch;            // of 64 x 128 tiles, by tiles a CU
    Linear tile64, tile128, tile128_many, wide, tile256;
};
// Fitted to 1370 calls (9 to 8192 rows, N 64 to 14336, K 128 to 14336, one matrix and
// two; up to six sets of operands in turn, in a graph), the eight-row kernel's to
// fewer and earlier ones.  Of 2400 others (perf/fit_gemm_f8.py, which fits them anew)
// the choice was on average 1.6% behind the best kernel for 16-bit outputs, 10% or
// more in one of twenty; for float32 4.1% and 18%, mostly where eight-row tiles are
// taken for more rows: they are estimated too low (50 x 588 x 2160 gated 7.2 us, 4.4
// in 16 x 16).  Where they
// decide: 64 x 4096 x 14336 takes 21.1 us in tiles of 32 x 32, 26.5 in 32 x 16, 28.5
// in 64 x 32 and 39.3 in 64 x 64; at 128 rows these are 32.2, 42.1, 27.3 and 38.1.
// 1024 x 4096 x 4096 takes 26.7 us in 128 x 128, 29.0 in 64 x 128 and 31.8 in 128 x
// 256, 8192 x 14336 x 4096 417 in 256 x 256, 488 in 128 x 256 and 553 in 128 x 128.
constexpr Costs kCosts16 = {{-0.344, 0.353, 0.045, 0.057, 0.963},
                            {-0.617, 0.596, 0.066, 0.086, 1.336},
                            {-0.221, 0.908, 0.105, 0.153, 1.345},
                            {0.806, 0.721, 0.117, 0., 2.430},
                            {-0.055, 0.895, 0.219, 0., 3.842},
                            0.129, 0.837, -1.496,
                            {4.659, 0.327},
                            1.105, {2.935, 0.521}, {3.929, 0.608}, {0.979, 0.855}, {7.065, 0.968}, {9.123, 1.712}};
constexpr Costs kCosts32 = {{-0.615, 0.142, 0.036, 0.046, 0.912},
                            {1.107, 0.547, 0.057, 0.086, 1.943},
                            {0.361, 0.782, 0.087, 0.131, 2.548},
                            {0.904, 0.849, 0.131, 0., 1.810},
                            {-0.338, 1.006, 0.236, 0., 3.920},
                            0.192, 0.565, -2.228,
                            {4.348, 0.437},
                            1.315, {4.539, 0.663}, {4.837, 0.996}, {5.928, 1.025}, {12.344, 1.549}, {0., 0.}};

// The kernel for a call's sizes: up to 8 rows the weights' stream decides; above,
// the least estimated time.
Kernel choose(const Args &p, int mats) {
    const int64_t steps = tiles_of(p.K, BK);
    const bool f16 = p.y_type == I8_F32, two = mats == 2;
    const Costs &c = f16 ? kCosts32 : kCosts16;
    if (p.M <= 8) return kFew8;
    if (p.K < BK) return p.M <= 16 ? kFew16 : kFew32;
    auto tiles = [&](int bm, int bw) { return tiles_of(p.M, bm) * tiles_of(p.N, bw / mats); };
    auto rounds = [&](int64_t t) { return (double)((t + kCUs - 1) / kCUs); };
    // Tiles a CU, 1 where there are fewer, and the time of one alone or of one among others.
    auto each = [&](int64_t t, const Linear &one, const Linear &many) {
        return t <= kCUs ? one.at(steps) : (double)t / kCUs * many.at(steps);
    };
    auto few = [&](int bm, int cols, int most, const FewCost &f) {
        const Split s = split_of(p, bm, cols, most);
        const int64_t tm = tiles_of(p.M, bm), wgs = tm * tiles_of(s.strips, s.waves >> s.log2);
        const double waves = (double)(tiles_of(wgs, kCUs) * s.waves);                   // of a CU
        const double block = std::max(f.block, (two ? f.shared_two : f.shared) * waves);
        const double mb = (double)mats * p.N * p.K * 1e-6;
        return std::max(f.start + block * (f.first + (double)tiles_of(steps, 1 << s.log2)),
                        c.mb * mb * (1. + c.again * (double)(tm - 1)) - c.off);
    };
    constexpr double kNever = 1e30;
    double cost[kKernels];
    cost[kFew8] = few(8, 16, 8, c.few8);
    cost[kFew16] = few(16, 16, 8, c.few16);
    cost[kFew32] = few(32, 16, 8, c.few32);
    cost[kFew32x32] = two ? kNever : few(32, 32, 8, c.few32x32);
    cost[kFew64] = two ? kNever : few(64, 32, 4, c.few64);
    cost[kTileDeep] = tiles(64, 64) <= kCUs ? c.deep.at(steps) : kNever;
    cost[kTile64] = std::max(1.0, (double)tiles(64, 128) / kCUs * c.stretch) * c.tile64.at(steps);
    cost[kTile128] = each(tiles(128, 128), c.tile128, c.tile128_many);
    cost[kTileWide] = rounds(tiles(128, 256)) * c.wide.at(steps);
    const int64_t t256 = tiles(256, 256), left = t256 % kCUs;
    const double divided = left > kQuartersMost ? c.wide.at(steps) : left ? c.tile128.at(steps) : 0.;
    cost[kTile256] = f16                                 ? kNever        // its fragments would not fit
                     : t256 < kCUs || left > kRestMost ? rounds(t256) * c.tile256.at(steps)
                                                       : (double)(t256 / kCUs) * c.tile256.at(steps) + divided;
    Kernel best = kFew8;
    for (Kernel k : {kFew16, kFew32, kFew32x32, kFew64, kTileDeep, kTile64, kTile128, kTileWide, kTile256})
        if (cost[k] < cost[best]) best = k;
    return best;
}

template <Mode MODE, bool F16>
int launch(const Args &p, Kernel k, const Target &to) {
    constexpr bool TWO = MODE != kPlain;
    // Where there is only one workgroup for each CU, its ring has more stages:
    // 512 x 4096 x 14336 gated takes 84 us with four, 117 with two.
    auto alone = [&](int bm, int bw) { return tiles_of(p.M, bm) * tiles_of(p.N, TWO ? bw / 2 : bw) <= kCUs; };
    // Two matrices halve the columns of a lane's run: four rows of wavefronts
    // then store whole lines of 16 bits (1999 x 14336 x 4096 gated, 128 x 256: 253 us
    // against 258).  To float32 they do in either order, and two rows convert fewer
    // operands (4096 x 8192 x 512 gated: 84 us against 92).
    constexpr int kM = TWO && !F16 ? 4 : 2, kN = TWO && !F16 ? 2 : 4;
    switch (k) {
    case kFew8: return launch_few<1, 1, MODE, F16>(p, to);
    case kFew16: return launch_few<2, 1, MODE, F16>(p, to);
    case kFew32: return launch_few<4, 1, MODE, F16>(p, to);
    case kFew32x32:
    case kFew64:
        if constexpr (TWO) return Q4_EINVAL;                                    // not chosen
        else return k == kFew64 ? launch_few<8, 2, MODE, F16, 4>(p, to) : launch_few<4, 2, MODE, F16>(p, to);
    case kTile64: return launch_block<64, 128, 2, 4, 1, 3, MODE, F16>(p, to);
    case kTileDeep: return launch_block<64, 64, 2, 2, 2, 4, MODE, F16>(p, to);
    case kTile128:
        if (alone(128, 128)) return launch_block<128, 128, kM, kN, 1, 4, MODE, F16>(p, to);
        // Four wavefronts, of 64 x 64: two workgroups a CU, neither of which
        // waits at the other's barriers, and a last round that is not full has
        // the CUs to itself.
        return launch_block<128, 128, 2, 2, 1, 2, MODE, F16>(p, to);
    case kTileWide: return launch_block<128, 256, kM, kN, 1, 3, MODE, F16>(p, to);
    default:
        if constexpr (F16) return Q4_EINVAL;         // not chosen
        else {
            Args q = p;
            // One tile a CU, in rounds.  Where the last would have few, it goes to a
            // launch of smaller tiles.  With six sets of operands in turn 4600 x 4096 x
            // 14336 (32 tiles left) takes 280 us so and 368 without, 5376 rows (80 left)
            // 311 and 358, 1999 x 14336 x 4096 gated (128 left) 227 and 235 (222 with
            // three sets, which the last cache holds in part).
            const int64_t all = tiles_of(p.M, 256) * tiles_of(p.N, TWO ? 128 : 256);
            const int whole = whole_rounds((int)all), left = (int)all - whole;
            if (all > kCUs && left) {
                q.part = kWhole;
                q.whole = whole;
            }
            if (int st = launch_block<256, 256, kM, kN, 1, 2, MODE, false>(q, to)) return st;
            if (q.part == kAll) return Q4_OK;
            if (left > kQuartersMost) {
                q.part = kHalves;
                return launch_block<128, 256, kM, kN, 1, 3, MODE, false>(q, to);
            }
            q.part = kQuarters;
            return launch_block<128, 128, kM, kN, 1, 4, MODE, false>(q, to);
        }
    }
}

int launch(const Args &p, Mode mode, const Target &to) {
    const Kernel k = choose(p, mode == kPlain ? 1 : 2);
    const bool f16 = p.y_type == I8_F32;
    switch (mode) {
    case kPlain: return f16 ? launch<kPlain, true>(p, k, to) : launch<kPlain, false>(p, k, to);
    case kGated: return f16 ? launch<kGated, true>(p, k, to) : launch<kGated, false>(p, k, to);
    default: return f16 ? launch<kBackward, true>(p, k, to) : launch<kBackward, false>(p, k, to);
    }
}

bool type_ok(int t) { return t == I8_F32 || t == I8_F16 || t == I8_BF16; }

int check_sizes(const Args &p) {
    if (p.M < 0 || p.M > kMaxRows || p.N < 0 || p.N > kMaxRows || p.K < 16 || p.K % 16 || p.K > kMaxK)
        return Q4_EINVAL;
    if (tiles_of(p.M, 16) * tiles_of(p.N, 16) > 0x7FFFFFFFll) return Q4_EINVAL;
    return type_ok(p.y_type) ? Q4_OK : Q4_EINVAL;
}

int run(Args p, int a_block, Mode mode, void *stream) {
    if (int st = check_sizes(p)) return st;
    if (a_block != 1 && a_block != 128) return Q4_EINVAL;
    if (p.sa_m < 0 || p.sa_m > (1 << 20) || p.sa_k < 0 || p.sa_k > (1ll << 31)) return Q4_EINVAL;
    if (mode == kBackward && !type_ok(p.dh_type)) return Q4_EINVAL;
    if (p.M == 0 || p.N == 0) return Q4_OK;
    if (!p.a || !p.sa || !p.w[0] || !p.sw[0] || !p.y) return Q4_ENULL;
    if (mode != kPlain && (!p.w[1] || !p.sw[1])) return Q4_ENULL;
    if (mode == kBackward && !p.dh) return Q4_ENULL;
    if (!q4::aligned(p.a, 16) || !q4::aligned(p.w[0], 16) || !q4::aligned(p.w[1], 16) || !q4::aligned(p.sa, 4) ||
        !q4::aligned(p.sw[0], 4) || !q4::aligned(p.sw[1], 4) || !q4::aligned(p.bias, 4) ||
        !elem_aligned(p.y, p.y_type) || !elem_aligned(p.dh, p.dh_type))
        return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    p.sa_shift = a_block == 128 ? 7 : 0;
    return launch(p, mode, {static_cast<hipStream_t>(stream), nullptr});
}

Args args_of(const uint8_t *a, const float *sa, int64_t sm, int64_t sk, const uint8_t *w0, const float *s0,
             const uint8_t *w1, const float *s1, void *y, int y_type, int M, int N, int K) {
    Args p = {};
    p.a = a, p.sa = sa, p.sa_m = sm, p.sa_k = sk;
    p.w[0] = w0, p.w[1] = w1, p.sw[0] = s0, p.sw[1] = s1;
    p.y = y, p.y_type = y_type, p.M = M, p.N = N, p.K = K;
    return p;
}

}  // namespace

extern "C" int gemm_f8(const uint8_t *a, const float *a_scales, int64_t stride_m, int64_t stride_k, int a_block,
                       const uint8_t *w, const float *w_scales, const float *bias, void *y, int y_type, int M, int N,
                       int K, void *stream) {
    Args p = args_of(a, a_scales, stride_m, stride_k, w, w_scales, nullptr, nullptr, y, y_type, M, N, K);
    p.bias = bias;
    return run(p, a_block, kPlain, stream);
}

extern "C" int gemm_f8_swiglu(const uint8_t *a, const float *a_scales, int64_t stride_m, int64_t stride_k, int a_block,
                              const uint8_t *w_gate, const float *scales_gate, const uint8_t *w_up,
                              const float *scales_up, void *y, int y_type, int M, int N, int K, void *stream) {
    return run(args_of(a, a_scales, stride_m, stride_k, w_gate, scales_gate, w_up, scales_up, y, y_type, M, N, K),
               a_block, kGated, stream);
}

extern "C" int gemm_f8_swiglu_backward(const void *dh, int dh_type, const uint8_t *a, const float *a_scales,
                                       int64_t stride_m, int64_t stride_k, int a_block, const uint8_t *w_gate,
                                       const float *scales_gate, const uint8_t *w_up, const float *scales_up, void *d,
                                       int y_type, int M, int N, int K, void *stream) {
    Args p = args_of(a, a_scales, stride_m, stride_k, w_gate, scales_gate, w_up, scales_up, d, y_type, M, N, K);
    p.dh = dh, p.dh_type = dh_type;
    return run(p, a_block, kBackward, stream);
}

extern "C" int gemm_f8_geometry(int matrices, int y_type, int M, int N, int K, int *tile_rows, int *tile_cols,
                                int *grid, int *block) {
    Args p = {};
    p.M = M, p.N = N, p.K = K, p.y_type = y_type;
    if (matrices != 1 && matrices != 2) return Q4_EINVAL;
    if (int st = check_sizes(p)) return st;
    Report r = {};
    if (M > 0 && N > 0)
        if (int st = launch(p, matrices == 1 ? kPlain : kGated, {nullptr, &r})) return st;
    if (tile_rows) *tile_rows = r.rows;
    if (tile_cols) *tile_cols = r.cols;
    if (grid) *grid = (int)r.grid;
    if (block) *block = r.block;
    return Q4_OK;
}
