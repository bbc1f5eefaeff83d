// gemm_i8.hip -- products of 8-bit activations with 8-bit weights for gfx950
// (see q4i8.h):
//
//     P[m, n] = (sum_k a[m, k] w[n, k]) * a_scales[m] * w_scales[n]
//
// plain, as a SwiGLU block of two matrices, and both grouped by expert.
//
// The sums run on v_mfma_i32_16x16x64_i8, exactly.  The weights are its first
// operand and the activations its second, so that a lane ends with several
// consecutive n of one row m; which weight row goes to which row of a
// fragment is chosen so that the fragments of a lane together hold one run
// of n (frag_row).
#include "q4_common.h"
#include "q4i8.h"

#include <algorithm>

namespace {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct Args {
    const int8_t *a;
    const float *sa;
    const int8_t *w[2];        // one matrix, or gate and up
    const float *sw[2];
    const float *bias;
    const int32_t *offsets;    // groups, or NULL
    void *y;
    int y_type, M, N, K, E;
    int tiles_m, tiles_n;
    bool vec;                  // rows of y may be written in 16-byte stores
};

// The fragment of 16 weight rows j (of F that share a run of 16 F rows) takes
// row frag_row<F>(j, i) of the run as its row i: lane group i / 4 then holds,
// over the F fragments, the 4 F consecutive rows from 4 F (i / 4) on.
template <int F>
__device__ __forceinline__ int frag_row(int j, int i) { return (i >> 2) * (4 * F) + 4 * j + (i & 3); }

__device__ __forceinline__ float silu(float v) { return v * __builtin_amdgcn_rcpf(1.f + __expf(-v)); }

__device__ __forceinline__ uint32_t bits16(float v, int type) {
    if (type == I8_F16) return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// Writes the run v[0 .. C) of row m from column n on, its columns past N
// left out.  16-byte stores where the rows allow them.
template <int C>
__device__ __forceinline__ void store_run(const Args &p, int m, int n, const float (&v)[C]) {
    if (n >= p.N) return;
    const size_t at = (size_t)m * p.N + n;
    const bool whole = n + C <= p.N;
    if (p.y_type == I8_F32) {
        float *y = static_cast<float *>(p.y) + at;
        if (p.vec && whole) {
#pragma unroll
            for (int c = 0; c < C; c += 4)
                *reinterpret_cast<u32x4_t *>(y + c) =
                    u32x4_t{__builtin_bit_cast(uint32_t, v[c]), __builtin_bit_cast(uint32_t, v[c + 1]),
                            __builtin_bit_cast(uint32_t, v[c + 2]), __builtin_bit_cast(uint32_t, v[c + 3])};
        } else {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (n + c < p.N) y[c] = v[c];
        }
        return;
    }
    uint16_t *y = static_cast<uint16_t *>(p.y) + at;
    uint32_t b[C];
#pragma unroll
    for (int c = 0; c < C; ++c) b[c] = bits16(v[c], p.y_type);
    if (p.vec && whole) {
        if constexpr (C % 8 == 0) {
#pragma unroll
            for (int c = 0; c < C; c += 8)
                *reinterpret_cast<u32x4_t *>(y + c) =
                    u32x4_t{b[c] | b[c + 1] << 16, b[c + 2] | b[c + 3] << 16, b[c + 4] | b[c + 5] << 16,
                            b[c + 6] | b[c + 7] << 16};
        } else {
#pragma unroll
            for (int c = 0; c < C; c += 4)
                *reinterpret_cast<u32x2_t *>(y + c) = u32x2_t{b[c] | b[c + 1] << 16, b[c + 2] | b[c + 3] << 16};
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c)
            if (n + c < p.N) y[c] = (uint16_t)b[c];
    }
}

// The rows of a workgroup's tile: m0 .. m0 + rows of y, with matrix e.
// rows == 0: no such tile.
struct Tile { int m0, rows, e; };

// Finds tile t of BM rows among the groups: 64 groups at a time, one a lane,
// the lanes' tile counts summed by a scan.  Offsets are held to 0 .. M.
template <int BM>
__device__ __forceinline__ Tile find_tile(const Args &p, int t) {
    if (!p.offsets) return {t * BM, min(BM, p.M - t * BM), 0};
    const int lane = threadIdx.x & 63;
    for (int e0 = 0; e0 < p.E; e0 += 64) {
        const int e = e0 + lane;
        int lo = 0, hi = 0;
        if (e < p.E) {
            lo = min(max(p.offsets[e], 0), p.M);
            hi = min(max(p.offsets[e + 1], lo), p.M);
        }
        const int mine = (hi - lo + BM - 1) / BM;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const int all = __builtin_amdgcn_readlane(upto, 63);
        if (t < all) {
            const int owner = __ffsll((unsigned long long)__ballot(upto > t)) - 1;
            const int m0 = __builtin_amdgcn_readlane(lo, owner) +
                           (t - __builtin_amdgcn_readlane(upto - mine, owner)) * BM;
            return {m0, min(BM, __builtin_amdgcn_readlane(hi, owner) - m0), e0 + owner};
        }
        t -= all;
    }
    return {0, 0, 0};
}

// Scales a wavefront's sums and writes them.  acc[i][..]: rows row0 + 16 i +
// lane % 16 of the tile; over its fragments a lane holds the C columns from n
// on (with SWI: C of gate in the first half of the fragments, C of up in the
// second).
template <int FM, int C, bool SWI>
__device__ __forceinline__ void finish(const Args &p, const i32x4_t (&acc)[FM][SWI ? C / 2 : C / 4], const Tile &tl,
                                       size_t mat, int row0, int n, int lane) {
    float sw[SWI ? 2 : 1][C], bias[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const bool in = n + c < p.N;
        sw[0][c] = in ? p.sw[0][mat + n + c] : 0.f;
        if constexpr (SWI) sw[SWI][c] = in ? p.sw[1][mat + n + c] : 0.f;
        bias[c] = !SWI && p.bias && in ? p.bias[n + c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = row0 + i * 16 + (lane & 15);
        if (r >= tl.rows) continue;
        const float sa = p.sa[tl.m0 + r];
        float v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (SWI) {
                const float g = (float)acc[i][c >> 2][c & 3] * sa * sw[0][c];
                const float u = (float)acc[i][(C + c) >> 2][c & 3] * sa * sw[SWI][c];
                v[c] = silu(g) * u;
            } else {
                v[c] = (float)acc[i][c >> 2][c & 3] * sa * sw[0][c] + bias[c];
            }
        }
        store_run<C>(p, tl.m0 + r, n, v);
    }
}

// The tile of this workgroup.  Workgroups are dealt to the eight XCDs in
// turn, each with its own L2: XCD x takes the x-th eighth of the tiles, and
// tiles are ordered in bands of eight tile rows, column by column, so that
// the tiles an XCD runs at one time share rows of a and of w.
__device__ __forceinline__ void tile_of(const Args &p, int &tm, int &tn) {
    const int all = gridDim.x, b = blockIdx.x, x = b & 7, per = all >> 3, more = all & 7;
    const int t = x * per + min(x, more) + (b >> 3);
    const int band = t / (8 * p.tiles_n), first = band * 8, rows = min(8, p.tiles_m - first);
    const int in = t - band * 8 * p.tiles_n;
    tm = first + in % rows;
    tn = in / rows;
}

// LDS tiles: rows of 128 bytes in eight 16-byte chunks; chunk c of row r
// sits at slot c ^ (r & 7), so that the 16 lanes of a fragment that read one
// chunk of 16 rows touch every bank alike.
constexpr int BK = 128;
__device__ __forceinline__ int slot(int r, int c) { return r * BK + ((c ^ (r & 7)) << 4); }

// One 64 x 64 tile (with SWI: 32 columns of each matrix), four wavefronts of
// 32 x 32 each.  Tiles pass through registers into one LDS buffer.
template <bool SWI>
__global__ __launch_bounds__(256) void gemm_i8_tile(Args p) {
    constexpr int BM = 64, BW = 64, BN = SWI ? 32 : 64;
    __shared__ __align__(16) char lds[(BM + BW) * BK];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave >> 1, wn = wave & 1;
    int tm, tn;
    tile_of(p, tm, tn);
    const Tile tl = find_tile<BM>(p, tm);
    if (tl.rows <= 0) return;
    const int n0 = tn * BN;
    const size_t mat = (size_t)tl.e * p.N;

    i32x4_t acc[2][2] = {};
    const int kc = p.K >> 4;       // 16-byte chunks of a row
    for (int k0 = 0; k0 < kc; k0 += 8) {
#pragma unroll
        for (int i = 0; i < (BM + BW) * 8 / 256; ++i) {
            const int q = i * 256 + tid, r = q >> 3, c = q & 7;
            i32x4_t v = {0, 0, 0, 0};
            if (k0 + c < kc) {
                if (r < BM) {
                    if (r < tl.rows)
                        v = *reinterpret_cast<const i32x4_t *>(p.a + (size_t)(tl.m0 + r) * p.K + (size_t)(k0 + c) * 16);
                } else {
                    // SWI: each wavefront's 32 weight rows are 16 of gate, then 16 of up.
                    const int b = r - BM, s = SWI ? (b >> 4) & 1 : 0;
                    const int n = n0 + (SWI ? (b >> 5) * 16 + (b & 15) : b);
                    if (n < p.N)
                        v = *reinterpret_cast<const i32x4_t *>(p.w[s] + (mat + n) * p.K + (size_t)(k0 + c) * 16);
                }
            }
            *reinterpret_cast<i32x4_t *>(lds + slot(r, c)) = v;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int c = kk * 4 + (lane >> 4);
            i32x4_t x[2], w[2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                x[i] = *reinterpret_cast<const i32x4_t *>(lds + slot(wm * 32 + i * 16 + (lane & 15), c));
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = SWI ? j * 16 + (lane & 15) : frag_row<2>(j, lane & 15);
                w[j] = *reinterpret_cast<const i32x4_t *>(lds + slot(BM + wn * 32 + r, c));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
        }
        __syncthreads();
    }

    constexpr int C = SWI ? 4 : 8;       // consecutive columns of a lane
    finish<2, C, SWI>(p, acc, tl, mat, wm * 32, n0 + (SWI ? wn * 16 : wn * 32) + (lane >> 4) * C, lane);
}

// ---------------------------------------------------------------- large tiles
//
// A 256 x 256 tile (with SWI: 128 columns of each matrix), eight wavefronts
// of 128 x 64.  Steps of 128 bytes of K pass through two LDS buffers, loaded
// straight from memory (buffer loads to LDS, 1 KiB an instruction: eight rows
// of 128 bytes, the lanes' chunk order making the swizzle).  A step has two
// halves of 64 bytes; the fragments of each half are read into registers
// while the other half's products run:
//
//     first half:   read (t, second half),  products of (t, first half)
//                   wait for step t + 1 in LDS and for this step's reads
//     second half:  load step t + 2 over step t,  read (t + 1, first half),
//                   products of (t, second half)
//
// so there is one barrier a step, and a step's loads have a whole step to
// arrive.  A last step that K does not fill is taken as the last 128 bytes
// of the rows, with the activations already used set to zero; every address
// stays inside the rows.  Rows past the tile's end repeat its last row, and
// their results are not stored.
typedef __attribute__((address_space(3))) void *lds_ptr_t;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(const int8_t *base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<int8_t *>(base), 0, (int)bytes, 0x00020000);
}

template <bool SWI>
__global__ __launch_bounds__(512, 2) void gemm_i8_large(Args p) {
    constexpr int BM = 256, BW = 256, BN = SWI ? 128 : 256;
    constexpr int STAGE = (BM + BW) * BK;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int tm, tn;
    tile_of(p, tm, tn);
    const Tile tl = find_tile<BM>(p, tm);
    if (tl.rows <= 0) return;
    const int n0 = tn * BN, cols = min(BN, p.N - n0);
    const size_t mat = (size_t)tl.e * p.N;

    // Loads: this wavefront brings rows 32 wave .. 32 wave + 31 of both
    // halves of a stage, eight rows an instruction.
    const __amdgpu_buffer_rsrc_t ra = rsrc_of(p.a + (size_t)tl.m0 * p.K, (uint32_t)tl.rows * p.K);
    // SWI: the 32 weight rows of one wavefront's loads are all gate or all up.
    const int8_t *wbase = SWI && (wave & 1) ? p.w[1] : p.w[0];
    const __amdgpu_buffer_rsrc_t rw = rsrc_of(wbase + (mat + n0) * p.K, (uint32_t)cols * p.K);
    uint32_t va[4], vw[4];
    const int chunk = ((lane & 7) ^ (lane >> 3)) << 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = wave * 32 + i * 8 + (lane >> 3);
        va[i] = (uint32_t)min(r, tl.rows - 1) * p.K + chunk;
        // Row r of the weight half belongs to wavefront column r / 64, its
        // fragment (r / 16) % 4, row r % 16 of it.
        const int c = r >> 6, j = (r >> 4) & 3, q = r & 15;
        const int n = SWI ? c * 32 + frag_row<2>(j & 1, q) : c * 64 + frag_row<4>(j, q);
        vw[i] = (uint32_t)min(n, cols - 1) * p.K + chunk;
    }
    auto load = [&](int buf, int koff) {
        char *at = lds + buf * STAGE + wave * 32 * BK;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(ra, (lds_ptr_t)(at + i * 8 * BK), 16, va[i], koff, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rw, (lds_ptr_t)(at + BM * BK + i * 8 * BK), 16, vw[i], koff, 0,
                                                     0);
    };

    // Fragment reads: lane l takes row l % 16, chunk l / 16 (+ 4 in the
    // second half, which flips bit 6 of the swizzled address).
    const int fr = (lane & 15) * BK + (((lane >> 4) ^ (lane & 7)) << 4);
    const char *xa = lds + wm * 128 * BK + fr, *wa = lds + (BM + wn * 64) * BK + fr;
    const char *xb = lds + wm * 128 * BK + (fr ^ 64), *wb = lds + (BM + wn * 64) * BK + (fr ^ 64);
    i32x4_t acc[8][4] = {};
    i32x4_t x0[8], w0[4], x1[8], w1[4];
    auto read = [&](i32x4_t (&x)[8], i32x4_t (&w)[4], const char *px, const char *pw) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const i32x4_t *>(pw + j * 16 * BK);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = *reinterpret_cast<const i32x4_t *>(px + i * 16 * BK);
    };
    auto products = [&](const i32x4_t (&x)[8], const i32x4_t (&w)[4]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
    };
    const int steps = (p.K + BK - 1) / BK;
    auto koff = [&](int t) { return min(t * BK, p.K - BK); };
    // Chunks of the last step that earlier steps have used.
    const int used = steps * 8 - (p.K >> 4);
    auto drop = [&](i32x4_t (&x)[8], int c) {
        if (c < used) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = i32x4_t{0, 0, 0, 0};
        }
    };

    load(0, koff(0));
    if (steps > 1) load(1, koff(1));
    if (steps > 1) asm volatile("s_waitcnt vmcnt(8)" ::: "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_barrier" ::: "memory");
    read(x0, w0, xa, wa);
    if (steps == 1 && used) drop(x0, lane >> 4);
    auto wait = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    int t = 0;
    auto whole = [&](int buf) {          // a step with two full ones behind it
        const int cur = buf * STAGE, nxt = STAGE - cur;
        read(x1, w1, xb + cur, wb + cur);
        products(x0, w0);
        wait();
        load(buf, (t + 2) * BK);
        read(x0, w0, xa + nxt, wa + nxt);
        products(x1, w1);
        __builtin_amdgcn_sched_barrier(0);
        ++t;
    };
    while (t + 4 < steps) {
        whole(0);
        whole(1);
    }
    for (; t < steps; ++t) {
        const int cur = (t & 1) * STAGE, nxt = STAGE - cur;
        read(x1, w1, xb + cur, wb + cur);
        if (t + 1 == steps && used) drop(x1, 4 + (lane >> 4));
        products(x0, w0);
        wait();
        if (t + 2 < steps) load(t & 1, koff(t + 2));
        if (t + 1 < steps) {
            read(x0, w0, xa + nxt, wa + nxt);
            if (t + 2 == steps && used) drop(x0, lane >> 4);
        }
        products(x1, w1);
        __builtin_amdgcn_sched_barrier(0);
    }

    constexpr int C = SWI ? 8 : 16;      // consecutive columns of a lane
    finish<8, C, SWI>(p, acc, tl, mat, wm * 128, n0 + (SWI ? wn * 32 : wn * 64) + (lane >> 4) * C, lane);
}

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxK = 131056;      // 16384 * 131056 < 2^31: the sum fits whatever the codes

bool elem_aligned(const void *y, int type) { return q4::aligned(y, type == I8_F32 ? 4 : 2); }

int run(Args p, int mats, hipStream_t stream) {
    if (p.M < 0 || p.M > kMaxRows || p.N < 0 || p.N > kMaxRows || p.K < 16 || p.K % 16 || p.K > kMaxK)
        return Q4_EINVAL;
    if (p.y_type != I8_F32 && p.y_type != I8_F16 && p.y_type != I8_BF16) return Q4_EINVAL;
    if ((int64_t)((p.M + 15) / 16) * ((p.N + 15) / 16) > 0x7FFFFFFFll) return Q4_EINVAL;
    if (p.E < 1 || p.E > 65536 || (int64_t)p.E * p.N > 0x7FFFFFFFll) return Q4_EINVAL;
    if (p.M == 0 || p.N == 0) return Q4_OK;
    if (!p.a || !p.sa || !p.w[0] || !p.sw[0] || !p.y || (mats == 2 && (!p.w[1] || !p.sw[1]))) return Q4_ENULL;
    if (!q4::aligned(p.a, 16) || !q4::aligned(p.w[0], 16) || !q4::aligned(p.sa, 4) || !q4::aligned(p.sw[0], 4) ||
        !q4::aligned(p.bias, 4) || !q4::aligned(p.offsets, 4) || !elem_aligned(p.y, p.y_type))
        return Q4_EALIGN;
    if (mats == 2 && (!q4::aligned(p.w[1], 16) || !q4::aligned(p.sw[1], 4))) return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    p.vec = q4::aligned(p.y, 16) && (size_t)p.N * (p.y_type == I8_F32 ? 4 : 2) % 16 == 0;
    const bool large = p.K >= BK && p.M > 128;
    const int bm = large ? 256 : 64, bn = bm / mats;
    p.tiles_n = (p.N + bn - 1) / bn;
    // Groups: every group may end inside a tile.
    const int64_t tiles_m = p.offsets ? p.M / bm + std::min(p.E, p.M) : (p.M + bm - 1) / bm;
    const int64_t grid = tiles_m * p.tiles_n;
    if (grid > 0x7FFFFFFFll) return Q4_EINVAL;
    p.tiles_m = (int)tiles_m;
    if (large) {
        constexpr int lds = 2 * 512 * BK;
        const void *f = mats == 2 ? (const void *)gemm_i8_large<true> : (const void *)gemm_i8_large<false>;
        if (hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, lds) != hipSuccess) return Q4_ELAUNCH;
        if (mats == 2) gemm_i8_large<true><<<(unsigned)grid, 512, lds, stream>>>(p);
        else gemm_i8_large<false><<<(unsigned)grid, 512, lds, stream>>>(p);
    } else if (mats == 2) {
        gemm_i8_tile<true><<<(unsigned)grid, 256, 0, stream>>>(p);
    } else {
        gemm_i8_tile<false><<<(unsigned)grid, 256, 0, stream>>>(p);
    }
    return q4::launch_status();
}

}  // namespace

extern "C" int gemm_i8(const int8_t *a, const float *a_scales, const int8_t *w, const float *w_scales,
                       const float *bias, void *y, int y_type, int M, int N, int K, void *stream) {
    return run({a, a_scales, {w, nullptr}, {w_scales, nullptr}, bias, nullptr, y, y_type, M, N, K, 1, 0, 0, false}, 1,
               static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_swiglu(const int8_t *a, const float *a_scales, const int8_t *w_gate,
                              const float *scales_gate, const int8_t *w_up, const float *scales_up, void *y,
                              int y_type, int M, int N, int K, void *stream) {
    return run({a, a_scales, {w_gate, w_up}, {scales_gate, scales_up}, nullptr, nullptr, y, y_type, M, N, K, 1, 0, 0,
                false},
               2, static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_grouped(const int8_t *a, const float *a_scales, const int8_t *w, const float *w_scales,
                               const int32_t *offsets, void *y, int y_type, int M, int E, int N, int K,
                               void *stream) {
    if (!offsets && M > 0 && N > 0) return Q4_ENULL;
    return run({a, a_scales, {w, nullptr}, {w_scales, nullptr}, nullptr, offsets, y, y_type, M, N, K, E, 0, 0, false}, 1,
               static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_grouped_swiglu(const int8_t *a, const float *a_scales, const int8_t *w_gate,
                                      const float *scales_gate, const int8_t *w_up, const float *scales_up,
                                      const int32_t *offsets, void *y, int y_type, int M, int E, int N, int K,
                                      void *stream) {
    if (!offsets && M > 0 && N > 0) return Q4_ENULL;
    return run({a, a_scales, {w_gate, w_up}, {scales_gate, scales_up}, nullptr, offsets, y, y_type, M, N, K, E, 0, 0,
                false},
               2, static_cast<hipStream_t>(stream));
}
