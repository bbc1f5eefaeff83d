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

constexpr int kCUs = 256;

// Tiles of 256 x 256 come in rounds of one for each CU.  Where the last round
// would have up to 128, they go to a launch of their own (kHalves, 128 rows
// each, where there are more than 64; kQuarters, 128 x 128, else), which takes
// one round of two thirds or a third of the time: 4600 x 4096 x 14336 (32 tiles
// left) takes 223 us so and 315 without, 5376 rows (80 left) 251 and 316 (287
// as quarters, in two rounds), 9000 x 8192 x 8192 (128 left) 461 and 481.
// With groups the count is the GPU's to know: both are launched, and one has
// no work.
enum Part { kAll, kWhole, kHalves, kQuarters };
constexpr int kRestMost = 128, kQuartersMost = 64;

struct Args {
    const int8_t *a;
    const float *sa;
    const int8_t *w[2];        // one matrix, or gate and up
    const float *sw[2];
    const float *bias;
    const int32_t *offsets;    // groups, or NULL
    void *y;
    int y_type, M, N, K, E;
    int tiles_m, tiles_n;      // kHalves, kQuarters: of the tiles that are divided
    Part part;
    bool once;                 // the weights' stream is more than a cache would keep
    bool share;                // several row tiles read the same weights
};

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

// Writes the run v[0 .. C) of row m from column n on, its columns past N
// left out.
template <int C>
__device__ __forceinline__ void store_run(const Args &p, int m, int n, const float (&v)[C]) {
    if (n >= p.N) return;
    const size_t at = (size_t)m * p.N + n;
    const bool whole = n + C <= p.N;
    if (p.y_type == I8_F32) {
        float *y = static_cast<float *>(p.y) + at;
        if (whole) {
#pragma unroll
            for (int c = 0; c < C; c += 4)
                *reinterpret_cast<u32x4_at4_t *>(y + c) =
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
    uint32_t b[C / 2];
#pragma unroll
    for (int c = 0; c < C / 2; ++c) b[c] = bits16(v[2 * c], p.y_type) | bits16(v[2 * c + 1], p.y_type) << 16;
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
            if (n + c < p.N) y[c] = (uint16_t)(b[c / 2] >> (16 * (c & 1)));
    }
}

// The rows of a workgroup's tile: m0 .. m0 + rows of y, with matrix e.
// rows == 0: no such tile.
struct Tile { int m0, rows, e; };

// Sums over the lanes up to and with each lane.
__device__ __forceinline__ int scan_lanes(int v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// The rows of group e, none past the last group.  Offsets are held to 0 .. M
// and to their order, so that whatever they are, rows stay inside a and y.
struct Rows { int lo, hi; };
__device__ __forceinline__ Rows rows_of(const Args &p, int e) {
    if (e >= p.E) return {0, 0};
    const int lo = min(max(p.offsets[e], 0), p.M);
    return {lo, min(max(p.offsets[e + 1], lo), p.M)};
}

// Groups for each lane: lane l sums the tiles of groups l * groups_each ..
__device__ __forceinline__ int groups_each(const Args &p) { return (p.E + 63) >> 6; }

// Of a lane: the tiles of bm rows of all groups up to and with its own, at most
// tiles_m for each lane (no more unless the offsets are out of order: the sums
// cannot overflow), and the rows of its first group.
struct Groups { int upto; Rows rows; };
__device__ __forceinline__ Groups groups_of(const Args &p, int bm) {
    if (!p.offsets) return {0, {0, 0}};
    const int each = groups_each(p), e0 = (threadIdx.x & 63) * each;
    const Rows first = rows_of(p, e0);
    int mine = min((int)((unsigned)(first.hi - first.lo + bm - 1) / (unsigned)bm), p.tiles_m);
#pragma unroll 4
    for (int e = e0 + 1; e < e0 + each; ++e) {
        const Rows r = rows_of(p, e);
        mine = min(mine + (int)((unsigned)(r.hi - r.lo + bm - 1) / (unsigned)bm), p.tiles_m);
    }
    return {scan_lanes(mine), first};
}

// The tiles that there are.
__device__ __forceinline__ int tile_count(const Args &p, const Groups &g) {
    return p.offsets ? min(__builtin_amdgcn_readlane(g.upto, 63), p.tiles_m) : p.tiles_m;
}

// Tile t of bm rows (rows == 0: there is none): the lane whose groups hold it,
// then the group among that lane's.
__device__ __forceinline__ Tile find_tile(const Args &p, int bm, const Groups &g, int t) {
    if (!p.offsets) return {t * bm, min(bm, p.M - t * bm), 0};
    const unsigned long long past = __ballot(g.upto > t);
    if (!past) return {0, 0, 0};
    const int owner = __ffsll(past) - 1, each = groups_each(p);
    if (owner) t -= __builtin_amdgcn_readlane(g.upto, owner - 1);
    int e = owner * each;
    Rows r = {__builtin_amdgcn_readlane(g.rows.lo, owner), __builtin_amdgcn_readlane(g.rows.hi, owner)};
    if (each > 1) {
        for (int c = 0;; c += 64) {
            if (c >= each) return {0, 0, 0};
            const int q = c + (threadIdx.x & 63);
            const Rows here_rows = q < each ? rows_of(p, e + q) : Rows{0, 0};
            const int mine = (int)((unsigned)(here_rows.hi - here_rows.lo + bm - 1) / (unsigned)bm);
            const int here = scan_lanes(min(mine, p.tiles_m));
            const unsigned long long in = __ballot(here > t);
            if (in) {
                const int l = __ffsll(in) - 1;
                if (l) t -= __builtin_amdgcn_readlane(here, l - 1);
                e += c + l;
                r = {__builtin_amdgcn_readlane(here_rows.lo, l), __builtin_amdgcn_readlane(here_rows.hi, l)};
                break;
            }
            t -= __builtin_amdgcn_readlane(here, 63);
        }
    }
    const int m0 = r.lo + t * bm;
    return {m0, min(bm, r.hi - m0), e};
}

// Scales a wavefront's sums and writes them.  acc[i][..]: rows row0 + 16 i +
// lane % 16 of the tile; over its fragments a lane holds the C columns from n
// on (with SWI: C of gate in the first half of the fragments, C of up in the
// second).  sa: the scales of its rows; sw0, sw1: of its columns (sw1: of up, or
// without SWI the bias where there is one), anything past N.
template <int FM, int C, bool SWI>
__device__ __forceinline__ void finish(const Args &p, const i32x4_t (&acc)[FM][SWI ? C / 2 : C / 4], const Tile &tl,
                                       const float (&sa)[FM], const float *sw0, const float *sw1, int row0, int n,
                                       int lane) {
    float w[2][C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        w[0][c] = sw0[c];
        w[1][c] = SWI || p.bias ? sw1[c] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int r = row0 + i * 16 + (lane & 15);
        if (r >= tl.rows) continue;
        const float s = sa[i];
        float v[C], least = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if constexpr (SWI) {
                const float g = (float)acc[i][c >> 2][c & 3] * s * w[0][c];
                const float u = (float)acc[i][(C + c) >> 2][c & 3] * s * w[1][c];
                v[c] = silu(g) * u;
                least = __builtin_fminf(least, g);
            } else {
                v[c] = (float)acc[i][c >> 2][c & 3] * s * w[0][c] + w[1][c];
            }
        }
        // Far gates are rare, and without one this costs nothing that shows (8192 x
        // 2 x 4096 x 512 46.9 us, 47.1 without the branch); one formula that holds
        // for all gates took 49.5 against 45.5 there.
        if (SWI && __builtin_expect(least < kFar, 0)) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const float g = (float)acc[i][c >> 2][c & 3] * s * w[0][c];
                const float u = (float)acc[i][(SWI ? C + c : c) >> 2][c & 3] * s * w[1][c];
                if (g < kFar) v[c] = far_silu(g, u);
            }
        }
        store_run<C>(p, tl.m0 + r, n, v);
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

// ---------------------------------------------------------------- tiles
//
// A tile of BM rows and BW weight rows (with SWI: BW / 2 of each matrix) by
// WM x WN wavefronts, or by G groups of as many that share out K: group g
// takes every G-th slice of 128 bytes, and the groups' sums meet in LDS at the
// end.  Steps of G slices pass through a ring of D stages in LDS, loaded
// straight from memory (buffer loads to LDS, 1 KiB an instruction: eight rows
// of 128 bytes, the lanes' chunk order making the swizzle).  A step has two
// halves of 64 bytes; the fragments of each half are read into registers while
// the other half's products run:
//
//     first half:   read (t, second half),  products of (t, first half)
//                   wait for step t + 1 in LDS and for this step's reads
//     second half:  load step t + D over step t,  read (t + 1, first half),
//                   products of (t, second half)
//
// so there is one barrier a step, and a step's loads have D - 1 steps to
// arrive.  The last D steps of a tile load the first D of the workgroup's
// next tile (one gridDim.x further), which arrive while this one is scaled and
// stored.  A last step that K does not fill is taken as the last 128 bytes
// of the rows, with the activations already used set to zero; every address
// stays inside the rows.  Rows past the tile's end repeat its last row, and
// their results are not stored.
//
// At large sizes the bound is how fast the card runs the products under load:
// with codes of a normal distribution 8192^3 takes 409 us (2690 TOP/s; the
// library's int8 product reaches 2130 on them), with all codes zero 378, and
// products alone, fed from registers, reach 3700 to 4000 TOP/s.
// v_mfma_i32_32x32x32_i8 reaches 2900 to 3300 there.  LDS reads are free of bank
// conflicts and take a quarter of the time; fetching into the L2 ahead changes
// nothing but the run on zeros.  In middle sizes it is what one CU can have
// under way to memory, 50 to 65 bytes a ns, so that tiles are as large as still
// leaves one for each CU.
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

// Orders the instructions of one half step: a product first, then the loads,
// then the LDS reads, each behind a product, then the products left.
template <int LOADS, int READS, int PRODUCTS>
__device__ __forceinline__ void interleave() {
    if constexpr (LOADS + READS <= PRODUCTS) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        }
#pragma unroll
        for (int i = 0; i < READS; ++i) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, PRODUCTS - LOADS - READS, 0);
    }
}

template <int BM, int BW, int WM, int WN, int G, int D, bool SWI>
__global__ __launch_bounds__(WM * WN * G * 64, 2) void gemm_i8_block(Args p) {
    constexpr int FM = BM / WM / 16, FW = BW / WN / 16, BN = SWI ? BW / 2 : BW;
    constexpr int W = WM * WN;                                      // wavefronts of a group
    constexpr int LX = BM / 8 / W, LW = BW / 8 / W, LOADS = LX + LW; // load instructions of one of them and step
    constexpr int SLICE = (BM + BW) * BK, STAGE = G * SLICE, SCALES = BM + 2 * BN;
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & 63, all_waves = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wave = all_waves % W, group = all_waves / W;
    const int wm = wave / WN, wn = wave % WN;
    const int steps = (p.K + G * BK - 1) / (G * BK);
    // Every wavefront leaves the same sums of the groups' tiles in LDS, and
    // finds its own there whenever it looks for a tile: a load from memory would
    // wait for all of the ring's.
    Groups *groups = reinterpret_cast<Groups *>(lds + D * STAGE + 2 * SCALES * 4) + lane;
    const int bm = p.part >= kHalves ? 2 * BM : BM;
    *groups = groups_of(p, bm);
    const int tiles_m = tile_count(p, *groups), all = tiles_m * p.tiles_n, whole = whole_rounds(all);
    if (p.part >= kHalves && (all - whole <= kQuartersMost) != (p.part == kQuarters)) return;
    struct Place { Tile tl; int n0; };
    auto place = [&](int id, Place &at) {
        const int b = p.part >= kHalves ? whole + (id >> (p.part - kHalves + 1)) : id;
        int tm, tn;
        if (b >= (p.part == kWhole ? whole : all) || !tile_of(b, tiles_m, p.tiles_n, tm, tn)) return false;
        at.tl = find_tile(p, bm, *groups, tm);
        at.n0 = tn * BN;
        if (p.part >= kHalves) {
            const int down = (id & 1) * BM;
            at.tl.m0 += down;
            at.tl.rows = min(BM, at.tl.rows - down);
            if (p.part == kQuarters) at.n0 = (2 * tn + (id >> 1 & 1)) * BN;
        }
        return at.tl.rows > 0 && at.n0 < p.N;
    };
    int id = blockIdx.x;
    Place cur;
    if (!place(id, cur)) return;

    // In the largest tiles, what a tile's start and end compute from the lane is
    // computed anew each time.  Kept, it takes registers that the fragments
    // need, and the spills' reloads wait for all of the ring's loads: 8192 x
    // 8192 x 512 58 us so and 66.  128 x 256 tiles are 1.5% slower with it.
    auto lane_anew = [&]() {
        int l = tid & 63;
        if constexpr (FM * FW >= 32) asm volatile("" : "+v"(l));
        return l;
    };

    // Loads: this wavefront brings 1 / W of the rows of a and of w.
    // SWI: its weight rows are all gate or all up.
    const int8_t *wbase = SWI && wave * LW / 2 % FW >= FW / 2 ? p.w[1] : p.w[0];
    __amdgpu_buffer_rsrc_t ra, rw;
    uint32_t va[LX], vw[LW];
    auto aim = [&](const Place &at) {
        const int lane = lane_anew();
        const int rows = at.tl.rows, cols = min(BN, p.N - at.n0), chunk = ((lane & 7) ^ (lane >> 3)) << 4;
        ra = rsrc_of(p.a + (size_t)at.tl.m0 * p.K, (uint32_t)rows * p.K);
        rw = rsrc_of(wbase + ((size_t)at.tl.e * p.N + at.n0) * p.K, (uint32_t)cols * p.K);
#pragma unroll
        for (int i = 0; i < LX; ++i)
            va[i] = (uint32_t)min((wave * LX + i) * 8 + (lane >> 3), rows - 1) * p.K + chunk;
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            // Row r belongs to wavefront column c, its fragment j, row q of it.
            const int r = (wave * LW + i) * 8 + (lane >> 3), c = r / (16 * FW), j = r / 16 % FW, q = r & 15;
            const int n = SWI ? c * (8 * FW) + frag_row<FW / 2>(j % (FW / 2), q) : c * (16 * FW) + frag_row<FW>(j, q);
            vw[i] = (uint32_t)min(n, cols - 1) * p.K + chunk;
        }
    };
    auto load = [&](int slot, int t) {
        char *at = lds + slot * STAGE + group * SLICE + wave * 1024;
        const int koff = min((t * G + group) * BK, p.K - BK);
#pragma unroll
        for (int i = 0; i < LX; ++i) load16(ra, at + (wave * (LX - 1) + i) * 1024, va[i], koff);
#pragma unroll
        for (int i = 0; i < LW; ++i) load16(rw, at + (BM / 8 + wave * (LW - 1) + i) * 1024, vw[i], koff);
    };

    // Fragment reads: lane l takes row l % 16, chunk l / 16 (+ 4 in the
    // second half, which flips bit 6 of the swizzled address).
    const int fr = (lane & 15) * BK + (((lane >> 4) ^ (lane & 7)) << 4);
    const int xat = wm * (16 * FM) * BK, wat = (BM + wn * (16 * FW)) * BK;
    i32x4_t acc[FM][FW];
    i32x4_t x0[FM], w0[FW], x1[FM], w1[FW];
    auto read = [&](i32x4_t (&x)[FM], i32x4_t (&w)[FW], int slot, int f) {
        const char *at = lds + slot * STAGE + group * SLICE + f;
#pragma unroll
        for (int j = 0; j < FW; ++j) w[j] = *reinterpret_cast<const i32x4_t *>(at + wat + j * 16 * BK);
#pragma unroll
        for (int i = 0; i < FM; ++i) x[i] = *reinterpret_cast<const i32x4_t *>(at + xat + i * 16 * BK);
    };
    // Neighbours share an operand, and rows run back and forth so that the
    // turns do too: the matrix cores are bound by power at large sizes, and
    // this order draws 1% less than one that returns to column 0.
    auto products = [&](const i32x4_t (&x)[FM], const i32x4_t (&w)[FW]) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int q = 0; q < FW; ++q) {
                const int j = i & 1 ? FW - 1 - q : q;
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
            }
    };
    // Chunks of this group's last slice that others have used.
    const int used = max(0, ((steps - 1) * G + group + 1) * 8 - (p.K >> 4));
    auto drop = [&](i32x4_t (&x)[FM], int c) {
        if (c < used) {
#pragma unroll
            for (int i = 0; i < FM; ++i) x[i] = i32x4_t{0, 0, 0, 0};
        }
    };
    auto barrier = [&]() {       // and this wavefront's LDS reads are done
        __builtin_amdgcn_sched_barrier(0);
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
    };
    // The scales of a tile's rows and columns, and the bias, go behind the ring,
    // 64 of them a wavefront: fetched at the end, they would cost a trip to
    // memory there.
    float *scales = reinterpret_cast<float *>(lds + D * STAGE);
    const int most = BM + BN + (SWI || p.bias ? BN : 0);
    auto load_scales = [&](const Place &at, float *to) {
        const int lane = lane_anew();
        for (int q = all_waves * 64; q < most; q += W * G * 64) {
            const int i = q + lane - BM, col = at.n0 + (i & (BN - 1));
            const float *sw = i < BN ? p.sw[0] : SWI ? p.sw[1] : p.bias;
            const float *from = i < 0 ? p.sa + at.tl.m0 + min(q + lane, at.tl.rows - 1)
                                      : sw + (size_t)at.tl.e * p.N + min(col, p.N - 1);
            load4(from, to + q);
        }
    };
    auto after = [](int slot) { return slot + 1 == D ? 0 : slot + 1; };

    aim(cur);
    int side = 0;                // of the two places for scales
    load_scales(cur, scales);
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (d < steps) load(d, d);
    wait_batches<LOADS, D - 1>(steps - 1);
    barrier();
    for (int slot = 0;;) {
        read(x0, w0, slot, fr);
        if (steps == 1 && used) drop(x0, lane >> 4);
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FW; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
        int t = 0;
        for (; t + D < steps; ++t) {
            read(x1, w1, slot, fr ^ 64);
            products(x0, w0);
            interleave<0, FM + FW, FM * FW>();
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<(D - 2) * LOADS>();
            barrier();
            const int next = after(slot);
            load(slot, t + D);
            read(x0, w0, next, fr);
            products(x1, w1);
            interleave<LOADS, FM + FW, FM * FW>();
            __builtin_amdgcn_sched_barrier(0);
            slot = next;
        }
        // The last D steps load the next tile's first.
        Place nxt = cur;
        const bool more = G == 1 && steps >= D && place(id + (int)gridDim.x, nxt);
        if (more) aim(nxt);
        for (; t < steps; ++t) {
            const int next = after(slot);
            read(x1, w1, slot, fr ^ 64);
            if (t + 1 == steps && used) drop(x1, 4 + (lane >> 4));
            products(x0, w0);
            __builtin_amdgcn_sched_barrier(0);
            // Step t + 1, or the next tile's first, has come.
            if (more) wait_loads<(D - 2) * LOADS>();
            else wait_batches<LOADS, D - 2>(steps - t - 2);
            barrier();
            if (more) {
                if (t + D == steps) load_scales(nxt, scales + (side ^ 1) * SCALES);
                load(slot, t + D - steps);
            }
            if (t + 1 < steps) {
                read(x0, w0, next, fr);
                if (t + 2 == steps && used) drop(x0, lane >> 4);
            }
            products(x1, w1);
            __builtin_amdgcn_sched_barrier(0);
            slot = next;
        }
        constexpr int C = SWI ? 2 * FW : 4 * FW;      // consecutive columns of a lane
        const int lane = lane_anew();
        const int col = wn * (4 * C) + (lane >> 4) * C;
        const float *mine = scales + side * SCALES, *sw0 = mine + BM + col, *sw1 = sw0 + BN;
        if constexpr (G == 1) {
            float sa[FM];
#pragma unroll
            for (int i = 0; i < FM; ++i) sa[i] = mine[wm * (16 * FM) + i * 16 + (lane & 15)];
            finish<FM, C, SWI>(p, acc, cur.tl, sa, sw0, sw1, wm * (16 * FM), cur.n0 + col, lane);
        } else {
            // The groups' sums meet in the ring's place, and group g finishes
            // rows g, g + G, .. of the fragments.
            static_assert(G * W * FM * FW * 1024 <= D * STAGE, "the sums fit the ring");
            __syncthreads();
            i32x4_t *part = reinterpret_cast<i32x4_t *>(lds) + wave * (FM * FW * 64) + lane;
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FW; ++j) part[(group * W * FM * FW + i * FW + j) * 64] = acc[i][j];
            __syncthreads();
            for (int i = group; i < FM; i += G) {
                i32x4_t sum[1][FW] = {};
#pragma unroll
                for (int g = 0; g < G; ++g)
#pragma unroll
                    for (int j = 0; j < FW; ++j) sum[0][j] += part[(g * W * FM * FW + i * FW + j) * 64];
                const float sa[1] = {mine[wm * (16 * FM) + i * 16 + (lane & 15)]};
                finish<1, C, SWI>(p, sum, cur.tl, sa, sw0, sw1, wm * (16 * FM) + i * 16, cur.n0 + col, lane);
            }
            return;
        }
        if (!more) return;
        id += gridDim.x;
        cur = nxt;
        side ^= 1;
    }
}

// ---------------------------------------------------------------- few rows
//
// Tiles of 8 NX rows: what counts is the bytes in flight, and that every CU
// has its share of them.  A wavefront takes FN strips of 16 weight rows (of
// each matrix) and every KS-th unit of 128 bytes of K; KS wavefronts of a
// workgroup meet in LDS at the end.  Its units pass through a ring of D
// slots of its own in LDS, loaded straight from memory eight rows of 128
// bytes an instruction (a fragment's own order, 16 rows of 64 bytes, loads
// the same bytes at 3/4 of the rate or less), the next unit issued as soon
// as a slot has been read: no barrier, and D - 1 units in flight while one
// is multiplied.  Units past K repeat the row's last 16 bytes against
// activations of zero.  Up to a few hundred rows, where larger tiles leave
// CUs idle, many such tiles are faster although each reads all its operands:
// 64 x 2048 x 8192 takes 10.0 us in tiles of 32 rows, 21.7 in 64 x 64, 1024
// columns of 4096 5.0 and 9.3.
constexpr int kFewDepth = 2;

template <int NX, int FN, bool SWI, int W>
__global__ __launch_bounds__(W * 64) void gemm_i8_few(Args p, int ks_log2) {
    constexpr int FM = (NX + 1) / 2, BM = 8 * NX, MATS = SWI ? 2 : 1, FW = FN * MATS;
    constexpr int D = kFewDepth, LOADS = 2 * FW + NX;                   // load instructions of a unit
    constexpr int SLOT = (2 * FW + 2 * FM) * 1024;                      // whole fragments, the last may be half loaded
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int KS = 1 << ks_log2, ks = wave & (KS - 1);
    // Row tiles that read the same weights lie side by side on one XCD, so that
    // its L2 brings them once; others take the XCDs in turn.
    const Groups groups = groups_of(p, BM);
    int tm = (int)blockIdx.x / p.tiles_n, tn = (int)blockIdx.x - tm * p.tiles_n;
    if (p.share) {
        const int tiles_m = tile_count(p, groups), id = eighth_of(blockIdx.x, tiles_m * p.tiles_n);
        if (id < 0) return;
        tn = id / tiles_m;
        tm = id - tn * tiles_m;
    }
    const Tile tl = find_tile(p, BM, groups, tm);
    if (tl.rows <= 0) return;
    const int n0 = (tn * (W >> ks_log2) + (wave >> ks_log2)) * (16 * FN);
    const size_t mat = (size_t)tl.e * p.N;
    const int kc = p.K >> 4, units = (kc + 7) >> 3;
    const int g = lane >> 4, r = lane & 15;
    i32x4_t acc[FM][FW] = {};
    // Scales and bias of the lane's rows and columns, fetched before the ring's
    // loads: at the end they would cost a trip to memory.
    constexpr int C = 4 * FN;
    const int n = n0 + g * C;
    float sa[FM], sw[2][C];
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = p.sa[tl.m0 + min(i * 16 + r, tl.rows - 1)];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int at = min(n + c, p.N - 1);
        sw[0][c] = p.sw[0][mat + at];
        sw[1][c] = SWI ? p.sw[1][mat + at] : p.bias ? p.bias[at] : 0.f;
    }

    if (n0 < p.N) {
        char *ring = lds + wave * (D * SLOT);
        const int cols = min(16 * FN, p.N - n0);
        const __amdgpu_buffer_rsrc_t rx = rsrc_of(p.a + (size_t)tl.m0 * p.K, (uint32_t)tl.rows * p.K);
        __amdgpu_buffer_rsrc_t rw[MATS];
#pragma unroll
        for (int s = 0; s < MATS; ++s) rw[s] = rsrc_of(p.w[s] + (mat + n0) * p.K, (uint32_t)cols * p.K);
        uint32_t vx[NX], vw[2 * FN];
#pragma unroll
        for (int i = 0; i < NX; ++i) vx[i] = (uint32_t)min(i * 8 + (lane >> 3), tl.rows - 1) * p.K;
#pragma unroll
        for (int i = 0; i < 2 * FN; ++i) {
            const int q = (i & 1) * 8 + (lane >> 3);               // row of fragment i / 2
            vw[i] = (uint32_t)min(frag_row<FN>(i >> 1, q), cols - 1) * p.K;
        }
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
        };
        const int fr = r * BK + ((g ^ (r & 7)) << 4);
        auto products = [&](int slot, int u) {
            const char *at = ring + slot * SLOT;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const char *f = at + (h ? fr ^ 64 : fr);
                i32x4_t w[FW], x[FM];
#pragma unroll
                for (int j = 0; j < FW; ++j) w[j] = *reinterpret_cast<const i32x4_t *>(f + j * 2048);
#pragma unroll
                for (int i = 0; i < FM; ++i) x[i] = *reinterpret_cast<const i32x4_t *>(f + (FW + i) * 2048);
                if (u * 8 + 8 > kc && u * 8 + h * 4 + g >= kc) {
#pragma unroll
                    for (int i = 0; i < FM; ++i) x[i] = i32x4_t{0, 0, 0, 0};
                }
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FW; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j], x[i], acc[i][j], 0, 0, 0);
            }
        };
        int left = (units - ks + KS - 1) >> ks_log2, u = ks, slot = 0;      // this wavefront's units
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < left) load(d, ks + d * KS);
        for (; left > D; --left, u += KS) {
            wait_loads<(D - 1) * LOADS>();
            products(slot, u);
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");      // the slot has been read
            load(slot, u + D * KS);
            if (++slot == D) slot = 0;
        }
        for (; left > 0; --left, u += KS) {
            if (left == 2) wait_loads<LOADS>();
            else wait_loads<0>();
            products(slot, u);
            if (++slot == D) slot = 0;
        }
    }
    if (KS > 1) {
        // Every wavefront has read its ring: the partial sums take its place.
        __syncthreads();
        i32x4_t *part = reinterpret_cast<i32x4_t *>(lds) + lane;
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
    finish<FM, C, SWI>(p, acc, tl, sa, sw[0], sw[1], 0, n, lane);
}

constexpr int kMaxRows = 1 << 24;
constexpr int kMaxK = 131056;      // 16384 * 131056 < 2^31: the sum fits whatever the codes

bool elem_aligned(const void *y, int type) { return q4::aligned(y, type == I8_F32 ? 4 : 2); }

constexpr int64_t kMaxThreads = 0xFFFFFFFFll;      // of one launch

int64_t tiles_of(int64_t n, int tile) { return (n + tile - 1) / tile; }

// Tiles of bm rows that a call may need: every group may end inside one.
int64_t row_tiles(const Args &p, int bm) {
    return p.offsets ? p.M / bm + std::min(p.E, p.M) : tiles_of(p.M, bm);
}

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
// of bm rows.  As many share K as it takes for 1536 wavefronts, 6 for each CU,
// while each has a unit: at 8 rows, 4096 -> 14336, 2 of them take 11.8 us and
// 8 take 13.6; at 24 rows, 14336 -> 4096, 8 take 12.0 and 2 take 26.1.
// Workgroups of 4 are spread more evenly than of 8: at 31 rows, 3840 -> 8512,
// 10.5 and 12.9 us; but 8 are as good where they come to no more than one a
// CU, and then 14.1 against 14.6 us at 16 rows, 4096 -> 14336.
struct Split { int64_t tiles, strips; int log2, waves; };
Split split_of(const Args &p, int bm, int cols, int most) {
    Split s = {row_tiles(p, bm), tiles_of(p.N, cols), 0, most};
    const int64_t units = tiles_of(p.K, BK);
    while ((2 << s.log2) <= most && (units >> s.log2) > 1 && (s.tiles * s.strips) << s.log2 < 1536) ++s.log2;
    const int64_t eights = most == 8 ? s.tiles * tiles_of(s.strips, 8 >> s.log2) : 0;
    if (s.log2 < 3 && (eights < kCUs / 2 || eights > kCUs)) s.waves = 4;
    return s;
}

template <int NX, int FN, bool SWI, int W>
int launch_few(Args p, const Split &s, const Target &to) {
    constexpr int FM = (NX + 1) / 2, FW = SWI ? 2 * FN : FN, kLds = W * kFewDepth * (2 * FW + 2 * FM) * 1024;
    // Weights of more than a quarter of the 256 MB cache are loaded
    // non-temporally.  Cycling 2 GB of matrices, one row through 4096 -> 14336
    // (59 MB) takes 12.6 us so and 14.2 without, the SwiGLU of two such 24.0
    // and 26.3; but a small model's matrices can be found in the cache, and
    // three of 59 MB in turn take 11.8 us so and 10.7 without.  Rows that do not
    // start on a 64-byte border share lines with their neighbours, which the
    // caches have to keep: 8 rows, 2 x 4080 -> 14336, 29.3 us so, 27.8 without.
    // Weights that several row tiles read are to be kept, too.
    p.share = p.offsets ? p.M > (int64_t)p.E * (8 * NX) : s.tiles > 1;
    p.once = p.K % 64 == 0 && !p.share && (int64_t)(SWI ? 2 : 1) * p.E * p.N * p.K > (int64_t)64 << 20;
    p.tiles_m = (int)s.tiles;
    p.tiles_n = (int)tiles_of(s.strips, W >> s.log2);
    const int64_t grid = s.tiles * p.tiles_n;
    if (grid * (W * 64) > kMaxThreads) return Q4_EINVAL;
    if (to.report) return planned(to, 8 * NX, (W >> s.log2) * 16 * FN, grid, W * 64);
    gemm_i8_few<NX, FN, SWI, W><<<(unsigned)grid, W * 64, kLds, to.stream>>>(p, s.log2);
    return q4::launch_status();
}

template <int NX, int FN, bool SWI, int MOST = 8>
int launch_few(const Args &p, const Target &to) {
    const Split s = split_of(p, 8 * NX, 16 * FN, MOST);
    if constexpr (MOST == 8)
        if (s.waves == 8) return launch_few<NX, FN, SWI, 8>(p, s, to);
    return launch_few<NX, FN, SWI, 4>(p, s, to);
}

template <int BM, int BW, int WM, int WN, int G, int D, bool SWI>
int launch_block(Args p, const Target &to) {
    constexpr int kBN = SWI ? BW / 2 : BW;
    constexpr int kLds = G * D * (BM + BW) * BK + 2 * (BM + 2 * kBN) * 4 + 64 * (int)sizeof(Groups);
    constexpr int kThreads = WM * WN * G * 64;
    p.tiles_m = (int)row_tiles(p, (p.part >= kHalves ? 2 : 1) * BM);
    p.tiles_n = (int)tiles_of(p.N, (p.part == kQuarters ? 2 : 1) * kBN);
    int64_t grid = (int64_t)p.tiles_m * p.tiles_n;
    if (grid > 1 << 30) return Q4_EINVAL;
    if (p.part == kWhole) grid = p.offsets ? grid : whole_rounds((int)grid);
    if (p.part >= kHalves) {
        const int most = p.part == kHalves ? kRestMost : kQuartersMost;
        grid = (p.offsets ? std::min<int64_t>(grid, most) : grid - whole_rounds((int)grid)) << (p.part - kHalves + 1);
    }
    // Workgroups that stay and go through the tiles, each loading its next one
    // while it finishes the last: 8192 x 8192 x 512 takes 58 us so, 66 with a
    // workgroup for each tile, x 1024 87 and 95; 8000 rows over 64 experts with
    // SwiGLU, K = 1024, 108 and 122.  At long K tiles change rarely, and dealing
    // them as CUs come free is better where they differ: 527 against 539 us
    // for 8190 rows over 8 experts, K = 14336.
    const int64_t steps = tiles_of(p.K, BK);
    if (G == 1 && p.part < kHalves && steps >= D && steps <= 64)
        grid = std::min<int64_t>(grid, kCUs * (160 * 1024 / kLds));
    else if (grid * kThreads > kMaxThreads) return Q4_EINVAL;
    if (to.report) return planned(to, BM, kBN, grid, kThreads);
    gemm_i8_block<BM, BW, WM, WN, G, D, SWI><<<(unsigned)grid, kThreads, kLds, to.stream>>>(p);
    return q4::launch_status();
}

enum Kernel { kFew8, kFew16, kFew32, kFew32x32, kFew64, kTile64, kTile128, kTileWide, kTile256, kTileDeep, kKernels };

// The kernel for a call's sizes.  Up to 8 rows the weights' stream decides.
// Above that, each kernel's time is estimated, with constants fitted to
// measured shapes (up to six matrices in turn, so that small ones came from the
// cache): the tiles to 320 (33 to 8192 rows, N 64 to 14336, K 256 to 14336, one
// matrix and two), in us a tile, us a step, and how far more tiles than CUs
// stretch it; tiles that have a CU to themselves come in whole rounds.
// The kernels of few rows to 1070 (9 to 3000 rows): us a unit of a wavefront
// alone and for each of the CU's, and, as they read weights past the L2 again
// for every row tile, us a MB of weights.  The choice is on average 1.2%
// behind the best of the nine there, but now and then far more: 512 x 4096 x
// 14336 goes to 128 x 128, 68.0 us, and takes 54.9 in 64 x 128.  64 x 4096 x 14336 takes 21.2 us in tiles
// of 32 x 32, 26.4 in 32 x 16, 28.4 in 64 x 32, 36.7 in 64 x 64; at 128 rows
// these are 32.9, 41.3, 26.8 and 36.3.
// Groups go by their average rows, their sizes being known to the GPU alone.
// Measured with uneven groups, as a router makes them, over 64 experts of 2 x
// 2816 x 1024, at 4, 32 and 128 rows on average: 16 rows a tile 49, 97, 248 us,
// 64 rows 63, 87, 138, 128 x 256 64, 91, 116, 256 rows 87, 116, 153.  Over 8
// experts of 4096 x 14336, at 256 rows: 128 x 256 226 us, 256 rows 187 (135 and
// 154 where all have 256); of 2 x 4096 x 4096, at 512 rows 168 and 165, at 2048
// 558 and 501.  Where that leaves CUs idle, the estimates decide, a group ending
// inside a tile half way: 769 rows over 3 experts of 643 x 3648 take 11.7 us in
// tiles of 64 x 64, 30.1 in 128 x 256.  Over 220
// calls (2 to 128 experts, 0.5 to 300 rows each) the choice is on average 2.7%
// behind the best.
Kernel choose(const Args &p, int mats) {
    const int64_t steps = tiles_of(p.K, BK), groups = p.offsets ? std::min(p.E, p.M) : 0;
    const int64_t rows = p.offsets ? tiles_of(p.M, p.E) : p.M;
    if (rows <= (p.offsets ? 2 : 8)) return kFew8;
    if ((p.offsets && rows <= 8) || (p.K < BK && rows <= 16)) return kFew16;
    if (p.K < BK) return kFew32;
    auto row_tiles_likely = [&](int bm) { return p.offsets ? p.M / bm + (groups + 1) / 2 : tiles_of(p.M, bm); };
    auto tiles = [&](int bm, int bw) { return row_tiles_likely(bm) * tiles_of(p.N, bw / mats); };
    if (p.offsets) {
        const int many = p.K < 8192 ? 1536 : 256;
        if (rows <= 48 && tiles(64, 128) >= kCUs) return kTile64;
        if (rows > 48 && rows < many && tiles(128, 256) >= 2 * kCUs) return kTileWide;
        if (rows >= many && tiles(256, 256) >= kCUs) return kTile256;
    }
    auto rounds = [&](int bm, int bw) { return (double)((tiles(bm, bw) + kCUs - 1) / kCUs); };
    // Tiles a CU, 1 where there are fewer, and the time of one alone or of one among others.
    auto each = [&](int64_t t, double one, double many) { return t <= kCUs ? one : (double)t / kCUs * many; };
    auto few = [&](int bm, int cols, int most, double start, double unit, double shared, double first) {
        const Split s = split_of(p, bm, cols, most);
        const int64_t tm = row_tiles_likely(bm), wgs = tm * tiles_of(s.strips, s.waves >> s.log2);
        const double a_unit = std::max(unit, shared * (double)(tiles_of(wgs, kCUs) * s.waves));
        const double mb = p.offsets ? 0. : (double)mats * p.N * p.K * 1e-6;
        return std::max(start + a_unit * (first + (double)tiles_of(steps, 1 << s.log2)),
                        0.32 * mb * (1. + 0.4 * (double)(tm - 1)) - 1.5);
    };
    const bool two = mats == 2;
    double cost[kKernels];
    cost[kFew8] = few(8, 16, 8, -0.5, 0.15, two ? 0.050 : 0.031, 0.81);
    cost[kFew16] = few(16, 16, 8, -0.7, 0.24, two ? 0.099 : 0.043, 0.5);
    cost[kFew32] = few(32, 16, 8, -0.4, 0.30, two ? 0.154 : 0.11, 0.74);
    cost[kFew32x32] = few(32, 32, 8, -0.23, 0.33, 0.14, 0.56);       // with one matrix
    cost[kFew64] = few(64, two ? 16 : 32, 4, 0.74, 0.63, 0.25, 0.75);
    cost[kTileDeep] = each(tiles(64, 64), 0.67 + steps * 0.38, 0.78 + steps * 0.40);
    cost[kTile64] = std::max(1.0, (double)tiles(64, 128) / kCUs * 1.2) * (0.67 + steps * 0.42);
    cost[kTile128] = each(tiles(128, 128), 2.25 + steps * 0.46, 0.63 + steps * 0.78);
    cost[kTileWide] = rounds(128, 256) * (6.54 + steps * 0.75);
    const int64_t t256 = tiles(256, 256), left = t256 % kCUs;
    const double divided = left > kQuartersMost ? 6.54 + steps * 0.75 : left ? 2.25 + steps * 0.46 : 0.;
    cost[kTile256] = t256 < kCUs || left > kRestMost ? rounds(256, 256) * (8.0 + steps * 1.33)
                                                     : (double)(t256 / kCUs) * (8.0 + steps * 1.33) + divided;
    // Of few rows, groups take 16 or 32 a tile: at 8, most are read in several.
    Kernel best = kFew16;
    for (Kernel k : {kFew32, kTileDeep, kTile64, kTile128, kTileWide, kTile256})
        if (cost[k] < cost[best]) best = k;
    if (p.offsets) return best;
    for (Kernel k : {kFew8, kFew32x32, kFew64})
        if (cost[k] < cost[best] && !(two && k == kFew32x32)) best = k;
    return best;
}

template <bool SWI>
int launch(const Args &p, Kernel k, const Target &to) {
    // Two workgroups share a CU with a ring of two stages; where there is only
    // one for each CU, it takes four: 1024 x 4096 x 4096 in 24.7 against 33.6
    // us, but 2048 x 4096 x 1024 in 16.8 against 14.5 (tiles of 128 x 128).
    auto alone = [&](int bm, int bw) { return row_tiles(p, bm) * tiles_of(p.N, SWI ? bw / 2 : bw) <= kCUs; };
    // Two matrices halve the columns of a lane's run: four rows of wavefronts
    // then store whole lines.  4096 x 2 x 14336 x 1024 takes 134 us so, 154 with
    // two rows of four; one matrix is faster in two (8192 x 14336 x 4096 404
    // and 460: the fragments of four spill).
    constexpr int kM = SWI ? 4 : 2, kN = SWI ? 2 : 4;
    switch (k) {
    case kFew8: return launch_few<1, 1, SWI>(p, to);
    case kFew16: return launch_few<2, 1, SWI>(p, to);
    case kFew32: return launch_few<4, 1, SWI>(p, to);
    case kFew32x32: return launch_few<4, SWI ? 1 : 2, SWI>(p, to);
    case kFew64: return launch_few<8, SWI ? 1 : 2, SWI, 4>(p, to);
    case kTile64: return launch_block<64, 128, 2, 4, 1, 3, SWI>(p, to);
    case kTileDeep:
        if (alone(64, 64)) return launch_block<64, 64, 2, 2, 2, 4, SWI>(p, to);
        return launch_block<64, 64, 2, 2, 2, 2, SWI>(p, to);
    case kTile128:
        if (alone(128, 128)) return launch_block<128, 128, kM, kN, 1, 4, SWI>(p, to);
        return launch_block<128, 128, kM, kN, 1, 2, SWI>(p, to);
    case kTileWide: return launch_block<128, 256, kM, kN, 1, 3, SWI>(p, to);
    default: {
        // Whole rounds, then the tiles that are left, divided.
        Args q = p;
        const int64_t all = row_tiles(p, 256) * tiles_of(p.N, SWI ? 128 : 256), left = all % kCUs;
        if (all >= kCUs && (p.offsets || (left && left <= kRestMost))) q.part = kWhole;
        if (int st = launch_block<256, 256, kM, kN, 1, 2, SWI>(q, to)) return st;
        if (q.part == kAll) return Q4_OK;
        if (p.offsets || left > kQuartersMost) {
            q.part = kHalves;
            if (int st = launch_block<128, 256, kM, kN, 1, 3, SWI>(q, to)) return st;
        }
        if (!p.offsets && left > kQuartersMost) return Q4_OK;
        q.part = kQuarters;
        return launch_block<128, 128, kM, kN, 1, 4, SWI>(q, to);
    }
    }
}

int check_sizes(const Args &p) {
    if (p.M < 0 || p.M > kMaxRows || p.N < 0 || p.N > kMaxRows || p.K < 16 || p.K % 16 || p.K > kMaxK)
        return Q4_EINVAL;
    if (tiles_of(p.M, 16) * tiles_of(p.N, 16) > 0x7FFFFFFFll) return Q4_EINVAL;
    if (p.E < 1 || p.E > 65536 || (int64_t)p.E * p.N > 0x7FFFFFFFll) return Q4_EINVAL;
    return Q4_OK;
}

int run(const Args &p, int mats, hipStream_t stream) {
    if (int st = check_sizes(p)) return st;
    if (p.y_type != I8_F32 && p.y_type != I8_F16 && p.y_type != I8_BF16) return Q4_EINVAL;
    if (p.M == 0 || p.N == 0) return Q4_OK;
    if (!p.a || !p.sa || !p.w[0] || !p.sw[0] || !p.y || (mats == 2 && (!p.w[1] || !p.sw[1]))) return Q4_ENULL;
    if (!q4::aligned(p.a, 16) || !q4::aligned(p.w[0], 16) || !q4::aligned(p.sa, 4) || !q4::aligned(p.sw[0], 4) ||
        !q4::aligned(p.bias, 4) || !q4::aligned(p.offsets, 4) || !elem_aligned(p.y, p.y_type))
        return Q4_EALIGN;
    if (mats == 2 && (!q4::aligned(p.w[1], 16) || !q4::aligned(p.sw[1], 4))) return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    const Kernel k = choose(p, mats);
    const Target to = {stream, nullptr};
    return mats == 2 ? launch<true>(p, k, to) : launch<false>(p, k, to);
}

}  // namespace

extern "C" int gemm_i8(const int8_t *a, const float *a_scales, const int8_t *w, const float *w_scales,
                       const float *bias, void *y, int y_type, int M, int N, int K, void *stream) {
    return run({a, a_scales, {w, nullptr}, {w_scales, nullptr}, bias, nullptr, y,
                y_type, M, N, K, 1, 0, 0, kAll, false, false},
               1, static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_swiglu(const int8_t *a, const float *a_scales, const int8_t *w_gate,
                              const float *scales_gate, const int8_t *w_up, const float *scales_up, void *y,
                              int y_type, int M, int N, int K, void *stream) {
    return run({a, a_scales, {w_gate, w_up}, {scales_gate, scales_up}, nullptr, nullptr, y,
                y_type, M, N, K, 1, 0, 0, kAll, false, false},
               2, static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_grouped(const int8_t *a, const float *a_scales, const int8_t *w, const float *w_scales,
                               const int32_t *offsets, void *y, int y_type, int M, int E, int N, int K,
                               void *stream) {
    if (!offsets && M > 0 && N > 0) return Q4_ENULL;
    return run({a, a_scales, {w, nullptr}, {w_scales, nullptr}, nullptr, offsets, y,
                y_type, M, N, K, E, 0, 0, kAll, false, false},
               1, static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_grouped_swiglu(const int8_t *a, const float *a_scales, const int8_t *w_gate,
                                      const float *scales_gate, const int8_t *w_up, const float *scales_up,
                                      const int32_t *offsets, void *y, int y_type, int M, int E, int N, int K,
                                      void *stream) {
    if (!offsets && M > 0 && N > 0) return Q4_ENULL;
    return run({a, a_scales, {w_gate, w_up}, {scales_gate, scales_up}, nullptr, offsets, y,
                y_type, M, N, K, E, 0, 0, kAll, false, false},
               2, static_cast<hipStream_t>(stream));
}

extern "C" int gemm_i8_geometry(int matrices, int M, int E, int N, int K, int *tile_rows, int *tile_cols, int *grid,
                                int *block) {
    static const int32_t kGrouped = 0;             // stands for offsets, never read
    Args p = {};
    p.M = M, p.N = N, p.K = K, p.E = E ? E : 1;
    p.offsets = E ? &kGrouped : nullptr;
    if (matrices != 1 && matrices != 2) return Q4_EINVAL;
    if (int st = check_sizes(p)) return st;
    Report r = {};
    if (M > 0 && N > 0) {
        const Kernel k = choose(p, matrices);
        const Target to = {nullptr, &r};
        if (int st = matrices == 2 ? launch<true>(p, k, to) : launch<false>(p, k, to)) return st;
    }
    if (tile_rows) *tile_rows = r.rows;
    if (tile_cols) *tile_cols = r.cols;
    if (grid) *grid = (int)r.grid;      // at most 2^30 and two parts of 256
    if (block) *block = r.block;
    return Q4_OK;
}
