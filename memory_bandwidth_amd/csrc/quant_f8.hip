// quant_f8.hip -- matrices to e4m3 codes with a scale for each block of 128,
// for gfx950 (see q4f8.h):
//
//     s = max(rn(max |x| / 448), 2^-126),  c = the e4m3 value nearest to x / s
//
// over 1 x 128 blocks (rows) or 128 x 128 ones.  Both are bound by memory: x is
// read once, held in registers between the largest magnitude and the codes.
// Sixteen lanes take the 128 values of a row's block, eight each, so that a
// lane's codes are one 8-byte store and the maximum needs four steps of DPP.
#include "q4_common.h"
#include "q4f8.h"

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct F32 {};
struct F16 {};
struct BF16 {};

// Eight consecutive values as they are loaded, and in fp32 (each conversion is exact).
template <typename T> struct Eight;
template <> struct Eight<F32> {
    u32x4_t r[2];
    __device__ void load(const char *p) {
        r[0] = reinterpret_cast<const u32x4_t *>(p)[0];
        r[1] = reinterpret_cast<const u32x4_t *>(p)[1];
    }
    __device__ void zero() { r[0] = r[1] = u32x4_t{0, 0, 0, 0}; }
    __device__ float get(int i) const {
        const uint32_t b = r[i >> 2][i & 3];
        return __builtin_bit_cast(float, b);
    }
    static constexpr int size = 4;
};
template <> struct Eight<F16> {
    u32x4_t r;
    __device__ void load(const char *p) { r = *reinterpret_cast<const u32x4_t *>(p); }
    __device__ void zero() { r = u32x4_t{0, 0, 0, 0}; }
    __device__ float get(int i) const {
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(r[i >> 1] >> (16 * (i & 1))));
    }
    static constexpr int size = 2;
};
template <> struct Eight<BF16> {
    u32x4_t r;
    __device__ void load(const char *p) { r = *reinterpret_cast<const u32x4_t *>(p); }
    __device__ void zero() { r = u32x4_t{0, 0, 0, 0}; }
    __device__ float get(int i) const {
        return __builtin_bit_cast(float, i & 1 ? r[i >> 1] & 0xFFFF0000u : r[i >> 1] << 16);
    }
    static constexpr int size = 2;
};

// Magnitudes are compared as their bit patterns, which order like the values
// and put Inf and NaN above all of them.
constexpr uint32_t kInfBits = 0x7F800000u;

template <typename T>
__device__ __forceinline__ uint32_t magnitude(const Eight<T> &x, uint32_t most) {
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, __builtin_bit_cast(uint32_t, x.get(i)) & 0x7FFFFFFFu);
    return most;
}

// The largest over 16 consecutive lanes, in all of them: partners 1 and 2 lanes
// away, then the mirrored half row and row.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, true));      // quad_perm 1 0 3 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, true));      // quad_perm 2 3 0 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, true));     // row_half_mirror
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, true));  // row_mirror
}

// The scale of a block; one that is not finite is divided by 1 and its codes
// are not used.
struct Scale { bool finite; float s, inv; };
__device__ __forceinline__ Scale scale_of(uint32_t most) {
    Scale c;
    c.finite = most < kInfBits;
    c.s = c.finite ? __builtin_fmaxf(__builtin_bit_cast(float, most) / 448.f, 0x1p-126f) : 1.f;
    c.inv = 1.f / c.s;
    return c;
}

// Codes of eight values.  q = x inv is within 2^-22.9 of the real quotient, and
// v_cvt_pk_fp8_f32 rounds q to the nearest code, ties to even: the code is right
// unless q and the quotient lie on two sides of a border between two codes, or
// one of them on it.  A border has at most 5 bits, so that its fp32 pattern ends
// in 19 zeros, and q is then within 4 of such a pattern (as are codes
// themselves, to no harm).  There (in 2^-16 of all values, and for zeros) the
// sign of x - border s decides, which doubles give exactly: the product has
// at most 29 bits.
template <typename T>
__device__ __forceinline__ u32x2_t codes8(const Eight<T> &x, const Scale &c) {
    float q[8];
    uint32_t least = ~0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        q[i] = x.get(i) * c.inv;
        least = min(least, (__builtin_bit_cast(uint32_t, q[i]) + 4u) << 13);
    }
    if (least <= 8u << 13) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __builtin_bit_cast(uint32_t, q[i]);
            if ((b + 4u) << 13 > 8u << 13) continue;
            const uint32_t border = (b + 4u) & ~0x7FFFFu;
            const float v = x.get(i), t = __builtin_bit_cast(float, border);
            const double over = ((double)v - (double)t * (double)c.s) * (t < 0.f ? -1.0 : 1.0);
            // Away from zero, towards it, or on the border.
            q[i] = __builtin_bit_cast(float, over > 0.0 ? border + 16u : over < 0.0 && t != 0.f ? border - 16u : border);
        }
    }
    u32x2_t w;
    int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    int hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[4], q[5], 0, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(q[6], q[7], hi, true);
    w[0] = c.finite ? (uint32_t)lo : 0u;
    w[1] = c.finite ? (uint32_t)hi : 0u;
    return w;
}

// 1 x 128 blocks, one for a team of 16 lanes.  A workgroup's 16 teams take one block
// of 2^rows_log2 rows, or several of fewer, so that with 16 rows the scales of a
// block are one run (stride_m = 1).  4099 rows of 14336 floats take 45.9 us, 6.4
// TB/s in and out; with two blocks a team 49.2, with four 52.5: more of them are
// on their way to memory with more, smaller wavefronts.
constexpr int kTeams = 16;
constexpr int64_t kMaxThreads = 0xFFFFFFFFll;      // of one launch

template <typename T>
__global__ __launch_bounds__(256) void quant_rows(const char *__restrict__ x, uint8_t *__restrict__ codes,
                                                  float *__restrict__ scales, int64_t stride_m, int64_t stride_k,
                                                  int M, int K, int rows_log2, int strips) {
    const int team = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int tile = (int)blockIdx.x / strips, strip = (int)blockIdx.x - tile * strips;
    const int m = (tile << rows_log2) + (team & ((1 << rows_log2) - 1));
    const int b = strip * (kTeams >> rows_log2) + (team >> rows_log2), k = b * 128 + lane * 8;
    if (m >= M || b * 128 >= K) return;
    const size_t at = (size_t)m * K + k;
    Eight<T> v;
    if (k < K) v.load(x + at * Eight<T>::size);
    else v.zero();
    const Scale c = scale_of(max16(magnitude(v, 0u)));
    if (lane == 0) scales[m * stride_m + b * stride_k] = c.finite ? c.s : __builtin_nanf("");
    if (k < K) *reinterpret_cast<u32x2_t *>(codes + at) = codes8(v, c);
}

template <typename T>
int launch_rows(const char *x, uint8_t *codes, float *scales, int64_t sm, int64_t sk, int M, int K, hipStream_t s) {
    int rows_log2 = 0;
    while (rows_log2 < 4 && (1 << rows_log2) < M) ++rows_log2;
    const int blocks = kTeams >> rows_log2, strips = ((K + 127) / 128 + blocks - 1) / blocks;
    const int64_t grid = (int64_t)((M + (1 << rows_log2) - 1) >> rows_log2) * strips;
    if (grid * 256 > kMaxThreads) return Q4_EINVAL;
    quant_rows<T><<<(unsigned)grid, 256, 0, s>>>(x, codes, scales, sm, sk, M, K, rows_log2, strips);
    return q4::launch_status();
}

// 128 x 128 blocks, one a workgroup.  A team of 16 lanes takes four rows, a lane
// a piece of 4 x 8 of the block.  For the transposed codes it turns the piece
// in registers, and the pieces meet in LDS: column c is 128 bytes in 32 pieces of
// four rows, piece p at slot p ^ 2 (c / 8), so that the lanes of a store (16
// different c / 8) spread over the banks; then every wavefront stores whole
// lines of eight columns.
//
// Byte i of row j of the piece to byte j of column i.
__device__ __forceinline__ void turn(const u32x2_t (&w)[4], uint32_t (&t)[8]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const uint32_t a = __builtin_amdgcn_perm(w[1][c], w[0][c], 0x05010400u);
        const uint32_t b = __builtin_amdgcn_perm(w[3][c], w[2][c], 0x05010400u);
        const uint32_t d = __builtin_amdgcn_perm(w[1][c], w[0][c], 0x07030602u);
        const uint32_t e = __builtin_amdgcn_perm(w[3][c], w[2][c], 0x07030602u);
        t[4 * c] = __builtin_amdgcn_perm(b, a, 0x05040100u);
        t[4 * c + 1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
        t[4 * c + 2] = __builtin_amdgcn_perm(e, d, 0x05040100u);
        t[4 * c + 3] = __builtin_amdgcn_perm(e, d, 0x07060302u);
    }
}

template <typename T>
__global__ __launch_bounds__(512) void quant_blocks(const char *__restrict__ x, uint8_t *__restrict__ codes,
                                                    float *__restrict__ scales, uint8_t *__restrict__ codes_t,
                                                    float *__restrict__ scales_t, int R, int C, int RB, int CB) {
    __shared__ uint32_t part[8];
    __shared__ __align__(16) uint32_t turned[128 * 32];
    const int tid = threadIdx.x, team = tid >> 4, lane = tid & 15;
    const int rb = (int)blockIdx.x / CB, cb = (int)blockIdx.x - rb * CB;
    const int r0 = rb * 128 + team * 4, c0 = cb * 128 + lane * 8;
    Eight<T> v[4];
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (r0 + j < R && c0 < C) v[j].load(x + ((size_t)(r0 + j) * C + c0) * Eight<T>::size);
        else v[j].zero();
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) most = magnitude(v[j], most);
    most = max16(most);
    most = max(most, (uint32_t)__shfl_xor((int)most, 16));
    most = max(most, (uint32_t)__shfl_xor((int)most, 32));
    if ((tid & 63) == 0) part[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) most = max(most, part[i]);
    const Scale c = scale_of(most);
    if (tid == 0) {
        const float s = c.finite ? c.s : __builtin_nanf("");
        if (codes) scales[(size_t)rb * CB + cb] = s;
        if (codes_t) scales_t[(size_t)cb * RB + rb] = s;
    }
    u32x2_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        w[j] = codes8(v[j], c);
        if (codes && r0 + j < R && c0 < C) *reinterpret_cast<u32x2_t *>(codes + (size_t)(r0 + j) * C + c0) = w[j];
    }
    if (!codes_t) return;
    uint32_t t[8];
    turn(w, t);
#pragma unroll
    for (int i = 0; i < 8; ++i) turned[(lane * 8 + i) * 32 + (team ^ (2 * lane))] = t[i];
    __syncthreads();
    const int R16 = (R + 15) & ~15, q = tid & 7;           // 16 rows from 16 q on
    if (rb * 128 + q * 16 >= R16) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int col = i * 64 + (tid >> 3), l = col >> 3;
        if (cb * 128 + col >= C) return;
        // Pieces 4 q .. at 4 (q ^ l / 2) .., with odd l the second pair first.
        const u32x4_t four = *reinterpret_cast<const u32x4_t *>(&turned[col * 32 + 4 * (q ^ (l >> 1))]);
        const u32x4_t out = l & 1 ? u32x4_t{four[2], four[3], four[0], four[1]} : four;
        *reinterpret_cast<u32x4_t *>(codes_t + (size_t)(cb * 128 + col) * R16 + rb * 128 + q * 16) = out;
    }
}

bool type_ok(int t) { return t == I8_F32 || t == I8_F16 || t == I8_BF16; }

}  // namespace

extern "C" int quant_f8(const void *x, int x_type, uint8_t *codes, float *scales, int64_t stride_m, int64_t stride_k,
                        int M, int K, void *stream) {
    if (M < 0 || M >= (1 << 22) || K < 16 || K % 16 || K > 131056 || !type_ok(x_type)) return Q4_EINVAL;
    if (stride_m < 0 || stride_m > (1 << 20) || stride_k < 0 || stride_k > (1ll << 31)) return Q4_EINVAL;
    // Each scale has a place of its own: runs along one dimension end before the next begins.
    const int64_t end_m = M > 0 ? (M - 1) * stride_m : 0, end_k = ((K + 127) / 128 - 1) * stride_k;
    const bool several_m = M > 1, several_k = K > 128;
    if ((several_m && stride_m < 1) || (several_k && stride_k < 1) ||
        (several_m && several_k && stride_k <= end_m && stride_m <= end_k))
        return Q4_EINVAL;
    if (M == 0) return Q4_OK;
    if (!x || !codes || !scales) return Q4_ENULL;
    if (!q4::aligned(x, 16) || !q4::aligned(codes, 16) || !q4::aligned(scales, 4)) return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    const auto *xb = static_cast<const char *>(x);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (x_type == I8_F32) return launch_rows<F32>(xb, codes, scales, stride_m, stride_k, M, K, s);
    if (x_type == I8_F16) return launch_rows<F16>(xb, codes, scales, stride_m, stride_k, M, K, s);
    return launch_rows<BF16>(xb, codes, scales, stride_m, stride_k, M, K, s);
}

extern "C" int quant_f8_block(const void *x, int x_type, uint8_t *codes, float *scales, uint8_t *codes_t,
                              float *scales_t, int R, int C, void *stream) {
    if (R < 0 || R >= (1 << 22) || C < 16 || C % 16 || C > 131056 || !type_ok(x_type)) return Q4_EINVAL;
    if (R == 0) return Q4_OK;
    if (!x || !codes != !scales || !codes_t != !scales_t || (!codes && !codes_t)) return Q4_ENULL;
    if (!q4::aligned(x, 16) || !q4::aligned(codes, 16) || !q4::aligned(scales, 4) || !q4::aligned(codes_t, 16) ||
        !q4::aligned(scales_t, 4))
        return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    const auto *xb = static_cast<const char *>(x);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const int RB = (R + 127) / 128, CB = (C + 127) / 128, grid = RB * CB;
    if ((int64_t)grid * 512 > kMaxThreads) return Q4_EINVAL;
    if (x_type == I8_F32) quant_blocks<F32><<<grid, 512, 0, s>>>(xb, codes, scales, codes_t, scales_t, R, C, RB, CB);
    else if (x_type == I8_F16) quant_blocks<F16><<<grid, 512, 0, s>>>(xb, codes, scales, codes_t, scales_t, R, C, RB, CB);
    else quant_blocks<BF16><<<grid, 512, 0, s>>>(xb, codes, scales, codes_t, scales_t, R, C, RB, CB);
    return q4::launch_status();
}
