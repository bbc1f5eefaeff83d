// quant_i8.hip -- rows of activations to 8-bit codes with one scale each, for
// gfx950 (see q4i8.h):
//
//     s[m] = max(rn(max_k |x[m, k]| / 127), 2^-126),  c[m, k] = nearest(x[m, k] / s[m])
//
// The operator is bound by memory.  T threads take a row and hold it in
// registers between the two passes over it (the largest magnitude, then the
// codes), 16-byte vectors NV to a thread; only rows past 8 vectors for each
// of 1024 threads are read twice.  4099 rows of 14336 floats take 49 us, 5.95
// TB/s in and out; reading every row twice took 93.
#include "q4_common.h"
#include "q4i8.h"

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

struct F32 {};
struct F16 {};
struct BF16 {};

// Values of one 16-byte load, in fp32 (each conversion is exact).
template <typename T> struct Vec;
template <> struct Vec<F32> {
    static constexpr int n = 4;
    __device__ static void get(u32x4_t r, float *v) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = r[i];       // bit_cast of the element itself would read element 0
            v[i] = __builtin_bit_cast(float, b);
        }
    }
};
template <> struct Vec<F16> {
    static constexpr int n = 8;
    __device__ static void get(u32x4_t r, float *v) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)(r[i / 2] >> (16 * (i % 2))));
    }
};
template <> struct Vec<BF16> {
    static constexpr int n = 8;
    __device__ static void get(u32x4_t r, float *v) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = __builtin_bit_cast(float, i % 2 ? r[i / 2] & 0xFFFF0000u : r[i / 2] << 16);
    }
};

// Codes of four values in the bytes of a word.  code = the integer nearest to
// x / s, ties to even, of the real quotient.  inv is 1 / s rounded, so x inv is
// within 127.5 * 2^-24 < 2^-17 of x / s: adding 1.5 * 2^23 to it in one fused
// multiply-add leaves its nearest integer n in the low bits, and n is right
// unless x inv lies within 2^-15 of n + 1/2 or n - 1/2.  There (in 2^-14 of
// all values) the sign of x - (n +- 1/2) s decides, which doubles give exactly:
// the product has at most 33 bits.
__device__ __forceinline__ uint32_t codes4(const float *v, float s, float inv) {
    constexpr float kMagic = 12582912.f;
    uint32_t t[4];
    float off = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = __builtin_fmaf(v[i], inv, kMagic);
        off = __builtin_fmaxf(off, __builtin_fabsf(__builtin_fmaf(v[i], inv, kMagic - r)));
        t[i] = __builtin_bit_cast(uint32_t, r);
    }
    if (off > 0.5f - 0x1p-15f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float n = __builtin_bit_cast(float, t[i]) - kMagic, d = __builtin_fmaf(v[i], inv, -n);
            if (__builtin_fabsf(d) <= 0.5f - 0x1p-15f) continue;
            const float to = d > 0.f ? 1.f : -1.f;                 // the other integer is n + to
            const double over = ((double)v[i] - (double)(n + 0.5f * to) * (double)s) * to;
            if (over > 0.0 || (over == 0.0 && ((int)n & 1))) t[i] += (uint32_t)(int)to;
        }
    }
    const uint32_t lo = __builtin_amdgcn_perm(t[1], t[0], 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(t[3], t[2], 0x0C0C0400u);
    return lo | hi << 16;
}

// Magnitudes are compared as their bit patterns, which order like the values
// and put Inf and NaN above all of them.
constexpr uint32_t kInfBits = 0x7F800000u;

template <typename T>
__device__ __forceinline__ uint32_t magnitude(u32x4_t r, uint32_t most) {
    float v[Vec<T>::n];
    Vec<T>::get(r, v);
#pragma unroll
    for (int k = 0; k < Vec<T>::n; ++k) most = max(most, __builtin_bit_cast(uint32_t, v[k]) & 0x7FFFFFFFu);
    return most;
}

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
    return v;
}

// The scale of a row; a row that is not finite is divided by 1 and its codes
// are not used.
struct Scale { bool finite; float s, inv; };
__device__ __forceinline__ Scale scale_of(uint32_t most) {
    Scale c;
    c.finite = most < kInfBits;
    c.s = c.finite ? __builtin_fmaxf(__builtin_bit_cast(float, most) / 127.f, 0x1p-126f) : 1.f;
    c.inv = 1.f / c.s;
    return c;
}

template <typename T>
__device__ __forceinline__ void store_codes(int8_t *row, int i, u32x4_t r, const Scale &c) {
    float v[Vec<T>::n];
    Vec<T>::get(r, v);
    uint32_t *out = reinterpret_cast<uint32_t *>(row) + i * (Vec<T>::n / 4);
    uint32_t w[Vec<T>::n / 4];
#pragma unroll
    for (int j = 0; j < Vec<T>::n / 4; ++j) w[j] = c.finite ? codes4(v + 4 * j, c.s, c.inv) : 0u;
    if constexpr (Vec<T>::n == 8) *reinterpret_cast<u32x2_t *>(out) = u32x2_t{w[0], w[1]};
    else out[0] = w[0];
}

// Largest of a row over its T threads.
template <int T>
__device__ __forceinline__ uint32_t row_max(uint32_t most, uint32_t *part) {
    most = wave_max(most);
    if constexpr (T > 64) {
        const int tid = threadIdx.x;
        if ((tid & 63) == 0) part[tid >> 6] = most;
        __syncthreads();
        most = part[tid & (T / 64 - 1)];
#pragma unroll
        for (int m = 1; m < T / 64; m <<= 1) most = max(most, (uint32_t)__shfl_xor((int)most, m));
    }
    return most;
}

// T = 64: four rows a workgroup, one for each wavefront; else one row.
template <typename T, int TPR, int NV>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR) void quant_rows(const u32x4_t *__restrict__ x,
                                                                   int8_t *__restrict__ codes,
                                                                   float *__restrict__ scales, int M, int K) {
    __shared__ uint32_t part[16];
    const int m = TPR == 64 ? (int)blockIdx.x * 4 + (int)(threadIdx.x >> 6) : (int)blockIdx.x;
    if (m >= M) return;                   // a whole wavefront; T > 64 has no such workgroup
    const int tid = threadIdx.x & (TPR - 1), nv = K / Vec<T>::n;
    const u32x4_t *row = x + (size_t)m * nv;
    u32x4_t r[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = j * TPR + tid;
        r[j] = i < nv ? row[i] : u32x4_t{0, 0, 0, 0};
    }
    uint32_t most = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) most = magnitude<T>(r[j], most);
    const Scale c = scale_of(row_max<TPR>(most, part));
    if (tid == 0) scales[m] = c.finite ? c.s : __builtin_nanf("");
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = j * TPR + tid;
        if (i < nv) store_codes<T>(codes + (size_t)m * K, i, r[j], c);
    }
}

// Rows too long for the registers of 1024 threads: read twice.
template <typename T>
__global__ __launch_bounds__(1024) void quant_long_rows(const u32x4_t *__restrict__ x, int8_t *__restrict__ codes,
                                                        float *__restrict__ scales, int K) {
    __shared__ uint32_t part[16];
    const int m = blockIdx.x, tid = threadIdx.x, nv = K / Vec<T>::n;
    const u32x4_t *row = x + (size_t)m * nv;
    uint32_t most = 0;
    for (int i = tid; i < nv; i += 1024) most = magnitude<T>(row[i], most);
    const Scale c = scale_of(row_max<1024>(most, part));
    if (tid == 0) scales[m] = c.finite ? c.s : __builtin_nanf("");
    for (int i = tid; i < nv; i += 1024) store_codes<T>(codes + (size_t)m * K, i, row[i], c);
}

template <typename T, int TPR>
void launch_vectors(const u32x4_t *x, int8_t *codes, float *scales, int M, int K, int nv, hipStream_t s) {
    const int grid = TPR == 64 ? (M + 3) / 4 : M, block = TPR == 64 ? 256 : TPR, each = (nv + TPR - 1) / TPR;
    if (each <= 1) quant_rows<T, TPR, 1><<<grid, block, 0, s>>>(x, codes, scales, M, K);
    else if (each <= 2) quant_rows<T, TPR, 2><<<grid, block, 0, s>>>(x, codes, scales, M, K);
    else if (TPR == 64 || each <= 4) quant_rows<T, TPR, 4><<<grid, block, 0, s>>>(x, codes, scales, M, K);
    else if constexpr (TPR > 64) quant_rows<T, TPR, 8><<<grid, block, 0, s>>>(x, codes, scales, M, K);
}

template <typename T>
void launch(const u32x4_t *x, int8_t *codes, float *scales, int M, int K, hipStream_t s) {
    const int nv = K / Vec<T>::n;
    // The fewest threads that hold a row (64 of them no more than 4 vectors
    // each: 8192 rows of 4096 bf16 take 19.1 us with 256 threads, 25.2 with 64
    // and 8 vectors), but more while the rows are too few to fill the chip
    // (2048 wavefronts) and each thread has several vectors.
    auto enough = [&](int t) { return nv <= (t == 64 ? 4 : 8) * t && (nv <= t || (int64_t)M * t >= 2048 * 64); };
    if (enough(64)) launch_vectors<T, 64>(x, codes, scales, M, K, nv, s);
    else if (enough(256)) launch_vectors<T, 256>(x, codes, scales, M, K, nv, s);
    else if (nv <= 8192) launch_vectors<T, 1024>(x, codes, scales, M, K, nv, s);
    else quant_long_rows<T><<<M, 1024, 0, s>>>(x, codes, scales, K);
}

}  // namespace

extern "C" int quant_i8(const void *x, int x_type, int8_t *codes, float *scales, int M, int K, void *stream) {
    if (M < 0 || M >= (1 << 22) || K < 16 || K % 16 || K > 131056) return Q4_EINVAL;
    if (x_type != I8_F32 && x_type != I8_F16 && x_type != I8_BF16) return Q4_EINVAL;
    if (M == 0) return Q4_OK;
    if (!x || !codes || !scales) return Q4_ENULL;
    if (!q4::aligned(x, 16) || !q4::aligned(codes, 16) || !q4::aligned(scales, 4)) return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    const auto *xv = static_cast<const u32x4_t *>(x);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (x_type == I8_F32) launch<F32>(xv, codes, scales, M, K, s);
    else if (x_type == I8_F16) launch<F16>(xv, codes, scales, M, K, s);
    else launch<BF16>(xv, codes, scales, M, K, s);
    return q4::launch_status();
}
