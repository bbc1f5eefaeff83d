// quant_i8.hip -- rows of activations to 8-bit codes with one scale each, for
// gfx950 (see q4i8.h):
//
//     s[m] = max(rn(max_k |x[m, k]| / 127), 2^-126),  c[m, k] = nearest(x[m, k] / s[m])
//
// One workgroup takes a row: it finds the row's largest magnitude, then reads
// the row again (from the caches) and writes its codes.
#include "q4_common.h"
#include "q4i8.h"

namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

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

// The integer nearest to x / s, ties to even, of the real quotient: inv is
// 1 / s rounded, so q = x * inv is within 2^-23 * 127.5 < 2^-16 of x / s, and
// rint(q) is right unless q lies that near to t = n + 1/2.  There the sign of
// x - t s decides, which doubles give exactly (t s has at most 33 bits).
__device__ __forceinline__ int code_of(float x, float s, float inv) {
    const float q = x * inv;
    float n = __builtin_rintf(q);
    const float below = __builtin_floorf(q);
    if (__builtin_fabsf(q - below - 0.5f) < 0x1p-14f) {
        const double d = (double)x - (double)(below + 0.5f) * (double)s;
        n = d > 0.0 ? below + 1.f : d < 0.0 ? below : 2.f * __builtin_rintf(0.5f * (below + 0.5f));
    }
    return (int)n;
}

// Magnitudes are compared as their bit patterns, which order like the values
// and put Inf and NaN above all of them.
constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, m));
    return v;
}

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void quant_rows(const u32x4_t *__restrict__ x, int8_t *__restrict__ codes,
                                                       float *__restrict__ scales, int K) {
    constexpr int V = Vec<T>::n;
    __shared__ uint32_t part[kThreads / 64];
    const int tid = threadIdx.x, nv = K / V;
    const u32x4_t *row = x + (size_t)blockIdx.x * nv;
    uint32_t most = 0;
    for (int i = tid; i < nv; i += kThreads) {
        float v[V];
        Vec<T>::get(row[i], v);
#pragma unroll
        for (int k = 0; k < V; ++k) most = max(most, __builtin_bit_cast(uint32_t, v[k]) & 0x7FFFFFFFu);
    }
    most = wave_max(most);
    if ((tid & 63) == 0) part[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 64; ++i) most = max(most, part[i]);
    const bool finite = most < kInfBits;
    const float s = finite ? __builtin_fmaxf(__builtin_bit_cast(float, most) / 127.f, 0x1p-126f) : 1.f;
    const float inv = 1.f / s;
    if (tid == 0) scales[blockIdx.x] = finite ? s : __builtin_nanf("");
    uint32_t *out = reinterpret_cast<uint32_t *>(codes + (size_t)blockIdx.x * K);
    for (int i = tid; i < nv; i += kThreads) {
        float v[V];
        Vec<T>::get(row[i], v);
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            uint32_t c = 0;
            if (finite) {
#pragma unroll
                for (int k = 0; k < 4; ++k) c |= (uint32_t)(code_of(v[4 * j + k], s, inv) & 255) << (8 * k);
            }
            out[i * (V / 4) + j] = c;
        }
    }
}

}  // namespace

extern "C" int quant_i8(const void *x, int x_type, int8_t *codes, float *scales, int M, int K, void *stream) {
    if (M < 0 || M > (1 << 24) || K < 16 || K % 16 || K > 131056) return Q4_EINVAL;
    if (x_type != I8_F32 && x_type != I8_F16 && x_type != I8_BF16) return Q4_EINVAL;
    if (M == 0) return Q4_OK;
    if (!x || !codes || !scales) return Q4_ENULL;
    if (!q4::aligned(x, 16) || !q4::aligned(codes, 16) || !q4::aligned(scales, 4)) return Q4_EALIGN;
    if (int st = q4::check_device()) return st;
    const auto *xv = static_cast<const u32x4_t *>(x);
    const hipStream_t s = static_cast<hipStream_t>(stream);
    if (x_type == I8_F32) quant_rows<F32><<<M, kThreads, 0, s>>>(xv, codes, scales, K);
    else if (x_type == I8_F16) quant_rows<F16><<<M, kThreads, 0, s>>>(xv, codes, scales, K);
    else quant_rows<BF16><<<M, kThreads, 0, s>>>(xv, codes, scales, K);
    return q4::launch_status();
}
