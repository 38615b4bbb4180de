// Microscaled 4-bit rows: quantisation and reading back.
//
// k_quant_fp4   one CTA per row, or per four short rows of a 128-row scale tile
//               (32 apart: their scale bytes are consecutive), 16 values
//               per thread and step.  NV needs the row's largest value first:
//               up to HELD steps of the row stay in registers between the two
//               uses, longer rows are read again (from L2).  One conversion
//               and one product or division per value are the least that the
//               definition allows.  Load, maximum, conversions and store of a
//               CTA follow one another, which 45 % occupancy covers in part:
//               4096 x 14336 bf16 to NV 34.8 us, 3.8 TB/s of bytes read and
//               written (floor 23 us), issue slots 60 % taken; one token of
//               14336 4.2 us, which is the latency of load, row maximum and
//               store.
// k_dequant_fp4 16 output bytes per thread and step: 4096 x 14336 to bf16
//               33.2 us, 4.5 TB/s (issue slots 66 % taken).
#include <type_traits>

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"

namespace as {

// Sixteen consecutive values; the return value is the bits of the largest
// |v| (for |v| the order of the bits is the order of the values, with
// infinities and NaN above all finite ones).
template <typename TX>
struct Raw16;
template <>
struct Raw16<__nv_bfloat16> {
    uint4 a, b;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p)
    {
        a = *reinterpret_cast<const uint4 *>(p);
        b = *reinterpret_cast<const uint4 *>(p + 8);
    }
    __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t amax() const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7FFF7FFFu);
        return max(m & 0xFFFF0000u, m << 16);
    }
    __device__ __forceinline__ void get(float (&v)[16]) const
    {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw16<float> {
    uint4 q[4];
    __device__ __forceinline__ void load(const float *p)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = *reinterpret_cast<const uint4 *>(p + 4 * i);
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ uint32_t amax() const
    {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            m = max(max(m, max(q[i].x & 0x7FFFFFFFu, q[i].y & 0x7FFFFFFFu)),
                    max(q[i].z & 0x7FFFFFFFu, q[i].w & 0x7FFFFFFFu));
        return m;
    }
    __device__ __forceinline__ void get(float (&v)[16]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[4 * i] = __uint_as_float(q[i].x);
            v[4 * i + 1] = __uint_as_float(q[i].y);
            v[4 * i + 2] = __uint_as_float(q[i].z);
            v[4 * i + 3] = __uint_as_float(q[i].w);
        }
    }
};

// ROWS rows of TPR threads each; a row is at least HELD steps of 16 * TPR
// values or is read once.
template <typename TX, int FMT, int ROWS, int TPR, int HELD>
__global__ void __launch_bounds__(ROWS *TPR, 1024 / (ROWS * TPR))
    k_quant_fp4(const TX *__restrict__ x, int rows, int K, int kt, uint8_t *__restrict__ codes,
                uint8_t *__restrict__ sf, float *__restrict__ row_scale)
{
    constexpr int NT = ROWS * TPR, GROUPS = 4 / ROWS;      // CTAs that share 32-row positions
    extern __shared__ __align__(16) unsigned char s_sf[];  // [kt][ROWS][4 blocks]
    __shared__ uint32_t s_max[ROWS][TPR / 32];
    const int rt = blockIdx.x / (32 * GROUPS), rem = blockIdx.x % (32 * GROUPS);
    const int p = rem & 31, j0 = (rem >> 5) * ROWS;         // row within its 32, first of the tile's four 32s
    const int j = threadIdx.x / TPR, i = threadIdx.x % TPR;  // row of the CTA, thread of the row
    const int row = rt * 128 + 32 * (j0 + j) + p;
    const bool row_ok = row < rows;
    const TX *xr = x + (size_t)(row_ok ? row : 0) * K;
    const int nu = K >> 4;                       // 16-value units of the row
    const int steps = (nu + TPR - 1) / TPR;

    // the scales past K stay zero
    for (int t = threadIdx.x; t < kt * ROWS; t += NT) reinterpret_cast<uint32_t *>(s_sf)[t] = 0u;

    Raw16<TX> held[HELD];
    float inv_row = 1.0f;
#pragma unroll
    for (int s = 0; s < HELD; ++s) {
        const int u = s * TPR + i;
        if (row_ok && u < nu) held[s].load(xr + 16 * (size_t)u);
        else held[s].zero();
    }
    if constexpr (FMT == AS_FP4_NV) {
        uint32_t m = 0;
#pragma unroll
        for (int s = 0; s < HELD; ++s) {
            const uint32_t b = held[s].amax();
            m = max(m, b < F32_INF_BITS ? b : 0u);
        }
        for (int s = HELD; s < steps; ++s) {
            const int u = s * TPR + i;
            if (row_ok && u < nu) {
                Raw16<TX> t;
                t.load(xr + 16 * (size_t)u);
                const uint32_t b = t.amax();
                m = max(m, b < F32_INF_BITS ? b : 0u);
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) s_max[j][i >> 5] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < TPR / 32; ++w) m = max(m, s_max[j][w]);
        const int e = nv_row_exponent(m);
        inv_row = pow2f(-e);
        if (i == 0 && row_ok && as_in(row, rows)) row_scale[row] = pow2f(e);
    } else {
        if (i == 0 && row_ok && row_scale && as_in(row, rows)) row_scale[row] = 1.0f;
        __syncthreads();  // the zeroed scales, before they are written
    }

    auto emit = [&](const Raw16<TX> &raw, int u) {
        const uint32_t am = fp4_block_amax<FMT>(raw.amax());
        if (!row_ok || u >= nu) return;
        float v[16];
        raw.get(v);
        const Fp4Block b = fp4_block_scale<FMT>(am, inv_row);
        const uint2 c = fp4_codes16<FMT, sizeof(TX) == 2>(v, b);
        if (as_in((long long)row * (K / 2) + 8 * u + 7, (long long)rows * (K / 2)))
            *reinterpret_cast<uint2 *>(codes + (size_t)row * (K / 2) + 8 * (size_t)u) = c;
        const int blk = FMT == AS_FP4_MX ? u >> 1 : u;
        if (FMT == AS_FP4_NV || (u & 1) == 0) s_sf[(blk >> 2) * (4 * ROWS) + j * 4 + (blk & 3)] = (unsigned char)b.byte;
    };
#pragma unroll
    for (int s = 0; s < HELD; ++s)
        if (s < steps) emit(held[s], s * TPR + i);
    for (int s = HELD; s < steps; ++s) {
        const int u = s * TPR + i;
        Raw16<TX> t;
        if (row_ok && u < nu) t.load(xr + 16 * (size_t)u);
        else t.zero();
        emit(t, u);
    }
    __syncthreads();
    const long long sf_bytes = (long long)((rows + 127) / 128) * kt * 512;
    using W = typename std::conditional<ROWS == 4, uint4, uint32_t>::type;
    for (int c = threadIdx.x; c < kt; c += NT)
        if (as_in(((long long)rt * kt + c) * 512 + p * 16 + 4 * (j0 + ROWS) - 1, sf_bytes))
            *reinterpret_cast<W *>(sf + ((size_t)rt * kt + c) * 512 + p * 16 + 4 * j0) =
                *reinterpret_cast<const W *>(s_sf + c * (4 * ROWS));
}

// Reading back: a thread turns DQ_U runs of N codes into 16 bytes each (N = 8
// bf16, 4 float32), so that a warp's stores are 512 consecutive bytes; every
// load of a thread is in flight at once.
constexpr int DQ_U = 8;
template <typename TO, int FMT>
__global__ void __launch_bounds__(256) k_dequant_fp4(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf,
                                                     const float *__restrict__ row_scale, int rows, int K, int kt,
                                                     TO *__restrict__ out)
{
    constexpr int N = 16 / sizeof(TO), B = fp4_block(FMT);
    const unsigned nu = (unsigned)K / N;
    const long long first = (long long)blockIdx.x * (256 * DQ_U);
    const int row0 = (int)(first / nu);
    const unsigned rem0 = (unsigned)(first % nu);
    uint32_t c[DQ_U], s[DQ_U];
    float rs[DQ_U];
    int row[DQ_U];
    unsigned u[DQ_U];
#pragma unroll
    for (int k = 0; k < DQ_U; ++k) {
        const unsigned v = rem0 + threadIdx.x + 256u * k;
        row[k] = row0 + (int)(v / nu);
        u[k] = v % nu;
        if (row[k] < rows) {
            const uint8_t *cp = codes + (size_t)row[k] * (K / 2) + (size_t)(N / 2) * u[k];
            c[k] = N == 8 ? __ldcs(reinterpret_cast<const uint32_t *>(cp))
                          : (uint32_t)__ldcs(reinterpret_cast<const uint16_t *>(cp));
            s[k] = sf[fp4_sf_byte(row[k], (int)(u[k] / (B / N)), kt)];
            rs[k] = row_scale ? row_scale[row[k]] : 1.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < DQ_U; ++k) {
        if (row[k] >= rows || !as_in((long long)row[k] * K + N * u[k] + N - 1, (long long)rows * K)) continue;
        const float sv = fp4_scale_value<FMT>(s[k]);
        float v[N];
#pragma unroll
        for (int b = 0; b < N / 2; ++b) {
            const float2 f = e2m1x2_value((c[k] >> (8 * b)) & 0xFFu);
            v[2 * b] = f.x * sv * rs[k];
            v[2 * b + 1] = f.y * sv * rs[k];
        }
        TO *o = out + (size_t)row[k] * K + (size_t)N * u[k];
        if constexpr (sizeof(TO) == 2) {
            uint32_t t[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * b], v[2 * b + 1]);
                t[b] = *reinterpret_cast<const uint32_t *>(&q);
            }
            __stcs(reinterpret_cast<uint4 *>(o), make_uint4(t[0], t[1], t[2], t[3]));
        } else {
            __stcs(reinterpret_cast<float4 *>(o), make_float4(v[0], v[1], v[2], v[3]));
        }
    }
}

size_t fp4_sf_bytes(int rows, int K, int fmt) { return (size_t)((rows + 127) / 128) * fp4_sf_ktiles(K, fmt) * 512; }

template <typename TX, int FMT, int ROWS, int TPR, int HELD>
static cudaError_t launch_quant_c(const void *x, int rows, int K, uint8_t *codes, uint8_t *sf, float *row_scale,
                                  cudaStream_t st)
{
    const int kt = fp4_sf_ktiles(K, FMT);
    const size_t smem = (size_t)kt * 4 * ROWS;  // at most 32 KB (K <= 131072)
    k_quant_fp4<TX, FMT, ROWS, TPR, HELD><<<(rows + 127) / 128 * (128 / ROWS), ROWS * TPR, smem, st>>>(
        static_cast<const TX *>(x), rows, K, kt, codes, sf, row_scale);
    return cudaGetLastError();
}

template <typename TX, int FMT>
static cudaError_t launch_quant_t(const void *x, int rows, int K, uint8_t *codes, uint8_t *sf, float *row_scale,
                                  cudaStream_t st)
{
    if (K <= 4096) return launch_quant_c<TX, FMT, 4, 64, sizeof(TX) == 2 ? 4 : 2>(x, rows, K, codes, sf, row_scale, st);
    return launch_quant_c<TX, FMT, 1, 256, sizeof(TX) == 2 ? 4 : 2>(x, rows, K, codes, sf, row_scale, st);
}

cudaError_t launch_quant_fp4(const void *x, int bf16, int rows, int K, int fmt, uint8_t *codes, uint8_t *sf,
                             float *row_scale, cudaStream_t st)
{
    if (bf16)
        return fmt == AS_FP4_NV ? launch_quant_t<__nv_bfloat16, AS_FP4_NV>(x, rows, K, codes, sf, row_scale, st)
                                : launch_quant_t<__nv_bfloat16, AS_FP4_MX>(x, rows, K, codes, sf, row_scale, st);
    return fmt == AS_FP4_NV ? launch_quant_t<float, AS_FP4_NV>(x, rows, K, codes, sf, row_scale, st)
                            : launch_quant_t<float, AS_FP4_MX>(x, rows, K, codes, sf, row_scale, st);
}

template <typename TO, int FMT>
static cudaError_t launch_dequant_t(const uint8_t *codes, const uint8_t *sf, const float *row_scale, int rows, int K,
                                    void *out, cudaStream_t st)
{
    const long long units = (long long)rows * (K / (16 / (int)sizeof(TO)));
    k_dequant_fp4<TO, FMT><<<(unsigned)((units + 256 * DQ_U - 1) / (256 * DQ_U)), 256, 0, st>>>(
        codes, sf, row_scale, rows, K, fp4_sf_ktiles(K, FMT), static_cast<TO *>(out));
    return cudaGetLastError();
}

cudaError_t launch_dequant_fp4(const uint8_t *codes, const uint8_t *sf, const float *row_scale, int rows, int K,
                               int fmt, int out_bf16, void *out, cudaStream_t st)
{
    if (out_bf16)
        return fmt == AS_FP4_NV
                   ? launch_dequant_t<__nv_bfloat16, AS_FP4_NV>(codes, sf, row_scale, rows, K, out, st)
                   : launch_dequant_t<__nv_bfloat16, AS_FP4_MX>(codes, sf, row_scale, rows, K, out, st);
    return fmt == AS_FP4_NV ? launch_dequant_t<float, AS_FP4_NV>(codes, sf, row_scale, rows, K, out, st)
                            : launch_dequant_t<float, AS_FP4_MX>(codes, sf, row_scale, rows, K, out, st);
}

}  // namespace as
