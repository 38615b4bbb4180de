// Microscaled 4-bit rows: quantisation, reading back, and the decode layout
// of a quantised weight.
//
// k_quant_fp4   one CTA per four rows of a 128-row scale tile (r, r+32, r+64,
//               r+96: their scale bytes of a tile are 16 consecutive bytes),
//               128 threads per row, 16 values per thread and step.  NV needs
//               the row's largest value first: the row stays in registers
//               between the two uses up to FP4_HELD steps and is read again
//               (from L2) beyond.
// k_dequant_fp4 16 codes per thread.
// k_fp4_rowf, k_fp4_decode_layout  see below.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"

namespace as {

constexpr int FP4_QTHREADS = 512;          // 4 rows x 128 threads
constexpr int FP4_STEP = 128 * 16;         // values of a row per step

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

template <typename TX>
constexpr int fp4_held() { return sizeof(TX) == 2 ? 7 : 3; }  // steps held in registers

template <typename TX, int FMT>
__global__ void __launch_bounds__(FP4_QTHREADS) k_quant_fp4(const TX *__restrict__ x, int rows, int K, int kt,
                                                            uint8_t *__restrict__ codes, uint8_t *__restrict__ sf,
                                                            float *__restrict__ row_scale)
{
    constexpr int HELD = fp4_held<TX>();
    extern __shared__ __align__(16) unsigned char s_sf[];  // [kt][4 rows][4 blocks]
    __shared__ uint32_t s_max[4][4];
    const int rt = blockIdx.x >> 5, p = blockIdx.x & 31;   // row tile, row within its 32
    const int j = threadIdx.x >> 7, i = threadIdx.x & 127;  // row of the four, thread of the row
    const int row = rt * 128 + 32 * j + p;
    const bool row_ok = row < rows;
    const TX *xr = x + (size_t)(row_ok ? row : 0) * K;
    const int nu = K >> 4;                       // 16-value units of the row
    const int steps = (nu + 127) >> 7;

    // the scales past K stay zero
    for (int t = threadIdx.x; t < kt * 4; t += FP4_QTHREADS) reinterpret_cast<uint32_t *>(s_sf)[t] = 0u;

    Raw16<TX> held[HELD];
    float inv_row = 1.0f;
#pragma unroll
    for (int s = 0; s < HELD; ++s) {
        const int u = s * 128 + i;
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
            const int u = s * 128 + i;
            if (row_ok && u < nu) {
                Raw16<TX> t;
                t.load(xr + 16 * (size_t)u);
                const uint32_t b = t.amax();
                m = max(m, b < F32_INF_BITS ? b : 0u);
            }
        }
        m = __reduce_max_sync(0xffffffffu, m);
        if ((threadIdx.x & 31) == 0) s_max[j][(threadIdx.x >> 5) & 3] = m;
        __syncthreads();
        m = max(max(s_max[j][0], s_max[j][1]), max(s_max[j][2], s_max[j][3]));
        const int e = nv_row_exponent(m);
        inv_row = pow2f(-e);
        if (i == 0 && row_ok && as_in(row, rows)) row_scale[row] = pow2f(e);
    } else {
        if (i == 0 && row_ok && row_scale) row_scale[row] = 1.0f;
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
        if (FMT == AS_FP4_NV || (u & 1) == 0) s_sf[(blk >> 2) * 16 + j * 4 + (blk & 3)] = (unsigned char)b.byte;
    };
#pragma unroll
    for (int s = 0; s < HELD; ++s)
        if (s < steps) emit(held[s], s * 128 + i);
    for (int s = HELD; s < steps; ++s) {
        const int u = s * 128 + i;
        Raw16<TX> t;
        if (row_ok && u < nu) t.load(xr + 16 * (size_t)u);
        else t.zero();
        emit(t, u);
    }
    __syncthreads();
    const long long sf_bytes = (long long)((rows + 127) / 128) * kt * 512;
    for (int c = threadIdx.x; c < kt; c += FP4_QTHREADS)
        if (as_in(((long long)rt * kt + c) * 512 + p * 16 + 15, sf_bytes))
            *reinterpret_cast<uint4 *>(sf + ((size_t)rt * kt + c) * 512 + p * 16) =
                *reinterpret_cast<const uint4 *>(s_sf + c * 16);
}

// Reading back: thread = 16 codes (one NV block, half an MX block).
template <typename TO, int FMT>
__global__ void __launch_bounds__(256) k_dequant_fp4(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ sf,
                                                     const float *__restrict__ row_scale, int rows, int K, int kt,
                                                     TO *__restrict__ out)
{
    const int nu = K >> 4;
    const long long total = (long long)rows * nu;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const int row = (int)(i / nu), u = (int)(i % nu);
        const uint2 c = *reinterpret_cast<const uint2 *>(codes + (size_t)row * (K / 2) + 8 * (size_t)u);
        const float s = fp4_scale_value<FMT>(sf[fp4_sf_byte(row, FMT == AS_FP4_MX ? u >> 1 : u, kt)]);
        const float rs = row_scale ? row_scale[row] : 1.0f;
        float v[16];
#pragma unroll
        for (int b = 0; b < 8; ++b) {
            const float2 f = e2m1x2_value(((b < 4 ? c.x : c.y) >> (8 * (b & 3))) & 0xFFu);
            v[2 * b] = f.x * s * rs;
            v[2 * b + 1] = f.y * s * rs;
        }
        TO *o = out + (size_t)row * K + 16 * (size_t)u;
        if (!as_in((long long)row * K + 16 * u + 15, (long long)rows * K)) continue;
        if constexpr (sizeof(TO) == 2) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 t = __floats2bfloat162_rn(v[8 * h + 2 * k], v[8 * h + 2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t *>(&t);
                }
                *reinterpret_cast<uint4 *>(o + 8 * h) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
#pragma unroll
            for (int h = 0; h < 4; ++h)
                *reinterpret_cast<float4 *>(o + 4 * h) = make_float4(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3]);
        }
    }
}

size_t fp4_sf_bytes(int rows, int K, int fmt) { return (size_t)((rows + 127) / 128) * fp4_sf_ktiles(K, fmt) * 512; }

template <typename TX, int FMT>
static cudaError_t launch_quant_t(const void *x, int rows, int K, uint8_t *codes, uint8_t *sf, float *row_scale,
                                  cudaStream_t st)
{
    const int kt = fp4_sf_ktiles(K, FMT);
    const size_t smem = (size_t)kt * 16;  // at most 32 KB (K <= 131072)
    k_quant_fp4<TX, FMT><<<(rows + 127) / 128 * 32, FP4_QTHREADS, smem, st>>>(static_cast<const TX *>(x), rows, K, kt,
                                                                             codes, sf, row_scale);
    return cudaGetLastError();
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
    const long long units = (long long)rows * (K / 16);
    const long long want = (units + 255) / 256;
    const int grid = (int)(want < 148 * 64 ? want : 148 * 64);
    k_dequant_fp4<TO, FMT><<<grid, 256, 0, st>>>(codes, sf, row_scale, rows, K, fp4_sf_ktiles(K, FMT),
                                                 static_cast<TO *>(out));
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
