// The step between two blocks of a transformer, one pass over the rows:
//   u  = y * rsqrt(mean(y^2) + eps) * (w_offset + post_w)
//   r' = res_scale * r + gate * u
//   h  = r' * rsqrt(mean(r'^2) + eps) * (w_offset + pre_w)
// h as bf16/float32 and/or as the microscaled 4-bit operand of the product.
//
// Bound: memory.  One CTA per row; the row of y, r and r' stays in registers
// (8-channel chunks, CH per thread), so every input is read once and the two
// sums cost one block reduction each.  Mean squares are sums of per-thread
// partials, lanes and warps in a fixed order.
#include <algorithm>

#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"
#include "select_util.cuh"

namespace as {

__device__ __forceinline__ void load8_any(const void *p, size_t i, int bf16, float (&v)[8])
{
    if (bf16) load8(static_cast<const __nv_bfloat16 *>(p) + i, v);
    else load8(static_cast<const float *>(p) + i, v);
}

__device__ __forceinline__ void store8_any(void *p, size_t i, int bf16, const float (&v)[8])
{
    if (bf16) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&t);
        }
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p) + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p) + i);
        o[0] = make_float4(v[0], v[1], v[2], v[3]);
        o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
}

// Sum over the block, the same bits in every thread (lanes by a fixed tree,
// warps in order).  `red` is not shared with another reduction in flight.
template <int NT>
__device__ __forceinline__ float block_sum(float v, float *red)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w) v += red[w];
    }
    return v;
}

// Four scale bytes of row t (up to the next multiple of 128 past T), tile i of kt.
__device__ __forceinline__ void norm_store_sf(const NormArgs &a, int t, int T, int i, int kt, uint32_t bytes)
{
    const size_t at = fp4_sf_byte(t, 4 * i, kt);
    if (as_in((long long)at + 3, (long long)((T + 127) / 128) * kt * 512))
        *reinterpret_cast<uint32_t *>(a.h_sf + at) = bytes;
}

// h -> codes and scales of row t (all threads of the block).
template <int NT, int CH, int FMT>
__device__ __forceinline__ void norm_store_fp4(const NormArgs &a, const float (&h)[CH][8], int t, int T, int D, int kt,
                                               unsigned char *s_sf, uint32_t *s_max)
{
    const int tid = threadIdx.x, nch = D >> 3;
    constexpr int LANES = fp4_block(FMT) / 8;  // threads that share a block
    for (int i = tid; i < kt; i += NT) reinterpret_cast<uint32_t *>(s_sf)[i] = 0u;
    uint32_t am[CH];
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < CH; ++r) {
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(h[r][e]) & 0x7FFFFFFFu);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        am[r] = m;
        if (m < F32_INF_BITS) top = max(top, m);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) s_max[tid >> 5] = top;
    __syncthreads();  // the zeroed scales too
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = max(top, s_max[w]);
    const int e = FMT == AS_FP4_NV ? nv_row_exponent(top) : 0;
    if (tid == 0 && a.h_scale && as_in(t, T)) a.h_scale[t] = pow2f(e);
    const float inv_row = pow2f(-e);
#pragma unroll
    for (int r = 0; r < CH; ++r) {
        const int c = r * NT + tid;
        if (c >= nch) continue;
        const Fp4Block b = fp4_block_scale<FMT>(am[r], inv_row);
        if (as_in((long long)t * (D / 2) + 4 * c + 3, (long long)T * (D / 2)))
            *reinterpret_cast<uint32_t *>(a.h_q + (size_t)t * (D / 2) + 4 * (size_t)c) =
                fp4_codes8<FMT, false>(h[r], b, 1.0f);
        if (c % LANES == 0) s_sf[c / LANES] = (unsigned char)b.byte;
    }
    __syncthreads();
    for (int i = tid; i < kt; i += NT) norm_store_sf(a, t, T, i, kt, reinterpret_cast<const uint32_t *>(s_sf)[i]);
}

template <int NT, int CH>
__global__ void __launch_bounds__(NT, NT * CH <= 1024 ? 1024 / NT : 1) k_norm_residual(NormArgs a, int T, int D, int kt)
{
    __shared__ float red[2][NT / 32];
    __shared__ uint32_t s_max[NT / 32];
    extern __shared__ __align__(16) unsigned char s_sf[];
    const int t = blockIdx.x, tid = threadIdx.x, nch = D >> 3;
    if (t >= T) {  // padding rows of the last 128-row scale tile
        for (int i = tid; i < kt; i += NT) norm_store_sf(a, t, T, i, kt, 0u);
        return;
    }
    const size_t row = (size_t)t * D;
    // one chunk per thread: the weights are loaded with the row, so that their
    // latency does not follow the reductions
    float pw[8], qw[8];
    if constexpr (CH == 1) {
        if (tid < nch && a.post_w) load8f(a.post_w + 8 * (size_t)tid, pw);
        if (tid < nch && a.pre_w) load8f(a.pre_w + 8 * (size_t)tid, qw);
    }
    float v[CH][8];  // r, then r', then h
#pragma unroll
    for (int r = 0; r < CH; ++r) {
        const int c = r * NT + tid;
        if (c < nch) load8_any(a.r, row + 8 * (size_t)c, a.r_bf16, v[r]);
        else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[r][e] = 0.0f;
        }
    }
    if (a.y) {
        float y[CH][8], g[CH][8];
        float ss = 0.0f;
        const float *gate = a.gate ? a.gate + (a.gate_rows == 1 ? 0 : row) : nullptr;
#pragma unroll
        for (int r = 0; r < CH; ++r) {
            const int c = r * NT + tid;
            if (c < nch) load8_any(a.y, row + 8 * (size_t)c, a.y_bf16, y[r]);
            else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[r][e] = 0.0f;
            }
            if (gate && c < nch) load8f(gate + 8 * (size_t)c, g[r]);  // before the reduction waits
        }
        float rms = 1.0f;
        if (a.post_norm) {
#pragma unroll
            for (int r = 0; r < CH; ++r)
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(y[r][e], y[r][e], ss);
            rms = __frsqrt_rn(block_sum<NT>(ss, red[0]) / (float)D + a.eps);
        }
#pragma unroll
        for (int r = 0; r < CH; ++r) {
            const int c = r * NT + tid;
            if (c >= nch) continue;
            if (CH > 1 && a.post_w) load8f(a.post_w + 8 * (size_t)c, pw);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u = y[r][e] * rms;
                if (a.post_w) u *= a.w_offset + pw[e];
                if (gate) u *= g[r][e];
                v[r][e] = fmaf(a.res_scale, v[r][e], u);
            }
            if (a.r_out && as_in((long long)row + 8 * c + 7, (long long)T * D))
                store8_any(a.r_out, row + 8 * (size_t)c, a.r_bf16, v[r]);
        }
    }
    if (!a.h && !a.h_q) return;
    float ss = 0.0f;
#pragma unroll
    for (int r = 0; r < CH; ++r)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[r][e], v[r][e], ss);
    const float rms = __frsqrt_rn(block_sum<NT>(ss, red[1]) / (float)D + a.eps);
#pragma unroll
    for (int r = 0; r < CH; ++r) {
        const int c = r * NT + tid;
        if (c >= nch) continue;
        if (CH > 1 && a.pre_w) load8f(a.pre_w + 8 * (size_t)c, qw);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[r][e] *= rms;
            if (a.pre_w) v[r][e] *= a.w_offset + qw[e];
        }
        if (a.h && as_in((long long)row + 8 * c + 7, (long long)T * D))
            store8_any(a.h, row + 8 * (size_t)c, a.h_bf16, v[r]);
    }
    if (a.h_q) {
        if (a.fmt == AS_FP4_NV) norm_store_fp4<NT, CH, AS_FP4_NV>(a, v, t, T, D, kt, s_sf, s_max);
        else norm_store_fp4<NT, CH, AS_FP4_MX>(a, v, t, T, D, kt, s_sf, s_max);
    }
}

// Many long rows: persistent CTAs with a ring of NR_STAGES rows (y, r and a
// per-token gate) that bulk copies fill, so that the next rows are on their way
// while this one is reduced and written; weights and a shared gate stay in
// registers.  8192 x 8192: 179 us against 215 us for one CTA per row (float32 r
// and per-token gate, bf16 y and h; 1.07 GB, 6.0 TB/s) and 106 against 165 us
// (bf16, gate of channels); 8192 x 4096: 90 against 104 and 56 against 80 us.
// From two rows per SM on (300 x 4096: 6.1 against 7.0 us, 1000 x 8192: 18 against
// 31 us); other D keep one CTA per row.
constexpr int NR_STAGES = 2;  // at most (one where a row of three float32 inputs fills a third of an SM)
template <int NT, int CH, int PER_SM>
__global__ void __launch_bounds__(NT, PER_SM) k_norm_ring(NormArgs a, int T, int D, int kt, int stages)
{
    __shared__ float red[2][NT / 32];
    __shared__ uint32_t s_max[NT / 32];
    __shared__ __align__(8) uint64_t full[NR_STAGES];
    extern __shared__ __align__(16) unsigned char smem[];
    const int tid = threadIdx.x, nch = D >> 3;
    const uint32_t rb = (uint32_t)D * (a.r_bf16 ? 2 : 4), yb = (uint32_t)D * (a.y_bf16 ? 2 : 4);
    const bool gtok = a.gate && a.gate_rows != 1;
    const uint32_t gb = gtok ? (uint32_t)D * 4 : 0u, stage_bytes = rb + yb + gb;
    unsigned char *s_sf = smem + (size_t)stages * stage_bytes;
    if (tid == 0) {
        for (int s = 0; s < stages; ++s) mbar_init(&full[s], 1);
        fence_mbar_init();
    }
    __syncthreads();
    auto issue = [&](int t, int s) {  // thread 0
        unsigned char *dst = smem + (size_t)s * stage_bytes;
        mbar_arrive_expect_tx(&full[s], stage_bytes);
        bulk_load(dst, static_cast<const char *>(a.y) + (size_t)t * yb, yb, &full[s]);
        bulk_load(dst + yb, static_cast<const char *>(a.r) + (size_t)t * rb, rb, &full[s]);
        if (gtok) bulk_load(dst + yb + rb, reinterpret_cast<const char *>(a.gate) + (size_t)t * gb, gb, &full[s]);
    };
    if (tid == 0)
        for (int s = 0; s < stages; ++s)
            if ((int)blockIdx.x + s * (int)gridDim.x < T) issue(blockIdx.x + s * gridDim.x, s);
    // constants of the columns: products of weights and a shared gate
    float pw[CH][8], qw[CH][8];
#pragma unroll
    for (int r = 0; r < CH; ++r) {
        const int c = r * NT + tid;
        float g[8];
        if (c < nch) {
            if (a.post_w) load8f(a.post_w + 8 * (size_t)c, pw[r]);
            if (a.pre_w) load8f(a.pre_w + 8 * (size_t)c, qw[r]);
            if (a.gate && !gtok) load8f(a.gate + 8 * (size_t)c, g);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            pw[r][e] = a.post_w && c < nch ? a.w_offset + pw[r][e] : 1.0f;
            qw[r][e] = a.pre_w && c < nch ? a.w_offset + qw[r][e] : 1.0f;
            if (a.gate && !gtok && c < nch) pw[r][e] *= g[e];
        }
    }
    int stage = 0;
    uint32_t phase = 0;
    for (int t = blockIdx.x; t < T; t += gridDim.x) {
        if (!__syncthreads_and(mbar_wait(&full[stage], phase))) break;  // every thread leaves together
        const unsigned char *src = smem + (size_t)stage * stage_bytes;
        const size_t row = (size_t)t * D;
        float v[CH][8], y[CH][8];
        float ss = 0.0f;
#pragma unroll
        for (int r = 0; r < CH; ++r) {
            const int c = r * NT + tid;
            if (c < nch) {
                load8_any(src, 8 * (size_t)c, a.y_bf16, y[r]);
                load8_any(src + yb, 8 * (size_t)c, a.r_bf16, v[r]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) y[r][e] = v[r][e] = 0.0f;
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(y[r][e], y[r][e], ss);
        }
        float rms = 1.0f;
        if (a.post_norm) rms = __frsqrt_rn(block_sum<NT>(ss, red[0]) / (float)D + a.eps);
#pragma unroll
        for (int r = 0; r < CH; ++r) {
            const int c = r * NT + tid;
            if (c >= nch) continue;
            float g[8];
            if (gtok) load8_any(src + yb + rb, 8 * (size_t)c, 0, g);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u = y[r][e] * rms * pw[r][e];
                if (gtok) u *= g[e];
                v[r][e] = fmaf(a.res_scale, v[r][e], u);
            }
            if (a.r_out && as_in((long long)row + 8 * c + 7, (long long)T * D))
                store8_any(a.r_out, row + 8 * (size_t)c, a.r_bf16, v[r]);
        }
        ss = 0.0f;
#pragma unroll
        for (int r = 0; r < CH; ++r)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[r][e], v[r][e], ss);
        rms = __frsqrt_rn(block_sum<NT>(ss, red[1]) / (float)D + a.eps);  // its barrier: the stage is read
        if (tid == 0 && t + stages * (int)gridDim.x < T) issue(t + stages * gridDim.x, stage);
        if (++stage == stages) { stage = 0; phase ^= 1; }
        if (a.h || a.h_q) {
#pragma unroll
            for (int r = 0; r < CH; ++r) {
                const int c = r * NT + tid;
                if (c >= nch) continue;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[r][e] *= rms * qw[r][e];
                if (a.h && as_in((long long)row + 8 * c + 7, (long long)T * D))
                    store8_any(a.h, row + 8 * (size_t)c, a.h_bf16, v[r]);
            }
        }
        if (a.h_q) {
            if (a.fmt == AS_FP4_NV) norm_store_fp4<NT, CH, AS_FP4_NV>(a, v, t, T, D, kt, s_sf, s_max);
            else norm_store_fp4<NT, CH, AS_FP4_MX>(a, v, t, T, D, kt, s_sf, s_max);
        }
    }
    if (a.h_q)  // padding rows of the last 128-row scale tile
        for (int t = T + blockIdx.x; t < (T + 127) / 128 * 128; t += gridDim.x)
            for (int i = tid; i < kt; i += NT) norm_store_sf(a, t, T, i, kt, 0u);
}

template <int NT, int CH, int PER_SM>
static cudaError_t launch_norm_ring(const NormArgs &a, int T, int D, cudaStream_t st)
{
    const int kt = a.h_q ? fp4_sf_ktiles(D, a.fmt) : 0;
    const size_t row = (size_t)D * ((a.r_bf16 ? 2 : 4) + (a.y_bf16 ? 2 : 4) + (a.gate && a.gate_rows != 1 ? 4 : 0));
    const size_t room = (PER_SM == 3 ? 72 : 220) * 1024 - (size_t)kt * 4;
    const int stages = (int)std::min<size_t>(NR_STAGES, room / row);
    const size_t smem = stages * row + (size_t)kt * 4;
    static RaisedLimit done;
    const cudaError_t e = smem_limit_once(k_norm_ring<NT, CH, PER_SM>, smem, done);
    if (e != cudaSuccess) return e;
    k_norm_ring<NT, CH, PER_SM><<<PER_SM * sm_count(), NT, smem, st>>>(a, T, D, kt, stages);
    return cudaGetLastError();
}

template <int NT, int CH>
static cudaError_t launch_norm_t(const NormArgs &a, int T, int D, cudaStream_t st)
{
    const int kt = a.h_q ? fp4_sf_ktiles(D, a.fmt) : 0;
    const int grid = a.h_q ? (T + 127) / 128 * 128 : T;
    k_norm_residual<NT, CH><<<grid, NT, (size_t)kt * 4, st>>>(a, T, D, kt);
    return cudaGetLastError();
}

cudaError_t launch_norm(const NormArgs &a, int T, int D, cudaStream_t st)
{
    const int nch = D / 8;
    if (a.y && T >= 2 * sm_count()) {
        if (nch > 256 && nch <= 512) return launch_norm_ring<256, 2, 3>(a, T, D, st);
        if (nch > 512 && nch <= 1024) return launch_norm_ring<512, 2, 1>(a, T, D, st);
    }
    if (nch <= 128) return launch_norm_t<128, 1>(a, T, D, st);
    if (nch <= 256) return launch_norm_t<256, 1>(a, T, D, st);
    if (nch <= 512) return launch_norm_t<512, 1>(a, T, D, st);
    if (nch <= 1024) return launch_norm_t<1024, 1>(a, T, D, st);
    if (nch <= 2048) return launch_norm_t<512, 4>(a, T, D, st);
    return launch_norm_t<1024, 4>(a, T, D, st);
}

}  // namespace as
