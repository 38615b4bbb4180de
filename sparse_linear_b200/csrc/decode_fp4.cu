// Decode on microscaled 4-bit weights: y = prune(x) W^T for 1..16 tokens,
// reading only the codes of the channels that some token keeps.
//
// Weight layout (k_fp4_decode_layout, once per layer).  Slices of 128 output
// columns; in a slice one unit per scale block of B channels: B rows of 64
// bytes (the block's channels), then the 128 outputs' scales.  Inside 16
// channels, row 4r + q holds channel 4q + r; its 8-byte piece g holds the codes
// of outputs o(p, g) = 16 (p >> 1) + 8 (p & 1) + g, p = 0..15, four bits each:
// exactly what lane (g, q) of an m16n8k16 fragment needs, so a lane's four
// pieces need no exchange with other lanes.  Two rows' words interleave (two
// shifts and two selects per 16 codes) into bytes that hold the codes of a
// channel pair for one output, and one conversion per byte (cvt f16x2.e2m1x2)
// gives the A fragment register: codes enter the tensor cores as they are.
//   Scales multiply the products of their 16 channels in float32:
//   acc += s * (codes x), one fused step per block and output, which also keeps
//   every sum of the tensor core short.  MX scales are stored relative to the
//   row's largest; a float32 factor per output carries that power of two and
//   the weight's row scale.
//   Kept values enter as one or two f16 parts after scaling each token by a
//   power of two that puts its largest |x| in the CTA's range of K at 2^14: bf16
//   values are exact from 2^-28 of the largest up, smaller ones err by at most
//   2^-39 of it; two parts hold 22 bits of a float32 value.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"
#include "select_util.cuh"

namespace as {

constexpr int DF_COLS = 128;     // output columns per slice
constexpr int DF_WARPS = 8;
constexpr int DF_THREADS = DF_WARPS * 32;
constexpr int DF_DEPTH = 8;      // 16-channel steps in flight per warp
constexpr int DF_STAGE = 1024 + 128;
constexpr int DF_RSTRIDE = DF_COLS + 4;  // padded row of the reduction buffer (no bank conflicts)

__host__ __device__ constexpr int df_unit(int fmt) { return fp4_block(fmt) * 64 + 128; }
static size_t df_codes_bytes(int n_out, int K, int fmt)
{
    return (size_t)((n_out + DF_COLS - 1) / DF_COLS) * (size_t)(K / fp4_block(fmt)) * df_unit(fmt);
}
// codes and scales, then the float32 factor and (MX) the largest scale byte
// of every output
size_t fp4_decode_bytes(int n_out, int K, int fmt)
{
    return df_codes_bytes(n_out, K, fmt) + (size_t)((n_out + DF_COLS - 1) / DF_COLS) * DF_COLS * 8;
}

// One warp per output: the row's largest scale and its factor.
__global__ void __launch_bounds__(256) k_fp4_rowf(const uint8_t *__restrict__ w_sf, const float *__restrict__ w_scale,
                                                  int n_out, int n_pad, int K, int fmt, float *__restrict__ rowf,
                                                  int *__restrict__ top)
{
    const int o = blockIdx.x * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (o >= n_pad) return;
    const int nb = K / fp4_block(fmt), kt = fp4_sf_ktiles(K, fmt);
    uint32_t m = 0, bad = 0;
    if (o < n_out)
        for (int b = lane; b < nb; b += 32) {
            const uint32_t s = w_sf[fp4_sf_byte(o, b, kt)];
            if (fmt == AS_FP4_MX ? s == 255u : (s & 127u) == 127u) bad = 1;
            else m = max(m, s);
        }
    m = __reduce_max_sync(0xffffffffu, m);
    bad = __reduce_max_sync(0xffffffffu, bad);
    if (lane == 0) {
        const float ws = o < n_out ? (w_scale ? w_scale[o] : 1.0f) : 0.0f;
        rowf[o] = bad ? __uint_as_float(0x7FFFFFFFu) : (fmt == AS_FP4_MX ? ldexpf(ws, (int)m - 127) : ws);
        top[o] = (int)m;
    }
}

// CTA = (scale block, slice), 128 threads = outputs.
template <int FMT>
__global__ void __launch_bounds__(DF_COLS) k_fp4_decode_layout(const uint8_t *__restrict__ Wq,
                                                              const uint8_t *__restrict__ w_sf,
                                                              const int *__restrict__ top, int n_out, int K,
                                                              uint8_t *__restrict__ Wd)
{
    constexpr int B = fp4_block(FMT);
    __shared__ uint8_t nib[B][DF_COLS];
    const int blk = blockIdx.x, slice = blockIdx.y, c = threadIdx.x, o = slice * DF_COLS + c;
    uint32_t scale = 0;
    uint32_t w[B / 8];
#pragma unroll
    for (int i = 0; i < B / 8; ++i) w[i] = 0u;
    if (o < n_out) {
        const uint32_t *src = reinterpret_cast<const uint32_t *>(Wq + (size_t)o * (K / 2) + (size_t)blk * (B / 2));
#pragma unroll
        for (int i = 0; i < B / 8; ++i) w[i] = src[i];
        const uint32_t s = w_sf[fp4_sf_byte(o, blk, fp4_sf_ktiles(K, FMT))];
        // a NaN scale shows in the output's factor
        if constexpr (FMT == AS_FP4_MX) scale = s == 255u ? 0u : (uint32_t)max((int)s - top[o] + 127, 0);
        else scale = (s & 127u) == 127u ? 0u : s & 127u;
    }
#pragma unroll
    for (int i = 0; i < B; ++i) nib[i][c] = (uint8_t)((w[i >> 3] >> (4 * (i & 7))) & 15u);
    __syncthreads();
    uint8_t *unit = Wd + ((size_t)slice * gridDim.x + blk) * df_unit(FMT);
    for (int i = threadIdx.x; i < B * 16; i += DF_COLS) {  // 16 words per row
        const int row = i >> 4, g = (i >> 1) & 7, wd = i & 1;
        const int r = (row & 15) >> 2, q = row & 3, ch = (row & ~15) + 4 * q + r;
        uint32_t word = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int p = wd * 8 + k;
            word |= (uint32_t)nib[ch][16 * (p >> 1) + 8 * (p & 1) + g] << (4 * k);
        }
        reinterpret_cast<uint32_t *>(unit)[i] = word;
    }
    const int p = 2 * (c >> 4) + ((c >> 3) & 1), g = c & 7;
    unit[B * 64 + g * 16 + p] = (uint8_t)scale;
}

cudaError_t launch_weight_prep_fp4(const uint8_t *Wq, const uint8_t *w_sf, const float *w_scale, int n_out, int K,
                                   int fmt, uint8_t *Wd, cudaStream_t st)
{
    const int slices = (n_out + DF_COLS - 1) / DF_COLS, n_pad = slices * DF_COLS;
    float *rowf = reinterpret_cast<float *>(Wd + df_codes_bytes(n_out, K, fmt));
    int *top = reinterpret_cast<int *>(rowf + n_pad);
    k_fp4_rowf<<<(n_pad + 7) / 8, 256, 0, st>>>(w_sf, w_scale, n_out, n_pad, K, fmt, rowf, top);
    const dim3 grid(K / fp4_block(fmt), slices);
    if (fmt == AS_FP4_NV)
        k_fp4_decode_layout<AS_FP4_NV><<<grid, DF_COLS, 0, st>>>(Wq, w_sf, top, n_out, K, Wd);
    else
        k_fp4_decode_layout<AS_FP4_MX><<<grid, DF_COLS, 0, st>>>(Wq, w_sf, top, n_out, K, Wd);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ decode
// CTA (rank of a cluster, slice): the slice's 128 columns and a contiguous
// part of K; its warps take 16-channel steps in turn.  A lane copies its own
// pieces of the kept rows (cp.async, a ring of its own in shared memory),
// turns them into A fragments and multiplies with the kept values of x, which
// the CTA stages in shared memory as PARTS f16 arrays (zero where a token
// dropped the channel, so rows that were not loaded do not matter).  The
// warps' sums are added in shared memory and the cluster's through
// distributed shared memory, both in a fixed order.
template <int NT, int PARTS>
struct DfCfg {
    static constexpr int TP = 8 * NT;
    static constexpr int KSUB = NT * PARTS <= 2 ? 2048 : 1024;  // channels of x staged at a time
    static constexpr int XS = KSUB + 16;                        // row stride: token rows 8 banks apart
    static constexpr size_t xbytes = (size_t)PARTS * TP * XS * 2;
    static constexpr size_t ring = (size_t)DF_WARPS * DF_DEPTH * DF_STAGE;
    static constexpr size_t red = (size_t)DF_WARPS * TP * DF_RSTRIDE * 4;
    static constexpr size_t big = ring > red ? ring : red;
    static constexpr size_t smem = big + xbytes;
    static constexpr int per_sm = smem <= 110 * 1024 ? 2 : 1;
};

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// Four bytes of two codes each -> four f16x2.
__device__ __forceinline__ void e2m1x8(uint32_t w, uint32_t (&r)[4])
{
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
        : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, const float (&c)[4])
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

// The scales of outputs p (bytes of sc) as float32.
template <int FMT>
__device__ __forceinline__ void df_scales(uint32_t sc, float (&f)[4])
{
    if constexpr (FMT == AS_FP4_MX) {
        f[0] = __uint_as_float((sc & 0xFFu) << 23);
        f[1] = __uint_as_float((sc & 0xFF00u) << 15);
        f[2] = __uint_as_float((sc & 0xFF0000u) << 7);
        f[3] = __uint_as_float((sc >> 24) << 23);
    } else {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(sc & 0xFFFFu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(sc >> 16), __NV_E4M3);
        const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    }
}

template <int NT, int PARTS, int FMT>
__global__ void __launch_bounds__(DF_THREADS, DfCfg<NT, PARTS>::per_sm) k_decode_fp4(DecodeFp4Args a)
{
    using C = DfCfg<NT, PARTS>;
    constexpr int TP = C::TP;
    extern __shared__ __align__(16) unsigned char smem[];
    float *red = reinterpret_cast<float *>(smem);  // after the main loop
    __half *xs = reinterpret_cast<__half *>(smem + C::big);
    __shared__ uint32_t s_keep[TP][C::KSUB / 32];
    __shared__ uint32_t s_union[C::KSUB / 32];
    __shared__ float s_eta[TP], s_mul[TP], s_inv[TP];  // shift; power of two into and out of f16's range
    __shared__ uint32_t s_max[TP];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, q4 = lane & 3;
    const int rank = (int)cluster_ctarank(), nranks = gridDim.x, slice = blockIdx.y;
    const int T = a.T, K = a.K, n_out = a.n_out;
    const int nwords = K >> 5, wper = (nwords + nranks - 1) / nranks;
    const int w0 = min(nwords, rank * wper), w1 = min(nwords, w0 + wper);
    const uint8_t *wslice = a.Wd + (size_t)slice * (size_t)(K / fp4_block(FMT)) * df_unit(FMT);
    const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (DF_DEPTH * DF_STAGE);

    // step s of this warp in the part that starts at word ws covers channels
    // 32 ws + 16 (DF_WARPS s + warp); it has `mine` of them
    auto steps_of = [&](int ws) {
        const int n = 2 * min(C::KSUB / 32, w1 - ws);
        return n > warp ? (n - warp + DF_WARPS - 1) / DF_WARPS : 0;
    };
    auto issue = [&](int ws, int s, int mine, bool all) {
        if (s < mine) {
            const int lb = DF_WARPS * s + warp, b = 2 * ws + lb;
            const uint32_t keep = all ? 0xFFFFu : (s_union[lb >> 1] >> (16 * (lb & 1))) & 0xFFFFu;
            const uint8_t *unit = FMT == AS_FP4_NV ? wslice + (size_t)b * df_unit(FMT)
                                                   : wslice + (size_t)(b >> 1) * df_unit(FMT) + (b & 1) * 1024;
            const uint32_t dst = ring + (uint32_t)(s % DF_DEPTH) * DF_STAGE;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if ((keep >> (4 * q4 + r)) & 1u) cp_async8(dst + r * 256 + lane * 8, unit + r * 256 + q4 * 64 + g8 * 8);
            const uint8_t *sc = FMT == AS_FP4_NV ? unit + 1024 : wslice + (size_t)(b >> 1) * df_unit(FMT) + 2048;
            if (lane < 8) cp_async16(dst + 1024 + lane * 16, sc + lane * 16, 16u);
        }
        cp_async_commit();
    };
    auto prologue = [&](int ws, bool all) {
        const int mine = steps_of(ws);
#pragma unroll
        for (int s = 0; s < DF_DEPTH - 1; ++s) issue(ws, s, mine, all);
    };
    auto load_x = [&](int t, int c, float (&v)[8]) {  // channels c .. c+7 of token t
        const size_t at = (size_t)t * K + (size_t)c;
        if (a.bf16) load8(static_cast<const __nv_bfloat16 *>(a.x) + at, v);
        else load8(static_cast<const float *>(a.x) + at, v);
    };

    // The select kernel lets this one start after its own wait, so everything
    // before that kernel in the stream (x and the weights) is complete.  What
    // does not depend on the selection comes before the wait for it: the
    // tokens' largest |x| and, if every channel is wanted, the first weights.
    if (!a.after_select) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (a.stream_all) prologue(w0, true);
    if (tid < TP) s_max[tid] = 0u;
    __syncthreads();
    {
        const int tiles = (w1 - w0 + 7) >> 3;  // 256 channels
        for (int i = warp; i < T * tiles; i += DF_WARPS) {
            const int t = i / tiles, c = 32 * w0 + 256 * (i % tiles) + 8 * lane;
            uint32_t m = 0;
            if (c < 32 * w1 && as_in((long long)t * K + c + 7, (long long)T * K)) {
                float v[8];
                load_x(t, c, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
                    m = max(m, b < F32_INF_BITS ? b : 0u);
                }
            }
            m = __reduce_max_sync(0xffffffffu, m);
            if (lane == 0) atomicMax(&s_max[t], m);
        }
    }
    __syncthreads();
    if (a.after_select) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid < TP) {
        const float eta = (a.eta && tid < T) ? a.eta[tid] : 0.0f;
        s_eta[tid] = eta;
        const uint32_t top = __float_as_uint(__uint_as_float(s_max[tid]) + fabsf(eta));  // bounds |x - eta|
        int e = top == 0u ? 0 : 14 - ((int)(top >> 23) - 127);
        e = e > 126 ? 126 : (e < -113 ? -113 : e);
        s_mul[tid] = pow2f(e);
        s_inv[tid] = pow2f(-e);
    }

    float acc[8][NT][4];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

    for (int ws = w0; ws < w1; ws += C::KSUB / 32) {
        const int nw = min(C::KSUB / 32, w1 - ws), mine = steps_of(ws);
        if (a.stream_all && ws > w0) prologue(ws, true);
        for (int w = tid; w < nw; w += DF_THREADS) {
            uint32_t u = 0;
#pragma unroll
            for (int t = 0; t < TP; ++t) {
                uint32_t k = 0u;
                if (t < T)
                    k = !a.mask ? 0xFFFFFFFFu
                                : (as_in((long long)t * nwords + ws + w, (long long)T * nwords)
                                       ? a.mask[(size_t)t * nwords + ws + w] : 0u);
                s_keep[t][w] = k;
                u |= k;
            }
            s_union[w] = u;
        }
        __syncthreads();
        if (!a.stream_all) prologue(ws, false);
        // kept values, scaled, in PARTS f16 parts, each the rounding of what
        // the one before left
        const int groups = 4 * nw;
        for (int i = tid; i < TP * groups; i += DF_THREADS) {
            const int t = i / groups, g = i % groups;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            const uint32_t keep = (s_keep[t][g >> 2] >> (8 * (g & 3))) & 0xFFu;
            if (t < T && keep && as_in((long long)t * K + 32 * ws + 8 * g + 7, (long long)T * K)) {
                load_x(t, 32 * ws + 8 * g, v);
                const float eta = s_eta[t], mul = s_mul[t];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    v[e] = (keep >> e) & 1u ? __fmul_rn(a.eta ? __fsub_rn(v[e], eta) : v[e], mul) : 0.0f;
            }
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __half2 h = __floats2half2_rn(v[2 * k], v[2 * k + 1]);
                    w[k] = *reinterpret_cast<const uint32_t *>(&h);
                    if (p + 1 < PARTS) {  // nothing is left of an infinity
                        const float h0 = __low2float(h), h1 = __high2float(h);
                        v[2 * k] = isinf(h0) ? 0.0f : v[2 * k] - h0;
                        v[2 * k + 1] = isinf(h1) ? 0.0f : v[2 * k + 1] - h1;
                    }
                }
                *reinterpret_cast<uint4 *>(xs + ((size_t)p * TP + t) * C::XS + 8 * g) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        __syncthreads();

        for (int s = 0; s < mine; ++s) {
            cp_async_wait<DF_DEPTH - 2>();
            __syncwarp();  // the scale bytes were copied by other lanes
            const uint32_t src = ring + (uint32_t)(s % DF_DEPTH) * DF_STAGE;
            uint32_t wv[4][2];
#pragma unroll
            for (int r = 0; r < 4; ++r)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wv[r][0]), "=r"(wv[r][1])
                             : "r"(src + r * 256 + lane * 8) : "memory");
            uint32_t sc[4];
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(sc[0]), "=r"(sc[1]), "=r"(sc[2]), "=r"(sc[3]) : "r"(src + 1024 + g8 * 16) : "memory");
            issue(ws, s + DF_DEPTH - 1, mine, a.stream_all);
            uint32_t bx[NT][PARTS][2];
            const int cl = 16 * (DF_WARPS * s + warp) + 4 * q4;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const uint2 v = *reinterpret_cast<const uint2 *>(xs + ((size_t)p * TP + 8 * n + g8) * C::XS + cl);
                    bx[n][p][0] = v.x;
                    bx[n][p][1] = v.y;
                }
#pragma unroll
            for (int wd = 0; wd < 2; ++wd) {
                // codes of a channel pair in one byte: outputs p = 8 wd + 2 b
                // (lo, byte b) and p + 1 (hi), channels 4q, 4q+1 | 4q+2, 4q+3
                uint32_t A[4][4];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t x0 = wv[2 * k][wd], x1 = wv[2 * k + 1][wd];
                    e2m1x8((x0 & 0x0F0F0F0Fu) | ((x1 << 4) & 0xF0F0F0F0u), A[2 * k]);
                    e2m1x8(((x0 >> 4) & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u), A[2 * k + 1]);
                }
                float f[8];
                df_scales<FMT>(sc[2 * wd], *reinterpret_cast<float (*)[4]>(f));
                df_scales<FMT>(sc[2 * wd + 1], *reinterpret_cast<float (*)[4]>(f + 4));
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int p = PARTS - 1; p >= 0; --p)  // the small part first
                            mma_f16(d, A[0][b], A[1][b], A[2][b], A[3][b], bx[n][p][0], bx[n][p][1], d);
                        float (&o)[4] = acc[4 * wd + b][n];
                        o[0] = fmaf(f[2 * b], d[0], o[0]);
                        o[1] = fmaf(f[2 * b], d[1], o[1]);
                        o[2] = fmaf(f[2 * b + 1], d[2], o[2]);
                        o[3] = fmaf(f[2 * b + 1], d[3], o[3]);
                    }
            }
        }
        cp_async_wait<0>();
        __syncthreads();  // x and the ring are free
    }

    // warps in order, then the cluster's CTAs in order
    __syncthreads();
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float *r0 = red + ((size_t)warp * TP + 8 * n + 2 * q4) * DF_RSTRIDE + 16 * m + g8;
            r0[0] = acc[m][n][0];
            r0[DF_RSTRIDE] = acc[m][n][1];
            r0[8] = acc[m][n][2];
            r0[DF_RSTRIDE + 8] = acc[m][n][3];
        }
    __syncthreads();
    for (int i = tid; i < T * DF_COLS; i += DF_THREADS) {
        const int t = i / DF_COLS, at = t * DF_RSTRIDE + i % DF_COLS;
        float s = red[at];
#pragma unroll
        for (int w = 1; w < DF_WARPS; ++w) s += red[w * TP * DF_RSTRIDE + at];
        red[at] = s * s_inv[t];
    }
    cluster_sync_all();
    for (int i = rank * DF_THREADS + tid; i < T * DF_COLS; i += nranks * DF_THREADS) {
        const int t = i / DF_COLS, o = slice * DF_COLS + i % DF_COLS;
        const uint32_t at = smem_u32(red + t * DF_RSTRIDE + i % DF_COLS);
        float s = 0.0f;
        for (int r = 0; r < nranks; ++r) s += ld_cluster_f32(mapa_u32(at, (uint32_t)r));
        if (o >= n_out || !as_in((long long)t * n_out + o, (long long)T * n_out)) continue;
        s *= a.rowf[o];
        if (a.eta) s = fmaf(s_eta[t], a.rowsum[o], s);
        if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.y)[(size_t)t * n_out + o] = __float2bfloat16_rn(s);
        else static_cast<float *>(a.y)[(size_t)t * n_out + o] = s;
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
}

// CTAs of a cluster (along K): as many as fill the GPU, at least one step per
// warp, at most the portable cluster size.
static int df_ranks(int K, int n_out, int per_sm)
{
    const int slices = (n_out + DF_COLS - 1) / DF_COLS;
    int c = sm_count() * per_sm / slices;
    const int most = K / (16 * DF_WARPS);
    if (c > most) c = most;
    return c < 1 ? 1 : (c > 8 ? 8 : c);
}

template <int NT, int PARTS, int FMT>
static cudaError_t launch_df(const DecodeFp4Args &a, cudaStream_t st)
{
    using C = DfCfg<NT, PARTS>;
    static int done[64];
    cudaError_t e = smem_limit_once(k_decode_fp4<NT, PARTS, FMT>, C::smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int ranks = df_ranks(a.K, a.n_out, C::per_sm);
    cfg.gridDim = dim3(ranks, (a.n_out + DF_COLS - 1) / DF_COLS);
    cfg.blockDim = dim3(DF_THREADS);
    cfg.dynamicSmemBytes = C::smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, k_decode_fp4<NT, PARTS, FMT>, a);
}

template <int NT, int FMT>
static cudaError_t launch_df_parts(const DecodeFp4Args &a, cudaStream_t st)
{
    // a bf16 value without a shift fits one f16 part
    return a.bf16 && !a.eta ? launch_df<NT, 1, FMT>(a, st) : launch_df<NT, 2, FMT>(a, st);
}

cudaError_t launch_decode_fp4(DecodeFp4Args a, int fmt, cudaStream_t st)
{
    a.rowf = reinterpret_cast<const float *>(a.Wd + df_codes_bytes(a.n_out, a.K, fmt));
    if (fmt == AS_FP4_NV)
        return a.T <= 8 ? launch_df_parts<1, AS_FP4_NV>(a, st) : launch_df_parts<2, AS_FP4_NV>(a, st);
    return a.T <= 8 ? launch_df_parts<1, AS_FP4_MX>(a, st) : launch_df_parts<2, AS_FP4_MX>(a, st);
}

}  // namespace as
