// Decode on microscaled 4-bit weights: y = prune(x) W^T for 1..16 tokens,
// reading only the codes of the channels that some token keeps.
//
// Weight layout (k_fp4_decode_layout, once per layer).  Slices of 128 output
// columns; in a slice one unit per scale block of B channels: B rows of 64
// bytes (the block's channels), then the 128 outputs' scales.  Inside 16
// channels, row 4r + q holds channel 4q + r; its 8-byte piece g holds outputs
// o(p, g) = 16 (p >> 1) + 8 (p & 1) + g, p = 0..15: exactly what lane
// (g, q) of an m16n8k16 fragment needs, so a lane's four pieces need no
// exchange with other lanes.
//   A 16-bit half of a piece holds four codes with their bits placed so that
// a shift and a mask give bf16 patterns: magnitude bits at 6..8 (the two
// lowest exponent bits and the top mantissa bit), sign at 15.  Such a pattern
// is the E2M1 value times 2^-126 (E2M1 subnormals are bf16 subnormals).
//   Scales are recoded to 8 bits that shift into a bf16 of scale * 2^119
// (NV: 5 exponent and 3 mantissa bits, which hold E4M3's subnormals as
// normal numbers; MX: the exponent, relative to the row's largest so that
// the range always fits).  pattern * scale is then the weight times 2^-7
// (MX: times a power of two of its row), exact in bf16: at most 2 + 4
// significant bits.  A float32 factor per output undoes the power of two and
// carries the weight's row scale.
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
        rowf[o] = bad ? __uint_as_float(0x7FFFFFFFu) : ldexpf(ws, fmt == AS_FP4_MX ? (int)m - 128 : 7);
        top[o] = (int)m;
    }
}

// Code j of a half: magnitude and sign bits at their places (see above).
__device__ __forceinline__ uint32_t df_place(uint32_t code, int j)
{
    const int mp[4] = {6, 9, 0, 3}, sp[4] = {15, 14, 13, 12};
    return ((code & 7u) << mp[j]) | ((code >> 3) << sp[j]);
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
        if constexpr (FMT == AS_FP4_MX) {
            const int f = s == 255u ? 0 : (int)s - top[o] + 254;  // a NaN scale shows in the output's factor
            scale = f > 0 ? (uint32_t)f : 0u;
        } else {
            const uint32_t e = (s >> 3) & 15u, m = s & 7u;
            if ((s & 127u) != 127u && (s & 127u) != 0u) {
                if (e > 0) {
                    scale = ((e + 15u) << 3) | m;  // exponent e - 7, field + 22
                } else {                            // m * 2^-9, normalised
                    const uint32_t h = 31u - (uint32_t)__clz((int)m);
                    scale = ((h + 13u) << 3) | ((m << (3u - h)) & 7u);
                }
            }
        }
        if (scale == 0u) {  // a zero scale stands for zeros
#pragma unroll
            for (int i = 0; i < B / 8; ++i) w[i] = 0u;
        }
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
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int p = wd * 8 + h * 4 + j;
                word |= df_place(nib[ch][16 * (p >> 1) + 8 * (p & 1) + g], j) << (16 * h);
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
// the CTA stages in shared memory as PARTS bf16 arrays (zero where a token
// dropped the channel, so rows that were not loaded do not matter).  The
// warps' sums are added in shared memory and the cluster's through
// distributed shared memory, both in a fixed order.
template <int NT, int PARTS>
struct DfCfg {
    static constexpr int TP = 8 * NT;
    static constexpr int KSUB = NT * PARTS == 1 ? 2048 : 1024;  // channels of x staged at a time
    static constexpr int XS = KSUB + 16;                        // row stride: token rows 8 banks apart
    static constexpr size_t xbytes = (size_t)PARTS * TP * XS * 2;
    static constexpr size_t ring = (size_t)DF_WARPS * DF_DEPTH * DF_STAGE;
    static constexpr size_t red = (size_t)DF_WARPS * TP * DF_RSTRIDE * 4;
    static constexpr size_t big = ring > red ? ring : red;
    static constexpr size_t smem = big + xbytes;
    static constexpr int per_sm = smem <= 110 * 1024 ? 2 : 1;
};

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

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

template <int NT, int PARTS, int FMT>
__global__ void __launch_bounds__(DF_THREADS, DfCfg<NT, PARTS>::per_sm) k_decode_fp4(DecodeFp4Args a)
{
    using C = DfCfg<NT, PARTS>;
    constexpr int TP = C::TP;
    extern __shared__ __align__(16) unsigned char smem[];
    float *red = reinterpret_cast<float *>(smem);  // after the main loop
    __nv_bfloat16 *xs = reinterpret_cast<__nv_bfloat16 *>(smem + C::big);
    __shared__ uint32_t s_keep[TP][C::KSUB / 32];
    __shared__ uint32_t s_union[C::KSUB / 32];
    __shared__ float s_eta[TP];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, q4 = lane & 3;
    const int rank = (int)cluster_ctarank(), nranks = gridDim.x, slice = blockIdx.y;
    const int T = a.T, K = a.K, n_out = a.n_out;
    const int nwords = K >> 5, wper = (nwords + nranks - 1) / nranks;
    const int w0 = min(nwords, rank * wper), w1 = min(nwords, w0 + wper);
    const uint8_t *wslice = a.Wd + (size_t)slice * (size_t)(K / fp4_block(FMT)) * df_unit(FMT);
    const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (DF_DEPTH * DF_STAGE);

    float acc[8][NT][4];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

    bool waited = false;
    for (int ws = w0; ws < w1; ws += C::KSUB / 32) {
        const int nw = min(C::KSUB / 32, w1 - ws), nsteps = 2 * nw;  // 16-channel steps of this part
        // step s of this warp covers channels 32 ws + 16 (DF_WARPS s + warp)
        const int mine = nsteps > warp ? (nsteps - warp + DF_WARPS - 1) / DF_WARPS : 0;
        auto issue = [&](int s, bool all) {
            if (s < mine) {
                const int lb = DF_WARPS * s + warp, b = 2 * ws + lb;
                const uint32_t keep = all ? 0xFFFFu : (s_union[lb >> 1] >> (16 * (lb & 1))) & 0xFFFFu;
                const uint8_t *unit = FMT == AS_FP4_NV ? wslice + (size_t)b * df_unit(FMT)
                                                       : wslice + (size_t)(b >> 1) * df_unit(FMT) + (b & 1) * 1024;
                const uint32_t dst = ring + (uint32_t)(s % DF_DEPTH) * DF_STAGE;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if ((keep >> (4 * q4 + r)) & 1u) cp_async8(dst + r * 256 + lane * 8, unit + r * 256 + q4 * 64 + g8 * 8);
                const uint8_t *sc = FMT == AS_FP4_NV ? unit + 1024
                                                     : wslice + (size_t)(b >> 1) * df_unit(FMT) + 2048;
                if (lane < 8) cp_async16(dst + 1024 + lane * 16, sc + lane * 16, 16u);
            }
            cp_async_commit();
        };
        // every channel is wanted: the stream does not depend on the selection.
        // The select kernel lets this one start after its own wait, so all
        // work before it in the stream, the weights among it, is complete.
        if (a.stream_all && (a.after_select || waited)) {
#pragma unroll
            for (int s = 0; s < DF_DEPTH - 1; ++s) issue(s, true);
        }
        if (!waited) {
            asm volatile("griddepcontrol.wait;" ::: "memory");
            waited = true;
            if (a.stream_all && !a.after_select) {
#pragma unroll
                for (int s = 0; s < DF_DEPTH - 1; ++s) issue(s, true);
            }
            if (tid < TP) s_eta[tid] = (a.eta && tid < T) ? a.eta[tid] : 0.0f;
        }
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
        if (!a.stream_all) {
#pragma unroll
            for (int s = 0; s < DF_DEPTH - 1; ++s) issue(s, false);
        }
        // kept values, in PARTS bf16 parts: v = p0 + p1 + p2, each the
        // rounding of what the ones before left
        const int groups = 4 * nw;
        for (int i = tid; i < TP * groups; i += DF_THREADS) {
            const int t = i / groups, g = i % groups;
            float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            const uint32_t keep = (s_keep[t][g >> 2] >> (8 * (g & 3))) & 0xFFu;
            if (t < T && keep && as_in((long long)t * K + 32 * ws + 8 * g + 7, (long long)T * K)) {
                const size_t at = (size_t)t * K + 32 * (size_t)ws + 8 * (size_t)g;
                if (a.bf16) load8(static_cast<const __nv_bfloat16 *>(a.x) + at, v);
                else load8(static_cast<const float *>(a.x) + at, v);
                const float eta = s_eta[t];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = (keep >> e) & 1u ? (a.eta ? __fsub_rn(v[e], eta) : v[e]) : 0.0f;
            }
#pragma unroll
            for (int p = 0; p < PARTS; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
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
            issue(s + DF_DEPTH - 1, a.stream_all);
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
            for (int wd = 0; wd < 2; ++wd)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t sel = h ? 0x7632u : 0x5410u;
                    const uint32_t X[2] = {__byte_perm(wv[0][wd], wv[1][wd], sel), __byte_perm(wv[2][wd], wv[3][wd], sel)};
                    uint32_t A[4][2];  // code j, channel pair
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        A[0][k] = X[k] & 0x81C081C0u;
                        A[1][k] = ((X[k] >> 3) & 0x01C001C0u) | ((X[k] << 1) & 0x80008000u);
                        A[2][k] = ((X[k] << 6) & 0x01C001C0u) | ((X[k] << 2) & 0x80008000u);
                        A[3][k] = (X[k] << 3) & 0x81C081C0u;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int p = wd * 8 + h * 4 + j;
                        const uint32_t dup = __byte_perm(sc[p >> 2], 0u, 0x4040u | (uint32_t)(p & 3) | ((uint32_t)(p & 3) << 8));
                        // byte in bits 0..7 and 16..23
                        const uint32_t s2 = FMT == AS_FP4_NV ? dup * 16u + 0x70007000u : dup * 128u;
                        A[j][0] = bf16x2_mul(A[j][0], s2);
                        A[j][1] = bf16x2_mul(A[j][1], s2);
                    }
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int p = 0; p < PARTS; ++p)
                                mma_16816(acc[wd * 4 + h * 2 + m][n], A[2 * m][0], A[2 * m + 1][0], A[2 * m][1],
                                          A[2 * m + 1][1], bx[n][p][0], bx[n][p][1]);
                }
        }
        cp_async_wait<0>();
        __syncthreads();  // x and the ring are free
    }
    if (!waited) {  // a rank without channels
        asm volatile("griddepcontrol.wait;" ::: "memory");
        if (tid < TP) s_eta[tid] = (a.eta && tid < T) ? a.eta[tid] : 0.0f;
        __syncthreads();
    }

    // warps in order, then the cluster's CTAs in order
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
        const int at = (i / DF_COLS) * DF_RSTRIDE + i % DF_COLS;
        float s = red[at];
#pragma unroll
        for (int w = 1; w < DF_WARPS; ++w) s += red[w * TP * DF_RSTRIDE + at];
        red[at] = s;
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
    // kept values: bf16 x without a shift is one bf16 part exactly; else
    // three parts hold a float32 (24 bits) exactly, and two are within 2^-17,
    // far inside the half step (2^-9) of a bf16 output
    if (a.bf16 && !a.eta) return launch_df<NT, 1, FMT>(a, st);
    return a.out_bf16 ? launch_df<NT, 2, FMT>(a, st) : launch_df<NT, 3, FMT>(a, st);
}

cudaError_t launch_decode_fp4(DecodeFp4Args a, int fmt, cudaStream_t st)
{
    a.rowf = reinterpret_cast<const float *>(a.Wd + df_codes_bytes(a.n_out, a.K, fmt));
    if (fmt == AS_FP4_NV)
        return a.T <= 8 ? launch_df_parts<1, AS_FP4_NV>(a, st) : launch_df_parts<2, AS_FP4_NV>(a, st);
    return a.T <= 8 ? launch_df_parts<1, AS_FP4_MX>(a, st) : launch_df_parts<2, AS_FP4_MX>(a, st);
}

}  // namespace as
