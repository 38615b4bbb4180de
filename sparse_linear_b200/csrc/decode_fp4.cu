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
//   power of two that puts its largest |x| at 2^14: bf16 values are exact from
//   2^-28 of the largest up, smaller ones err by at most 2^-39 of it; two parts
//   hold 22 bits of a float32 value.
//
// Kernels of a call: (top-k: the selection kernel,) k_fp4_stage, k_decode_fp4,
// chained by programmatic dependent launch.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"
#include "select_util.cuh"

namespace as {

constexpr int DF_COLS = 128;     // output columns per slice
constexpr int DF_WARPS = 8;
constexpr int DF_THREADS = DF_WARPS * 32;
constexpr int DF_CODES = 1024 + 128;  // bytes of a 16-channel step: codes and scales
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

// ------------------------------------------------------------------ staging
// Grid (token, 2048-channel chunk).  Every CTA of a token reads the whole row
// (the same code and order as k_select_nm_decode: identical bits) for the mean
// and the largest |x|, selects its own channels (or takes a mask) and writes
// the keep words and the kept values as f16 parts, in the order the decode
// reads them: [16-channel step][column][16], part p of token t in column
// p * pstride + t.  Columns of no token are not written: they only reach sums
// that are not read.
constexpr int DS_THREADS = 256;
constexpr int DS_CHUNK = DS_THREADS * 8;
constexpr int DS_ROWREG = 8;  // row loads in flight per thread

struct StageArgs {
    const void *x;
    int T, K, cols, pstride;
    int score_f, sel, n, m, dpts;  // score_f: multiply |x| by f
    float tau;
    const float *eta_static, *f;
    const uint32_t *mask_in;  // selection made before, with its eta in eta_in; or nullptr
    const float *eta_in;
    uint32_t *mask;  // keep words, written unless mask_in
    float *eta;      // [T], written unless mask_in (with a shift)
    float *inv;      // [T] power of two that undoes the scaling
    __half *xh;
};

template <typename TX, int PARTS>
__global__ void __launch_bounds__(DS_THREADS) k_fp4_stage(StageArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // after the wait: see k_select_nm_decode
    __shared__ double red[DS_THREADS / 32];
    __shared__ uint32_t redm[DS_THREADS / 32];
    const int t = blockIdx.x, chunk = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int K = a.K, ng = K >> 3, words = (K + 31) >> 5;
    const TX *xr = static_cast<const TX *>(a.x) + (size_t)t * K;
    const int c0 = chunk * DS_CHUNK + warp * 256 + 8 * lane;  // this lane's 8 channels
    const bool act = c0 < K;

    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0}, f[8];
    if (act) load8(xr + c0, v);
    const bool has_f = a.score_f && act && !a.mask_in;
    if (has_f) load8f(a.f + c0, f);
    uint32_t word = 0xFFFFFFFFu;
    if (a.mask_in && act) word = a.mask_in[(size_t)t * words + (c0 >> 5)];
    float eta = !a.dpts ? 0.0f : (a.mask_in ? a.eta_in[t] : (a.dpts == AS_PTS_STATIC ? a.eta_static[t] : 0.0f));
    const bool mean = a.dpts == AS_PTS_DYNAMIC && !a.mask_in;

    double sum = 0.0;
    uint32_t top = 0;  // largest finite |x| (bits)
    for (int g0 = 0; g0 < ng; g0 += DS_ROWREG * DS_THREADS) {
        float w[DS_ROWREG][8];
#pragma unroll
        for (int r = 0; r < DS_ROWREG; ++r) {
            const int g = g0 + tid + r * DS_THREADS;
            if (g < ng) load8(xr + 8 * (size_t)g, w[r]);
        }
#pragma unroll
        for (int r = 0; r < DS_ROWREG; ++r) {
            const int g = g0 + tid + r * DS_THREADS;
            if (g < ng) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (mean) sum += (double)w[r][e];
                    const uint32_t b = __float_as_uint(w[r][e]) & 0x7FFFFFFFu;
                    top = max(top, b < F32_INF_BITS ? b : 0u);
                }
            }
        }
    }
    if (mean) {
        sum = warp_sum_f64(sum);
        if (lane == 0) red[warp] = sum;
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0) redm[warp] = top;
    __syncthreads();
    if (mean) {
        double tot = 0.0;
#pragma unroll
        for (int w = 0; w < DS_THREADS / 32; ++w) tot += red[w];
        eta = (float)(tot / (double)K);
    }
#pragma unroll
    for (int w = 0; w < DS_THREADS / 32; ++w) top = max(top, redm[w]);
    const uint32_t bound = __float_as_uint(__uint_as_float(top) + fabsf(eta));  // |x - eta| is at most this
    int e = bound == 0u ? 0 : 14 - ((int)(bound >> 23) - 127);
    e = e > 126 ? 126 : (e < -113 ? -113 : e);
    if (chunk == 0 && tid == 0) {
        a.inv[t] = pow2f(-e);
        if (a.dpts && !a.mask_in) a.eta[t] = eta;
    }
    float xh[8], sc[8];
    score8(v, a.dpts, eta, has_f ? f : nullptr, 0, xh, sc);
    uint32_t keep;
    if (a.mask_in) {
        keep = (word >> (8 * (lane & 3))) & 0xFFu;
    } else {
        keep = a.sel == AS_SEL_NM ? nm_keep_dispatch(sc, lane, a.n, a.m)
                                  : (a.sel == AS_SEL_THRESH ? keep_thresh(sc, a.tau) : 0xFFu);
        if (!act) keep = 0;
        word = keep << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        const int wi = c0 >> 5;
        if ((lane & 3) == 0 && act && as_in((long long)t * words + wi, (long long)a.T * words))
            a.mask[(size_t)t * words + wi] = word;
    }
    if (!act) return;
    // two or one f16 parts, the second the rounding of what the first left
    const float mul = pow2f(e);
#pragma unroll
    for (int k = 0; k < 8; ++k) xh[k] = (keep >> k) & 1u ? __fmul_rn(xh[k], mul) : 0.0f;
    __half *out = a.xh + ((size_t)(c0 >> 4) * a.cols + t) * 16 + (c0 & 8);
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const __half2 h = __floats2half2_rn(xh[2 * k], xh[2 * k + 1]);
            w[k] = *reinterpret_cast<const uint32_t *>(&h);
            if (p + 1 < PARTS) {  // nothing is left of an infinity
                const float h0 = __low2float(h), h1 = __high2float(h);
                xh[2 * k] = isinf(h0) ? 0.0f : xh[2 * k] - h0;
                xh[2 * k + 1] = isinf(h1) ? 0.0f : xh[2 * k + 1] - h1;
            }
        }
        *reinterpret_cast<uint4 *>(out + (size_t)p * a.pstride * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// ------------------------------------------------------------------ decode
// CTA (rank of a cluster, slice): the slice's 128 columns and a contiguous
// part of K; its warps take 16-channel steps in turn, each with a cp.async
// ring of its own (codes of kept rows, scales, staged x of a step).  Rows that
// no token keeps are not loaded (but for the first steps, which are asked for
// before the selection is known): their kept values are zero and a code is
// finite whatever its bits.  The warps' sums are added in shared memory; each
// CTA then sends every other its share of them and adds up what it receives,
// both in a fixed order.
//
// NT: 8-column tiles of staged values.  A value of two parts takes two columns
// of one tile while both fit (up to 4 tokens in one tile, up to 8 in two);
// PARTS = 2 (9 to 16 tokens) runs the second part as MMAs of its own.
template <int NT, int PARTS>
struct DfCfg {
    static constexpr int TP = 8 * NT;
    static constexpr int XB = PARTS * TP * 32;       // staged x of a step, bytes
    static constexpr int STAGE = DF_CODES + XB;
    static constexpr int DEPTH = NT * PARTS == 4 ? 5 : (NT == 2 ? 7 : 8);  // steps in flight per warp: two CTAs per SM fit
    static constexpr size_t ring = (size_t)DF_WARPS * DEPTH * STAGE;
    static constexpr size_t red = (size_t)DF_WARPS * TP * DF_RSTRIDE * 4;
    static constexpr size_t big = ring > red ? ring : red;
    static constexpr size_t recv = (size_t)TP * DF_COLS * 4 + 16 * 8 * 4;  // the shares of 8 CTAs, rounded up
    static constexpr size_t smem = big + recv;
    static_assert(smem + 4 * 1024 + 1024 <= 113 * 1024, "two CTAs per SM");
};

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
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

// D = A B and D += A B.
__device__ __forceinline__ void mma_f16_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ void mma_f16_add(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

constexpr int DF_MAXW = 512;  // keep words of a CTA's range held in shared memory

template <int NT, int PARTS, int FMT>
__global__ void __launch_bounds__(DF_THREADS, 2) k_decode_fp4(DecodeFp4Args a)
{
    using C = DfCfg<NT, PARTS>;
    constexpr int TP = C::TP, DEPTH = C::DEPTH;
    extern __shared__ __align__(16) unsigned char smem[];
    float *red = reinterpret_cast<float *>(smem);  // after the main loop
    __shared__ uint32_t s_union[DF_MAXW];

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g8 = lane >> 2, q4 = lane & 3;
    const int rank = (int)cluster_ctarank(), nranks = gridDim.x, slice = blockIdx.y;
    const int T = a.T, K = a.K, n_out = a.n_out;
    const int nwords = K >> 5, wper = (nwords + nranks - 1) / nranks;
    const int w0 = min(nwords, rank * wper), w1 = min(nwords, w0 + wper);
    const uint8_t *wslice = a.Wd + (size_t)slice * (size_t)(K / fp4_block(FMT)) * df_unit(FMT);
    const uint32_t ring = smem_u32(smem) + (uint32_t)warp * (DEPTH * C::STAGE);
    // step s of this warp: channels 32 w0 + 16 (DF_WARPS s + warp) ..
    const int nsteps = 2 * (w1 - w0);
    const int mine = nsteps > warp ? (nsteps - warp + DF_WARPS - 1) / DF_WARPS : 0;
    // 16-byte piece `lane` (and lane + 32) of the 16 rows: row 4r + q of channel 4q + r
    const int bit0 = 4 * ((lane >> 2) & 3) + (lane >> 4), bit1 = bit0 + 2;
    // sources of the step that is issued next, and its slot
    const int b0 = 2 * w0 + warp;
    constexpr size_t CSTEP = (size_t)DF_WARPS * (FMT == AS_FP4_NV ? df_unit(FMT) : df_unit(FMT) / 2);
    const uint8_t *cp = (FMT == AS_FP4_NV ? wslice + (size_t)b0 * df_unit(FMT)
                                          : wslice + (size_t)(b0 >> 1) * df_unit(FMT) + (b0 & 1) * 1024) + 16 * lane;
    const size_t sc_off = FMT == AS_FP4_NV ? 1024 : 2048 - (b0 & 1) * 1024;  // scales from the step's codes
    const uint8_t *xp = reinterpret_cast<const uint8_t *>(a.xh) + (size_t)b0 * C::XB + 16 * lane;

    auto issue_codes = [&](uint32_t dst, uint32_t keep) {
        if ((keep >> bit0) & 1u) cp_async16(dst, cp, 16u);
        if ((keep >> bit1) & 1u) cp_async16(dst + 512, cp + 512, 16u);
        if (lane < 8) cp_async16(dst + 1024, cp + sc_off, 16u);
        cp += CSTEP;
    };
    auto issue_x = [&](uint32_t dst) {
#pragma unroll
        for (int i = 0; i < (C::XB + 511) / 512; ++i)
            if (512 * i + 16 * lane < C::XB) cp_async16(dst + DF_CODES + 512 * i, xp + 512 * i, 16u);
        xp += (size_t)DF_WARPS * C::XB;
    };
    const uint32_t my = ring + 16 * lane;

    // Remote stores need their CTA to be running: the wait for these arrivals
    // comes before the first of them.
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    // The staging kernel lets this one start after its own wait, so everything
    // before that kernel in the stream (the weights among it) is complete: the
    // codes of the first steps come before the wait for the staged x, whole,
    // since the selection is not known yet.
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s)
        if (s < mine) issue_codes(my + s * C::STAGE, 0xFFFFu);
    asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
    for (int s = 0; s < DEPTH - 1; ++s) {
        if (s < mine) issue_x(my + s * C::STAGE);
        cp_async_commit();  // the first group also holds the codes before the wait
    }
    // rows that some token keeps, for the steps that are still to be issued
    if (!a.stream_all && nsteps > DF_WARPS * (DEPTH - 1)) {
        for (int w = tid; w < min(w1 - w0, DF_MAXW); w += DF_THREADS) {
            uint32_t u = 0;
            for (int t = 0; t < T; ++t)
                if (as_in((long long)t * nwords + w0 + w, (long long)T * nwords))
                    u |= a.mask[(size_t)t * nwords + w0 + w];
            s_union[w] = u;
        }
        __syncthreads();
    }
    auto kept_rows = [&](int s) -> uint32_t {
        const int lb = DF_WARPS * s + warp, w = lb >> 1;
        if (a.stream_all || w >= DF_MAXW) return 0xFFFFu;
        return (s_union[w] >> (16 * (lb & 1))) & 0xFFFFu;
    };

    float acc[8][NT][4];
#pragma unroll
    for (int m = 0; m < 8; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.0f;

    uint32_t src = ring, dst = my + (DEPTH - 1) * C::STAGE;
    for (int s = 0; s < mine; ++s) {
        cp_async_wait<DEPTH - 2>();
        __syncwarp();  // a step's pieces were copied by all lanes
        uint32_t wv[4][2];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(wv[r][0]), "=r"(wv[r][1])
                         : "r"(src + r * 256 + q4 * 64 + g8 * 8) : "memory");
        uint32_t sc[4];
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(sc[0]), "=r"(sc[1]), "=r"(sc[2]), "=r"(sc[3]) : "r"(src + 1024 + g8 * 16) : "memory");
        uint32_t bx[NT][PARTS][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(bx[n][p][0]), "=r"(bx[n][p][1])
                             : "r"(src + DF_CODES + (p * TP + 8 * n + g8) * 32 + q4 * 8) : "memory");
        if (s + DEPTH - 1 < mine) {  // into the slot read at s - 1
            issue_codes(dst, kept_rows(s + DEPTH - 1));
            issue_x(dst);
        }
        cp_async_commit();
        dst = src + 16 * lane;  // free after this step
        src += C::STAGE;
        if (src == ring + DEPTH * C::STAGE) src = ring;
#pragma unroll
        for (int wd = 0; wd < 2; ++wd) {
            // codes of a channel pair in one byte: outputs p = 8 wd + 2 b (A[0],
            // A[2], byte b) and p + 1 (A[1], A[3]); channels 4q, 4q+1 | 4q+2, 4q+3
            uint32_t A[4][4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t x0 = wv[2 * k][wd], x1 = wv[2 * k + 1][wd];
                e2m1x8((x0 & 0x0F0F0F0Fu) | ((x1 << 4) & 0xF0F0F0F0u), A[2 * k]);
                e2m1x8(((x0 >> 4) & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u), A[2 * k + 1]);
            }
            float f[2][4];
            df_scales<FMT>(sc[2 * wd], f[0]);
            df_scales<FMT>(sc[2 * wd + 1], f[1]);
#pragma unroll
            for (int b = 0; b < 4; ++b)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float d[4];  // the small part first
                    mma_f16_zero(d, A[0][b], A[1][b], A[2][b], A[3][b], bx[n][PARTS - 1][0], bx[n][PARTS - 1][1]);
                    if constexpr (PARTS == 2) mma_f16_add(d, A[0][b], A[1][b], A[2][b], A[3][b], bx[n][0][0], bx[n][0][1]);
                    float (&o)[4] = acc[4 * wd + b][n];
                    const float f0 = f[b >> 1][2 * (b & 1)], f1 = f[b >> 1][2 * (b & 1) + 1];
                    o[0] = fmaf(f0, d[0], o[0]);
                    o[1] = fmaf(f0, d[1], o[1]);
                    o[2] = fmaf(f1, d[2], o[2]);
                    o[3] = fmaf(f1, d[3], o[3]);
                }
        }
    }
    cp_async_wait<0>();

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
    // element i of the T * 128 sums belongs to CTA i / share; rank r's share of
    // it lands in slot r of that CTA
    const int total = T * DF_COLS, share = (total + nranks - 1) / nranks;
    float *recv = reinterpret_cast<float *>(smem + C::big);
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster has started
    for (int i = tid; i < total; i += DF_THREADS) {
        const int t = i / DF_COLS, at = t * DF_RSTRIDE + i % DF_COLS;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < DF_WARPS; ++w) {
            s += red[w * TP * DF_RSTRIDE + at];
            if (a.part_cols) s += red[w * TP * DF_RSTRIDE + at + a.part_cols * DF_RSTRIDE];  // the second part
        }
        const int owner = i / share;
        st_cluster_f32(mapa_u32(smem_u32(recv + rank * share + i - owner * share), (uint32_t)owner), s * a.inv[t]);
    }
    cluster_sync_all();
    for (int k = tid; k < share; k += DF_THREADS) {
        const int i = rank * share + k;
        if (i >= total) break;
        const int t = i / DF_COLS, o = slice * DF_COLS + i % DF_COLS;
        if (o >= n_out || !as_in((long long)t * n_out + o, (long long)T * n_out)) continue;
        float s = 0.0f;
        for (int r = 0; r < nranks; ++r) s += recv[r * share + k];
        s *= a.rowf[o];
        if (a.eta) s = fmaf(a.eta[t], a.rowsum[o], s);
        if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.y)[(size_t)t * n_out + o] = __float2bfloat16_rn(s);
        else static_cast<float *>(a.y)[(size_t)t * n_out + o] = s;
    }
}

// CTAs of a cluster (along K): as many as fill the GPU (two per SM), at least
// one step per warp, at most the portable cluster size.
static int df_ranks(int K, int n_out)
{
    const int slices = (n_out + DF_COLS - 1) / DF_COLS;
    int c = 2 * sm_count() / slices;
    const int most = K / (16 * DF_WARPS);
    if (c > most) c = most;
    return c < 1 ? 1 : (c > 8 ? 8 : c);
}

static void df_launch(cudaLaunchConfig_t &cfg, cudaLaunchAttribute *attr, dim3 grid, int threads, size_t smem,
                      int ranks, cudaStream_t st)
{
    cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ranks;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ranks > 0 ? 2 : 1;
}

template <int NT, int PARTS, int FMT>
static cudaError_t launch_df(const DecodeFp4Args &a, cudaStream_t st)
{
    using C = DfCfg<NT, PARTS>;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    static int done[64];
    cudaError_t e = smem_limit_once(k_decode_fp4<NT, PARTS, FMT>, C::smem, done);
    if (e != cudaSuccess) return e;
    const int ranks = df_ranks(a.K, a.n_out);
    df_launch(cfg, attr, dim3(ranks, (a.n_out + DF_COLS - 1) / DF_COLS), DF_THREADS, C::smem, ranks, st);
    return cudaLaunchKernelEx(&cfg, k_decode_fp4<NT, PARTS, FMT>, a);
}

template <int PARTS>
static cudaError_t launch_stage(const StageArgs &s, int bf16, cudaStream_t st)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    df_launch(cfg, attr, dim3(s.T, (s.K + DS_CHUNK - 1) / DS_CHUNK), DS_THREADS, 0, 0, st);
    return bf16 ? cudaLaunchKernelEx(&cfg, k_fp4_stage<__nv_bfloat16, PARTS>, s)
                : cudaLaunchKernelEx(&cfg, k_fp4_stage<float, PARTS>, s);
}

// columns that staged values take: parts of a token side by side while they
// fit two tiles
static int df_cols(int T, int parts) { return T * parts <= 8 ? 8 : (T * parts <= 16 ? 16 : 32); }

template <int FMT>
static cudaError_t launch_df_cols(const DecodeFp4Args &a, int cols, cudaStream_t st)
{
    if (cols == 8) return launch_df<1, 1, FMT>(a, st);
    return cols == 16 ? launch_df<2, 1, FMT>(a, st) : launch_df<2, 2, FMT>(a, st);
}

// keep words, eta, scale factors, staged x (for two parts)
DecodeFp4Layout decode_fp4_layout(int T, int K)
{
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    DecodeFp4Layout l{};
    l.eta = up((size_t)T * ((K + 31) / 32) * sizeof(uint32_t));
    l.inv = l.eta + up((size_t)T * sizeof(float));
    l.xh = l.inv + up((size_t)T * sizeof(float));
    l.bytes = l.xh + up((size_t)K * df_cols(T, 2) * sizeof(__half));
    return l;
}

cudaError_t launch_decode_fp4(DecodeFp4Args a, const SelectArgs &sel, bool selected, void *ws, int fmt, cudaStream_t st)
{
    const DecodeFp4Layout l = decode_fp4_layout(a.T, a.K);
    char *w = static_cast<char *>(ws);
    a.rowf = reinterpret_cast<const float *>(a.Wd + df_codes_bytes(a.n_out, a.K, fmt));
    a.inv = reinterpret_cast<const float *>(w + l.inv);
    a.xh = w + l.xh;
    StageArgs s{};
    s.x = a.x;
    s.T = a.T;
    s.K = a.K;
    // a bf16 value without a shift fits one f16 part
    const int parts = a.bf16 && !a.eta ? 1 : 2;
    s.cols = df_cols(a.T, parts);
    s.pstride = s.cols / 2;
    a.part_cols = parts == 2 && s.cols <= 16 ? s.pstride : 0;
    s.score_f = sel.f != nullptr;
    s.sel = sel.sel;
    s.n = sel.n;
    s.m = sel.m;
    s.dpts = sel.dpts;
    s.tau = sel.tau;
    s.eta_static = sel.eta_static;
    s.f = sel.f;
    s.mask_in = selected ? sel.bitmask : nullptr;
    s.eta_in = selected ? sel.eta : nullptr;
    s.mask = sel.bitmask;
    s.eta = sel.eta;
    s.inv = reinterpret_cast<float *>(w + l.inv);
    s.xh = reinterpret_cast<__half *>(w + l.xh);
    const cudaError_t e = parts == 1 ? launch_stage<1>(s, a.bf16, st) : launch_stage<2>(s, a.bf16, st);
    if (e != cudaSuccess) return e;
    return fmt == AS_FP4_NV ? launch_df_cols<AS_FP4_NV>(a, s.cols, st) : launch_df_cols<AS_FP4_MX>(a, s.cols, st);
}

}  // namespace as
