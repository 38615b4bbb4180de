// Decode on microscaled 4-bit weights: y = prune(x) W^T for 1..16 tokens.
//
// The weights go to the tensor cores as they are stored, codes and block
// scales (tcgen05.mma kind::mxf4nvf4), with the outputs on the M = 128 side,
// so that nothing is unpacked and the kernel is bound by the bytes of W.  The
// kept values of x enter as a sum of P four-bit parts,
//   xhat m = S sum_p s_b 8^-p code_p  (+ rest),
// with a power of two S per token (MX: 1) and one scale s_b per block: the
// smallest E4M3 value (NV) or power of two (MX) that leaves no value of the
// block above 4 s_b S.  Up to 4 the codes' steps are at most 1, so that a part
// leaves at most 1/2, which is 4 for the next one: P parts leave at most
// s_b S 8^-(P-1) / 2.  MX: s_b is below half the block's largest value M (its
// smallest scale is 2^-126).  NV: s_b S is at most 9/32 M, and for scales among
// E4M3's subnormals at most M/4 + 2^-9 S with S < amax/896 of the token's
// largest, below 0.54 M where M is at least 2^-17 amax.  So P parts leave at
// most 0.27 8^-(P-1) M: 8 parts for bf16 output 2^-22 M, 10 parts for float32
// output 2^-28 M.  All factors are powers of two: only the parts themselves
// and their sum in the epilogue round.  Each part of each token is a column of the
// product (T P <= 160 of at most 256); the epilogue adds a token's columns in
// float32, smallest first.
//   (Powers of 6 with the block's largest value at 6 were used first, 7 and 10
// parts: 2^-17.7 M and 2^-25.5 M, with a rounded factor per part.)
//   Every channel's codes are read.  Reading only the rows of kept channels
// was built first (channel-major codes, cp.async, unpacking for mma.sync):
// 8:16 with one token halves the bytes, but the unpacking bound it: 14.5 us a
// call at 11008 x 4096 with one token and 21.9 us at 14336 x 4096 with 16,
// against 25 MB / 6.5 TB/s = 3.9 us and 5.0 us of weight bytes here.
//
// Kernels of a call, chained by programmatic dependent launch: (top-k: the
// selection kernel,) k_fp4_stage, which makes the selection and the parts,
// and k_decode_fp4, whose weight copies start before the parts are ready.  (One
// kernel, every CTA making the parts of its own channels, took 15.0 us against
// 10.7 us of both in a set-up of its own: the row's mean and the parts are then
// computed 32 times over, beside the weight stream.)
//   Calls one after another in a graph over weights of 400 MB, bf16 with 8:16:
// 11008 x 4096 NV, one token, 9.9 us (25 MB: 2.5 TB/s), with the token shift
// 10.3 us; 14336 x 4096 MX, 16 tokens, 12.3 us (float32 output 13.5); 14336 x
// 11008 NV, one token, 19.1 us (89 MB: 4.6 TB/s).  What is not weight stream is
// the staging (about 5 us), the first loads' latency and the exchange.
#include "common.cuh"
#include "fp4.cuh"
#include "kernels.cuh"
#include "select_util.cuh"

namespace as {

constexpr int DF_ROWS = 128;  // outputs per tile
constexpr int DF_KB = 256;    // channels per stage
constexpr int DF_WTILE = DF_ROWS * DF_KB / 2;
constexpr int DF_PARTS_BF16 = 8, DF_PARTS_F32 = 10;  // by the output's type

static int df_kblocks(int K) { return (K + DF_KB - 1) / DF_KB; }
static int df_mtiles(int n_out) { return (n_out + DF_ROWS - 1) / DF_ROWS; }
// A tile of Wd: 128 rows x 128 bytes of codes as the 128-byte-swizzled operand
// image, then the scale tiles of the K block.
__host__ __device__ constexpr int df_unit(int fmt) { return DF_WTILE + (fmt == AS_FP4_NV ? 4 : 2) * 512; }

// tiles, then the float32 row scale of every output
size_t fp4_decode_bytes(int n_out, int K, int fmt)
{
    return (size_t)df_mtiles(n_out) * ((size_t)df_kblocks(K) * df_unit(fmt) + DF_ROWS * sizeof(float));
}

// CTA = (K block, tile of outputs).
template <int FMT>
__global__ void __launch_bounds__(256) k_fp4_decode_layout(const uint8_t *__restrict__ Wq,
                                                          const uint8_t *__restrict__ w_sf,
                                                          const float *__restrict__ w_scale, int n_out, int K,
                                                          uint8_t *__restrict__ Wd)
{
    using C = Fp4Cfg<FMT>;
    const int kb = blockIdx.x, mt = blockIdx.y, nkb = gridDim.x, kt = fp4_sf_ktiles(K, FMT);
    uint8_t *unit = Wd + ((size_t)mt * nkb + kb) * df_unit(FMT);
    // every write below is at a constant bound inside the unit
    if (!as_in(kb, (K + DF_KB - 1) / DF_KB) || !as_in((long long)mt * DF_ROWS, n_out)) return;
    // MX rows whose largest scale is above 2^8 are stored smaller by a power
    // of two that their row factor carries, so that sums of products stay in
    // float32; by no more than leaves their smallest scale a scale
    __shared__ int s_shift[DF_ROWS];
    if (threadIdx.x < DF_ROWS) {
        const int o = mt * DF_ROWS + threadIdx.x;
        int top = 0, low = 254;
        if (FMT == AS_FP4_MX && o < n_out)
            for (int t = 0; t < kt; ++t) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(w_sf + fp4_sf_byte(o, 4 * t, kt));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int b = (int)((w >> (8 * k)) & 0xFFu);
                    if (b == 255 || 4 * t + k >= K / 32) continue;
                    top = max(top, b);
                    low = min(low, b);
                }
            }
        s_shift[threadIdx.x] = top > 135 ? min(top - 135, low) : 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < DF_ROWS * 8; i += 256) {  // 16-byte chunk c of row r
        const int r = i >> 3, c = i & 7, o = mt * DF_ROWS + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (o < n_out && kb * 128 + c * 16 < K / 2)
            v = *reinterpret_cast<const uint4 *>(Wq + (size_t)o * (K / 2) + kb * 128 + c * 16);
        *reinterpret_cast<uint4 *>(unit + r * 128 + ((c ^ (r & 7)) << 4)) = v;
    }
    for (int i = threadIdx.x; i < C::SFT * 32; i += 256) {  // 16 bytes of a scale tile
        const int t = kb * C::SFT + (i >> 5);
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t < kt) v = *reinterpret_cast<const uint4 *>(w_sf + ((size_t)mt * kt + t) * 512 + (i & 31) * 16);
        if (FMT == AS_FP4_MX) {  // word k: row (i & 31) + 32 k
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int sh = s_shift[(i & 31) + 32 * k];
                uint32_t out = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int b = (int)((w[k] >> (8 * j)) & 0xFFu);
                    out |= (uint32_t)(b == 255 ? 255 : max(b - sh, 0)) << (8 * j);  // below sh: past K
                }
                w[k] = out;
            }
            v = make_uint4(w[0], w[1], w[2], w[3]);
        }
        *reinterpret_cast<uint4 *>(unit + DF_WTILE + i * 16) = v;
    }
    if (kb == 0 && threadIdx.x < DF_ROWS) {
        float *rowf = reinterpret_cast<float *>(Wd + (size_t)gridDim.y * nkb * df_unit(FMT));
        const int o = mt * DF_ROWS + threadIdx.x;
        rowf[o] = o < n_out ? ldexpf(w_scale ? w_scale[o] : 1.0f, s_shift[threadIdx.x]) : 0.0f;
    }
}

cudaError_t launch_weight_prep_fp4(const uint8_t *Wq, const uint8_t *w_sf, const float *w_scale, int n_out, int K,
                                   int fmt, uint8_t *Wd, cudaStream_t st)
{
    const dim3 grid(df_kblocks(K), df_mtiles(n_out));
    if (fmt == AS_FP4_NV)
        k_fp4_decode_layout<AS_FP4_NV><<<grid, 256, 0, st>>>(Wq, w_sf, w_scale, n_out, K, Wd);
    else
        k_fp4_decode_layout<AS_FP4_MX><<<grid, 256, 0, st>>>(Wq, w_sf, w_scale, n_out, K, Wd);
    return cudaGetLastError();
}

// ------------------------------------------------------------------ staging
// A cluster per token, its CTAs and their warps share the row's 256-channel
// tiles: mean and largest |x| are exchanged through distributed shared memory,
// then every warp selects its own channels (or takes a mask), writes the keep
// words and turns the kept values into P parts.  Part p of token t is
// column t P + P - 1 - p (the small parts first).  The columns of a K block are
// the operand image that the decode copies in one piece: N rows of 128 bytes
// (128-byte swizzle), then the scale tiles of 128 rows.  Rows past T P are not
// written: they only reach sums that are not read.
// The mean is a float64 sum in a fixed order (of bf16 values it is exact, so
// its order does not show).
// Bound: latency.
constexpr int DS_WARPS = 8;

struct StageArgs {
    const void *x;
    int bf16;
    int T, K, P, N;
    int score_f, sel, n, m, dpts;  // score_f: multiply |x| by f
    float tau;
    const float *eta_static, *f;
    const uint32_t *mask_in;  // selection made before, with its eta in eta_in; or nullptr
    const float *eta_in;
    uint32_t *mask;  // keep words, written unless mask_in
    float *eta;      // [T], written unless mask_in (with a shift)
    float *scale;    // [T] S of every token
    uint8_t *xq;     // the columns' images, xb bytes per K block
    size_t xb;
};

// 8 values of token t from channel c0 on.
__device__ __forceinline__ void df_load8(const StageArgs &a, int t, int c0, float (&v)[8])
{
    const size_t at = (size_t)t * a.K + c0;
    if (a.bf16) load8(static_cast<const __nv_bfloat16 *>(a.x) + at, v);
    else load8(static_cast<const float *>(a.x) + at, v);
}

// Exponent of S: the smallest e >= -126 with m <= 4 * 448 * 2^e for the token's
// largest possible |x - eta|, m = top + |eta|.  1792 = 1.75 * 2^10.
template <int FMT>
__device__ __forceinline__ int df_exponent(uint32_t top, float eta)
{
    if (FMT == AS_FP4_MX) return 0;
    const uint32_t m = min(__float_as_uint(__uint_as_float(top) + fabsf(eta)), F32_INF_BITS - 1u);
    if (m == 0u) return 0;
    return max((int)(m >> 23) - 127 - 10 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0), -126);
}

// What a lane needs of its 8 channels (a warp: 256 channels from a multiple of
// 256 on; act: below K).
struct DfRaw {
    float v[8], f[8];
    uint32_t word;  // keep word of mask_in
};
__device__ __forceinline__ void df_load_raw(const StageArgs &a, int t, int c0, bool act, DfRaw &r)
{
#pragma unroll
    for (int e = 0; e < 8; ++e) r.v[e] = 0.0f, r.f[e] = 1.0f;
    r.word = 0u;
    if (!act) return;
    df_load8(a, t, c0, r.v);
    if (a.mask_in) r.word = a.mask_in[(size_t)t * ((a.K + 31) >> 5) + (c0 >> 5)];
    else if (a.score_f) load8f(a.f + c0, r.f);
}

// Kept values, selected here unless mask_in.
__device__ __forceinline__ void df_keep8(const StageArgs &a, const DfRaw &r, int t, int c0, bool act, float eta,
                                         float (&xh)[8])
{
    const int lane = threadIdx.x & 31, words = (a.K + 31) >> 5;
    float sc[8];
    score8(r.v, a.dpts, eta, nullptr, 0, xh, sc);
    uint32_t keep;
    if (a.mask_in) {
        keep = (r.word >> (8 * (lane & 3))) & 0xFFu;
    } else {
        if (a.score_f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) sc[e] = __fmul_rn(sc[e], r.f[e]);
        }
        keep = a.sel == AS_SEL_NM ? nm_keep_dispatch(sc, lane, a.n, a.m)
                                  : (a.sel == AS_SEL_THRESH ? keep_thresh(sc, a.tau) : 0xFFu);
        if (!act) keep = 0;
        uint32_t word = keep << (8 * (lane & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 1);
        word |= __shfl_xor_sync(0xffffffffu, word, 2);
        const int wi = c0 >> 5;
        if ((lane & 3) == 0 && act && as_in((long long)t * words + wi, (long long)a.T * words))
            a.mask[(size_t)t * words + wi] = word;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) xh[k] = act && ((keep >> k) & 1u) ? xh[k] : 0.0f;
}

// The P parts of 8 kept values into their K block's image `img` (rows of 128
// bytes, scale tiles at sf).  Channels up to the next multiple of 64 past K are
// written (zeros): an instruction covers 64.
template <int FMT>
__device__ __forceinline__ void df_parts8(const StageArgs &a, int t, int c0, int e0, float (&xh)[8], uint8_t *img,
                                          uint8_t *sf)
{
    using C = Fp4Cfg<FMT>;
    const int lane = threadIdx.x & 31;
    const bool write = c0 < (a.K + 63) / 64 * 64;
    const int off = (c0 & 255) >> 1;                          // byte of the row
    constexpr int LANES = fp4_block(FMT) / 8;                 // lanes of a block
    const int blk = (c0 & 255) / fp4_block(FMT);              // block of the K block
    uint32_t top = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) top = max(top, __float_as_uint(xh[k]) & 0x7FFFFFFFu);
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
    // a block that holds an infinity or a NaN takes the NaN scale, and with it
    // the outputs
    const bool bad = top >= F32_INF_BITS;
    float sv = 1.0f;  // scale in units of 2^e (NV: S, MX: the block's own)
    int e = e0;
    uint32_t byte;
    if constexpr (FMT == AS_FP4_NV) {
        // up to the next of 4 significant bits, or of 2^-9 below the normal numbers
        const float q = __uint_as_float(top) * pow2f(-e0) * 0.25f;
        if (q >= 0.015625f) {
            const uint32_t r = min((__float_as_uint(q) + 0xFFFFFu) & 0xFFF00000u, __float_as_uint(448.0f));
            sv = __uint_as_float(r);
            byte = (r >> 20) - 8 * 120;
        } else {
            byte = (uint32_t)ceilf(q * 512.0f);
            sv = (float)byte * (1.0f / 512.0f);
        }
        if (bad) byte = 127u;
    } else {
        // up to the next power of two (normal ones): the quantiser's, or twice
        // that for a largest value that is no power of two
        byte = (uint32_t)min(max((int)(top >> 23) - 2 + ((top & 0x7FFFFFu) != 0u ? 1 : 0), 1), 253);
        e = (int)byte - 127;
        if (bad) byte = 255u;
    }
    // values in units of 2^e: exact, and far from both ends of float32
    const float unit = pow2f(-e);
#pragma unroll
    for (int k = 0; k < 8; ++k) xh[k] *= unit;
    const bool none = bad || !(sv > 0.0f);
    float back = none ? 0.0f : sv, fwd = none ? 0.0f : __frcp_rn(sv);
    uint8_t *sfb = sf + (blk >> 2) * 512 + (blk & 3);
    const bool sf_lane = write && (lane & (LANES - 1)) == 0;
#pragma unroll 2
    for (int p = 0; p < a.P; ++p) {
        uint32_t codes = 0u;
#pragma unroll
        for (int k = 0; k < 4; ++k) codes |= e2m1x2(xh[2 * k] * fwd, xh[2 * k + 1] * fwd) << (8 * k);
#pragma unroll
        for (int k = 0; k < 4; ++k) {  // the rest (one rounding)
            const float2 q = e2m1x2_value((codes >> (8 * k)) & 0xFFu);
            xh[2 * k] = fmaf(-q.x, back, xh[2 * k]);
            xh[2 * k + 1] = fmaf(-q.y, back, xh[2 * k + 1]);
        }
        const int row = t * a.P + a.P - 1 - p;
        uint8_t *code_at = img + row * 128 + ((((off >> 4) ^ (row & 7)) << 4) | (off & 15));
        uint8_t *sf_at = sfb + (row >> 7) * C::SFB + (row & 31) * 16 + ((row >> 5) & 3) * 4;
        if (write && as_in(code_at + 3 - img, a.N * 128)) *reinterpret_cast<uint32_t *>(code_at) = bad ? 0u : codes;
        if (sf_lane && as_in(sf_at - sf, (long long)a.xb - a.N * 128)) *sf_at = (uint8_t)byte;
        back *= 0.125f;
        fwd *= 8.0f;
    }
}

__device__ __forceinline__ float df_given_eta(const StageArgs &a, int t)
{
    return !a.dpts ? 0.0f : (a.mask_in ? a.eta_in[t] : (a.dpts == AS_PTS_STATIC ? a.eta_static[t] : 0.0f));
}

__device__ __forceinline__ void st_cluster_b64(uint32_t addr, uint64_t v)
{
    asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <int FMT>
__global__ void __launch_bounds__(DS_WARPS * 32) k_fp4_stage(StageArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __shared__ double w_sum[DS_WARPS];
    __shared__ uint32_t w_max[DS_WARPS];
    __shared__ __align__(8) uint64_t c_sum[8], c_max[8];  // of every CTA
    const int t = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int rank = (int)cluster_ctarank(), ranks = gridDim.x;
    const int nkb = (a.K + 255) >> 8, per = (nkb + ranks - 1) / ranks;
    const int kb0 = min(nkb, rank * per), kb1 = min(nkb, kb0 + per);
    float eta = df_given_eta(a, t);
    uint32_t top = 0;
    const bool mean = a.dpts == AS_PTS_DYNAMIC && !a.mask_in;
    // a warp's first tile stays in registers (it is the only one up to K =
    // 16384): later loads would queue behind the decode kernel's weights
    DfRaw raw;
    {
        const int c0 = 256 * (kb0 + warp) + 8 * lane;
        df_load_raw(a, t, c0, kb0 + warp < kb1 && c0 < a.K, raw);
    }
    // after the wait (see k_select_nm_decode) and after those loads
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (mean || FMT == AS_FP4_NV) {  // uniform over the cluster
        double sum = 0.0;
        for (int kb = kb0 + warp; kb < kb1; kb += warps) {
            const int c0 = 256 * kb + 8 * lane;
            if (c0 < a.K) {
                float v[8];
                if (kb == kb0 + warp) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[e] = raw.v[e];
                } else {
                    df_load8(a, t, c0, v);
                }
                if (mean)
                    sum += (((double)v[0] + (double)v[1]) + ((double)v[2] + (double)v[3])) +
                           (((double)v[4] + (double)v[5]) + ((double)v[6] + (double)v[7]));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t b = __float_as_uint(v[e]) & 0x7FFFFFFFu;
                    top = max(top, b < F32_INF_BITS ? b : 0u);
                }
            }
        }
        if (mean) sum = warp_sum_f64(sum);
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) {
            w_sum[warp] = sum;
            w_max[warp] = top;
        }
        asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");  // this CTA runs
        __syncthreads();
        sum = 0.0;
        for (int w = 0; w < warps; ++w) {
            sum += w_sum[w];
            top = max(top, w_max[w]);
        }
        asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        if ((int)threadIdx.x < ranks) {
            st_cluster_b64(mapa_u32(smem_u32(&c_sum[rank]), threadIdx.x), (uint64_t)__double_as_longlong(sum));
            st_cluster_b64(mapa_u32(smem_u32(&c_max[rank]), threadIdx.x), (uint64_t)top);
        }
        cluster_sync_all();
        sum = 0.0;
        for (int r = 0; r < ranks; ++r) {
            sum += __longlong_as_double((long long)c_sum[r]);
            top = max(top, (uint32_t)c_max[r]);
        }
        if (mean) eta = (float)(sum / (double)a.K);
    }
    const int e0 = df_exponent<FMT>(top, eta);
    if (rank == 0 && threadIdx.x == 0 && as_in(t, a.T)) {
        a.scale[t] = pow2f(e0);
        if (a.dpts && !a.mask_in) a.eta[t] = eta;
    }
    for (int kb = kb0 + warp; kb < kb1; kb += warps) {
        const int c0 = 256 * kb + 8 * lane;
        float xh[8];
        if (kb != kb0 + warp) df_load_raw(a, t, c0, c0 < a.K, raw);
        df_keep8(a, raw, t, c0, c0 < a.K, eta, xh);
        if (!as_in(kb, nkb)) break;  // the whole warp: images of nkb K blocks
        uint8_t *img = a.xq + (size_t)kb * a.xb;
        df_parts8<FMT>(a, t, c0, e0, xh, img, img + (size_t)a.N * 128);
    }
}

// ------------------------------------------------------------------ decode
// CTA (rank of a cluster, tile of 128 outputs): a contiguous part of the K
// blocks, one accumulator.  warp 0 copies (1-D bulk copies of whole tiles),
// warp 1 issues the MMAs, warps 2-5 take the accumulator, add a token's
// columns and send every CTA of the cluster its share of the outputs, which it
// sums in rank order.
constexpr int DF_THREADS = 192;
template <int FMT, int NB>  // NB: columns that a stage has room for
struct DfCfg {
    static constexpr int NSB = (NB + 127) / 128;
    static constexpr int W = DF_WTILE, SA = Fp4Cfg<FMT>::SFB;
    static constexpr int XB = NB * 128 + NSB * Fp4Cfg<FMT>::SFB;
    static constexpr int SCOLS = 4 * (1 + NSB) * Fp4Cfg<FMT>::SFT;
    // up to 64 columns two CTAs fit an SM, of one call or of two in a row
    // (one token, 11008 x 4096: 9.9 us against 15.0 with a CTA that takes all of
    // tensor memory)
    static constexpr int PER_SM = NB <= 64 ? 2 : 1;
    static constexpr int STAGES = NB <= 32 ? 4 : (NB <= 64 ? 3 : (NB <= 128 ? 5 : 4));
    static constexpr uint32_t TCOLS = PER_SM == 2 ? 256 : 512;
    static constexpr size_t smem = 1024 + (size_t)STAGES * (W + SA + XB) + 256;
    static_assert(smem + 12 * 1024 <= 227 * 1024 / PER_SM, "shared memory");
    static_assert(NB + STAGES * SCOLS <= TCOLS, "tensor memory");
};
constexpr int DF_RECV = 16 * (128 + 8);  // floats: T outputs' shares from up to 8 CTAs

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// The sum of a token's P columns (column P - 1 - p times 8^-p), for every token,
// to the owner of this lane's output.  (P is a constant so that the columns stay
// in registers.)
template <int P>
__device__ __forceinline__ void df_send(uint32_t acc, bool some, int T, int width, uint32_t to)
{
    for (int t0 = 0; t0 < T; t0 += 2) {
        uint32_t r[2][16];  // columns past P, and of a token T, belong to others and are not used
        if (some) {
#pragma unroll
            for (int u = 0; u < 2; ++u)
                asm volatile(
                    "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                    "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                    : "=r"(r[u][0]), "=r"(r[u][1]), "=r"(r[u][2]), "=r"(r[u][3]), "=r"(r[u][4]), "=r"(r[u][5]),
                      "=r"(r[u][6]), "=r"(r[u][7]), "=r"(r[u][8]), "=r"(r[u][9]), "=r"(r[u][10]), "=r"(r[u][11]),
                      "=r"(r[u][12]), "=r"(r[u][13]), "=r"(r[u][14]), "=r"(r[u][15])
                    : "r"(acc + (uint32_t)((t0 + u) * P)));
            tmem_ld_wait();
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) r[0][i] = r[1][i] = 0u;
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (t0 + u >= T) break;
            float v = __uint_as_float(r[u][0]);
#pragma unroll
            for (int p = 1; p < P; ++p) v = fmaf(v, 0.125f, __uint_as_float(r[u][p]));
            st_cluster_f32(to + 4u * (uint32_t)((t0 + u) * width), v);
        }
    }
}

template <int FMT, int NB>
__global__ void __launch_bounds__(DF_THREADS, DfCfg<FMT, NB>::PER_SM) k_decode_fp4(DecodeFp4Args a)
{
    using C = Fp4Cfg<FMT>;
    using P = DfCfg<FMT, NB>;
    constexpr int S = P::STAGES;
    extern __shared__ unsigned char smem_raw[];
    __shared__ __align__(16) float recv[DF_RECV];
    __shared__ float s_scale[16], s_rowf[DF_ROWS], s_rowsum[DF_ROWS], s_eta[16];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                            ~uintptr_t(1023));
    // every W and X image is 1024-byte aligned
    unsigned char *sW = smem, *sX = sW + S * P::W, *sSA = sX + S * P::XB;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sSA + S * P::SA);
    uint64_t *full = bars, *empty = bars + S, *done = bars + 2 * S;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * S + 1);
    int *abort_flag = reinterpret_cast<int *>(tmem_slot + 1);

    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int warp = uniform_warp(), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), nranks = gridDim.x, mt = blockIdx.y;
    const int nkb = (a.K + DF_KB - 1) / DF_KB, per = (nkb + nranks - 1) / nranks;
    const int kb0 = min(nkb, rank * per), kb1 = min(nkb, kb0 + per);

    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, P::TCOLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    // remote stores need their CTA to be running: the wait for these arrivals
    // comes before the first of them
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    if (warp == 0) {
        if (lane == 0) {
            const uint8_t *w = a.Wd + (size_t)mt * nkb * df_unit(FMT);
            const uint32_t xbytes = (uint32_t)a.N * 128 + P::NSB * C::SFB;
            auto load_w = [&](int kb, int s) {
                mbar_arrive_expect_tx(&full[s], P::W + P::SA + xbytes);
                const uint8_t *src = w + (size_t)kb * df_unit(FMT);
                bulk_load(sW + s * P::W, src, P::W, &full[s]);
                bulk_load(sSA + s * P::SA, src + P::W, P::SA, &full[s]);
            };
            auto load_x = [&](int kb, int s) {  // rows, then the scale tiles
                const uint8_t *src = a.xq + (size_t)kb * xbytes;
                bulk_load(sX + s * P::XB, src, (uint32_t)a.N * 128, &full[s]);
                bulk_load(sX + s * P::XB + NB * 128, src + (size_t)a.N * 128, P::NSB * C::SFB, &full[s]);
            };
            // The kernel before this one in its call lets it start after its
            // own wait, so everything before that, the weights among it, is
            // complete: only x waits for it.
            const int first = min(S, kb1 - kb0);
            for (int i = 0; i < first; ++i) load_w(kb0 + i, i);
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = 0; i < first; ++i) load_x(kb0 + i, i);
            int stage = 0;
            uint32_t phase = 0;
            for (int kb = kb0 + S; kb < kb1; ++kb) {
                if (!mbar_wait(&empty[stage], phase)) { *(volatile int *)abort_flag = 1; break; }
                load_w(kb, stage);
                load_x(kb, stage);
                if (++stage == S) { stage = 0; phase ^= 1; }
            }
        }
    } else if (warp == 1) {
        const uint32_t lead = elect_lane();
        const uint32_t idesc = idesc_fp4<FMT>(128, a.N);
        int stage = 0;
        uint32_t phase = 0;
        bool ready = false;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!ready && !mbar_wait(&full[stage], phase)) { *(volatile int *)abort_flag = 1; break; }
            tc_fence_after();
            const int next = stage + 1 == S ? 0 : stage + 1;
            const uint32_t nphase = stage + 1 == S ? phase ^ 1 : phase;
            // test_wait: this stage's MMAs are ready and do not wait for the next's
            // (8 tokens 4096 x 14336 NV bf16: 12.6 us against 13.5 with try_wait)
            ready = kb + 1 < kb1 && mbar_test(&full[next], nphase);
            const int steps = min(4, (a.K - kb * DF_KB + 63) >> 6);
            const uint32_t sfa = tmem + NB + stage * P::SCOLS, sfb = sfa + 4 * C::SFT;
            const unsigned char *x = sX + stage * P::XB;
            const uint32_t xsf = smem_u32(x + NB * 128);
#pragma unroll
            for (int t = 0; t < C::SFT; ++t) {
                tmem_cp_sf(lead, sfa + 4 * t, sdesc_rows16(smem_u32(sSA + stage * P::SA + 512 * t)));
#pragma unroll
                for (int c = 0; c < P::NSB; ++c)
                    tmem_cp_sf(lead, sfb + 4 * P::NSB * t + 4 * c, sdesc_rows16(xsf + c * C::SFB + 512 * t));
            }
            const uint64_t a_desc = sdesc_kmajor_sw128(smem_u32(sW + stage * P::W));
            const uint64_t b_desc = sdesc_kmajor_sw128(smem_u32(x));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j < steps)
                    mma_fp4<FMT, false>(lead, tmem, a_desc + (uint64_t)((32 * j) >> 4), b_desc + (uint64_t)((32 * j) >> 4),
                                        idesc | C::ids(j), sfa + 4 * C::tile(j), sfb + 4 * P::NSB * C::tile(j),
                                        (kb > kb0 || j > 0));
            tc_commit_lead<false>(lead, &empty[stage]);
            stage = next;
            phase = nphase;
        }
        tc_commit_lead<false>(lead, done);  // every MMA above has completed
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every CTA of the cluster has started
    // outputs [first(r), first(r + 1)) of the tile belong to rank r
    auto first_of = [&](int r) { return (r * 128 + nranks - 1) / nranks; };
    const int width = (127 + nranks) / nranks;  // room per CTA and token
    if (warp >= 2) {
        // factors, while the MMAs run
        const int u = (int)threadIdx.x - 64, uo = mt * DF_ROWS + u;
        s_rowf[u] = a.rowf[uo];
        s_rowsum[u] = a.eta && uo < a.n_out ? a.rowsum[uo] : 0.0f;
        asm volatile("griddepcontrol.wait;" ::: "memory");  // the staging kernel's columns and means
        if (u < a.T) {
            s_scale[u] = a.scale[u];
            s_eta[u] = a.eta ? a.eta[u] : 0.0f;
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const bool ok = mbar_wait(done, 0);
        tc_fence_after();
        const int q = warp & 3, o = 32 * q + lane;
        const int owner = o * nranks >> 7;
        const uint32_t to = mapa_u32(smem_u32(recv + (size_t)rank * a.T * width + o - first_of(owner)), (uint32_t)owner);
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
        const bool some = ok && kb1 > kb0;
        if (a.P == DF_PARTS_BF16) df_send<DF_PARTS_BF16>(acc, some, a.T, width, to);
        else df_send<DF_PARTS_F32>(acc, some, a.T, width, to);
        tc_fence_before();
    }
    __syncwarp();
    cluster_sync_all();
    tc_fence_after();
    const int o0 = first_of(rank), no = first_of(rank + 1) - o0;
    const int t1 = (int)threadIdx.x / no, c = (int)threadIdx.x - t1 * no, tstep = max(1, DF_THREADS / no);
    const int o = mt * DF_ROWS + o0 + c;
    if (t1 < tstep && o < a.n_out)
    for (int t = t1; t < a.T; t += tstep) {
        if (!as_in((long long)t * a.n_out + o, (long long)a.T * a.n_out)) continue;
        float s = 0.0f;
        for (int r = 0; r < nranks; ++r) s += recv[(r * a.T + t) * width + c];
        // in double: S, the row factor and the sum may leave float32 while their
        // product does not
        double d = (double)s * s_scale[t] * s_rowf[o0 + c];
        if (a.eta) d += (double)s_eta[t] * s_rowsum[o0 + c];
        s = (float)d;
        if (a.out_bf16) static_cast<__nv_bfloat16 *>(a.y)[(size_t)t * a.n_out + o] = __float2bfloat16_rn(s);
        else static_cast<float *>(a.y)[(size_t)t * a.n_out + o] = s;
    }
    if (warp == 1) tmem_dealloc(tmem, P::TCOLS);
}

// ---------------------------------------------------------------- host side
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
    cfg.numAttrs = 2;
}

template <int FMT, int NB>
static cudaError_t launch_df(const DecodeFp4Args &a, cudaStream_t st)
{
    using P = DfCfg<FMT, NB>;
    static RaisedLimit done;
    const cudaError_t e = smem_limit_once(k_decode_fp4<FMT, NB>, P::smem, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    static DeviceAnswer fit[9];
    df_launch(cfg, attr, dim3(1), DF_THREADS, P::smem, 1, st);
    const int ranks =
        cluster_that_fits(k_decode_fp4<FMT, NB>, cfg, df_mtiles(a.n_out), P::PER_SM, df_kblocks(a.K), fit);
    df_launch(cfg, attr, dim3(ranks, df_mtiles(a.n_out)), DF_THREADS, P::smem, ranks, st);
    return cudaLaunchKernelEx(&cfg, k_decode_fp4<FMT, NB>, a);
}

template <int FMT>
static cudaError_t launch_df_fmt(const DecodeFp4Args &a, const StageArgs &s, cudaStream_t st)
{
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    const int nkb = df_kblocks(s.K), ranks = std::min(8, nkb), warps = std::min(DS_WARPS, (nkb + ranks - 1) / ranks);
    df_launch(cfg, attr, dim3(ranks, s.T), 32 * warps, 0, ranks, st);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, k_fp4_stage<FMT>, s);
    if (e != cudaSuccess) return e;
    if (a.N <= 16) return launch_df<FMT, 16>(a, st);
    if (a.N <= 32) return launch_df<FMT, 32>(a, st);
    if (a.N <= 64) return launch_df<FMT, 64>(a, st);
    if (a.N <= 128) return launch_df<FMT, 128>(a, st);
    return launch_df<FMT, 160>(a, st);
}

static int df_parts(bool out_bf16) { return out_bf16 ? DF_PARTS_BF16 : DF_PARTS_F32; }
static int df_cols(int T, int parts) { return (T * parts + 15) / 16 * 16; }
static size_t df_xbytes(int N, int fmt) { return (size_t)N * 128 + (size_t)((N + 127) / 128) * (fmt == AS_FP4_NV ? 2048 : 1024); }

// keep words, eta, the tokens' S, staged columns (the larger of both formats)
DecodeFp4Layout decode_fp4_layout(int T, int K, int out_bf16)
{
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const int n = df_cols(T, df_parts(out_bf16));
    const size_t xb = df_xbytes(n, AS_FP4_NV);
    DecodeFp4Layout l{};
    l.eta = up((size_t)T * ((K + 31) / 32) * sizeof(uint32_t));
    l.scale = l.eta + up((size_t)T * sizeof(float));
    l.xq = l.scale + up((size_t)T * sizeof(float));
    l.bytes = l.xq + up((size_t)df_kblocks(K) * xb);
    return l;
}

cudaError_t launch_decode_fp4(DecodeFp4Args a, const SelectArgs &sel, bool selected, void *ws, int fmt, cudaStream_t st)
{
    const DecodeFp4Layout l = decode_fp4_layout(a.T, a.K, a.out_bf16);
    char *w = static_cast<char *>(ws);
    a.P = df_parts(a.out_bf16);
    a.N = df_cols(a.T, a.P);
    a.rowf = reinterpret_cast<const float *>(a.Wd + (size_t)df_mtiles(a.n_out) * df_kblocks(a.K) * df_unit(fmt));
    a.scale = reinterpret_cast<const float *>(w + l.scale);
    a.xq = reinterpret_cast<const uint8_t *>(w + l.xq);
    StageArgs s{};
    s.x = a.x;
    s.bf16 = a.bf16;
    s.T = a.T;
    s.K = a.K;
    s.P = a.P;
    s.N = a.N;
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
    s.scale = reinterpret_cast<float *>(w + l.scale);
    s.xq = reinterpret_cast<uint8_t *>(w + l.xq);
    s.xb = df_xbytes(a.N, fmt);
    return fmt == AS_FP4_NV ? launch_df_fmt<AS_FP4_NV>(a, s, st) : launch_df_fmt<AS_FP4_MX>(a, s, st);
}

}  // namespace as
