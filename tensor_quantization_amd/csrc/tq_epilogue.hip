// tq_epilogue.hip -- the W8A8 product with bias, activation and residual in
// its epilogue, from one token to thousands, and the backward of that epilogue.
//
//   z[m][n] = ((float)sum_k qx[m][k] qw[n][k]) sx[m] sw[n] + bias[n]
//   y[m][n] = act(z[m][n]) + residual[m][n]
//   backward: dz = dy act'(z), dbias[n] = sum_m dz[m][n]
//
// The integer sums are exact on the matrix cores; z is binary32, in that
// order of operations, and y (and z, where it is asked for) is rounded once.
#include "tq_product.h"

namespace tq {

// ------------------------------------------------------------- a few tokens
// k_epi_few: a few tokens, bound by the weights, which are read once; or an
// output of few elements.  A workgroup of NWV waves owns 16 CT output columns of
// 16 MT tokens (few_product); the waves' sums meet in LDS, one thread per output.  What
// an output's epilogue needs is loaded before the weights are.  With 256 workgroups
// each CU has one slice of 16 columns, whose first loads and last sums nothing covers:
// 16 x 4096 x 11008 10.6 us (4.3 TB/s of weights).
template <int YT, int MT, int CT, int NWV, int U>
__global__ __launch_bounds__(64 * NWV) void k_epi_few(const int8_t* __restrict__ qx, const int8_t* __restrict__ qw,
                                                      int64_t K, Epi e)
{
    constexpr int NT = 64 * NWV, COLS = 16 * CT, STEP = NT / COLS;           // rows of outputs per step of all threads
    constexpr int PER = 16 * MT > STEP ? 16 * MT / STEP : 1;                 // outputs per thread
    // rows 4 apart beyond their sums: 16-byte steps that spread over the banks
    __shared__ int sums[NWV][MT * 16][COLS + 4];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * COLS, m0 = (int64_t)blockIdx.y * (16 * MT);

    // thread t finishes column t % COLS of tokens t / COLS, + STEP, ...
    const int64_t on = n0 + t % COLS;
    float osx[PER], ores[PER], osw = 0.0f, ob = 0.0f;
    bool mine[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int m = t / COLS + i * STEP;
        mine[i] = m < 16 * MT && m0 + m < e.M && on < e.N;
        osx[i] = mine[i] ? e.sx[m0 + m] : 0.0f;
        ores[i] = mine[i] && e.res ? load1<YT>(e.res, (m0 + m) * e.ldr + on) : 0.0f;
    }
    if (mine[0]) {
        osw = e.sw[on];
        ob = load1_rt(e.bias, e.bias_dt, on, 0.0f);
    }

    Rows16 weights[CT], tokens[MT];
#pragma unroll
    for (int j = 0; j < CT; ++j) weights[j] = rows16_of(qw, e.N, n0 + 16 * j, K);
#pragma unroll
    for (int i = 0; i < MT; ++i) tokens[i] = rows16_of(qx, e.M, m0 + 16 * i, K);
    v4i acc[MT][CT];
    few_product<MT, CT, NWV, U>(weights, tokens, K, acc);
    // lane l holds columns 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) *reinterpret_cast<v4i*>(&sums[w][16 * i + l16][16 * j + 4 * g4]) = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int m = t / COLS + i * STEP;
        if (!mine[i]) continue;
        int s = 0;
#pragma unroll
        for (int v = 0; v < NWV; ++v) s += sums[v][m][t % COLS];
        float v = (float)s * osx[i] * osw;
        if (e.bias) v += ob;
        const int64_t at = (m0 + m) * e.N + on;
        if (e.z) store1<YT>(e.z, at, v);
        with_act(e.act, [&](auto a) { v = act1<decltype(a)::value>(v); });
        if (e.res) v += ores[i];
        store1<YT>(e.y, at, v);
    }
}

// -------------------------------------------------------------- many tokens
// 256 x 256 with 2 x 4 waves of 128 x 64: on [8192, 4096] x [11008, 4096] 308-319
// us without and 327-340 us with bias and gelu_tanh, by the card and its clock (the
// first 20 ms of matrix work run at 350-450; 2350 / 2220 TOP/s; the platform
// library's plain int8 product of that size 400 us, its best size 2336 TOP/s),
// 2560 TOP/s at 8192^3.  Bound by the matrix cores at the clock that the chip
// holds under them, and by what stands between them: per block a SIMD's products
// take 2048 clocks, its two waves' sixteen direct loads 928 of issue (about 58
// each), the CU's operand reads 917 of LDS (counted).  Four waves of 128 x 128
// read a third less but leave each SIMD one wave, whose loads then stop its
// products: 326 / 346 us.  About 45 us are the epilogue, which one workgroup per
// CU cannot lay under the products of another.  The 256 x 256 tile's stores are
// non-temporal (an output of 180 MB passes every cache): 10 us less; smaller
// products keep plain stores, since what follows reads them.
//
// 128 x 128, one workgroup per CU and 9 units: 777 x 4096 x 4096 f16 with bias,
// silu and residual 20-21 us; 64 x 64, two per CU: 128 x 4096 x 4096 11.2 us.
// There a block of 128 codes takes 0.48 and 0.3 us.  For the 128 tile that is some
// 1100 clocks, of which a SIMD's products need 512, its two waves' eight direct
// loads 464 of issue, and the CU's operand reads 420 of LDS (counted): with two waves
// to a SIMD they run side by side only in part.  Longer rings change nothing, and
// neither does sharing a block's two steps between two sets of waves (23.2 and 10.5
// us).
//
// Operands of any alignment (k_epi_tile): 777 x 4096 x 4095 35 us (aligned operands: 20), 8192 x 11008 x 4088 416 us (330): bound
// by the loads, whose 16 bytes per lane straddle lines.  One block ahead only: 52 /
// 485 us.
template <int YT>
struct EpiTile : Epi {
    static constexpr bool GATED = false;
    static __device__ __forceinline__ const int8_t* second_weight(const int8_t* first) { return first; }
    template <int TILE, int WM, int WN>
    static constexpr int staging()
    {
        return 4 * WM * WN * Stage<TILE / WM / 16, TILE / WN / 16>::INTS;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ int early(const Epi&, int64_t)
    {
        return 0;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ void finish(const Epi& e, int64_t m0, int64_t n0,
                                                  const v4i (&acc)[TILE / WM / 16][TILE / WN / 16], uint8_t* lds, int)
    {
        constexpr int NM = TILE / WM / 16, NN = TILE / WN / 16;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        finish_part<YT, NM, NN, TILE == 256>(e, m0 + TILE / WM * (w / WN), n0 + TILE / WN * (w % WN), acc,
                                             reinterpret_cast<int*>(lds) + w * Stage<NM, NN>::INTS);
    }
};

// ------------------------------------------------------ backward of epilogue
// k_epi_bwd: dz = dy act'(z) and its column sums: 4 bytes read and 2 written
// per bf16 element, bound by HBM: [8192, 11008] bf16 with gelu_tanh 101.7 us
// (5.3 TB/s) and 4.9 us for the column sums.  A wave owns 512 columns, a workgroup's four
// waves take a chunk of the rows in turn, U rows in flight each; their column
// sums meet in LDS in wave order and leave as one row of partials per chunk.  dz
// may be dy or z: an element's output depends on that element alone and is stored
// by the lane that owns it after its load; what a moved-back vector or a chunk's
// last rows read besides may be new already, and is not used.
template <int FT>
__global__ __launch_bounds__(256) void k_epi_bwd(const void* dy, const void* z, int64_t M, int64_t N, int64_t chunk,
                                                 int act, void* dz, float* __restrict__ part, int64_t ldp)
{
    constexpr int U = 4;
    __shared__ float fold[3][8][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)blockIdx.x * 512;
    const int n = N - c0 < 512 ? (int)(N - c0) : 512;
    const int64_t r0 = (int64_t)blockIdx.y * chunk, r1 = r0 + chunk < M ? r0 + chunk : M;
    // N >= 8: a last slab of fewer than 8 columns starts earlier, and counts only its own
    const int64_t cs = n >= 8 ? c0 : N - 8;
    const int skip = (int)(c0 - cs);
    Vec8 at = vec8(lane, n + skip);
    if (skip) at.lo = lane == 0 ? skip : 8;
    float db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) db[i] = 0.0f;
    for (int64_t r = r0 + w; r < r1; r += 4 * U) {
        Raw8<FT> a[U], b[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r + 4 * u < r1 ? r + 4 * u : r1 - 1;
            a[u] = load8_any<FT>(dy, row * N + cs + at.at);
            b[u] = load8_any<FT>(z, row * N + cs + at.at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + 4 * u >= r1) break;
            float d[8], v[8];
            widen8<FT>(a[u], d);
            widen8<FT>(b[u], v);
            slope8(act, v, d);
#pragma unroll
            for (int i = 0; i < 8; ++i) db[i] += d[i];
            if (at.lo < 8) store8_own<FT>(dz, (r + 4 * u) * N + cs, at, d);
        }
    }
    if (!part) return;
    if (w > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) fold[w - 1][i][lane] = db[i];
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) db[i] += fold[k][i][lane];
    if (at.lo < 8) store8_own<F32>(part, (int64_t)blockIdx.y * ldp + cs, at, db);
}

// Fewer than 8 columns: a thread per row and step, the columns in turn.
template <int FT>
__global__ __launch_bounds__(256) void k_epi_bwd_thin(const void* dy, const void* z, int64_t M, int64_t N,
                                                      int64_t chunk, int act, void* dz, float* __restrict__ part,
                                                      int64_t ldp)
{
    __shared__ float fold[4][8];
    const int t = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.y * chunk, r1 = r0 + chunk < M ? r0 + chunk : M;
    float db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) db[i] = 0.0f;
    for (int64_t r = r0 + t; r < r1; r += 256) {
        float d[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] = i < N ? load1<FT>(dy, r * N + i) : 0.0f;
            v[i] = i < N ? load1<FT>(z, r * N + i) : 0.0f;
        }
        slope8(act, v, d);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < N) {
                db[i] += d[i];
                store1<FT>(dz, r * N + i, d[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float s = wave_sum(db[i]);
        if ((t & 63) == 0) fold[t >> 6][i] = s;
    }
    __syncthreads();
    if (part && t < N) part[(int64_t)blockIdx.y * ldp + t] = fold[0][t] + fold[1][t] + fold[2][t] + fold[3][t];
}

// ---------------------------------------------------------------- launches
// Rows per chunk of the backward pass: whole rounds of the four waves' four
// rows, in about EPI_GROUPS workgroups over the slabs of 512 columns (measured on
// [8192, 11008] bf16: 1400 workgroups 115 us, 4096 109, 8192 106).
constexpr int64_t EPI_GROUPS = 8192;
// Up to EPI_ONE rows are one chunk, whose sums are dbias itself: one launch.
constexpr int64_t EPI_ONE = 64;
inline int64_t epi_chunk(int64_t M, int64_t N)
{
    if (M <= EPI_ONE) return EPI_ONE;
    const int64_t chunks = std::max<int64_t>(1, EPI_GROUPS / cdiv(N, 512));
    return cdiv(cdiv(M, chunks), 16) * 16;
}

// The kernel of a product, by its shape.  Measured (us, K = 4096; 64 / 128 / 256 tile):
//   512 x 4096     16.6 / 19.5 / -     640 x 4096     24.5 / 20.0 / -
//   2048 x 4096       - / 35 / 51      4096 x 4096       - / 87 / 60
// A tile kernel takes a time of its own per round of resident workgroups (two 64 x 64
// tiles or, up to 256 of them, one 128 x 128 tile per CU), so the smallest tile that
// needs one round is taken, and the largest once it fills the chip.  128 x 128 tiles
// beyond one round run two to a CU on shorter rings.  Where the output is so small that
// tiles leave most CUs idle, its 32 x 16 or 32 x 32 pieces, each with the K axis split
// over eight waves, do not (few_tokens; us, 32 x 16 / 32 x 32 / 64 tile):
//   24 x 4096 x 4096    8.5 /  8.4 / 11.7     220 x 507 x 10256   10.2 / 12.2 / 27.2
//   24 x 11008 x 4096  13.4 / 14.6 / 12.7     40 x 1024 x 8192     8.2 /  8.7 / 18.1
//   48 x 11008 x 4096  20.5 / 18.9 / 12.7     1260 x 140 x 10688  23.3 / 16.4 / 23.3
//   64 x 4096 x 4096   10.5 /  8.3 / 11.3     48 x 4096 x 11008      - / 13.8 / 25.8
//   128 x 4096 x 4096  15.5 / 12.5 / 11.2     512 x 512 x 90       8.4 /    - /  8.3
// and with rows at odd addresses
//   24 x 11008 x 4090  26.4 / 27.0 / 23.4     48 x 4096 x 4095       - / 15.5 / 19.6
//   220 x 507 x 10250  13.6 / 17.2 / 34.2     243 x 1000 x 9000      - / 12.6 / 26.1
// Operands of other alignments (k_epi_tile, us; 64 / 128 / 256 tile):
//   243 x 2546 x 9000    26.7 / 51 / -      777 x 4096 x 4095     57 / 35 / 81
//   2564 x 614 x 2708    20.5 / 21.8 / -    2048 x 4096 x 4098    87 / 58 / 75
//   1024 x 11008 x 4088    - / 71 / 67      4096 x 4096 x 4088     - / 96 / 75
// where the largest tile pays a little before it fills the chip.
template <int YT>
static void product_launch(const int8_t* qx, const int8_t* qw, int64_t K, const Epi& e, hipStream_t st)
{
    const bool rows16 = K >= ET && K % 16 == 0 && aligned16(qx) && aligned16(qw);
#define TQ_FEW(MT, CT, NWV, U)                                                                              \
    do {                                                                                                    \
        const dim3 grid((unsigned)cdiv(e.N, 16 * CT), (unsigned)cdiv(e.M, 16 * MT));                        \
        hipLaunchKernelGGL((k_epi_few<YT, MT, CT, NWV, U>), grid, dim3(64 * NWV), 0, st, qx, qw, K, e);     \
        return;                                                                                             \
    } while (0)
    if (few_tokens(e.M, e.N)) {
        if (e.M <= 16) TQ_FEW(1, 1, 8, 2);
        if (few_columns(e.M, e.N)) TQ_FEW(2, 1, 8, 1);
        TQ_FEW(2, 2, 8, 1);
    }
#undef TQ_FEW
    if (rows16) {
#define TQ_RING(TILE, RING, WM, WN, WGS)                                                                     \
    do {                                                                                                     \
        const int64_t nt = cdiv(e.N, TILE), mt = cdiv(e.M, TILE);                                            \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                            \
        hipLaunchKernelGGL((k_epi_ring<EpiTile<YT>, TILE, RING, WM, WN, WGS>), dim3((unsigned)(nt * mt)),             \
                           dim3(64 * WM * WN), 0, st, qx, qw, K, nt, mt, slab, EpiTile<YT>{e});                           \
    } while (0)
        const int64_t t128 = cdiv(e.M, 128) * cdiv(e.N, 128);
        if (cdiv(e.M, 256) * cdiv(e.N, 256) >= 256) TQ_RING(256, 5, 2, 4, 1);
        else if (t128 > 256) TQ_RING(128, 5, 2, 4, 2);
        else if (cdiv(e.M, 64) * cdiv(e.N, 64) > 512) TQ_RING(128, 9, 2, 4, 1);
        else TQ_RING(64, 9, 2, 2, 2);
#undef TQ_RING
        return;
    }
#define TQ_TILE(TILE, WM, WN, D, WGS)                                                                        \
    do {                                                                                                     \
        const int64_t nt = cdiv(e.N, TILE), mt = cdiv(e.M, TILE);                                            \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                            \
        hipLaunchKernelGGL((k_epi_tile<EpiTile<YT>, TILE, WM, WN, D, WGS>), dim3((unsigned)(nt * mt)),                \
                           dim3(64 * WM * WN), 0, st, qx, qw, K, nt, mt, slab, EpiTile<YT>{e});                           \
    } while (0)
    if (cdiv(e.M, 256) * cdiv(e.N, 256) > 160) TQ_TILE(256, 2, 4, 2, 1);
    else if (cdiv(e.M, 64) * cdiv(e.N, 64) > 512) TQ_TILE(128, 2, 4, 2, 2);
    else TQ_TILE(64, 2, 2, 4, 2);
#undef TQ_TILE
}

static bool natural(const void* p, int dt) { return ((uintptr_t)p & (uintptr_t)(ftype_size(dt) - 1)) == 0; }
static bool valid_act(int a) { return a >= TQ_ACT_NONE && a <= TQ_ACT_GELU_TANH; }

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_w8a8_linear_epilogue(const int8_t* qx, const float* sx, const int8_t* qw, const float* sw, int64_t M,
                                  int64_t N, int64_t K, const void* bias, int bias_dtype, int act,
                                  const void* residual, int64_t residual_row_stride, void* y, void* preact,
                                  int y_dtype, void* stream)
{
    if (!valid_ftype(y_dtype) || !valid_act(act) || M < 0 || N < 0 || K < 0) return TQ_ERR_INVALID;
    if (bias && !valid_ftype(bias_dtype)) return TQ_ERR_INVALID;
    if (M == 0 || N == 0) return TQ_OK;
    if (!y || !sx || !sw || (K > 0 && (!qx || !qw)) || (residual && residual_row_stride < N)) return TQ_ERR_INVALID;
    // a grid holds fewer than 2^32 threads: 512 per slice of 16 columns or per 256 x 256 tile
    if (K > 131071 || cdiv(M, ET) > 65535 || cdiv(N, 16) > 0x7fffff || cdiv(M, 256) * cdiv(N, 256) > 0x7fffff)
        return TQ_ERR_UNSUPPORTED;
    if (!natural(sx, TQ_F32) || !natural(sw, TQ_F32) || (bias && !natural(bias, bias_dtype)) ||
        !natural(residual, y_dtype) || !natural(y, y_dtype) || !natural(preact, y_dtype))
        return TQ_ERR_ALIGN;
    const Epi e = {sx, sw, bias, bias_dtype, act, residual, residual_row_stride, y, preact, M, N};
    TQ_LLM_FT_SWITCH(y_dtype, product_launch<FTV>(qx, qw, K, e, as_stream(stream)));
    return launch_status();
}

size_t tq_linear_epilogue_backward_workspace_bytes(int64_t M, int64_t N)
{
    if (M <= EPI_ONE || N <= 0) return 0;
    return (size_t)cdiv(M, epi_chunk(M, N)) * (size_t)colsum_ld(N) * sizeof(float);
}

tq_status tq_linear_epilogue_backward(const void* dy, const void* preact, int dtype, int64_t M, int64_t N, int act,
                                      void* dz, float* dbias, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_ftype(dtype) || !valid_act(act) || M < 0 || N < 0) return TQ_ERR_INVALID;
    if (N == 0) return TQ_OK;
    if (!natural(dbias, TQ_F32)) return TQ_ERR_ALIGN;
    hipStream_t st = as_stream(stream);
    if (M == 0) {                        // no rows: the sums are empty, not unwritten
        zero_vec_launch(dbias, TQ_F32, N, st);
        return launch_status();
    }
    if (!dy || !preact || !dz) return TQ_ERR_INVALID;
    if (!natural(dy, dtype) || !natural(preact, dtype) || !natural(dz, dtype)) return TQ_ERR_ALIGN;
    if (cdiv(N, 512) > 0xffffff) return TQ_ERR_UNSUPPORTED;     // 256 threads each, fewer than 2^32 in a grid
    if (dbias && M > EPI_ONE) {
        if (!workspace || workspace_bytes < tq_linear_epilogue_backward_workspace_bytes(M, N)) return TQ_ERR_INVALID;
        if (!aligned16(workspace)) return TQ_ERR_ALIGN;
    }
    const int64_t chunk = epi_chunk(M, N), chunks = cdiv(M, chunk), ld = colsum_ld(N);
    float* part = dbias && chunks > 1 ? static_cast<float*>(workspace) : dbias;
    const dim3 grid((unsigned)cdiv(N, 512), (unsigned)chunks);
    TQ_LLM_FT_SWITCH(dtype, {
        if (N < 8)
            hipLaunchKernelGGL((k_epi_bwd_thin<FTV>), grid, dim3(256), 0, st, dy, preact, M, N, chunk, act, dz, part,
                               ld);
        else
            hipLaunchKernelGGL((k_epi_bwd<FTV>), grid, dim3(256), 0, st, dy, preact, M, N, chunk, act, dz, part, ld);
    });
    if (dbias && chunks > 1) colsum_launch(part, chunks, 1, ld, N, dbias, nullptr, TQ_F32, st);
    return launch_status();
}

}  // extern "C"
