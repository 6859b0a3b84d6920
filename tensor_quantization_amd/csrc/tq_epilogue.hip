// tq_epilogue.hip -- the W8A8 product with bias, activation and residual in
// its epilogue, from one token to thousands, and the backward of that epilogue.
//
//   z[m][n] = ((float)sum_k qx[m][k] qw[n][k]) sx[m] sw[n] + bias[n]
//   y[m][n] = act(z[m][n]) + residual[m][n]
//   backward: dz = dy act'(z), dbias[n] = sum_m dz[m][n]
//
// The integer sums are exact on the matrix cores; z is binary32, in that
// order of operations, and y (and z, where it is asked for) is rounded once.
#include "tq_llm.h"

namespace tq {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));

// -------------------------------------------------------------- activations
// v / (1 + 2^x): where 2^x overflows the quotient is v's zero.
__device__ __forceinline__ float times_logistic(float v, float x)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
}

constexpr float GELU_C = 0.79788456080286535588f;      // sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;
constexpr float SQRT_HALF = 0.70710678118654752440f;

// act(v).  The tanh form of gelu is v times a logistic: (1 + tanh u) / 2 = 1 /
// (1 + exp(-2u)).
template <int ACT>
__device__ __forceinline__ float act1(float v)
{
    if constexpr (ACT == TQ_ACT_RELU) return v > 0.0f || v != v ? v : 0.0f;
    else if constexpr (ACT == TQ_ACT_SILU) return times_logistic(v, -LOG2E * v);
    else if constexpr (ACT == TQ_ACT_GELU) return 0.5f * v * erfcf(-v * SQRT_HALF);
    else if constexpr (ACT == TQ_ACT_GELU_TANH)
        return times_logistic(v, v * __builtin_fmaf(-2.0f * LOG2E * GELU_C * GELU_A * v, v, -2.0f * LOG2E * GELU_C));
    else return v;
}

// f(integral constant of `act`): one uniform branch for what f does with it.
template <class F>
__device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case TQ_ACT_RELU: f(std::integral_constant<int, TQ_ACT_RELU>()); break;
    case TQ_ACT_SILU: f(std::integral_constant<int, TQ_ACT_SILU>()); break;
    case TQ_ACT_GELU: f(std::integral_constant<int, TQ_ACT_GELU>()); break;
    case TQ_ACT_GELU_TANH: f(std::integral_constant<int, TQ_ACT_GELU_TANH>()); break;
    default: f(std::integral_constant<int, TQ_ACT_NONE>()); break;
    }
}

__device__ __forceinline__ void act8(int act, float v[8])
{
    with_act(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = act1<decltype(a)::value>(v[i]);
    });
}

// d[i] *= act'(z[i]).  A slope's second term v p' vanishes with p' (a value
// so large that p' underflows would otherwise meet an overflow there).
__device__ __forceinline__ void slope8(int act, const float z[8], float d[8])
{
    switch (act) {
    case TQ_ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = z[i] > 0.0f ? d[i] : z[i] <= 0.0f ? 0.0f : z[i];    // a NaN stays
        break;
    case TQ_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * z[i]));
            d[i] *= __builtin_fmaf(z[i], __builtin_fmaf(-p, p, p), p);
        }
        break;
    case TQ_ACT_GELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = __builtin_amdgcn_exp2f(-0.5f * LOG2E * z[i] * z[i]) * (GELU_C * 0.5f);
            d[i] *= 0.5f * erfcf(-z[i] * SQRT_HALF) + (f == 0.0f ? 0.0f : z[i] * f);
        }
        break;
    case TQ_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            constexpr float A = -2.0f * LOG2E * GELU_C;
            const float zz = z[i] * z[i];
            const float x = z[i] * __builtin_fmaf(zz, A * GELU_A, A);
            const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
            const float pq = __builtin_fmaf(-p, p, p);
            const float u = z[i] * __builtin_fmaf(zz, 6.0f * GELU_C * GELU_A, 2.0f * GELU_C);
            d[i] *= __builtin_fmaf(pq == 0.0f ? 0.0f : u, pq, p);
        }
        break;
    default: break;
    }
}

// ----------------------------------------------------------------- epilogue
struct Epi {
    const float* sx;
    const float* sw;
    const void* bias;
    int bias_dt, act;
    const void* res;
    int64_t ldr;
    void* y;
    void* z;
    int64_t M, N;
};

template <int YT>
__device__ __forceinline__ void store8_first(void* p, int64_t at, int n, const float v[8])
{
    if (n == 8) {
        store8_any<YT>(p, at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) store1<YT>(p, at + i, v[i]);
    }
}

// What eight columns col .. col + 7 need for every row: scales and bias (zeros
// past N), and how many of them there are.
struct Cols8 {
    int64_t col;
    int n;
    float sw[8], b[8];
};
__device__ __forceinline__ Cols8 cols8(const Epi& e, int64_t col)
{
    Cols8 c;
    c.col = col;
    c.n = e.N - col >= 8 ? 8 : e.N - col > 0 ? (int)(e.N - col) : 0;
    if (c.n == 8) {
        widen8<F32>(load8_any<F32>(e.sw, col), c.sw);
        widen8_rt(load8_rt(e.bias, e.bias_dt, col), e.bias, e.bias_dt, 0.0f, c.b);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            c.sw[i] = i < c.n ? e.sw[col + i] : 0.0f;
            c.b[i] = i < c.n ? load1_rt(e.bias, e.bias_dt, col + i, 0.0f) : 0.0f;
        }
    }
    return c;
}

// The residual of those columns in one row (apart from its use, so that it can
// be loaded ahead); e.res is not null.
template <int YT>
__device__ __forceinline__ Raw8<YT> residual8(const Epi& e, const Cols8& c, int64_t row)
{
    if (c.n == 8) return load8_any<YT>(e.res, row * e.ldr + c.col);
    Raw8<YT> r = {};
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < c.n) {
            if constexpr (YT == F32) w[i] = as_u(load1<F32>(e.res, row * e.ldr + c.col + i));
            else w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(e.res)[row * e.ldr + c.col + i] << (16 * (i & 1));
        }
    return r;
}

// Finishes eight columns of one row from their sums.
template <int YT>
__device__ __forceinline__ void epilogue8(const Epi& e, const Cols8& c, int64_t row, float sx, const int acc[8],
                                          const Raw8<YT>& res)
{
    const int64_t at = row * e.N + c.col;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)acc[i] * sx * c.sw[i];
    if (e.bias) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += c.b[i];
    }
    if (e.z) store8_first<YT>(e.z, at, c.n, v);
    act8(e.act, v);
    if (e.res) {
        float r[8];
        widen8<YT>(res, r);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] += r[i];
    }
    store8_first<YT>(e.y, at, c.n, v);
}

// Sixteen codes at any byte address.
__device__ __forceinline__ v4i codes16_whole(const int8_t* p)
{
    const u32x4_byte v = *reinterpret_cast<const u32x4_byte*>(p);
    return v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
}

// The same, zeros from code K of the row on.
__device__ __forceinline__ v4i codes16(const int8_t* row, int64_t k, int64_t K)
{
    if (k + 16 <= K) return codes16_whole(row + k);
    v4i r = v4i{};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int b = k + i < K ? (int)(uint8_t)row[k + i] << (8 * (i & 3)) : 0;
        r[i >> 2] |= b;
    }
    return r;
}

// ------------------------------------------------------------- a few tokens
// k_epi_few: a few tokens, bound by the weights, which are read once; or an
// output of few elements.  A workgroup of NWV waves owns 16 CT output columns of
// 16 MT tokens; the waves take the K axis in turn, 128 codes at a time, so that a wave's two loads use whole 128-byte
// lines; the sums meet in LDS, one thread per output.  The weights are the
// matrix core's first operand (16 columns), the tokens its second (16 tokens;
// rows past the end repeat the last), U blocks of both in flight per wave.  What an
// output's epilogue needs is loaded before the weights are.  Kernel times: 1 x
// 11008 x 4096 10.2 us (4.4 TB/s of weights), 16 x 4096 x 11008 12.2 (3.7): with
// 256 workgroups each CU has one slice of 16 columns, whose first loads and
// last sums nothing covers.  Refilling each of the U slots as it is used instead
// of all at once: 13.3 -> 12.2 us.
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

    const int8_t* pw[CT];
    const int8_t* px[MT];
#pragma unroll
    for (int j = 0; j < CT; ++j) {
        const int64_t n = n0 + 16 * j + l16;
        pw[j] = qw + (n < e.N ? n : e.N - 1) * K;
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = m0 + 16 * i + l16;
        px[i] = qx + (m < e.M ? m : e.M - 1) * K;
    }
    v4i acc[MT][CT];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = v4i{};
    // this wave's whole blocks are w, w + NWV, ...: U of them under way, each slot refilled as it is used
    const int nkb = (int)((K + 127) / 128), whole = (int)(K / 128);
    v4i a[U][2][CT], b[U][2][MT];
    auto fetch = [&](int u, int kb) {
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int k = kb * 128 + 64 * s + 16 * g4;
#pragma unroll
            for (int j = 0; j < CT; ++j) a[u][s][j] = codes16_whole(pw[j] + k);
#pragma unroll
            for (int i = 0; i < MT; ++i) b[u][s][i] = codes16_whole(px[i] + k);
        }
    };
    auto products = [&](const v4i (&x)[CT], const v4i (&y)[MT]) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[j], y[i], acc[i][j], 0, 0, 0);
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (w + u * NWV < whole) fetch(u, w + u * NWV);
    for (int kb = w; kb < whole; kb += U * NWV)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (kb + u * NWV >= whole) break;
#pragma unroll
            for (int s = 0; s < 2; ++s) products(a[u][s], b[u][s]);
            if (kb + (u + U) * NWV < whole) fetch(u, kb + (u + U) * NWV);
        }
    if (whole < nkb && whole % NWV == w)     // the rest of K
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t k = (int64_t)whole * 128 + 64 * s + 16 * g4;
            v4i x[CT], y[MT];
#pragma unroll
            for (int j = 0; j < CT; ++j) x[j] = codes16(pw[j], k, K);
#pragma unroll
            for (int i = 0; i < MT; ++i) y[i] = codes16(px[i], k, K);
            products(x, y);
        }
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
// Output tiles of TILE x TILE, K in blocks of 128 codes.  A row of a block is
// 128 bytes of LDS in eight 16-byte chunks, their order turned by the row so
// that the sixteen rows of a matrix operand meet all banks.  The product is
// taken as D^T, so a lane holds four consecutive columns of a row; at the end
// each wave lays its part out in LDS and finishes it eight columns at a time,
// so that stores are whole and the epilogue's code exists once.
constexpr int ET = 128;
__device__ __forceinline__ int eslot(int row, int chunk) { return row * ET + ((chunk ^ ((row >> 1) & 7)) << 4); }

// A wave's own part of a staged half: 32 rows of 16 NN sums, 4 apart beyond
// them so that sixteen rows' 16-byte stores spread over the banks, and the row
// scales of all 16 NM rows behind them.
template <int NM, int NN>
struct Stage {
    static constexpr int PITCH = 16 * NN + 4, LPR = 2 * NN, RPI = 64 / LPR;   // lanes per row, rows per instruction
    static constexpr int INTS = 32 * PITCH + 16 * NM;
};

template <int NM, int NN>
__device__ __forceinline__ void stage_scales(const Epi& e, int64_t m0, int* stage)
{
    const int lane = threadIdx.x & 63;
    float* sx = reinterpret_cast<float*>(stage + 32 * Stage<NM, NN>::PITCH);
#pragma unroll
    for (int i = 0; i < NM; i += 4) {
        const int64_t row = m0 + 16 * i + lane;
        if (16 * i + lane < 16 * NM) sx[16 * i + lane] = e.sx[row < e.M ? row : e.M - 1];
    }
}

// acc[i][j][r] = row 16 i + l % 16, column 16 j + 4 (l / 16) + r.  A wave's LDS
// accesses stay in order; the fences keep the compiler's in order too.
template <int NM, int NN>
__device__ __forceinline__ void stage_half(int h, const v4i (&acc)[NM][NN], int* stage)
{
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < NN; ++j)
            *reinterpret_cast<v4i*>(&stage[(16 * i + l16) * Stage<NM, NN>::PITCH + 16 * j + 4 * g4]) =
                acc[2 * h + i][j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
}

// A part that lies inside the output: no bounds, the activation and the
// residual known, 32-bit offsets from its corner, two rows' worth of
// independent work at a time.
template <int YT, int NM, int NN, int ACT, bool RES, bool NTS>
__device__ __forceinline__ void finish_inside(const Epi& e, const Cols8& cc, int64_t m0, int64_t n0,
                                              const v4i (&acc)[NM][NN], int* stage)
{
    using S = Stage<NM, NN>;
    constexpr int ES = YT == F32 ? 4 : 2;
    const int lane = threadIdx.x & 63;
    const int c = 8 * (lane % S::LPR), r0 = lane / S::LPR;
    const float* sx = reinterpret_cast<const float*>(stage + 32 * S::PITCH);
    char* y = static_cast<char*>(e.y) + (m0 * e.N + n0) * ES;
    const char* res = RES ? static_cast<const char*>(e.res) + (m0 * e.ldr + n0) * ES : nullptr;
    const uint32_t ystep = (uint32_t)e.N * ES, rstep = (uint32_t)e.ldr * ES;
#pragma unroll
    for (int h = 0; h < NM / 2; ++h) {
        stage_half<NM, NN>(h, acc, stage);
        uint32_t yo = (uint32_t)(32 * h + r0) * ystep + c * ES, ro = (uint32_t)(32 * h + r0) * rstep + c * ES;
#pragma unroll 1
        for (int r = r0; r < 32; r += 2 * S::RPI) {
            Raw8<YT> rr[2];
            float v[2][8];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if constexpr (RES) rr[k] = load8_off<YT>(res, ro + k * S::RPI * rstep);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int* p = &stage[(r + k * S::RPI) * S::PITCH + c];
                const v4i s0 = *reinterpret_cast<const v4i*>(p), s1 = *reinterpret_cast<const v4i*>(p + 4);
                const float sc = sx[32 * h + r + k * S::RPI];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = (float)(i < 4 ? s0[i] : s1[i - 4]) * sc * cc.sw[i];
            }
            if (e.bias) {
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[k][i] += cc.b[i];
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[k][i] = act1<ACT>(v[k][i]);
                if constexpr (RES) {
                    float w[8];
                    widen8<YT>(rr[k], w);
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[k][i] += w[i];
                }
                store8_off<YT, NTS>(y, yo + k * S::RPI * ystep, v[k]);
            }
            yo += 2 * S::RPI * ystep;
            ro += 2 * S::RPI * rstep;
        }
    }
}

// Any part: bounds, and the value before the activation where it is asked for
// (8192 x 11008 x 4096 with gelu_tanh and that value 366 us, 327 without: the 180 MB
// more take 36 at a large copy's rate).
template <int YT, int NM, int NN>
__device__ __forceinline__ void finish_any(const Epi& e, const Cols8& cc, int64_t m0, const v4i (&acc)[NM][NN],
                                           int* stage)
{
    using S = Stage<NM, NN>;
    const int lane = threadIdx.x & 63;
    const int c = 8 * (lane % S::LPR), r0 = lane / S::LPR;
    const float* sx = reinterpret_cast<const float*>(stage + 32 * S::PITCH);
#pragma unroll
    for (int h = 0; h < NM / 2; ++h) {
        const int64_t mh = m0 + 32 * h;
        if (mh >= e.M) return;           // uniform
        stage_half<NM, NN>(h, acc, stage);
        const int rows = cc.n == 0 ? 0 : e.M - mh < 32 ? (int)(e.M - mh) : 32;
#pragma unroll 1
        for (int r = r0; r < rows; r += S::RPI) {
            Raw8<YT> res = {};
            if (e.res) res = residual8<YT>(e, cc, mh + r);
            const v4i s0 = *reinterpret_cast<const v4i*>(&stage[r * S::PITCH + c]);
            const v4i s1 = *reinterpret_cast<const v4i*>(&stage[r * S::PITCH + c + 4]);
            const int s[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
            epilogue8<YT>(e, cc, mh + r, sx[32 * h + r], s, res);
        }
    }
}

// A wave's 16 NM x 16 NN sums, 32 rows at a time through the wave's own part
// of LDS, so that its stores are whole rows of its part and the epilogue's
// code exists once per activation.  A lane keeps its eight columns for all
// rows, so their scales and bias are read once.
template <int YT, int NM, int NN, bool NTS = false>
__device__ __forceinline__ void finish_part(const Epi& e, int64_t m0, int64_t n0, const v4i (&acc)[NM][NN],
                                               int* stage)
{
    const Cols8 cc = cols8(e, n0 + 8 * ((threadIdx.x & 63) % Stage<NM, NN>::LPR));
    if (m0 >= e.M) return;               // uniform
    stage_scales<NM, NN>(e, m0, stage);
    const bool inside = m0 + 16 * NM <= e.M && n0 + 16 * NN <= e.N && e.N <= 1 << 22 && e.ldr <= 1 << 22;
    if (inside && !e.z)
        with_act(e.act, [&](auto a) {
            if (e.res) finish_inside<YT, NM, NN, decltype(a)::value, true, NTS>(e, cc, m0, n0, acc, stage);
            else finish_inside<YT, NM, NN, decltype(a)::value, false, NTS>(e, cc, m0, n0, acc, stage);
        });
    else finish_any<YT, NM, NN>(e, cc, m0, acc, stage);
}

// k_epi_ring: operands whose rows start at 16-byte addresses.  A TILE x TILE
// output tile per workgroup of WM x WN waves, a wave a TILE / WM x TILE / WN
// part of it.  LDS is a ring of RING units, a unit one operand's [TILE x 128
// codes] slice: unit 2 kb holds the activations of block kb, unit 2 kb + 1 its
// weights.  Units arrive by direct global -> LDS loads (lane l of an
// instruction writes 16 bytes at base + 16 l, so the swizzle of eslot is
// applied to the address it reads).  A block is two 64-code steps; while the
// matrix cores work on one step's operands the next step's are read from LDS
// into a second set of registers.  One barrier per block, between its steps:
// there every wave has read both units, so their slots are refilled with the
// units RING ahead, and the next block's units have landed (those after it may
// still be on their way: the wait counts loads, it does not drain them).
//
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
// Where K is no multiple of 128, the block that the rest makes comes first
// (integer sums have no order): its missing chunks come from sixteen zero
// bytes on the weights' side, and the activations' side reads any valid chunk
// there.  All later loads are whole.
//
// The products are issued from asm that adds in place: the compiler, left to
// choose, gives the sums new registers and moves them back.
typedef __attribute__((address_space(3))) void lds_void;
__device__ const uint4 zero_codes = {0, 0, 0, 0};

// The loads are issued from asm, so that the compiler adds no wait of its own
// for them (they count in vmcnt; the kernel waits explicitly): every lane
// writes 16 bytes at M0 + 16 * lane.  Nothing else uses M0.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ uint64_t uniform_address(const void* p)
{
    const uint64_t v = (uint64_t)(size_t)p;
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
    return (uint64_t)hi << 32 | lo;
}
__device__ __forceinline__ void lds_load(uint64_t base, uint32_t off, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
                 : "memory", "m0");
}
__device__ __forceinline__ void lds_load_at(const void* g, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(lds) : "memory", "m0");
}
#pragma clang diagnostic pop

// c += w x, 16 x 16 x 64 codes.  The sums of one tile are next added to after
// every other tile of the wave, three products later or more.
__device__ __forceinline__ void add_product(v4i& c, v4i w, v4i x)
{
    asm volatile("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(c) : "v"(w), "v"(x));
}

// The wait instruction's operand: at most `vm` loads and `lgkm` LDS accesses
// still under way.
constexpr int WAIT(int vm, int lgkm) { return (vm & 15) | (vm >> 4) << 14 | 0x70 | lgkm << 8; }

// Tile of a workgroup.  Workgroup i of a launch goes to XCD i % 8; the launch
// index is renumbered so that each XCD (each L2) takes one contiguous run of
// tiles, walked in slabs of up to `slab` column tiles, columns fastest.
__device__ __forceinline__ void tile_of(int64_t nt, int64_t mt, int slab, int64_t& tm, int64_t& tn)
{
    const int64_t T = nt * mt, i = blockIdx.x;
    const int64_t xcd = i % 8, loc = i / 8, q = T / 8, r = T % 8;
    const int64_t L = xcd < r ? xcd * (q + 1) + loc : r * (q + 1) + (xcd - r) * q + loc;
    const int64_t per = (int64_t)slab * mt, first = (L / per) * slab;
    const int64_t wide = nt - first < slab ? nt - first : slab;
    const int64_t at = L % per;
    tn = first + at % wide;
    tm = at / wide;
}

// k_epi_tile: operands of any alignment and K.  Direct loads to LDS take
// 16-byte addresses only, so the codes pass through registers: a thread loads
// its chunks of both operands at any byte address D blocks ahead (the loop is
// unrolled by D, each block's registers refilled as they are written out) and
// the blocks alternate between two LDS buffers, one barrier per block.
// Measured, 777 x 4096 x 4095 35 us (aligned operands: 20), 8192 x 11008 x
// 4088 416 us (330): bound by the loads, whose 16 bytes per lane straddle
// lines.  One block ahead only: 52 / 485 us.
template <int YT, int TILE, int WM, int WN, int D, int WGS>
__global__ __launch_bounds__(64 * WM * WN, WGS * WM * WN / 4) void k_epi_tile(const int8_t* __restrict__ qx,
                                                                              const int8_t* __restrict__ qw, int64_t K,
                                                                              int64_t nt, int64_t mt, int slab, Epi e)
{
    constexpr int WAVES = WM * WN, NT = 64 * WAVES;
    constexpr int QM = TILE / WM, QN = TILE / WN, NM = QM / 16, NN = QN / 16;   // a wave's part and its 16-wide tiles
    constexpr int RPL = NT / 8, L = TILE / RPL;                                 // rows per load, loads per operand
    static_assert(D % 2 == 0, "blocks alternate between two buffers");
    __shared__ __attribute__((aligned(16))) union {
        uint8_t in[2][2][TILE * ET];
        int out[WAVES][Stage<NM, NN>::INTS];
    } lds;
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4, wm = w / WN, wn = w % WN;
    int64_t tm, tn;
    tile_of(nt, mt, slab, tm, tn);
    const int64_t m0 = tm * TILE, n0 = tn * TILE;
    const int fr = t >> 3, fc = t & 7;   // chunk fc of rows fr, fr + RPL, ...
    const int8_t* ga = qx + m0 * K;
    const int8_t* gb = qw + n0 * K;
    uint32_t oa[L], ob[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int r = fr + RPL * i;
        oa[i] = (uint32_t)(m0 + r < e.M ? r : (int)(e.M - 1 - m0)) * (uint32_t)K;
        ob[i] = (uint32_t)(n0 + r < e.N ? r : (int)(e.N - 1 - n0)) * (uint32_t)K;
    }
    v4i ra[D][L], rb[D][L];
    auto fetch = [&](int u, int kb) {    // a whole block
        const int k = kb * ET + 16 * fc;
#pragma unroll
        for (int i = 0; i < L; ++i) {
            ra[u][i] = codes16_whole(ga + k + oa[i]);
            rb[u][i] = codes16_whole(gb + k + ob[i]);
        }
    };
    v4i acc[NM][NN];
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < NN; ++j) acc[i][j] = v4i{};
    auto block = [&](int buf, const v4i (&a)[L], const v4i (&b)[L], auto refill) {
        uint8_t* la = lds.in[buf][0];
        uint8_t* lb = lds.in[buf][1];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            *reinterpret_cast<v4i*>(&la[eslot(fr + RPL * i, fc)]) = a[i];
            *reinterpret_cast<v4i*>(&lb[eslot(fr + RPL * i, fc)]) = b[i];
        }
        // the buffer written next was last read before this barrier
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        refill();
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v4i av[NM], bv[NN];
#pragma unroll
            for (int i = 0; i < NM; ++i)
                av[i] = *reinterpret_cast<const v4i*>(&la[eslot(wm * QM + i * 16 + l16, 4 * s + g4)]);
#pragma unroll
            for (int j = 0; j < NN; ++j)
                bv[j] = *reinterpret_cast<const v4i*>(&lb[eslot(wn * QN + j * 16 + l16, 4 * s + g4)]);
#pragma unroll
            for (int i = 0; i < NM; ++i)
#pragma unroll
                for (int j = 0; j < NN; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[j], av[i], acc[i][j], 0, 0, 0);
        }
    };
    const int whole = (int)(K / ET);
    if (whole > 0) {
#pragma unroll
        for (int u = 0; u < D; ++u) fetch(u, u < whole ? u : whole - 1);
        int kb = 0;
        for (; kb + D <= whole; kb += D)
#pragma unroll
            for (int u = 0; u < D; ++u)
                // past the end the last block again: an unconditional load leaves the waits of the others exact
                block(u & 1, ra[u], rb[u], [&] { fetch(u, kb + u + D < whole ? kb + u + D : whole - 1); });
#pragma unroll
        for (int u = 0; u < D - 1; ++u)
            if (kb + u < whole) block(u & 1, ra[u], rb[u], [] {});
    }
    __syncthreads();
    if (K % ET) {                        // the rest of K, zeros past it
        const int64_t k = (int64_t)whole * ET + 16 * fc;
        v4i a[L], b[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            a[i] = codes16(ga + oa[i], k, K);
            b[i] = codes16(gb + ob[i], k, K);
        }
        block(0, a, b, [] {});
        __syncthreads();
    }
    // the operands give way to the staged sums
    finish_part<YT, NM, NN>(e, m0 + QM * wm, n0 + QN * wn, acc, lds.out[w]);
}

template <int YT, int TILE, int RING, int WM, int WN, int WGS>
__global__ __launch_bounds__(64 * WM * WN, WGS * WM * WN / 4) void k_epi_ring(const int8_t* __restrict__ qx,
                                                                              const int8_t* __restrict__ qw, int64_t K,
                                                                              int64_t nt, int64_t mt, int slab, Epi e)
{
    constexpr int UNIT = TILE * ET;      // bytes of a unit
    constexpr int WAVES = WM * WN;
    constexpr int U = TILE / (8 * WAVES);          // loads per wave and unit
    constexpr int QM = TILE / WM, QN = TILE / WN;  // rows and columns of a wave's part
    constexpr int NM = QM / 16, NN = QN / 16;      // 16-wide tiles along its sides
    constexpr int AHEAD = (RING - 4) * U;          // loads that may be in flight behind the next block's
    constexpr int GROUPS = NM * NN >= 32 ? 16 : NM * NN >= 8 ? 8 : 4;   // products go in groups, loads between them
    constexpr int PER = NM * NN / GROUPS;
    static_assert(NM + NN <= 2 * GROUPS && 2 * U <= GROUPS && RING % 2 == 1 && TILE % (8 * WAVES) == 0, "schedule");
    static_assert(4 * WAVES * Stage<NM, NN>::INTS <= RING * UNIT, "staging");
    __shared__ __attribute__((aligned(16))) uint8_t ring[RING * UNIT];

    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4, wm = w / WN, wn = w % WN;
    int64_t tm, tn;
    tile_of(nt, mt, slab, tm, tn);
    const int64_t m0 = tm * TILE, n0 = tn * TILE;
    const int nkb = (int)((K + ET - 1) / ET);

    // loads of a unit: instruction q of wave w fills rows 8 (U w + q) .. + 7, lane l row l / 8, slot l % 8
    const int fr = 8 * U * w + (lane >> 3);
    const int8_t* ga = qx + m0 * K;
    const int8_t* gb = qw + n0 * K;
    uint32_t oa[U], ob[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
        const int r = fr + 8 * q;
        const int ra = m0 + r < e.M ? r : (int)(e.M - 1 - m0), rb = n0 + r < e.N ? r : (int)(e.N - 1 - n0);
        const uint32_t chunk = (uint32_t)(((lane & 7) ^ ((r >> 1) & 7)) << 4);
        oa[q] = (uint32_t)ra * (uint32_t)K + chunk;
        ob[q] = (uint32_t)rb * (uint32_t)K + chunk;
    }
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(size_t)(lds_void*)ring) + (uint32_t)w * (1024 * U);
    const int rest = K % ET != 0;        // block 0 is the rest, block kb > 0 starts at code (kb - rest) 128
    const int64_t k_rest = K / ET * ET;
    auto load_unit = [&](int unit, int slot) {
        const int b = unit >> 1;
        const int64_t k0 = rest && b == 0 ? k_rest : (int64_t)(b - rest) * ET;
        const bool weights = unit & 1;
        const int8_t* base = (weights ? gb : ga) + k0;
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int chunk = (lane & 7) ^ (((fr + 8 * q) >> 1) & 7);
            const int8_t* p = base + (weights ? ob[q] : oa[q]);
            const bool in = k0 + 16 * chunk < K;
            const void* from = in ? (const void*)p : weights ? (const void*)&zero_codes : (const void*)(p - 16 * chunk);
            lds_load_at(from, lds0 + (uint32_t)slot * UNIT + 1024u * q);
        }
    };

    // The zeros are set here, ahead of the loads and their barrier (volatile statements keep their order): a write of
    // an accumulation register needs wait states before a product reads it, which the compiler cannot see in asm.
    v4i acc[NM][NN];
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            acc[i][j] = v4i{};
            asm volatile("" : "+a"(acc[i][j]));
        }

    // lane l reads row l % 16, chunk 4 s + l / 16 of a tile of 16 rows
    const int key = l16 >> 1;
    const int la[2] = {(QM * wm + l16) * ET + ((g4 ^ key) << 4), (QM * wm + l16) * ET + (((4 + g4) ^ key) << 4)};
    const int lb[2] = {(QN * wn + l16) * ET + ((g4 ^ key) << 4), (QN * wn + l16) * ET + (((4 + g4) ^ key) << 4)};
    v4i av[2][NM], bv[2][NN];
    auto read = [&](int set, int x, const uint8_t* pa, const uint8_t* pb) {   // operand x of a step: weights first
        if (x < NN) bv[set][x] = *reinterpret_cast<const v4i*>(pb + 16 * ET * x);
        else if (x < NN + NM) av[set][x - NN] = *reinterpret_cast<const v4i*>(pa + 16 * ET * (x - NN));
    };
    auto products = [&](int set, int g) {
#pragma unroll
        for (int x = PER * g; x < PER * (g + 1); ++x)
            add_product(acc[x / NN][x % NN], bv[set][x % NN], av[set][x / NN]);
        __builtin_amdgcn_sched_barrier(0);
    };

    const int units = 2 * nkb;
    int sa = 0, sb = 1;                  // slots of the present block's units
    for (int u = 0; u < (units < RING ? units : RING); ++u) load_unit(u, u);
    if (units >= RING) __builtin_amdgcn_s_waitcnt(WAIT((RING - 2) * U, 15));
    else __builtin_amdgcn_s_waitcnt(WAIT(0, 15));
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int x = 0; x < NM + NN; ++x) read(0, x, ring + sa * UNIT + la[0], ring + sb * UNIT + lb[0]);
    // RING is odd: the units to come at block kb are the weights of block kb + RING / 2 and the activations after
    uint64_t wnext = uniform_address(gb + (int64_t)(RING / 2 - rest) * ET);
    uint64_t xnext = uniform_address(ga + (int64_t)(RING / 2 + 1 - rest) * ET);
    for (int kb = 0; kb < nkb; ++kb, wnext += ET, xnext += ET) {
        const uint8_t* pa = ring + sa * UNIT + la[1];
        const uint8_t* pb = ring + sb * UNIT + lb[1];
        __builtin_amdgcn_s_waitcnt(WAIT(63, 0));   // the first step's operands, before more reads join them
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {   // first step's products, second step's operands
            read(1, 2 * g, pa, pb);
            read(1, 2 * g + 1, pa, pb);
            products(0, g);
        }
        // both units read (lgkmcnt 0); the next block's two have landed
        const int next = 2 * kb + RING;
        if (next <= units) __builtin_amdgcn_s_waitcnt(WAIT(AHEAD, 0));
        else __builtin_amdgcn_s_waitcnt(WAIT(0, 0));
        asm volatile("s_barrier" ::: "memory");
        const uint32_t fa = lds0 + (uint32_t)sa * UNIT, fb = lds0 + (uint32_t)sb * UNIT;
        const bool more_w = next < units, more_x = next + 1 < units;
        sa = sa + 2 < RING ? sa + 2 : sa + 2 - RING;
        sb = sb + 2 < RING ? sb + 2 : sb + 2 - RING;
        // after the last block these slots hold older units, whose operands no product takes
        const uint8_t* na = ring + sa * UNIT + la[0];
        const uint8_t* nb = ring + sb * UNIT + lb[0];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {   // second step's products, the next block's first operands
            read(0, 2 * g, na, nb);
            read(0, 2 * g + 1, na, nb);
            if (g < U) {
                if (more_w) lds_load(wnext, ob[g], fa + 1024u * g);
            } else if (g < 2 * U) {
                if (more_x) lds_load(xnext, oa[g - U], fb + 1024u * (g - U));
            }
            products(1, g);
        }
    }
    // The last products' sums need up to 19 wait states before they are read, which the compiler cannot see behind
    // asm; the empty statements after the wait, in order as volatile asm is, keep every read behind it.
    asm volatile("s_nop 15\n\ts_nop 7");
#pragma unroll
    for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int j = 0; j < NN; ++j) asm volatile("" : "+a"(acc[i][j]));
    __builtin_amdgcn_s_waitcnt(0x0070);
    asm volatile("s_barrier" ::: "memory");   // the ring gives way to the staged sums
    finish_part<YT, NM, NN, TILE == 256>(e, m0 + QM * wm, n0 + QN * wn, acc,
                                         reinterpret_cast<int*>(ring) + w * Stage<NM, NN>::INTS);
}

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

// The kernel of a product, by its shape.  Measured (us, K = 4096 unless given;
// few tokens / 64 / 128 / 256 tile):
//   24 x 4096      8.3 / 11.9 / 18 / 46      32 x 11008    19.2 / 11.9 / 21 / 47
//   64 x 11008      30 / 12.0 / 21 / 49      512 x 4096       - / 16.6 / 19.5 / -
//   640 x 4096       - / 24.5 / 20.0 / -     2048 x 4096      - / - / 35 / 51
//   4096 x 4096      - / - / 87 / 60
// The few-token kernel reads the tokens again for every 16 columns, which costs
// more the more columns there are.  A tile kernel takes a time of its own per
// round of resident workgroups (two 64 x 64 tiles or, up to 256 of them, one
// 128 x 128 tile per CU), so the smallest tile that needs one round is taken,
// and the largest once it fills the chip.  128 x 128 tiles beyond one round run
// two to a CU on shorter rings.  Where the output is so small that tiles leave
// most CUs idle, its 32 x 16 or 32 x 32 pieces, each with the K axis split over
// eight waves, do not (tiles / 32 x 16 / 32 x 32):
//   220 x 507 x 10256   27 / 13.4 / 17.1     40 x 1024 x 8192     17.8 / 12.9 / 16.6
//   64 x 4096 x 4096  11.1 / 13.3 / 9.9      1260 x 140 x 10688   23.4 / 26 / 17.2
//   128 x 4096 x 4096 11.2 / 24 / 16.9       220 x 507 x 10250    34 / 42 / 55
// (the last with rows at odd addresses, whose loads cost these kernels more).
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
    if (e.M <= 16) TQ_FEW(1, 1, 8, 4);
    if ((e.M <= 32 && (e.N <= 6144 || !rows16)) || (rows16 && cdiv(e.M, 32) * cdiv(e.N, 16) <= 256))
        TQ_FEW(2, 1, 8, 2);
    if (rows16 && cdiv(e.M, 32) * cdiv(e.N, 32) <= 256) TQ_FEW(2, 2, 8, 2);
#undef TQ_FEW
    if (rows16) {
#define TQ_RING(TILE, RING, WM, WN, WGS)                                                                     \
    do {                                                                                                     \
        const int64_t nt = cdiv(e.N, TILE), mt = cdiv(e.M, TILE);                                            \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                            \
        hipLaunchKernelGGL((k_epi_ring<YT, TILE, RING, WM, WN, WGS>), dim3((unsigned)(nt * mt)),             \
                           dim3(64 * WM * WN), 0, st, qx, qw, K, nt, mt, slab, e);                           \
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
        hipLaunchKernelGGL((k_epi_tile<YT, TILE, WM, WN, D, WGS>), dim3((unsigned)(nt * mt)),                \
                           dim3(64 * WM * WN), 0, st, qx, qw, K, nt, mt, slab, e);                           \
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
