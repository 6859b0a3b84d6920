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
// 1 / (1 + exp(-u)) from t = exp(-|u|) <= 1, which cannot overflow.
struct Logistic {
    float p, pq;                         // the value and its slope p (1 - p)
};
__device__ __forceinline__ Logistic logistic(float u)
{
    const float t = __builtin_amdgcn_exp2f(-__builtin_fabsf(u) * LOG2E);
    const float h = __builtin_amdgcn_rcpf(1.0f + t);
    Logistic r;
    r.p = u >= 0.0f ? h : t * h;
    r.pq = t * h * h;
    return r;
}

constexpr float GELU_C = 0.79788456080286535588f;      // sqrt(2 / pi)
constexpr float GELU_A = 0.044715f;
constexpr float SQRT_HALF = 0.70710678118654752440f;

// act(v) of eight values; the branch on `act` is uniform.  The tanh form of
// gelu is v times a logistic: (1 + tanh u) / 2 = 1 / (1 + exp(-2u)).
__device__ __forceinline__ void act8(int act, float v[8])
{
    switch (act) {
    case TQ_ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] > 0.0f || v[i] != v[i] ? v[i] : 0.0f;
        break;
    case TQ_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * logistic(v[i]).p;
        break;
    case TQ_ACT_GELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.5f * v[i] * erfcf(-v[i] * SQRT_HALF);
        break;
    case TQ_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < 8; ++i)
            v[i] = v[i] * logistic(2.0f * GELU_C * v[i] * __builtin_fmaf(GELU_A * v[i], v[i], 1.0f)).p;
        break;
    default: break;
    }
}

// d[i] *= act'(z[i]).  A slope's second term v p' vanishes with p' (a value
// so large that p' underflows would otherwise meet an overflow there).
__device__ __forceinline__ void slope8(int act, const float z[8], float d[8])
{
    switch (act) {
    case TQ_ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = z[i] > 0.0f ? d[i] : 0.0f;
        break;
    case TQ_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const Logistic l = logistic(z[i]);
            d[i] *= l.p + (l.pq == 0.0f ? 0.0f : z[i] * l.pq);
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
            const float zz = GELU_A * z[i] * z[i];
            const Logistic l = logistic(2.0f * GELU_C * z[i] * (1.0f + zz));
            d[i] *= l.p + (l.pq == 0.0f ? 0.0f : z[i] * (2.0f * GELU_C) * (1.0f + 3.0f * zz) * l.pq);
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

// Eight consecutive columns col .. col + 7 of one row, from their sums.
template <int YT>
__device__ __forceinline__ void epilogue8(const Epi& e, int64_t row, int64_t col, const int acc[8])
{
    const float sx = e.sx[row];
    const int64_t at = row * e.N + col;
    float v[8];
    if (col + 8 <= e.N) {
        float sw[8], b[8];
        widen8<F32>(load8_any<F32>(e.sw, col), sw);
        const RawAny rb = load8_rt(e.bias, e.bias_dt, col);
        Raw8<YT> rr;
        if (e.res) rr = load8_any<YT>(e.res, row * e.ldr + col);
        widen8_rt(rb, e.bias, e.bias_dt, 0.0f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (float)acc[i] * sx * sw[i];
        if (e.bias) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += b[i];
        }
        if (e.z) store8_any<YT>(e.z, at, v);
        act8(e.act, v);
        if (e.res) {
            float r[8];
            widen8<YT>(rr, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
        }
        store8_any<YT>(e.y, at, v);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = 0.0f;
            if (col + i < e.N) {
                v[i] = (float)acc[i] * sx * e.sw[col + i];
                if (e.bias) v[i] += load1_rt(e.bias, e.bias_dt, col + i, 0.0f);
                if (e.z) store1<YT>(e.z, at + i, v[i]);
            }
        }
        act8(e.act, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (col + i < e.N) {
                if (e.res) v[i] += load1<YT>(e.res, row * e.ldr + col + i);
                store1<YT>(e.y, at + i, v[i]);
            }
    }
}

// Sixteen codes at any byte address, zeros from code K of the row on.
__device__ __forceinline__ v4i codes16(const int8_t* row, int64_t k, int64_t K)
{
    if (k + 16 <= K) {
        const u32x4_byte v = *reinterpret_cast<const u32x4_byte*>(row + k);
        return v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
    }
    v4i r = v4i{};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int b = k + i < K ? (int)(uint8_t)row[k + i] << (8 * (i & 3)) : 0;
        r[i >> 2] |= b;
    }
    return r;
}

// ------------------------------------------------------------- a few tokens
// k_epi_few (M <= 16 MT): bound by the weights, which are read once.  A
// workgroup of NWV waves owns 16 output columns; the waves take the K axis in
// turn, 128 codes at a time, so that a wave's two loads use whole 128-byte
// lines; the sums meet in LDS.  The weights are the matrix core's first
// operand (16 columns), the tokens its second (16 tokens, rows past M repeat
// row M - 1), U blocks of both in flight per wave.
template <int YT, int MT, int NWV>
__global__ __launch_bounds__(64 * NWV) void k_epi_few(const int8_t* __restrict__ qx, const int8_t* __restrict__ qw,
                                                      int64_t K, Epi e)
{
    constexpr int U = MT == 1 ? 4 : 2;
    __shared__ int sums[NWV][MT * 16][20];   // rows of 16 sums, 20 apart (16-byte steps that spread over the banks)
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t n = n0 + l16 < e.N ? n0 + l16 : e.N - 1;
    const int8_t* pw = qw + n * K;
    const int8_t* px[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) {
        const int64_t m = 16 * i + l16 < e.M ? 16 * i + l16 : e.M - 1;
        px[i] = qx + m * K;
    }
    v4i acc[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) acc[i] = v4i{};
    const int64_t nkb = (K + 127) / 128, whole = K / 128;
    int64_t kb = w;
    for (; kb + (U - 1) * NWV < whole; kb += U * NWV) {
        v4i a[U][2], b[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int64_t k = (kb + u * NWV) * 128 + 64 * s + 16 * g4;
                const u32x4_byte v = *reinterpret_cast<const u32x4_byte*>(pw + k);
                a[u][s] = v4i{(int)v.x, (int)v.y, (int)v.z, (int)v.w};
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const u32x4_byte x = *reinterpret_cast<const u32x4_byte*>(px[i] + k);
                    b[u][s][i] = v4i{(int)x.x, (int)x.y, (int)x.z, (int)x.w};
                }
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int s = 0; s < 2; ++s)
#pragma unroll
                for (int i = 0; i < MT; ++i)
                    acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][s], b[u][s][i], acc[i], 0, 0, 0);
    }
    for (; kb < nkb; kb += NWV)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            const int64_t k = kb * 128 + 64 * s + 16 * g4;
            const v4i a = codes16(pw, k, K);
#pragma unroll
            for (int i = 0; i < MT; ++i)
                acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, codes16(px[i], k, K), acc[i], 0, 0, 0);
        }
    // lane l holds columns 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
    for (int i = 0; i < MT; ++i) *reinterpret_cast<v4i*>(&sums[w][16 * i + l16][4 * g4]) = acc[i];
    __syncthreads();
    for (int j = t; j < MT * 32; j += 64 * NWV) {
        const int m = j >> 1, c = 8 * (j & 1);
        if (m >= e.M || n0 + c >= e.N) continue;
        int s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = 0;
        for (int v = 0; v < NWV; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) s[i] += sums[v][m][c + i];
        epilogue8<YT>(e, m, n0 + c, s);
    }
}

// -------------------------------------------------------------- many tokens
// k_epi_tile: a 128 x 128 output tile per 256-thread workgroup, wave w the
// 64 x 64 quarter (w / 2, w % 2) as 4 x 4 tiles of 16 x 16.  Any K and any
// alignment: a thread loads four 16-code chunks of each operand into registers
// one 128-code block ahead and writes them to LDS (zeros past K).  The product
// is taken as D^T, so a lane holds four consecutive columns of a row; at the
// end each wave lays its quarter out in LDS and finishes it eight columns at a
// time, so that stores are whole and the epilogue's code exists once.
constexpr int ET = 128;
constexpr int EPITCH = 68;               // ints between rows of a staged quarter
__device__ __forceinline__ int eslot(int row, int chunk) { return row * ET + ((chunk ^ ((row >> 1) & 7)) << 4); }

// Finishes a wave's 64 x 64 sums acc[i][j][r] = row 16 i + l % 16, column
// 16 j + 4 (l / 16) + r through its own part of LDS.
template <int YT>
__device__ __forceinline__ void finish64(const Epi& e, int64_t m0, int64_t n0, const v4i (&acc)[4][4], int* stage)
{
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            *reinterpret_cast<v4i*>(&stage[(16 * i + l16) * EPITCH + 16 * j + 4 * g4]) = acc[i][j];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    const int c = 8 * (lane & 7);
    if (n0 + c >= e.N) return;
    for (int r = lane >> 3; r < 64; r += 8) {
        if (m0 + r >= e.M) break;
        int s[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const v4i v = *reinterpret_cast<const v4i*>(&stage[r * EPITCH + c + 4 * h]);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[4 * h + i] = v[i];
        }
        epilogue8<YT>(e, m0 + r, n0 + c, s);
    }
}

template <int YT>
__global__ __launch_bounds__(256) void k_epi_tile(const int8_t* __restrict__ qx, const int8_t* __restrict__ qw,
                                                  int64_t K, Epi e)
{
    __shared__ __attribute__((aligned(16))) union {
        uint8_t in[2][2][ET * ET];
        int out[4][64 * EPITCH];
    } lds;
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4, wm = w >> 1, wn = w & 1;
    const int64_t m0 = (int64_t)blockIdx.y * ET, n0 = (int64_t)blockIdx.x * ET;
    const int64_t nkb = (K + ET - 1) / ET;
    const int fr = t >> 3, fc = t & 7;   // chunk fc of rows fr, fr + 32, + 64, + 96
    const int8_t* pa[4];
    const int8_t* pb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + fr + 32 * i, n = n0 + fr + 32 * i;
        pa[i] = qx + (m < e.M ? m : e.M - 1) * K;
        pb[i] = qw + (n < e.N ? n : e.N - 1) * K;
    }
    v4i ra[4], rb[4];
    auto fetch = [&](int64_t kb) {
        const int64_t k = kb * ET + 16 * fc;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            ra[i] = codes16(pa[i], k, K);
            rb[i] = codes16(pb[i], k, K);
        }
    };
    v4i acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = v4i{};
    fetch(0);
    for (int64_t kb = 0; kb < nkb; ++kb) {
        uint8_t* la = lds.in[kb & 1][0];
        uint8_t* lb = lds.in[kb & 1][1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            *reinterpret_cast<v4i*>(&la[eslot(fr + 32 * i, fc)]) = ra[i];
            *reinterpret_cast<v4i*>(&lb[eslot(fr + 32 * i, fc)]) = rb[i];
        }
        // the buffer written next was last read before this barrier
        __syncthreads();
        if (kb + 1 < nkb) fetch(kb + 1);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            v4i av[4], bv[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                av[i] = *reinterpret_cast<const v4i*>(&la[eslot(wm * 64 + i * 16 + l16, 4 * s + g4)]);
                bv[i] = *reinterpret_cast<const v4i*>(&lb[eslot(wn * 64 + i * 16 + l16, 4 * s + g4)]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bv[j], av[i], acc[i][j], 0, 0, 0);
        }
    }
    __syncthreads();                     // the operands give way to the staged sums
    finish64<YT>(e, m0 + 64 * wm, n0 + 64 * wn, acc, lds.out[w]);
}

// ------------------------------------------------------ backward of epilogue
// k_epi_bwd: dz = dy act'(z) and its column sums: 4 bytes read and 2 written
// per bf16 element, bound by HBM.  A wave owns 512 columns, a workgroup's four
// waves take a chunk of the rows in turn, U rows in flight each; their column
// sums meet in LDS in wave order and leave as one row of partials per chunk.
template <int FT>
__global__ __launch_bounds__(256) void k_epi_bwd(const void* __restrict__ dy, const void* __restrict__ z, int64_t M,
                                                 int64_t N, int64_t chunk, int act, void* __restrict__ dz,
                                                 float* __restrict__ part, int64_t ldp)
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
__global__ __launch_bounds__(256) void k_epi_bwd_thin(const void* __restrict__ dy, const void* __restrict__ z,
                                                      int64_t M, int64_t N, int64_t chunk, int act,
                                                      void* __restrict__ dz, float* __restrict__ part, int64_t ldp)
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
constexpr int64_t EPI_CHUNKS = 64;       // row chunks of the backward pass
inline int64_t epi_chunk(int64_t M)      // rows per chunk: whole rounds of the four waves' four rows
{
    return cdiv(cdiv(M, EPI_CHUNKS), 16) * 16;
}

template <int YT>
static void product_launch(const int8_t* qx, const int8_t* qw, int64_t K, const Epi& e, hipStream_t st)
{
#define TQ_FEW(MT, NWV)                                                                                    \
    hipLaunchKernelGGL((k_epi_few<YT, MT, NWV>), dim3((unsigned)cdiv(e.N, 16)), dim3(64 * NWV), 0, st, qx, qw, K, e)
    if (e.M <= 64) {
        if (e.M <= 16) TQ_FEW(1, 8);
        else if (e.M <= 32) TQ_FEW(2, 8);
        else TQ_FEW(4, 8);
        return;
    }
#undef TQ_FEW
    const dim3 grid((unsigned)cdiv(e.N, ET), (unsigned)cdiv(e.M, ET));
    hipLaunchKernelGGL((k_epi_tile<YT>), grid, dim3(256), 0, st, qx, qw, K, e);
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
    if (K > 131071 || cdiv(M, ET) > 65535 || cdiv(N, 16) > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    if (!natural(sx, TQ_F32) || !natural(sw, TQ_F32) || (bias && !natural(bias, bias_dtype)) ||
        !natural(residual, y_dtype) || !natural(y, y_dtype) || !natural(preact, y_dtype))
        return TQ_ERR_ALIGN;
    const Epi e = {sx, sw, bias, bias_dtype, act, residual, residual_row_stride, y, preact, M, N};
    TQ_LLM_FT_SWITCH(y_dtype, product_launch<FTV>(qx, qw, K, e, as_stream(stream)));
    return launch_status();
}

size_t tq_linear_epilogue_backward_workspace_bytes(int64_t M, int64_t N)
{
    if (M <= 0 || N <= 0) return 0;
    return (size_t)cdiv(M, epi_chunk(M)) * (size_t)colsum_ld(N) * sizeof(float);
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
    if (cdiv(N, 512) > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    if (dbias) {
        if (!workspace || workspace_bytes < tq_linear_epilogue_backward_workspace_bytes(M, N)) return TQ_ERR_INVALID;
        if (!aligned16(workspace)) return TQ_ERR_ALIGN;
    }
    float* part = dbias ? static_cast<float*>(workspace) : nullptr;
    const int64_t chunk = epi_chunk(M), chunks = cdiv(M, chunk), ld = colsum_ld(N);
    const dim3 grid((unsigned)cdiv(N, 512), (unsigned)chunks);
    TQ_LLM_FT_SWITCH(dtype, {
        if (N < 8)
            hipLaunchKernelGGL((k_epi_bwd_thin<FTV>), grid, dim3(256), 0, st, dy, preact, M, N, chunk, act, dz, part, ld);
        else
            hipLaunchKernelGGL((k_epi_bwd<FTV>), grid, dim3(256), 0, st, dy, preact, M, N, chunk, act, dz, part, ld);
    });
    if (dbias) colsum_launch(part, chunks, 1, ld, N, dbias, nullptr, TQ_F32, st);
    return launch_status();
}

}  // extern "C"
