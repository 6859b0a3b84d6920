// tq_product.h -- what the W8A8 products share: the sums of codes with codes on
// the matrix cores (a few tokens, tiles fed by direct loads to LDS, tiles of any
// alignment), activations, and the epilogue that finishes eight columns of a row.
//
//   z[m][n] = ((float)sum_k qx[m][k] qw[n][k]) sx[m] sw[n] + bias[n]
//   y[m][n] = act(z[m][n]) + residual[m][n]
//
// A gated product takes the rows of two weights into one tile, sixteen of one
// and sixteen of the other in turn, so that a lane holds both sums of an output.
#pragma once

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
// ------------------------------------------------------------- operand loads
// A matrix operand wants row l % 16 in lane l, so lanes side by side read rows apart, and
// the address unit takes such a load one lane per clock: 64 clocks for 1 KB, which
// bounds a CU to 16 bytes per clock wherever operands come straight from memory (48 x
// 4096 x 11008 codes took 21.8 us for it, a few tokens' weights 10 of their 12).  So four
// lanes side by side read 64 bytes of one row at a time, four rows in turn, and change
// places afterwards: 256 bytes of sixteen rows, in four operands of 64.  Lane l's j-th
// then holds bytes 64 (l / 16) + 16 j of row l % 16: the same order of K for every
// operand so loaded.
struct Quad {
    v4i r[4];
};

// x and y of the lanes l ^ 1 (XOR1) or l ^ 2 trade places: where that bit of l is 0, y
// becomes the neighbour's x, where it is 1, x the neighbour's y.  (The same as one
// selecting instruction per value, from asm, which the compiler does not find, was
// slower: 48 x 4096 x 11008 15.7 us against 13.3.)
template <int CTRL>
__device__ __forceinline__ void trade(v4i& x, v4i& y, bool bit)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int u = x[i], v = y[i];
        const int of_u = (int)dpp<CTRL>((uint32_t)u), of_v = (int)dpp<CTRL>((uint32_t)v);
        x[i] = bit ? of_v : u;
        y[i] = bit ? v : of_u;
    }
}

// Lane 4 a + b's r[u] goes to lane 4 a + u's r[b].  Every lane takes part.
__device__ __forceinline__ void change_places(Quad& q)
{
    const bool odd = threadIdx.x & 1, high = threadIdx.x & 2;
    trade<DPP_XOR1>(q.r[0], q.r[1], odd);
    trade<DPP_XOR1>(q.r[2], q.r[3], odd);
    trade<DPP_XOR2>(q.r[0], q.r[2], high);
    trade<DPP_XOR2>(q.r[1], q.r[3], high);
}

// Where a lane's four loads of sixteen rows begin, relative to the first of them:
// rows past `last` are the last again.
template <class Off>
struct QuadAt {
    Off at[4];
};
template <class Off>
__device__ __forceinline__ QuadAt<Off> quad_at(int last, Off row_bytes)
{
    const int l = threadIdx.x & 63, first = (l & 15) & ~3;
    QuadAt<Off> q;
#pragma unroll
    for (int u = 0; u < 4; ++u)
        q.at[u] = (Off)(first + u < last ? first + u : last) * row_bytes + (Off)(64 * (l >> 4) + 16 * (l & 3));
    return q;
}
template <class Off>
__device__ __forceinline__ void quad_load(Quad& q, const void* rows, const QuadAt<Off>& a)
{
#pragma unroll
    for (int u = 0; u < 4; ++u) q.r[u] = codes16_whole(static_cast<const int8_t*>(rows) + a.at[u]);
}

// ------------------------------------------------------------- a few tokens
// Whether the few-token kernels take a product: they read the tokens again for every 16
// columns, which costs more the more columns there are, but give work to every CU
// where an output has few 32 x 32 pieces.
inline bool few_tokens(int64_t M, int64_t N)
{
    return M <= 16 || (M <= 32 && N <= 6144) || cdiv(M, 32) * cdiv(N, 32) <= 256;
}
// And, beyond 16 tokens, whether in 32 x 16 pieces rather than 32 x 32.
inline bool few_columns(int64_t M, int64_t N) { return (M <= 32 && N <= 6144) || cdiv(M, 32) * cdiv(N, 16) <= 256; }

// Sixteen rows of an operand: the first (uniform) and the last of them that is there.
struct Rows16 {
    const int8_t* first;
    int last;
};
// Rows from `from` on of a matrix of n rows of K codes; past its end the last one.
__device__ __forceinline__ Rows16 rows16_of(const int8_t* m, int64_t n, int64_t from, int64_t K)
{
    const int64_t f = from < n ? from : n - 1;
    return Rows16{m + f * K, n - 1 - f < 15 ? (int)(n - 1 - f) : 15};
}

// The sums of 16 CT weight rows with 16 MT tokens by a workgroup of NWV waves,
// which take the K axis in turn, 256 codes at a time: acc holds this wave's share.
// The weights are the matrix core's first operand, the tokens its second.  U groups of
// both are in flight per wave, each slot refilled as it is used.
template <int MT, int CT, int NWV, int U>
__device__ __forceinline__ void few_product(const Rows16 (&weights)[CT], const Rows16 (&tokens)[MT], int64_t K,
                                            v4i (&acc)[MT][CT])
{
    const int t = threadIdx.x, w = __builtin_amdgcn_readfirstlane(t >> 6), l16 = t & 15, g4 = (t & 63) >> 4;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) acc[i][j] = v4i{};
    QuadAt<uint32_t> wa[CT], xa[MT];
#pragma unroll
    for (int j = 0; j < CT; ++j) wa[j] = quad_at(weights[j].last, (uint32_t)K);
#pragma unroll
    for (int i = 0; i < MT; ++i) xa[i] = quad_at(tokens[i].last, (uint32_t)K);
    // this wave's whole groups are w, w + NWV, ...
    const int groups = (int)(K / 256);
    Quad a[U][CT], b[U][MT];
    auto fetch = [&](int u, int g) {
#pragma unroll
        for (int j = 0; j < CT; ++j) quad_load(a[u][j], weights[j].first + g * 256, wa[j]);
#pragma unroll
        for (int i = 0; i < MT; ++i) quad_load(b[u][i], tokens[i].first + g * 256, xa[i]);
    };
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (w + u * NWV < groups) fetch(u, w + u * NWV);
    for (int g = w; g < groups; g += U * NWV)
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (g + u * NWV >= groups) break;
#pragma unroll
            for (int j = 0; j < CT; ++j) change_places(a[u][j]);
#pragma unroll
            for (int i = 0; i < MT; ++i) change_places(b[u][i]);
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int j = 0; j < CT; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[u][j].r[s], b[u][i].r[s], acc[i][j], 0, 0, 0);
            if (g + (u + U) * NWV < groups) fetch(u, g + (u + U) * NWV);
        }
    if (groups % NWV != w) return;
    for (int64_t k = (int64_t)groups * 256 + 16 * g4; k - 16 * g4 < K; k += 64) {    // the rest of K
        v4i x[CT], y[MT];
#pragma unroll
        for (int j = 0; j < CT; ++j)
            x[j] = codes16(weights[j].first + (int64_t)(l16 < weights[j].last ? l16 : weights[j].last) * K, k, K);
#pragma unroll
        for (int i = 0; i < MT; ++i)
            y[i] = codes16(tokens[i].first + (int64_t)(l16 < tokens[i].last ? l16 : tokens[i].last) * K, k, K);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < CT; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(x[j], y[i], acc[i][j], 0, 0, 0);
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

// The weights of a product are the rows of one [N, K] matrix, or of two (a gate's and
// the other projection's).  Row r of a tile's weights is this row from the tile's
// first on, of weight (r / 16) % 2 where there are two.
template <bool GATED>
__device__ __forceinline__ int tile_row(int r) { return GATED ? (r >> 5) * 16 + (r & 15) : r; }

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

// ------------------------------------------------------------ the tile kernels
// An epilogue E gives M and N (rows of a weight), GATED (two weights, the second
// from second_weight, sixteen rows of either in turn: a tile is TILE / 2 columns
// wide), staging() bytes of LDS and finish(), which takes a wave's sums, the tile's
// place and what early() read before the first block.
//
// k_epi_ring: operands whose rows start at 16-byte addresses.  A TILE x TILE tile
// per workgroup of WM x WN waves, a wave a TILE / WM x TILE /
// WN part of it.  LDS is a ring of RING units, a unit one operand's [TILE x 128
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
// Where K is no multiple of 128, the block that the rest makes comes first
// (integer sums have no order): its missing chunks come from sixteen zero
// bytes on the weights' side, and the activations' side reads any valid chunk
// there.  All later loads are whole.
//
// The products are issued from asm that adds in place: the compiler, left to
// choose, gives the sums new registers and moves them back.
template <class E, int TILE, int RING, int WM, int WN, int WGS>
__global__ __launch_bounds__(64 * WM * WN, WGS * WM * WN / 4) void k_epi_ring(const int8_t* __restrict__ qx,
                                                                              const int8_t* __restrict__ qw, int64_t K,
                                                                              int64_t nt, int64_t mt, int slab, E e)
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
    static_assert(!E::GATED || U == 2 || U == 4, "the weight of an instruction's rows");
    static_assert(E::template staging<TILE, WM, WN>() <= RING * UNIT, "staging");
    __shared__ __attribute__((aligned(16))) uint8_t ring[RING * UNIT];

    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4, wm = w / WN, wn = w % WN;
    int64_t tm, tn;
    tile_of(nt, mt, slab, tm, tn);
    const int64_t m0 = tm * TILE, n0 = tn * (E::GATED ? TILE / 2 : TILE);
    const int nkb = (int)((K + ET - 1) / ET);

    // loads of a unit: instruction q of wave w fills rows 8 (U w + q) .. + 7, lane l row l / 8, slot l % 8
    const int fr = 8 * U * w + (lane >> 3);
    const int8_t* ga = qx + m0 * K;
    // with two weights an instruction's eight rows are all of one: with U = 4 it follows from q, with U = 2 from the wave
    const int8_t* gb = (E::GATED && U == 2 && (w & 1) ? e.second_weight(qw) : qw) + n0 * K;
    const int8_t* gb2 = E::GATED && U == 4 ? e.second_weight(qw) + n0 * K : gb;
    auto second = [](int q) { return E::GATED && U == 4 && q >= 2; };
    uint32_t oa[U], ob[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
        const int r = fr + 8 * q;
        const int f = tile_row<E::GATED>(r);
        const int ra = m0 + r < e.M ? r : (int)(e.M - 1 - m0), rb = n0 + f < e.N ? f : (int)(e.N - 1 - n0);
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
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int8_t* base = (weights ? second(q) ? gb2 : gb : ga) + k0;
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

    const auto early = E::template early<TILE, WM, WN>(e, m0);
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
    uint64_t wnext2 = uniform_address(gb2 + (int64_t)(RING / 2 - rest) * ET);
    uint64_t xnext = uniform_address(ga + (int64_t)(RING / 2 + 1 - rest) * ET);
    for (int kb = 0; kb < nkb; ++kb, wnext += ET, wnext2 += ET, xnext += ET) {
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
                if (more_w) lds_load(second(g) ? wnext2 : wnext, ob[g], fa + 1024u * g);
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
    E::template finish<TILE, WM, WN>(e, m0, n0, acc, ring, early);
}

// k_epi_tile: operands of any alignment and K.  Direct loads to LDS take 16-byte addresses only, so the codes pass through
// registers: a thread loads its chunks of both operands at any byte address D
// blocks ahead (the loop is unrolled by D, each block's registers refilled as
// they are written out) and the blocks alternate between two LDS buffers, one
// barrier per block.
template <class E, int TILE, int WM, int WN, int D, int WGS>
__global__ __launch_bounds__(64 * WM * WN, WGS * WM * WN / 4) void k_epi_tile(const int8_t* __restrict__ qx,
                                                                              const int8_t* __restrict__ qw, int64_t K,
                                                                              int64_t nt, int64_t mt, int slab, E e)
{
    constexpr int NT = 64 * WM * WN;
    constexpr int QM = TILE / WM, QN = TILE / WN, NM = QM / 16, NN = QN / 16;   // a wave's part and its 16-wide tiles
    constexpr int RPL = NT / 8, L = TILE / RPL;                                 // rows per load, loads per operand
    static_assert(D % 2 == 0, "blocks alternate between two buffers");
    static_assert(RPL % 32 == 0, "the weight of a wave's rows");
    __shared__ __attribute__((aligned(16))) union {
        uint8_t in[2][2][TILE * ET];
        uint8_t out[E::template staging<TILE, WM, WN>()];
    } lds;
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4, wm = w / WN, wn = w % WN;
    int64_t tm, tn;
    tile_of(nt, mt, slab, tm, tn);
    const int64_t m0 = tm * TILE, n0 = tn * (E::GATED ? TILE / 2 : TILE);
    const int fr = t >> 3, fc = t & 7;   // chunk fc of rows fr, fr + RPL, ...
    const int8_t* ga = qx + m0 * K;
    // the rows of wave w's loads are 8 w .. 8 w + 7 and those RPL, a multiple of 32, further on: all of one weight
    const int8_t* gb = (E::GATED && (w >> 1 & 1) ? e.second_weight(qw) : qw) + n0 * K;
    uint32_t oa[L], ob[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
        const int r = fr + RPL * i;
        oa[i] = (uint32_t)(m0 + r < e.M ? r : (int)(e.M - 1 - m0)) * (uint32_t)K;
        const int f = tile_row<E::GATED>(r);
        ob[i] = (uint32_t)(n0 + f < e.N ? f : (int)(e.N - 1 - n0)) * (uint32_t)K;
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
    const auto early = E::template early<TILE, WM, WN>(e, m0);
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
    E::template finish<TILE, WM, WN>(e, m0, n0, acc, lds.out, early);
}

}  // namespace tq
