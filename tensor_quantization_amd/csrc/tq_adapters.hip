// tq_adapters.hip -- the W8A8 product beside low-rank adapters of many requests:
// token m has the adapter c = adapter[m] of its request, or none.
//
//   h[m][r] = scale[c] sum_k x[m][k] a[c][r][k]
//   z[m][n] = ((float)sum_k qx[m][k] qw[n][k]) sx[m] sw[n] + sum_r h[m][r] b[c][n][r] + bias[n]
//   y = act(z) + residual
//
// x and the adapters are of one type, their products summed in binary32.  h goes from
// its kernel to the product's through the workspace, and the product adds its part in
// the epilogue.  For a few tokens that is a scalar loop per output, and h is
// binary32.  For tiles it is the matrix cores' work, and h comes in their operand order,
// 16 tokens and a step of 32 ranks (binary32: 16) in one piece.  A 16-bit operand of h
// would lose what h holds beyond 8 or 11 bits, so it goes in twice: h = hi + lo in the
// adapters' type, 16 or more bits in all (f16, whose range is short, takes a token's
// step relative to a power of two near its largest value).
//
// The tokens of one sixteen-row operand may have several adapters.  Each takes its
// turn, the other tokens' h cleared, and only its own tokens take the result, so
// that what another adapter holds (infinities, NaN) does not reach them.  An infinity in
// a token's own b makes NaN where it meets hi and lo apart, one of which may be 0 or of the
// other sign; outputs that are NaN are therefore looked at once more on their way out
// (which costs the call 0.2 to 1.5%; b looked through as it is loaded, 2 to 6%).
#include "tq_product.h"

namespace tq {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

struct Adapters {
    const int32_t* id;                   // [M]: an adapter, or none where outside [0, count)
    const void* a;                       // [count, R, K]
    const void* b;                       // [count, N, R]
    const float* scale;                  // [count], or null
    void* h;                             // for a few tokens binary32 [M, ldh], else in operand order
    int* up;                             // f16 in operand order: a token's and step's exponent [M, steps]
    int count, R, ldh, dt;
};

// In operand order a piece of 1024 bytes holds, for lane l, E ranks from E (l / 16) on of
// token l % 16; 16-bit types have two pieces, hi and lo.
template <int AT>
struct Low {
    static constexpr int STEP = AT == F32 ? 16 : 32, E = STEP / 4, PIECES = AT == F32 ? 1 : 2;
    static __device__ __forceinline__ int steps(const Adapters& ad) { return (ad.R + STEP - 1) / STEP; }
    static __device__ __forceinline__ uint4* piece(const Adapters& ad, int64_t tile, int step)
    {
        return static_cast<uint4*>(ad.h) + (tile * steps(ad) + step) * (64 * PIECES);
    }
    // h of token m and rank r.
    static __device__ __forceinline__ float value(const Adapters& ad, int64_t m, int r)
    {
        const uint4* p = piece(ad, m / 16, r / STEP) + 16 * (r % STEP / E) + m % 16;
        float h = load1<AT>(p, r % E);
        if constexpr (PIECES > 1) h += load1<AT>(p + 64, r % E);
        if constexpr (AT == F16) h = __builtin_amdgcn_ldexpf(h, ad.up[m * steps(ad) + r / STEP]);
        return h;
    }
};

__device__ __forceinline__ int adapter_of(const Adapters& ad, int64_t row, int64_t M)
{
    const int c = row < M ? ad.id[row] : -1;
    return (unsigned)c < (unsigned)ad.count ? c : -1;
}

constexpr int AD_R = 256;                // largest rank

// Sixteen bytes of elements.
template <int AT>
__device__ __forceinline__ uint4 whole_chunk(const void* p, int64_t at)
{
    return ld16_any(static_cast<const char*>(p) + at * (AT == F32 ? 4 : 2));
}

// Elements r .. of a vector of n (16 bytes of them), zeros past its end.
template <int AT>
__device__ __forceinline__ uint4 chunk_of(const void* p, int64_t at, int r, int n)
{
    constexpr int E = AT == F32 ? 4 : 8;
    if (r + E <= n) return whole_chunk<AT>(p, at + r);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E - 1; ++i)
        if (r + i < n) {
            if constexpr (AT == F32) w[i] = static_cast<const uint32_t*>(p)[at + r + i];
            else w[i / 2] |= (uint32_t)static_cast<const uint16_t*>(p)[at + r + i] << (16 * (i & 1));
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// d += w x on the matrix cores: 16 x 16 x 32 of 16 bits, or 16 x 16 x 16 of 32
// (whose four steps take the operands' elements in turn).
template <int AT>
__device__ __forceinline__ v4f add_low(uint4 w, uint4 x, v4f d)
{
    if constexpr (AT == F32) {
        const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x4f32(as_f(a[i]), as_f(b[i]), d, 0, 0, 0);
        return d;
    } else if constexpr (AT == F16) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, w), __builtin_bit_cast(v8h, x), d, 0, 0,
                                                      0);
    } else {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w), __builtin_bit_cast(v8bf, x), d, 0,
                                                       0, 0);
    }
}

template <int AT>
__device__ __forceinline__ v4f add_low(v4i w, v4i x, v4f d)
{
    return add_low<AT>(__builtin_bit_cast(uint4, w), __builtin_bit_cast(uint4, x), d);
}

// ------------------------------------------------------------------------- h
// Writes E ranks of token m, from rank E g of the step on, in operand order; the four
// threads of a token's step stand side by side.
template <int AT>
__device__ __forceinline__ void put_low(const Adapters& ad, int64_t m, int step, int g, float v[Low<AT>::E])
{
    uint4* to = Low<AT>::piece(ad, m / 16, step) + 16 * g + m % 16;
    if constexpr (AT == F32) {
        *to = make_uint4(as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3]));
    } else {
        if constexpr (AT == F16) {
            float most = 0.0f;
#pragma unroll
            for (int k = 0; k < 8; ++k) {        // an infinity needs no room; what is beside it does
                const float size = __builtin_fabsf(v[k]);
                most = size < __builtin_inff() ? __builtin_fmaxf(most, size) : most;
            }
            most = __builtin_fmaxf(most, as_f(dpp<DPP_XOR1>(as_u(most))));
            most = __builtin_fmaxf(most, as_f(dpp<DPP_XOR2>(as_u(most))));
            const int up = most > 0.0f ? __builtin_amdgcn_frexp_expf(most) : 0;
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __builtin_amdgcn_ldexpf(v[k], -up);
            if (g == 0) ad.up[m * Low<AT>::steps(ad) + step] = up;
        }
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            hi[k] = narrow2<AT>(v[2 * k], v[2 * k + 1]);
            Raw8<AT> back = {};
            back.w[0].x = hi[k];
            float wide[8];
            widen8<AT>(back, wide);
            // an infinite or NaN hi is all there is
            lo[k] = narrow2<AT>(__builtin_fabsf(wide[0]) < __builtin_inff() ? v[2 * k] - wide[0] : 0.0f,
                                __builtin_fabsf(wide[1]) < __builtin_inff() ? v[2 * k + 1] - wide[1] : 0.0f);
        }
        to[0] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        to[64] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    }
}

// A wave's share of the sum of x a over vectors v0, v0 + step, ... of K elements.
template <int AT>
__device__ __forceinline__ float low_dot(const void* x, int64_t xr, const void* a, int64_t ar, int K, int v0, int step)
{
    constexpr int U = AT == F32 ? 4 : 8;
    float s = 0.0f;
    if (K < 8) {
        if (v0 < K) s = load1<AT>(x, xr + v0) * load1<AT>(a, ar + v0);
        return s;
    }
    const int nvec = (K + 7) / 8;
    for (; v0 < nvec; v0 += step * U) {
        Raw8<AT> p[U], q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = vec8(v0 + step * u, K).at;
            p[u] = load8_any<AT>(x, xr + at);
            q[u] = load8_any<AT>(a, ar + at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int lo = vec8(v0 + step * u, K).lo;
            float f[8], g[8];
            widen8<AT>(p[u], f);
            widen8<AT>(q[u], g);
#pragma unroll
            for (int i = 0; i < 8; ++i) s = i >= lo ? __builtin_fmaf(f[i], g[i], s) : s;
        }
    }
    return s;
}

// k_low_few: h of a few tokens in binary32; two waves per token and rank.  Bound by
// the latency of its few loads: 1 x 4096, rank 16 3.9 us, 48 x 11008 7.1.  Four waves per
// token and rank: no faster for few of them, the call of 128 x 4096 x 4096, rank 64, 45 us
// instead of 35.
template <int AT>
__global__ __launch_bounds__(512) void k_low_few(const void* __restrict__ x, int64_t ldx, int K, Adapters ad)
{
    __shared__ float half[4];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = blockIdx.x * 4 + (w & 3);
    const int64_t m = blockIdx.y;
    const int c = adapter_of(ad, m, m + 1);
    if (c < 0) return;                   // uniform
    float s = 0.0f;
    if (r < ad.R)
        s = wave_sum(low_dot<AT>(x, m * ldx, ad.a, ((int64_t)c * ad.R + r) * K, K, 64 * (w >> 2) + lane, 128));
    if (w >= 4 && lane == 0) half[w - 4] = s;
    __syncthreads();
    if (w < 4 && lane == 0 && r < ad.R)
        static_cast<float*>(ad.h)[m * ad.ldh + r] = (s + half[w]) * (ad.scale ? ad.scale[c] : 1.0f);
}

// k_low_tokens: the same in operand order, a workgroup per token, whose sixteen waves
// take the ranks in turn (the whole call 20-26 us for 128 to 512 tokens of rank 64 to 16,
// K = 4096, low_by_token).
template <int AT>
__global__ __launch_bounds__(1024) void k_low_tokens(const void* __restrict__ x, int64_t ldx, int K, Adapters ad)
{
    __shared__ float h[AD_R];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t m = blockIdx.x;
    const int c = adapter_of(ad, m, m + 1);
    if (c < 0) return;                   // uniform
    const float f = ad.scale ? ad.scale[c] : 1.0f;
    for (int r = w; r < ad.R; r += 16) {
        const float s = wave_sum(low_dot<AT>(x, m * ldx, ad.a, ((int64_t)c * ad.R + r) * K, K, lane, 64));
        if (lane == 0) h[r] = s * f;
    }
    __syncthreads();
    constexpr int E = Low<AT>::E;
    if (t < 4 * Low<AT>::steps(ad)) {
        float v[E];
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = E * t + k < ad.R ? h[E * t + k] : 0.0f;
        put_low<AT>(ad, m, t / 4, t & 3, v);
    }
}

// k_low_many: many tokens, on the matrix cores.  A workgroup takes 16 of them; its waves
// take the K axis in turn, 256 bytes of every row at a time (Quad), and their sums meet
// in LDS.  Workgroups of neighbouring tokens go to one XCD, whose L2 then holds their
// adapters alone.  Without operand order (ORDER) h is binary32, for the few-token product
// of a small output.  4096 x 4096, rank 64, f16 23 us, bound by what one workgroup per CU
// has in flight: 650 KB of x and a pass through every CU at 12 bytes per clock, 43 MB of
// them from HBM.  Sixteen waves for 64 ranks cost 14 us more, two groups in flight per
// wave 7 (their registers spill); K split over workgroups was no faster.  Every further
// adapter among the 16 tokens is another pass over K: with 48 adapters in turn 152 us, and
// the product beside them, whose 32 tokens take theirs in turn too, 451 instead of 80.
template <int AT, int RT, int NWV, bool ORDER>
__global__ __launch_bounds__(64 * NWV) void k_low_many(const void* __restrict__ x, int64_t ldx, int64_t M, int K,
                                                       Adapters ad)
{
    constexpr int ES = AT == F32 ? 4 : 2, STEP = Low<AT>::STEP, E = Low<AT>::E;
    constexpr int STEPS = 16 * RT > STEP ? 16 * RT / STEP : 1;               // steps of the ranks at a time
    __shared__ float sums[NWV][16][16 * RT + 4];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int64_t T = gridDim.x, xcd = blockIdx.x % 8, left = T % 8;
    const int64_t m0 = 16 * ((xcd < left ? xcd * (T / 8 + 1) : left + xcd * (T / 8)) + blockIdx.x / 8);
    const int xlast = M - 1 - m0 < 15 ? (int)(M - 1 - m0) : 15, groups = (int)((int64_t)K * ES / 256);
    const char* xrows = static_cast<const char*>(x) + m0 * ldx * ES;
    const int id = adapter_of(ad, m0 + l16, M);
    for (int r0 = 0; r0 < ad.R; r0 += 16 * RT) {
        int todo = (int)(__ballot(id >= 0) & 0xffff);
        while (todo) {                   // uniform
            const int c = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
            todo &= ~(int)__ballot(id == c);
            const float f = ad.scale ? ad.scale[c] : 1.0f;
            v4f acc[RT];
            const char* arows[RT];
            int alast[RT];
#pragma unroll
            for (int j = 0; j < RT; ++j) {
                const int r = r0 + 16 * j < ad.R ? r0 + 16 * j : ad.R - 1;
                acc[j] = v4f{};
                arows[j] = static_cast<const char*>(ad.a) + ((int64_t)c * ad.R + r) * K * ES;
                alast[j] = ad.R - 1 - r < 15 ? ad.R - 1 - r : 15;
            }
            const auto xa = quad_at(xlast, (uint64_t)(ldx * ES));
            for (int g = w; g < groups; g += NWV) {
                Quad xv, av[RT];
                quad_load(xv, xrows + g * 256, xa);
#pragma unroll
                for (int j = 0; j < RT; ++j)
                    quad_load(av[j], arows[j] + g * 256, quad_at(alast[j], (uint32_t)(K * ES)));
                __builtin_amdgcn_sched_barrier(0);       // every load is on its way
                change_places(xv);
#pragma unroll
                for (int j = 0; j < RT; ++j) {
                    change_places(av[j]);
#pragma unroll
                    for (int s = 0; s < 4; ++s) acc[j] = add_low<AT>(av[j].r[s], xv.r[s], acc[j]);
                }
            }
            if (groups % NWV == w)
                for (int k = groups * (256 / ES); k < K; k += STEP) {        // the rest of K
                    const uint4 xv = chunk_of<AT>(xrows, (int64_t)(l16 < xlast ? l16 : xlast) * ldx, k + g4 * E, K);
#pragma unroll
                    for (int j = 0; j < RT; ++j)
                        acc[j] = add_low<AT>(chunk_of<AT>(arows[j], (int64_t)(l16 < alast[j] ? l16 : alast[j]) * K,
                                                          k + g4 * E, K), xv, acc[j]);
                }
            // lane l holds ranks 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
            for (int j = 0; j < RT; ++j) *reinterpret_cast<v4f*>(&sums[w][l16][16 * j + 4 * g4]) = acc[j];
            __syncthreads();
            auto value = [&](int m, int r) {
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < NWV; ++i) v += sums[i][m][r];
                return v * f;
            };
            if constexpr (ORDER) {
                const int m = t / (4 * STEPS), g = t % (4 * STEPS);
                if (m < 16 && adapter_of(ad, m0 + m, M) == c && r0 + g / 4 * STEP < ad.R) {
                    float v[E];
#pragma unroll
                    for (int k = 0; k < E; ++k) {
                        const int r = E * g + k;
                        v[k] = r < 16 * RT && r0 + r < ad.R ? value(m, r) : 0.0f;
                    }
                    put_low<AT>(ad, m0 + m, r0 / STEP + g / 4, g & 3, v);
                }
            } else {
                for (int o = t; o < 256 * RT; o += 64 * NWV) {
                    const int m = o / (16 * RT), r = o % (16 * RT);
                    if (adapter_of(ad, m0 + m, M) == c && r0 + r < ad.R)
                        static_cast<float*>(ad.h)[(m0 + m) * ad.ldh + r0 + r] = value(m, r);
                }
            }
            __syncthreads();
        }
    }
}

// -------------------------------------------------- the product, a few tokens
// k_adapt_few: the product's kernel for a few tokens or small outputs (few_product);
// the thread that finishes an output adds its adapter's part, rank by rank, while the
// other waves' sums arrive.  1 x 11008 x 4096, rank 16 10.9 us (plain product 10.2), 48 x
// 4096 x 11008 16.0 (13.3), where every token's rows of b come from memory for it alone.
template <int AT>
__device__ __forceinline__ float low_output(const Adapters& ad, int64_t m, int c, int64_t n, int64_t N)
{
    const float* h = static_cast<const float*>(ad.h) + m * ad.ldh;
    const int64_t at = ((int64_t)c * N + n) * ad.R;
    float s = 0.0f;
#pragma unroll 2
    for (int r = 0; r + 8 <= ad.R; r += 8) {
        float b[8];
        widen8<AT>(load8_any<AT>(ad.b, at + r), b);
        const float4 p = *reinterpret_cast<const float4*>(h + r), q = *reinterpret_cast<const float4*>(h + r + 4);
        const float v[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) s = __builtin_fmaf(v[i], b[i], s);
    }
    for (int r = ad.R & ~7; r < ad.R; ++r) s = __builtin_fmaf(h[r], load1<AT>(ad.b, at + r), s);
    return s;
}

template <int YT, int MT, int CT, int NWV, int U>
__global__ __launch_bounds__(64 * NWV) void k_adapt_few(const int8_t* __restrict__ qx, const int8_t* __restrict__ qw,
                                                        int64_t K, Epi e, Adapters ad)
{
    constexpr int NT = 64 * NWV, COLS = 16 * CT, STEP = NT / COLS;           // rows of outputs per step of all threads
    constexpr int PER = 16 * MT > STEP ? 16 * MT / STEP : 1;                 // outputs per thread
    __shared__ int sums[NWV][MT * 16][COLS + 4];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * COLS, m0 = (int64_t)blockIdx.y * (16 * MT);

    const int64_t on = n0 + t % COLS;
    float osx[PER], ores[PER], low[PER], osw = 0.0f, ob = 0.0f;
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
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t m = m0 + t / COLS + i * STEP;
        const int c = mine[i] ? adapter_of(ad, m, e.M) : -1;
        low[i] = -0.0f;                  // added to any value, -0 among them, it changes nothing
        if (c >= 0) low[i] = ad.dt == F32 ? low_output<F32>(ad, m, c, on, e.N)
                             : ad.dt == BF16 ? low_output<BF16>(ad, m, c, on, e.N) : low_output<F16>(ad, m, c, on, e.N);
    }
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
        v += low[i];
        const int64_t at = (m0 + m) * e.N + on;
        if (e.z) store1<YT>(e.z, at, v);
        with_act(e.act, [&](auto a) { v = act1<decltype(a)::value>(v); });
        if (e.res) v += ores[i];
        store1<YT>(e.y, at, v);
    }
}

// --------------------------------------------------- the product, many tokens
// A wave finishes its part 32 tokens at a time, in its own part of LDS: the scaled sums
// and the bias go there, the matrix cores' adapter parts are added to them, an adapter
// and a step of ranks at a time, and from there the values leave in whole rows.  A step's
// h is loaded while the tokens before it leave; b's rows, whose loads cost the address
// unit a lane per clock, stay in registers, up to HELD steps of them, while the adapter
// does.  4096 x 4096 x 4096, rank 64, f16 86 us, plain product 60: with one tile of 256
// per CU nothing covers the epilogue, whose sums pass through LDS once for each step of
// ranks.  Adding to the sums in their own registers instead does not fit them.
template <int NM>
struct Ids {
    int of[(NM + 3) / 4];                // lane l: the adapter of token 64 i + l of a wave's part
};

template <int YT, int AT, int NM, int NN>
struct AdaptPart {
    using S = Stage<NM, NN>;
    static constexpr int STEP = Low<AT>::STEP, E = Low<AT>::E, PIECES = Low<AT>::PIECES;
    static constexpr int HELD = NN >= 4 && AT != F32 && YT != F32 ? 2 : 1;   // steps of b that fit in registers
    static constexpr int IDS = S::INTS, SW = IDS + 16 * NM, BIAS = SW + 16 * NN, INTS = BIAS + 16 * NN;   // in ints

    const Epi& e;
    const Adapters& ad;
    const int64_t m0, n0;
    int* const stage;
    const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
    // the present step: of which 32 tokens, whose, from which rank on; the tokens still to be looked at, and their adapters
    int half = 0, c = 0, r0 = 0, id[2] = {};
    uint32_t todo = 0;
    bool have = false;
    int whose = -1, from = -1;           // b: this adapter's HELD steps from this rank on
    uint4 b[HELD][NN], h[2][PIECES];
    int up[2];

    __device__ __forceinline__ uint32_t tokens(bool first, bool second) const
    {
        return (uint32_t)(__ballot(first) & 0xffff) | (uint32_t)(__ballot(second) & 0xffff) << 16;
    }
    __device__ __forceinline__ void enter()
    {
        id[0] = stage[IDS + 32 * half + l16];
        id[1] = stage[IDS + 32 * half + 16 + l16];
        todo = tokens(id[0] >= 0, id[1] >= 0);
    }
    // The next adapter (uniform).
    __device__ __forceinline__ void pop()
    {
        while (!todo) {
            if (++half >= NM / 2) {
                have = false;
                return;
            }
            enter();
        }
        const int lead = __builtin_ctz(todo);
        c = lead < 16 ? __builtin_amdgcn_readlane(id[0], lead) : __builtin_amdgcn_readlane(id[1], lead - 16);
        todo &= ~tokens(id[0] == c, id[1] == c);
        r0 = 0;
        have = true;
    }
    __device__ __forceinline__ void fetch()
    {
        if (!have) return;
        const int pair = r0 / (HELD * STEP) * (HELD * STEP);
        if (whose != c || from != pair) {        // uniform
            whose = c;
            from = pair;
#pragma unroll
            for (int s = 0; s < HELD; ++s) {
                const int r = pair + STEP * s + E * g4;
                if (pair + STEP * s < ad.R)
#pragma unroll
                    for (int j = 0; j < NN; ++j) {
                        const int64_t n = n0 + 16 * j + l16, at = ((int64_t)c * e.N + (n < e.N ? n : e.N - 1)) * ad.R;
                        // without a branch; only a rank that is no multiple of a chunk ends inside one
                        if (ad.R % E == 0) b[s][j] = whole_chunk<AT>(ad.b, at + (r < ad.R ? r : 0));    // uniform
                        else b[s][j] = chunk_of<AT>(ad.b, at, r, ad.R);
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int64_t row = m0 + 32 * half + 16 * t, tile = (row < e.M ? row : e.M - 1) / 16;
            const uint4* p = Low<AT>::piece(ad, tile, r0 / STEP) + lane;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) h[t][i] = p[64 * i];
            if constexpr (AT == F16) {
                const int64_t m = row + l16 < e.M ? row + l16 : e.M - 1;
                up[t] = ad.up[m * Low<AT>::steps(ad) + r0 / STEP];
            }
        }
    }
    __device__ __forceinline__ void add_step(uint4 (&w)[NN])
    {
        if (r0 + E * g4 >= ad.R)
#pragma unroll
            for (int j = 0; j < NN; ++j) w[j] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const bool mine = stage[IDS + 32 * half + 16 * t + l16] == c;
            uint4 x[PIECES];
#pragma unroll
            for (int i = 0; i < PIECES; ++i)
                x[i] = make_uint4(mine ? h[t][i].x : 0, mine ? h[t][i].y : 0, mine ? h[t][i].z : 0, mine ? h[t][i].w : 0);
#pragma unroll
            for (int j = 0; j < NN; ++j) {
                v4f d = v4f{};
#pragma unroll
                for (int i = 0; i < PIECES; ++i) d = add_low<AT>(w[j], x[i], d);
                if constexpr (AT == F16) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) d[k] = __builtin_amdgcn_ldexpf(d[k], up[t]);
                }
                v4f* z = reinterpret_cast<v4f*>(&stage[(16 * t + l16) * S::PITCH + 16 * j + 4 * g4]);
                if (mine) *z += d;
            }
            __builtin_amdgcn_sched_barrier(0);   // sixteen tokens at a time, in few registers
        }
    }
    // Adds the present step, and asks for the next.
    __device__ __forceinline__ void add()
    {
        if (r0 / STEP % HELD == 0) add_step(b[0]);       // uniform
        else add_step(b[HELD - 1]);
        r0 += STEP;
        if (r0 >= ad.R) pop();
        fetch();
    }

    // Eight columns of a row, some of them NaN: a sum over the ranks that is infinite with h
    // in one piece stands.
    __device__ __forceinline__ void infinite_sums(int row, int col, int n, int* at) const
    {
        constexpr float INF = __builtin_inff();
#pragma unroll 1
        for (int i = 0; i < n; ++i, ++col, ++at) {
            if (as_f((uint32_t)*at) == as_f((uint32_t)*at)) continue;
            float s = 0.0f;
#pragma unroll 1
            for (int r = 0; r < ad.R && s == s; ++r) {
                // from the start each time: a held address costs the common path its registers
                const int m = afresh(row), c = adapter_of(ad, m, e.M);
                if (c >= 0) s += Low<AT>::value(ad, m, r) * load1<AT>(ad.b, ((int64_t)c * e.N + afresh(col)) * ad.R + r);
            }
            if (__builtin_fabsf(s) == INF && __builtin_fabsf(e.sx[row] * e.sw[col]) < INF)
                *at = (int)as_u(s + load1_rt(e.bias, e.bias_dt, col, 0.0f));
        }
    }

    // Eight columns of a row on their way out.
    template <bool NTS>
    __device__ __forceinline__ void leave(const Cols8& cc, int64_t row, int* from) const
    {
        Raw8<YT> res = {};
        if (YT != F32 && e.res) res = residual8<YT>(e, cc, row);
        v4f s0 = *reinterpret_cast<const v4f*>(from), s1 = *reinterpret_cast<const v4f*>(from + 4);
        if constexpr (PIECES > 1) {
            bool nan = false;
#pragma unroll
            for (int i = 0; i < 4; ++i) nan |= __builtin_isunordered(s0[i], s1[i]);
            if (__builtin_expect(nan, 0)) {
                infinite_sums((int)row, (int)cc.col, cc.n, from);
                s0 = *reinterpret_cast<const v4f*>(from);
                s1 = *reinterpret_cast<const v4f*>(from + 4);
            }
        }
        float v[8] = {s0[0], s0[1], s0[2], s0[3], s1[0], s1[1], s1[2], s1[3]};
        const int64_t at = row * e.N + cc.col;
        if (e.z) store8_first<YT>(e.z, at, cc.n, v);
        act8(e.act, v);
        if (e.res) {
            if constexpr (YT == F32) res = residual8<YT>(e, cc, row);    // its registers are taken until here
            float w[8];
            widen8<YT>(res, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += w[i];
        }
        if (cc.n == 8) store8_any<YT, NTS>(e.y, at, v);
        else store8_first<YT>(e.y, at, cc.n, v);
    }

    template <bool NTS>
    __device__ __forceinline__ void finish(const v4i (&acc)[NM][NN], const Ids<NM>& ids)
    {
        if (m0 >= e.M) return;           // uniform
#pragma unroll
        for (int i = 0; i < NM; i += 4)
            if (16 * i + lane < 16 * NM) stage[IDS + 16 * i + lane] = ids.of[i / 4];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        enter();
        pop();
        fetch();
        stage_scales<NM, NN>(e, m0, stage);
        if (lane < 16 * NN) {
            const int64_t n = n0 + lane < e.N ? n0 + lane : e.N - 1;
            stage[SW + lane] = (int)as_u(e.sw[n]);
            stage[BIAS + lane] = (int)as_u(load1_rt(e.bias, e.bias_dt, n, 0.0f));
        }
        const float* sx = reinterpret_cast<const float*>(stage + 32 * S::PITCH);
        Cols8 cc = {};
        cc.col = n0 + 8 * (lane % S::LPR);
        cc.n = e.N - cc.col >= 8 ? 8 : e.N - cc.col > 0 ? (int)(e.N - cc.col) : 0;
#pragma unroll
        for (int p = 0; p < NM / 2; ++p) {
            const int64_t mh = m0 + 32 * p;
            if (mh >= e.M) return;       // uniform
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const float f = sx[32 * p + 16 * t + l16];
#pragma unroll
                for (int j = 0; j < NN; ++j) {
                    const v4f sw = *reinterpret_cast<const v4f*>(stage + SW + 16 * j + 4 * g4);
                    v4f z;
#pragma unroll
                    for (int k = 0; k < 4; ++k) z[k] = (float)acc[2 * p + t][j][k] * f * sw[k];
                    if (e.bias) {
                        const v4f bias = *reinterpret_cast<const v4f*>(stage + BIAS + 16 * j + 4 * g4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) z[k] += bias[k];
                    }
                    *reinterpret_cast<v4f*>(&stage[(16 * t + l16) * S::PITCH + 16 * j + 4 * g4]) = z;
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 1
            while (have && half == p) add();
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            const int rows = cc.n == 0 ? 0 : e.M - mh < 32 ? (int)(e.M - mh) : 32;
#pragma unroll 1
            for (int r = lane / S::LPR; r < rows; r += S::RPI)
                leave<NTS>(cc, mh + r, stage + r * S::PITCH + 8 * (lane % S::LPR));
        }
    }
};

template <int YT>
struct AdaptTile : Epi {
    static constexpr bool GATED = false;
    Adapters ad;
    static __device__ __forceinline__ const int8_t* second_weight(const int8_t* first) { return first; }
    template <int TILE, int WM, int WN>
    static constexpr int staging()
    {
        return 4 * WM * WN * AdaptPart<YT, F32, TILE / WM / 16, TILE / WN / 16>::INTS;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ Ids<TILE / WM / 16> early(const AdaptTile& e, int64_t m0)
    {
        Ids<TILE / WM / 16> ids;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
#pragma unroll
        for (int i = 0; i < (TILE / WM / 16 + 3) / 4; ++i)
            ids.of[i] = adapter_of(e.ad, m0 + TILE / WM * (w / WN) + 64 * i + (threadIdx.x & 63), e.M);
        return ids;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ void finish(const AdaptTile& e, int64_t m0, int64_t n0,
                                                  const v4i (&acc)[TILE / WM / 16][TILE / WN / 16], uint8_t* lds,
                                                  const Ids<TILE / WM / 16>& ids)
    {
        constexpr int NM = TILE / WM / 16, NN = TILE / WN / 16;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int64_t m = m0 + TILE / WM * (w / WN), n = n0 + TILE / WN * (w % WN);
        int* stage = reinterpret_cast<int*>(lds) + w * AdaptPart<YT, F32, NM, NN>::INTS;
        constexpr bool NTS = TILE == 256;
        if (e.ad.dt == F32) AdaptPart<YT, F32, NM, NN>{e, e.ad, m, n, stage}.template finish<NTS>(acc, ids);
        else if (e.ad.dt == BF16) AdaptPart<YT, BF16, NM, NN>{e, e.ad, m, n, stage}.template finish<NTS>(acc, ids);
        else AdaptPart<YT, F16, NM, NN>{e, e.ad, m, n, stage}.template finish<NTS>(acc, ids);
    }
};

// ---------------------------------------------------------------- launches
// Up to LOW_FEW tokens times ranks, or twice as many where the tokens' tiles of 16 are too
// few for the chip, every token reads its adapter's rows for itself, which does not mind whose
// they are; beyond, the matrix cores, which take the adapters of a tile in turn.  The call
// with 128 columns, tokens of eight adapters in turn | in runs, by token / by tile, us:
//   48 x 11008, rank 16  16 / 70 | 16 / 38      512 x 4096, rank 16  20 / 33 | 20 / 16
//   128 x 4096, rank 64  20 / 76 | 20 / 18     1024 x 4096, rank 16  32 / 41 | 32 / 16
//   200 x 4096, rank 64  26 / 74 | 26 / 26      512 x 4096, rank 64  52 / 74 | 52 / 19
// (the last goes by tile, for batches whose tokens of one adapter stand together).
constexpr int64_t LOW_FEW = 8192;
inline bool low_by_token(int64_t M, int64_t rank) { return M * rank <= (M <= 256 ? 2 : 1) * LOW_FEW; }

// Whether the few-token kernel takes the product: by the product's rule, and for so few
// tokens times ranks also with two pieces of 32 x 32 per CU, since a tile takes the
// adapters of its tokens in turn.  Few tokens / tiles, us, rank 16, each token with an
// adapter of its own | all with one:
//   100 x 4096 x 11008   36 / 66 | 33 / 35     128 x 4096 x 4096   21 / 45 | 19.5 / 18
//   64 x 11008 x 4096    30 / 51 | 26 / 19     200 x 4096 x 4096   35 / 47 | 32.5 / 18
// (the last two go to the tiles: what tokens with an adapter each lose there, tokens that
// share one gain).
inline bool adapt_few(int64_t M, int64_t N, int64_t rank)
{
    return few_tokens(M, N) || (M * rank <= LOW_FEW && cdiv(M, 32) * cdiv(N, 32) <= 512);
}

template <int AT>
static void low_launch(const void* x, int64_t ldx, int64_t M, int64_t K, bool few, const Adapters& ad, hipStream_t st)
{
    if (low_by_token(M, ad.R)) {
        if (few)
            hipLaunchKernelGGL((k_low_few<AT>), dim3((unsigned)cdiv(ad.R, 4), (unsigned)M), dim3(512), 0, st, x, ldx,
                               (int)K, ad);
        else hipLaunchKernelGGL((k_low_tokens<AT>), dim3((unsigned)M), dim3(1024), 0, st, x, ldx, (int)K, ad);
        return;
    }
    const dim3 grid((unsigned)cdiv(M, 16));
#define TQ_LOW(RT, NWV)                                                                                             \
    do {                                                                                                            \
        if (few)                                                                                                    \
            hipLaunchKernelGGL((k_low_many<AT, RT, NWV, false>), grid, dim3(64 * NWV), 0, st, x, ldx, M, (int)K, ad);   \
        else                                                                                                        \
            hipLaunchKernelGGL((k_low_many<AT, RT, NWV, true>), grid, dim3(64 * NWV), 0, st, x, ldx, M, (int)K, ad);    \
    } while (0)
    if (ad.R <= 16) TQ_LOW(1, 16);
    else if (ad.R <= 32) TQ_LOW(2, 8);
    else TQ_LOW(4, 8);
#undef TQ_LOW
}

// The kernel of a product, by the rule of the product without adapters
// (product_launch).
template <int YT>
static void adapt_launch(const int8_t* qx, const int8_t* qw, int64_t K, const Epi& e, const Adapters& ad,
                         hipStream_t st)
{
    const bool rows16 = K >= ET && K % 16 == 0 && aligned16(qx) && aligned16(qw);
#define TQ_FEW(MT, CT, NWV, U)                                                                                  \
    do {                                                                                                        \
        const dim3 grid((unsigned)cdiv(e.N, 16 * CT), (unsigned)cdiv(e.M, 16 * MT));                            \
        hipLaunchKernelGGL((k_adapt_few<YT, MT, CT, NWV, U>), grid, dim3(64 * NWV), 0, st, qx, qw, K, e, ad);   \
        return;                                                                                                 \
    } while (0)
    if (adapt_few(e.M, e.N, ad.R)) {
        if (e.M <= 16) TQ_FEW(1, 1, 8, 2);
        if (few_columns(e.M, e.N)) TQ_FEW(2, 1, 8, 1);
        TQ_FEW(2, 2, 8, 1);
    }
#undef TQ_FEW
    const AdaptTile<YT> tile = {e, ad};
    if (rows16) {
#define TQ_RING(TILE, RING, WM, WN, WGS)                                                                        \
    do {                                                                                                        \
        const int64_t nt = cdiv(e.N, TILE), mt = cdiv(e.M, TILE);                                               \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                               \
        hipLaunchKernelGGL((k_epi_ring<AdaptTile<YT>, TILE, RING, WM, WN, WGS>), dim3((unsigned)(nt * mt)),     \
                           dim3(64 * WM * WN), 0, st, qx, qw, K, nt, mt, slab, tile);                           \
    } while (0)
        const int64_t t128 = cdiv(e.M, 128) * cdiv(e.N, 128);
        if (cdiv(e.M, 256) * cdiv(e.N, 256) >= 256) TQ_RING(256, 5, 2, 4, 1);
        else if (t128 > 256) TQ_RING(128, 5, 2, 4, 2);
        else if (cdiv(e.M, 64) * cdiv(e.N, 64) > 512) TQ_RING(128, 9, 2, 4, 1);
        else TQ_RING(64, 9, 2, 2, 2);
#undef TQ_RING
        return;
    }
#define TQ_TILE(TILE, WM, WN, D, WGS)                                                                           \
    do {                                                                                                        \
        const int64_t nt = cdiv(e.N, TILE), mt = cdiv(e.M, TILE);                                               \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                               \
        hipLaunchKernelGGL((k_epi_tile<AdaptTile<YT>, TILE, WM, WN, D, WGS>), dim3((unsigned)(nt * mt)),        \
                           dim3(64 * WM * WN), 0, st, qx, qw, K, nt, mt, slab, tile);                           \
    } while (0)
    if constexpr (YT != F32)             // with binary32 outputs the 256 tile's registers do not suffice
        if (cdiv(e.M, 256) * cdiv(e.N, 256) > 160) {
            TQ_TILE(256, 2, 4, 2, 1);
            return;
        }
    if (cdiv(e.M, 64) * cdiv(e.N, 64) > 512) TQ_TILE(128, 2, 4, 2, 2);
    else TQ_TILE(64, 2, 2, 4, 2);
#undef TQ_TILE
}

static bool natural(const void* p, int dt) { return ((uintptr_t)p & (uintptr_t)(ftype_size(dt) - 1)) == 0; }
static bool valid_act(int a) { return a >= TQ_ACT_NONE && a <= TQ_ACT_GELU_TANH; }
// Bytes of h: whole tiles of 16 tokens and steps of 32 ranks in 4 bytes each, which also
// holds binary32 rows of a multiple of 8 ranks, and an exponent per token and step behind.
inline int64_t low_ld(int64_t rank) { return cdiv(rank, 8) * 8; }
inline size_t low_bytes(int64_t M, int64_t rank) { return (size_t)(cdiv(M, 16) * 16) * (size_t)(cdiv(rank, 32) * 32) * 4; }

}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_w8a8_linear_adapters_workspace_bytes(int64_t M, int64_t rank)
{
    return M > 0 && rank > 0 ? low_bytes(M, rank) + (size_t)M * (size_t)cdiv(rank, 32) * sizeof(int) : 0;
}

tq_status tq_w8a8_linear_adapters(const void* x, int x_dtype, int64_t x_row_stride, const int8_t* qx, const float* sx,
                                  const int8_t* qw, const float* sw, int64_t M, int64_t N, int64_t K,
                                  const int32_t* adapter, int64_t adapters, int64_t rank, const void* a, const void* b,
                                  const float* scale, const void* bias, int bias_dtype, int act, const void* residual,
                                  int64_t residual_row_stride, void* y, void* preact, int y_dtype, void* workspace,
                                  size_t workspace_bytes, void* stream)
{
    if (!valid_ftype(x_dtype) || adapters < 0 || rank < 1 || M < 0 || N < 0 || K < 0) return TQ_ERR_INVALID;
    if (adapters == 0 || K == 0 || M == 0 || N == 0)
        return tq_w8a8_linear_epilogue(qx, sx, qw, sw, M, N, K, bias, bias_dtype, act, residual, residual_row_stride, y,
                                       preact, y_dtype, stream);
    if (!valid_ftype(y_dtype) || !valid_act(act) || (bias && !valid_ftype(bias_dtype))) return TQ_ERR_INVALID;
    if (!x || x_row_stride < K || !adapter || !a || !b || !y || !sx || !sw || !qx || !qw ||
        (residual && residual_row_stride < N))
        return TQ_ERR_INVALID;
    if (K > 131071 || cdiv(M, ET) > 65535 || cdiv(N, 16) > 0x7fffff || cdiv(M, 256) * cdiv(N, 256) > 0x7fffff ||
        rank > AD_R || adapters > 0x7fffffff)
        return TQ_ERR_UNSUPPORTED;
    if (!natural(x, x_dtype) || !natural(a, x_dtype) || !natural(b, x_dtype) || !natural(scale, TQ_F32) ||
        !natural(adapter, TQ_F32) || !natural(sx, TQ_F32) || !natural(sw, TQ_F32) ||
        (bias && !natural(bias, bias_dtype)) || !natural(residual, y_dtype) || !natural(y, y_dtype) ||
        !natural(preact, y_dtype))
        return TQ_ERR_ALIGN;
    if (!workspace || workspace_bytes < tq_w8a8_linear_adapters_workspace_bytes(M, rank)) return TQ_ERR_INVALID;
    if (!aligned16(workspace)) return TQ_ERR_ALIGN;
    const Epi e = {sx, sw, bias, bias_dtype, act, residual, residual_row_stride, y, preact, M, N};
    const Adapters ad = {adapter, a, b, scale, workspace, reinterpret_cast<int*>(static_cast<char*>(workspace) +
                         low_bytes(M, rank)), (int)adapters, (int)rank, (int)low_ld(rank), x_dtype};
    hipStream_t st = as_stream(stream);
    const bool few = adapt_few(M, N, rank);
    TQ_LLM_FT_SWITCH(x_dtype, low_launch<FTV>(x, x_row_stride, M, K, few, ad, st));
    TQ_LLM_FT_SWITCH(y_dtype, adapt_launch<FTV>(qx, qw, K, e, ad, st));
    return launch_status();
}

}  // extern "C"
