// tq_adapters.hip -- the W8A8 product beside low-rank adapters of many requests:
// token m has the adapter c = adapter[m] of its request, or none.
//
//   h[m][r] = scale[c] sum_k x[m][k] a[c][r][k]
//   z[m][n] = ((float)sum_k qx[m][k] qw[n][k]) sx[m] sw[n] + sum_r h[m][r] b[c][n][r] + bias[n]
//   y = act(z) + residual
//
// x and the adapters are of one type, their products summed in binary32; h stays
// in binary32 between its kernel and the product's, which takes it in its
// epilogue: as a scalar loop per output for a few tokens, on the matrix cores for
// tiles.  There a 16-bit operand of h would lose what h holds beyond 8 or 11 bits,
// so it goes in twice: h = hi + lo in the adapters' type, 16 or more bits in all
// (f16, whose range is short, takes h relative to a power of two near the row's
// largest value).
//
// The tokens of one sixteen-row operand may have several adapters.  Each takes its
// turn, the other tokens' h cleared, and only its own tokens take the result, so
// that what another adapter holds (infinities, NaN) does not reach them.
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
    float* h;                            // [M, ldh]
    int count, R, ldh, dt;
};

__device__ __forceinline__ int adapter_of(const Adapters& ad, int64_t row, int64_t M)
{
    const int c = row < M ? ad.id[row] : -1;
    return (unsigned)c < (unsigned)ad.count ? c : -1;
}

constexpr int AD_R = 256;                // largest rank

// Elements r .. of a vector of n (16 bytes of them), zeros past its end.
template <int AT>
__device__ __forceinline__ uint4 chunk_of(const void* p, int64_t at, int r, int n)
{
    constexpr int E = AT == F32 ? 4 : 8;
    if (r + E <= n) return AT == F32 ? ld16_any(static_cast<const float*>(p) + at + r)
                                     : ld16_any(static_cast<const uint16_t*>(p) + at + r);
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

// ------------------------------------------------------------- h, a few tokens
// k_low_few: a wave per token and rank.
template <int AT>
__global__ __launch_bounds__(256) void k_low_few(const void* __restrict__ x, int64_t ldx, int K, Adapters ad)
{
    constexpr int U = 4;
    const int lane = threadIdx.x & 63, r = blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t m = blockIdx.y;
    const int c = adapter_of(ad, m, m + 1);
    if (r >= ad.R || c < 0) return;
    const int64_t xr = m * ldx, ar = ((int64_t)c * ad.R + r) * K;
    float s = 0.0f;
    if (K < 8) {
        if (lane < K) s = load1<AT>(x, xr + lane) * load1<AT>(ad.a, ar + lane);
    } else {
        const int nvec = (K + 7) / 8;
        for (int v0 = lane; v0 < nvec; v0 += 64 * U) {
            Raw8<AT> p[U], q[U];
            Vec8 at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                at[u] = vec8(v0 + 64 * u, K);
                p[u] = load8_any<AT>(x, xr + at[u].at);
                q[u] = load8_any<AT>(ad.a, ar + at[u].at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[8], g[8];
                widen8<AT>(p[u], f);
                widen8<AT>(q[u], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) s = i >= at[u].lo ? __builtin_fmaf(f[i], g[i], s) : s;
            }
        }
    }
    s = wave_sum(s);
    if (lane == 0) ad.h[m * ad.ldh + r] = ad.scale ? s * ad.scale[c] : s;
}

// ------------------------------------------------------------ h, many tokens
// k_low_many: a workgroup per 16 tokens, on the matrix cores; its waves take the K
// axis in turn, two steps' 128 bytes of every row at a time, and their sums meet in LDS.
template <int AT, int RT, int NWV>
__global__ __launch_bounds__(64 * NWV) void k_low_many(const void* __restrict__ x, int64_t ldx, int64_t M, int K,
                                                       Adapters ad)
{
    constexpr int STEP = AT == F32 ? 16 : 32, E = STEP / 4, U = 4;    // elements per step and per lane; steps at a time
    __shared__ float sums[NWV][16][16 * RT + 4];
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int64_t m0 = (int64_t)blockIdx.x * 16;
    const int64_t row = m0 + l16 < M ? m0 + l16 : M - 1;
    const int id = adapter_of(ad, m0 + l16, M);
    const int steps = (K + STEP - 1) / STEP;
    for (int r0 = 0; r0 < ad.R; r0 += 16 * RT) {
        int64_t todo = __ballot(id >= 0) & 0xffff;
        while (todo) {                   // uniform
            const int c = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
            todo &= ~__ballot(id == c);
            v4f acc[RT];
#pragma unroll
            for (int j = 0; j < RT; ++j) acc[j] = v4f{};
            for (int s0 = w * U; s0 < steps; s0 += NWV * U) {
                uint4 xv[U], av[U][RT];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int k = (s0 + u) * STEP + g4 * E;
                    xv[u] = chunk_of<AT>(x, row * ldx, k, K);
#pragma unroll
                    for (int j = 0; j < RT; ++j) {
                        const int r = r0 + 16 * j + l16;
                        av[u][j] = chunk_of<AT>(ad.a, ((int64_t)c * ad.R + (r < ad.R ? r : ad.R - 1)) * K, k, K);
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[j] = add_low<AT>(av[u][j], xv[u], acc[j]);
            }
            // lane l holds ranks 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
            for (int j = 0; j < RT; ++j) *reinterpret_cast<v4f*>(&sums[w][l16][16 * j + 4 * g4]) = acc[j];
            __syncthreads();
            const float f = ad.scale ? ad.scale[c] : 1.0f;
            for (int o = t; o < 256 * RT; o += 64 * NWV) {
                const int m = o / (16 * RT), r = o % (16 * RT);
                if (adapter_of(ad, m0 + m, M) != c || r0 + r >= ad.R) continue;
                float v = 0.0f;
#pragma unroll
                for (int i = 0; i < NWV; ++i) v += sums[i][m][r];
                ad.h[(m0 + m) * ad.ldh + r0 + r] = v * f;
            }
            __syncthreads();
        }
    }
}

// -------------------------------------------------- the product, a few tokens
// k_adapt_few: the product's kernel for a few tokens or small outputs (few_product);
// the thread that finishes an output adds its adapter's part, rank by rank.
template <int AT>
__device__ __forceinline__ float low_output(const Adapters& ad, int64_t m, int c, int64_t n, int64_t N)
{
    const float* h = ad.h + m * ad.ldh;
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
    few_product<MT, CT, NWV, U>(pw, px, K, acc);
    // lane l holds columns 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < CT; ++j) *reinterpret_cast<v4i*>(&sums[w][16 * i + l16][16 * j + 4 * g4]) = acc[i][j];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int64_t m = m0 + t / COLS + i * STEP;
        const int c = mine[i] ? adapter_of(ad, m, e.M) : -1;
        low[i] = 0.0f;
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
        float v = (float)s * osx[i] * osw + low[i];
        if (e.bias) v += ob;
        const int64_t at = (m0 + m) * e.N + on;
        if (e.z) store1<YT>(e.z, at, v);
        with_act(e.act, [&](auto a) { v = act1<decltype(a)::value>(v); });
        if (e.res) v += ores[i];
        store1<YT>(e.y, at, v);
    }
}

// --------------------------------------------------- the product, many tokens
// A staged half of a wave's sums, 32 tokens of 16 NN columns: scaled where it lies,
// and their adapters' parts added, an adapter and a step of ranks at a time.
struct AdaptDelta {
    static constexpr bool ADDS = true;
    Adapters ad;

    // `at` is the lane's first value of a tile of 16 tokens and 16 columns, `tile` apart to the next 16 tokens.
    template <int AT, int NN>
    __device__ __forceinline__ void add(const Epi& e, const int (&id)[2], int64_t row0, int64_t n0, float* at,
                                        int tile) const
    {
        constexpr int STEP = AT == F32 ? 16 : 32, E = STEP / 4;
        const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
        // f16: h relative to a power of two near its row's largest value
        int up[2] = {0, 0};
        if constexpr (AT == F16) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                float most = 0.0f;
                if (id[t] >= 0)
                    for (int r = g4; r < ad.R; r += 4)
                        most = __builtin_fmaxf(most, __builtin_fabsf(ad.h[(row0 + 16 * t) * ad.ldh + r]));
                most = __builtin_fmaxf(most, lane_get(most, 16));
                most = __builtin_fmaxf(most, lane_get(most, 32));
                up[t] = most > 0.0f && most < __builtin_inff() ? __builtin_amdgcn_frexp_expf(most) : 0;
            }
        }
        uint32_t todo = (uint32_t)(__ballot(id[0] >= 0) & 0xffff) | (uint32_t)(__ballot(id[1] >= 0) & 0xffff) << 16;
        while (todo) {                   // uniform
            const int lead = __builtin_ctz(todo);
            const int c = lead < 16 ? __builtin_amdgcn_readlane(id[0], lead)
                                    : __builtin_amdgcn_readlane(id[1], lead - 16);
            todo &= ~((uint32_t)(__ballot(id[0] == c) & 0xffff) | (uint32_t)(__ballot(id[1] == c) & 0xffff) << 16);
#pragma unroll 1
            for (int r0 = 0; r0 < ad.R; r0 += STEP) {
                const int r = r0 + E * g4;
                uint4 b[NN];
#pragma unroll
                for (int j = 0; j < NN; ++j) {
                    const int64_t n = n0 + 16 * j + l16;
                    b[j] = chunk_of<AT>(ad.b, ((int64_t)c * e.N + (n < e.N ? n : e.N - 1)) * ad.R, r, ad.R);
                }
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    const bool mine = id[t] == c;
                    float h[E];
#pragma unroll
                    for (int i = 0; i < E; i += 4) {
                        float4 v = make_float4(0, 0, 0, 0);
                        if (mine && r + i < ad.R)
                            v = *reinterpret_cast<const float4*>(ad.h + (row0 + 16 * t) * ad.ldh + r + i);
                        h[i] = v.x;
                        h[i + 1] = r + i + 1 < ad.R ? v.y : 0.0f;
                        h[i + 2] = r + i + 2 < ad.R ? v.z : 0.0f;
                        h[i + 3] = r + i + 3 < ad.R ? v.w : 0.0f;
                    }
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (AT == F32) {
                            hi[i] = as_u(h[i]);
                        } else {
                            float p = h[2 * i], q = h[2 * i + 1];
                            if constexpr (AT == F16) {
                                p = __builtin_amdgcn_ldexpf(p, -up[t]);
                                q = __builtin_amdgcn_ldexpf(q, -up[t]);
                            }
                            hi[i] = narrow2<AT>(p, q);
                            Raw8<AT> back = {};
                            back.w[0].x = hi[i];
                            float wide[8];
                            widen8<AT>(back, wide);
                            // an infinite or NaN hi is all there is
                            lo[i] = narrow2<AT>(__builtin_fabsf(wide[0]) < __builtin_inff() ? p - wide[0] : 0.0f,
                                                __builtin_fabsf(wide[1]) < __builtin_inff() ? q - wide[1] : 0.0f);
                        }
                    }
#pragma unroll
                    for (int j = 0; j < NN; ++j) {
                        v4f d = add_low<AT>(b[j], make_uint4(hi[0], hi[1], hi[2], hi[3]), v4f{});
                        if constexpr (AT != F32) d = add_low<AT>(b[j], make_uint4(lo[0], lo[1], lo[2], lo[3]), d);
                        v4f* z = reinterpret_cast<v4f*>(at + t * tile + 16 * j);
                        if constexpr (AT == F16) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_ldexpf(d[i], up[t]);
                        }
                        if (mine) *z += d;
                    }
                }
            }
        }
    }

    template <int NM, int NN>
    __device__ __forceinline__ void apply(const Epi& e, int64_t m0, int64_t n0, int half, int* stage) const
    {
        using S = Stage<NM, NN>;
        const int lane = threadIdx.x & 63, l16 = lane & 15, g4 = lane >> 4;
        const int64_t row0 = m0 + 32 * half + l16;
        const int id[2] = {adapter_of(ad, row0, e.M), adapter_of(ad, row0 + 16, e.M)};
        int* at = stage + l16 * S::PITCH + 4 * g4;
        const float* sx = reinterpret_cast<const float*>(stage + 32 * S::PITCH) + 32 * half + l16;
#pragma unroll
        for (int j = 0; j < NN; ++j) {
            const int64_t n = n0 + 16 * j + 4 * g4;
            float sw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) sw[i] = n + i < e.N ? e.sw[n + i] : 0.0f;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const v4i s = *reinterpret_cast<const v4i*>(at + 16 * t * S::PITCH + 16 * j);
                const float f = sx[16 * t];
                v4i z;
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] = (int)as_u((float)s[i] * f * sw[i]);
                *reinterpret_cast<v4i*>(at + 16 * t * S::PITCH + 16 * j) = z;
            }
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        float* zf = reinterpret_cast<float*>(at);
        if (ad.dt == F32) add<F32, NN>(e, id, row0, n0, zf, 16 * S::PITCH);
        else if (ad.dt == BF16) add<BF16, NN>(e, id, row0, n0, zf, 16 * S::PITCH);
        else add<F16, NN>(e, id, row0, n0, zf, 16 * S::PITCH);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
};

template <int YT>
struct AdaptTile : Epi {
    static constexpr bool GATED = false;
    AdaptDelta delta;
    static __device__ __forceinline__ const int8_t* second_weight(const int8_t* first) { return first; }
    template <int TILE, int WM, int WN>
    static constexpr int staging()
    {
        return 4 * WM * WN * Stage<TILE / WM / 16, TILE / WN / 16>::INTS;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ void finish(const AdaptTile& e, int64_t m0, int64_t n0,
                                                  const v4i (&acc)[TILE / WM / 16][TILE / WN / 16], uint8_t* lds)
    {
        constexpr int NM = TILE / WM / 16, NN = TILE / WN / 16;
        const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        finish_part<YT, NM, NN, TILE == 256>(e, m0 + TILE / WM * (w / WN), n0 + TILE / WN * (w % WN), acc,
                                             reinterpret_cast<int*>(lds) + w * Stage<NM, NN>::INTS, e.delta);
    }
};

// ---------------------------------------------------------------- launches
// A wave per token and rank reads an adapter's rows anew for every token; the matrix
// cores take sixteen tokens at once, but in M / 16 workgroups only.
constexpr int64_t LOW_FEW = 128;

template <int AT>
static void low_launch(const void* x, int64_t ldx, int64_t M, int64_t K, const Adapters& ad, hipStream_t st)
{
    if (M <= LOW_FEW) {
        hipLaunchKernelGGL((k_low_few<AT>), dim3((unsigned)cdiv(ad.R, 4), (unsigned)M), dim3(256), 0, st, x, ldx, (int)K,
                           ad);
        return;
    }
    const dim3 grid((unsigned)cdiv(M, 16));
    if (ad.R <= 16) hipLaunchKernelGGL((k_low_many<AT, 1, 16>), grid, dim3(1024), 0, st, x, ldx, M, (int)K, ad);
    else if (ad.R <= 32) hipLaunchKernelGGL((k_low_many<AT, 2, 16>), grid, dim3(1024), 0, st, x, ldx, M, (int)K, ad);
    else hipLaunchKernelGGL((k_low_many<AT, 4, 8>), grid, dim3(512), 0, st, x, ldx, M, (int)K, ad);
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
    if (e.M <= 16) TQ_FEW(1, 1, 8, 4);
    if ((e.M <= 32 && (e.N <= 6144 || !rows16)) || (rows16 && cdiv(e.M, 32) * cdiv(e.N, 16) <= 256))
        TQ_FEW(2, 1, 8, 2);
    if (rows16 && cdiv(e.M, 32) * cdiv(e.N, 32) <= 256) TQ_FEW(2, 2, 8, 2);
#undef TQ_FEW
    const AdaptTile<YT> tile = {e, {ad}};
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
    if (cdiv(e.M, 256) * cdiv(e.N, 256) > 160) TQ_TILE(256, 2, 4, 2, 1);
    else if (cdiv(e.M, 64) * cdiv(e.N, 64) > 512) TQ_TILE(128, 2, 4, 2, 2);
    else TQ_TILE(64, 2, 2, 4, 2);
#undef TQ_TILE
}

static bool natural(const void* p, int dt) { return ((uintptr_t)p & (uintptr_t)(ftype_size(dt) - 1)) == 0; }
static bool valid_act(int a) { return a >= TQ_ACT_NONE && a <= TQ_ACT_GELU_TANH; }
inline int64_t low_ld(int64_t rank) { return cdiv(rank, 8) * 8; }

}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_w8a8_linear_adapters_workspace_bytes(int64_t M, int64_t rank)
{
    return M > 0 && rank > 0 ? (size_t)M * (size_t)low_ld(rank) * sizeof(float) : 0;
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
    const Adapters ad = {adapter, a, b, scale, static_cast<float*>(workspace), (int)adapters, (int)rank,
                         (int)low_ld(rank), x_dtype};
    hipStream_t st = as_stream(stream);
    TQ_LLM_FT_SWITCH(x_dtype, low_launch<FTV>(x, x_row_stride, M, K, ad, st));
    TQ_LLM_FT_SWITCH(y_dtype, adapt_launch<FTV>(qx, qw, K, e, ad, st));
    return launch_status();
}

}  // extern "C"
