// tq_gated.hip -- a gated block on codes: both W8A8 projections, the activation
// and the product in one kernel, and the gate by itself, forwards and back.
//
//   g[m][f] = ((float)sum_k qx[m][k] qg[f][k]) sx[m] sg[f] + bg[f],  u likewise
//   y = act(g) u;   backward: dg = dy u act'(g), du = dy act(g)
//
// The integer sums are exact on the matrix cores; g, u and their product are
// binary32, and y (and z = [g | u], where it is asked for) is rounded once.
#include "tq_product.h"

namespace tq {

struct Gate {
    const float* sx;
    const float* sw[2];
    const void* bias[2];                 // gate, up; each may be null
    int bias_dt, act;
    void* y;
    void* z;                             // [M, 2 F], or null
    int64_t M, N;                        // tokens, features
};

// ------------------------------------------------------------- a few tokens
// k_gate_few: a workgroup of NWV waves owns 16 features of 16 MT tokens, the 16
// rows of either weight side by side (few_product), so that the thread that
// finishes an output finds both sums in LDS.  Bound by the weights, which are read
// once: 1 x 11008 x 4096 17.2 us (90 MB of codes, 5.2 TB/s).
template <int YT, int MT, int NWV, int U>
__global__ __launch_bounds__(64 * NWV) void k_gate_few(const int8_t* __restrict__ qx, const int8_t* __restrict__ wg,
                                                       const int8_t* __restrict__ wu, int64_t K, Gate e)
{
    constexpr int NT = 64 * NWV, STEP = NT / 16, PER = 16 * MT > STEP ? 16 * MT / STEP : 1;
    __shared__ int sums[NWV][MT * 16][36];   // rows 4 apart beyond their sums, which spreads them over the banks
    const int t = threadIdx.x, lane = t & 63, w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int l16 = lane & 15, g4 = lane >> 4;
    const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * MT);

    // thread t finishes feature t % 16 of tokens t / 16, + STEP, ...: what that takes is asked for first
    const int64_t on = n0 + t % 16;
    float osx[PER], osw[2] = {0.0f, 0.0f}, ob[2] = {0.0f, 0.0f};
    bool mine[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int m = t / 16 + i * STEP;
        mine[i] = m < 16 * MT && m0 + m < e.M && on < e.N;
        osx[i] = mine[i] ? e.sx[m0 + m] : 0.0f;
    }
    if (mine[0])
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            osw[j] = e.sw[j][on];
            ob[j] = load1_rt(e.bias[j], e.bias_dt, on, 0.0f);
        }

    const Rows16 weights[2] = {rows16_of(wg, e.N, n0, K), rows16_of(wu, e.N, n0, K)};
    Rows16 tokens[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) tokens[i] = rows16_of(qx, e.M, m0 + 16 * i, K);
    v4i acc[MT][2];
    few_product<MT, 2, NWV, U>(weights, tokens, K, acc);
    // lane l holds features 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) *reinterpret_cast<v4i*>(&sums[w][16 * i + l16][16 * j + 4 * g4]) = acc[i][j];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int m = t / 16 + i * STEP;
        if (!mine[i]) continue;
        float v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            int s = 0;
#pragma unroll
            for (int x = 0; x < NWV; ++x) s += sums[x][m][16 * j + t % 16];
            v[j] = (float)s * osx[i] * osw[j] + ob[j];
            if (e.z) store1<YT>(e.z, (m0 + m) * 2 * e.N + j * e.N + on, v[j]);
        }
        float y = 0.0f;
        with_act(e.act, [&](auto a) { y = act1<decltype(a)::value>(v[0]) * v[1]; });
        store1<YT>(e.y, (m0 + m) * e.N + on, y);
    }
}

// -------------------------------------------------------------- many tokens
// A tile's outputs are finished in registers, where a lane holds both sums of four
// consecutive features of a row, and pass through LDS, so that stores are whole
// lines: half as many values to stage as there are sums, and the whole tile's at
// once (rows 16 features apart beyond theirs, which meets all banks).  For that a tile's
// weight rows are 16 of the gate and 16 of the other in turn (tile_row), and nothing
// else differs from the plain product with 2 F columns: 8192 x 11008 x 4096 bf16 590-621
// us (2 x 8192 x 22016 x 4096 operations at 2380-2500 TOP/s; matrix cores busy 61%,
// 1444 MB read past the L2s for 124 MB of codes), 694 with z kept (361 MB more to
// write, 72 us at a large copy's rate), 777 x 4096 x 4096 f16 36 us: 448 tiles of 128
// in one round of two to a CU, a seventh of which hold no token.  Any alignment with z
// kept: 1021 x 2501 x 5003 f32 80 us, 320 tiles for 256 CUs and the loads of k_epi_tile.
template <int YT, int TILE>
struct GateStage {
    static constexpr int ES = YT == F32 ? 4 : 2, PITCH = (TILE / 2 + 16) * ES, BYTES = TILE * PITCH;
};

// Four features' scales or biases from feature n on, those past F zero.
__device__ __forceinline__ void four_rt(const void* p, int dt, int64_t n, int64_t F, float v[4])
{
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = n + r < F ? load1_rt(p, dt, n + r, 0.0f) : 0.0f;
}

// Writes a staged tile to columns n0 .. of `out`, whose rows are `ld` elements apart.
template <int YT, int TILE, int NT>
__device__ __forceinline__ void gate_store(const Gate& e, const uint8_t* stage, int64_t m0, int64_t n0, void* out,
                                           int64_t ld, int64_t at)
{
    using S = GateStage<YT, TILE>;
    constexpr int EPC = 16 / S::ES, CPR = TILE / 2 / EPC, RPI = NT / CPR;   // elements per chunk, chunks per row
    const int c = threadIdx.x % CPR, r0 = threadIdx.x / CPR;
    const int64_t n = n0 + c * EPC;
    const int have = e.N - n >= EPC ? EPC : e.N - n > 0 ? (int)(e.N - n) : 0;
#pragma unroll
    for (int i = 0; i < TILE / RPI; ++i) {
        const int r = r0 + i * RPI;
        if (m0 + r >= e.M || have == 0) break;
        const uint4 v = *reinterpret_cast<const uint4*>(stage + r * S::PITCH + c * 16);
        char* to = static_cast<char*>(out) + ((m0 + r) * ld + at + n) * S::ES;
        if (have == EPC) {
            st16_any<TILE == 256>(to, v);
        } else {
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < EPC; ++k)
                if (k < have) {
                    if constexpr (YT == F32) reinterpret_cast<uint32_t*>(to)[k] = u[k];
                    else reinterpret_cast<uint16_t*>(to)[k] = (uint16_t)(u[k / 2] >> (16 * (k & 1)));
                }
        }
    }
}

template <int YT, int TILE, int WM, int WN>
__device__ __forceinline__ void finish_gate(const Gate& e, int64_t m0, int64_t n0,
                                            const v4i (&acc)[TILE / WM / 16][TILE / WN / 16], uint8_t* stage)
{
    using S = GateStage<YT, TILE>;
    constexpr int QM = TILE / WM, QF = TILE / WN / 2, NM = QM / 16, NP = QF / 16, NT = 64 * WM * WN;
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int l16 = lane & 15, g4 = lane >> 4, wm = w / WN, wn = w % WN;
    float sx[NM];
#pragma unroll
    for (int i = 0; i < NM; ++i) {
        const int64_t row = m0 + QM * wm + 16 * i + l16;
        sx[i] = e.sx[row < e.M ? row : e.M - 1];
    }
    // f(g, u) of every output, four features of a row at a time, staged
    auto stage_all = [&](auto f) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            asm volatile("" ::: "memory");       // one step's parameters at a time
            __builtin_amdgcn_sched_barrier(0);
            const int64_t n = n0 + QF * wn + 16 * p + 4 * g4;
            float sg[4], su[4], bg[4], bu[4];
            four_rt(e.sw[0], F32, n, e.N, sg);
            four_rt(e.sw[1], F32, n, e.N, su);
            four_rt(e.bias[0], e.bias_dt, n, e.N, bg);
            four_rt(e.bias[1], e.bias_dt, n, e.N, bu);
#pragma unroll
            for (int i = 0; i < NM; ++i) {
                float v[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float g = (float)acc[i][2 * p][r] * sx[i] * sg[r] + bg[r];
                    const float u = (float)acc[i][2 * p + 1][r] * sx[i] * su[r] + bu[r];
                    v[r] = f(g, u);
                }
                uint8_t* to = stage + (QM * wm + 16 * i + l16) * S::PITCH + (QF * wn + 16 * p + 4 * g4) * S::ES;
                if constexpr (YT == F32)
                    *reinterpret_cast<uint4*>(to) = make_uint4(as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3]));
                else
                    *reinterpret_cast<uint2*>(to) = make_uint2(narrow2<YT>(v[0], v[1]), narrow2<YT>(v[2], v[3]));
            }
        }
        __syncthreads();
    };
    if (e.z) {
        stage_all([](float g, float) { return g; });
        gate_store<YT, TILE, NT>(e, stage, m0, n0, e.z, 2 * e.N, 0);
        __syncthreads();
        stage_all([](float, float u) { return u; });
        gate_store<YT, TILE, NT>(e, stage, m0, n0, e.z, 2 * e.N, e.N);
        __syncthreads();
    }
    with_act(e.act, [&](auto a) {
        stage_all([](float g, float u) { return act1<decltype(a)::value>(g) * u; });
    });
    gate_store<YT, TILE, NT>(e, stage, m0, n0, e.y, e.N, 0);
}

template <int YT>
struct GateTile : Gate {
    static constexpr bool GATED = true;
    const int8_t* wu;
    __device__ __forceinline__ const int8_t* second_weight(const int8_t*) const { return wu; }
    template <int TILE, int WM, int WN>
    static constexpr int staging()
    {
        return GateStage<YT, TILE>::BYTES;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ int early(const Gate&, int64_t)
    {
        return 0;
    }
    template <int TILE, int WM, int WN>
    static __device__ __forceinline__ void finish(const Gate& e, int64_t m0, int64_t n0,
                                                  const v4i (&acc)[TILE / WM / 16][TILE / WN / 16], uint8_t* lds, int)
    {
        finish_gate<YT, TILE, WM, WN>(e, m0, n0, acc, lds);
    }
};

// ----------------------------------------------------------- gate by itself
// a = act(g) and s = act'(g), with one exponential for both.  As in the epilogue's
// slope, a second term vanishes with its factor, and relu's slope keeps a NaN.
__device__ __forceinline__ void act_slope8(int act, const float g[8], float a[8], float s[8])
{
    switch (act) {
    case TQ_ACT_RELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = g[i] > 0.0f || g[i] != g[i] ? g[i] : 0.0f;
            s[i] = g[i] > 0.0f ? 1.0f : g[i] <= 0.0f ? 0.0f : g[i];
        }
        break;
    case TQ_ACT_SILU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-LOG2E * g[i]));
            const float pq = __builtin_fmaf(-p, p, p);
            a[i] = g[i] * p;
            s[i] = __builtin_fmaf(pq == 0.0f ? 0.0f : g[i], pq, p);
        }
        break;
    case TQ_ACT_GELU:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float p = 0.5f * erfcf(-g[i] * SQRT_HALF);
            const float f = __builtin_amdgcn_exp2f(-0.5f * LOG2E * g[i] * g[i]) * (GELU_C * 0.5f);
            a[i] = g[i] * p;
            s[i] = p + (f == 0.0f ? 0.0f : g[i] * f);
        }
        break;
    case TQ_ACT_GELU_TANH:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            constexpr float A = -2.0f * LOG2E * GELU_C;
            const float gg = g[i] * g[i];
            const float p = __builtin_amdgcn_rcpf(
                1.0f + __builtin_amdgcn_exp2f(g[i] * __builtin_fmaf(gg, A * GELU_A, A)));
            const float pq = __builtin_fmaf(-p, p, p);
            const float u = g[i] * __builtin_fmaf(gg, 6.0f * GELU_C * GELU_A, 2.0f * GELU_C);
            a[i] = g[i] * p;
            s[i] = __builtin_fmaf(pq == 0.0f ? 0.0f : u, pq, p);
        }
        break;
    default:
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = g[i];
            s[i] = 1.0f;
        }
        break;
    }
}

// k_gate_act: a thread per eight features of a row (F >= 8), or per feature.  Bound by
// HBM: [8192, 2 x 11008] bf16 93.1 us (541 MB, 5.8 TB/s).
template <int FT>
__global__ __launch_bounds__(256) void k_gate_act(const void* __restrict__ z, uint32_t M, int64_t F, uint32_t per,
                                                  int act, void* __restrict__ y)
{
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, row = i / per, v = i % per;
    if (row >= M) return;
    const int64_t from = (int64_t)row * 2 * F, to = (int64_t)row * F;
    if (F < 8) {
        const float g = load1<FT>(z, from + v), u = load1<FT>(z, from + F + v);
        float a = 0.0f;
        with_act(act, [&](auto k) { a = act1<decltype(k)::value>(g); });
        store1<FT>(y, to + v, a * u);
        return;
    }
    // the last vector of a row is moved back to end with it
    Vec8 q;
    q.at = 8 * (int64_t)v < F - 8 ? (int)(8 * v) : (int)(F - 8);
    q.lo = (int)(8 * (int64_t)v - q.at);
    float g[8], u[8];
    widen8<FT>(load8_any<FT>(z, from + q.at), g);
    widen8<FT>(load8_any<FT>(z, from + F + q.at), u);
    act8(act, g);
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] *= u[k];
    store8_own<FT>(y, to, q, g);
}

// k_gate_bwd: dg, du and their column sums.  A wave owns 512 features, a
// workgroup's four waves take a chunk of the rows in turn, U rows in flight each;
// their column sums meet in LDS in wave order and leave as one row of partials per
// chunk, the gate's F and then the other's.  dz may be z: an element's output
// depends on its own row's pair and dy alone and is stored by the lane that owns
// them after their load; what a moved-back vector or a chunk's last rows read
// besides may be new already, and is not used.  Bound by HBM: [8192, 2 x 11008] bf16
// 168.6 us (902 MB, 5.35 TB/s) and 10.4 us for the sums of the chunks' partials.
template <int FT>
__global__ __launch_bounds__(256) void k_gate_bwd(const void* dy, const void* z, int64_t M, int64_t F, int64_t chunk,
                                                  int act, void* dz, float* __restrict__ part, int64_t ldp)
{
    constexpr int U = 2;
    __shared__ float fold[3][16][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t c0 = (int64_t)blockIdx.x * 512;
    const int n = F - c0 < 512 ? (int)(F - c0) : 512;
    const int64_t r0 = (int64_t)blockIdx.y * chunk, r1 = r0 + chunk < M ? r0 + chunk : M;
    // F >= 8: a last slab of fewer than 8 columns starts earlier, and counts only its own
    const int64_t cs = n >= 8 ? c0 : F - 8;
    const int skip = (int)(c0 - cs);
    Vec8 at = vec8(lane, n + skip);
    if (skip) at.lo = lane == 0 ? skip : 8;
    float db[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) db[i] = 0.0f;
    for (int64_t r = r0 + w; r < r1; r += 4 * U) {
        Raw8<FT> a[U], b[U], c[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r + 4 * u < r1 ? r + 4 * u : r1 - 1;
            a[u] = load8_any<FT>(dy, row * F + cs + at.at);
            b[u] = load8_any<FT>(z, row * 2 * F + cs + at.at);
            c[u] = load8_any<FT>(z, row * 2 * F + F + cs + at.at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + 4 * u >= r1) break;
            float d[8], g[8], x[8], dg[8], du[8];
            widen8<FT>(a[u], d);
            widen8<FT>(b[u], g);
            widen8<FT>(c[u], x);
            act_slope8(act, g, du, dg);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // where the slope is 0 so is dg, whatever dy and u hold
                dg[i] = dg[i] == 0.0f ? 0.0f : d[i] * x[i] * dg[i];
                du[i] *= d[i];
                db[i] += dg[i];
                db[8 + i] += du[i];
            }
            if (at.lo < 8) {
                store8_own<FT>(dz, (r + 4 * u) * 2 * F + cs, at, dg);
                store8_own<FT>(dz, (r + 4 * u) * 2 * F + F + cs, at, du);
            }
        }
    }
    if (!part) return;
    if (w > 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i) fold[w - 1][i][lane] = db[i];
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 16; ++i) db[i] += fold[k][i][lane];
    if (at.lo < 8) {
        store8_own<F32>(part, (int64_t)blockIdx.y * ldp + cs, at, db);
        store8_own<F32>(part, (int64_t)blockIdx.y * ldp + F + cs, at, db + 8);
    }
}

// Fewer than 8 features: a thread per row and step, the features in turn.
template <int FT>
__global__ __launch_bounds__(256) void k_gate_bwd_thin(const void* dy, const void* z, int64_t M, int64_t F,
                                                       int64_t chunk, int act, void* dz, float* __restrict__ part,
                                                       int64_t ldp)
{
    __shared__ float fold[4][16];
    const int t = threadIdx.x, n = (int)F;
    const int64_t r0 = (int64_t)blockIdx.y * chunk, r1 = r0 + chunk < M ? r0 + chunk : M;
    float db[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) db[i] = 0.0f;
    for (int64_t r = r0 + t; r < r1; r += 256) {
        float g[8], dg[8], du[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = i < n ? load1<FT>(z, r * 2 * F + i) : 0.0f;
        act_slope8(act, g, du, dg);
        float x[8], d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            d[i] = i < n ? load1<FT>(dy, r * F + i) : 0.0f;
            x[i] = i < n ? load1<FT>(z, r * 2 * F + F + i) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                dg[i] = dg[i] == 0.0f ? 0.0f : d[i] * x[i] * dg[i];
                du[i] *= d[i];
                db[i] += dg[i];
                db[8 + i] += du[i];
                store1<FT>(dz, r * 2 * F + i, dg[i]);
                store1<FT>(dz, r * 2 * F + F + i, du[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const float s = wave_sum(db[i]);
        if ((t & 63) == 0) fold[t >> 6][i] = s;
    }
    __syncthreads();
    if (part && t < 16 && (t & 7) < n)
        part[(int64_t)blockIdx.y * ldp + (t >> 3) * F + (t & 7)] = fold[0][t] + fold[1][t] + fold[2][t] + fold[3][t];
}

// ---------------------------------------------------------------- launches
// Rows per chunk of the backward pass: whole rounds of the four waves' two rows,
// in about GATE_GROUPS workgroups over the slabs of 512 features ([8192, 2 x 11008]:
// 4096 178.0 us, 8192 179.5, 16384 179.6); up to GATE_ONE rows are one chunk, whose sums
// are dbias itself: one launch.
constexpr int64_t GATE_GROUPS = 8192;
constexpr int64_t GATE_ONE = 64;
inline int64_t gate_chunk(int64_t M, int64_t F)
{
    if (M <= GATE_ONE) return GATE_ONE;
    const int64_t chunks = std::max<int64_t>(1, GATE_GROUPS / cdiv(F, 512));
    return cdiv(cdiv(M, chunks), 8) * 8;
}

// The kernel of a gated product, by its shape: as for the product with one weight of
// 2 F rows (product_launch), whose rounds and rates it shares.  Few tokens / 64 tile, us:
//   24 x 4096 x 4096    9.4 / 11.7     48 x 4096 x 4096   14.7 / 11.7
//   24 x 4096 x 11008  17.7 / 24.2     48 x 4096 x 11008  31.9 / 25.8
//   24 x 11008 x 4096  24.2 / 19.2     96 x 1024 x 4096    9.0 / 11.4
//   24 x 4096 x 4095   16.6 / 21.6     220 x 507 x 10250  17.3 / 33.6
template <int YT>
static void gate_launch(const int8_t* qx, const int8_t* wg, const int8_t* wu, int64_t K, const Gate& e, hipStream_t st)
{
    const bool rows16 = K >= ET && K % 16 == 0 && aligned16(qx) && aligned16(wg) && aligned16(wu);
    const int64_t N = 2 * e.N;
#define TQ_FEW(MT, NWV, U)                                                                                  \
    do {                                                                                                    \
        const dim3 grid((unsigned)cdiv(e.N, 16), (unsigned)cdiv(e.M, 16 * MT));                             \
        hipLaunchKernelGGL((k_gate_few<YT, MT, NWV, U>), grid, dim3(64 * NWV), 0, st, qx, wg, wu, K, e);        \
        return;                                                                                             \
    } while (0)
    if (few_tokens(e.M, N)) {
        if (e.M <= 16) TQ_FEW(1, 8, 1);
        TQ_FEW(2, 8, 1);
    }
#undef TQ_FEW
    if (rows16) {
#define TQ_RING(TILE, RING, WM, WN, WGS)                                                                     \
    do {                                                                                                     \
        const int64_t nt = cdiv(e.N, TILE / 2), mt = cdiv(e.M, TILE);                                        \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                            \
        hipLaunchKernelGGL((k_epi_ring<GateTile<YT>, TILE, RING, WM, WN, WGS>), dim3((unsigned)(nt * mt)),   \
                           dim3(64 * WM * WN), 0, st, qx, wg, K, nt, mt, slab, GateTile<YT>{e, wu});         \
    } while (0)
        const int64_t t128 = cdiv(e.M, 128) * cdiv(N, 128);
        if (cdiv(e.M, 256) * cdiv(N, 256) >= 256) TQ_RING(256, 5, 2, 4, 1);
        else if (t128 > 256) TQ_RING(128, 5, 2, 4, 2);
        else if (cdiv(e.M, 64) * cdiv(N, 64) > 512) TQ_RING(128, 9, 2, 4, 1);
        else TQ_RING(64, 9, 2, 2, 2);
#undef TQ_RING
        return;
    }
#define TQ_TILE(TILE, WM, WN, D, WGS)                                                                        \
    do {                                                                                                     \
        const int64_t nt = cdiv(e.N, TILE / 2), mt = cdiv(e.M, TILE);                                        \
        const int slab = (int)std::min<int64_t>(cdiv(nt, 8), 16);                                            \
        hipLaunchKernelGGL((k_epi_tile<GateTile<YT>, TILE, WM, WN, D, WGS>), dim3((unsigned)(nt * mt)),      \
                           dim3(64 * WM * WN), 0, st, qx, wg, K, nt, mt, slab, GateTile<YT>{e, wu});         \
    } while (0)
    if (cdiv(e.M, 256) * cdiv(N, 256) > 160) TQ_TILE(256, 2, 4, 2, 1);
    else if (cdiv(e.M, 64) * cdiv(N, 64) > 512) TQ_TILE(128, 2, 4, 2, 2);
    else TQ_TILE(64, 2, 2, 4, 2);
#undef TQ_TILE
}

static bool natural(const void* p, int dt) { return ((uintptr_t)p & (uintptr_t)(ftype_size(dt) - 1)) == 0; }
static bool valid_act(int a) { return a >= TQ_ACT_NONE && a <= TQ_ACT_GELU_TANH; }

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_w8a8_gated_linear(const int8_t* qx, const float* sx, const int8_t* qw_gate, const float* sw_gate,
                               const int8_t* qw_up, const float* sw_up, int64_t M, int64_t F, int64_t K,
                               const void* bias_gate, const void* bias_up, int bias_dtype, int act, void* y,
                               void* preact, int y_dtype, void* stream)
{
    if (!valid_ftype(y_dtype) || !valid_act(act) || M < 0 || F < 0 || K < 0) return TQ_ERR_INVALID;
    if ((bias_gate || bias_up) && !valid_ftype(bias_dtype)) return TQ_ERR_INVALID;
    if (M == 0 || F == 0) return TQ_OK;
    if (!y || !sx || !sw_gate || !sw_up || (K > 0 && (!qx || !qw_gate || !qw_up))) return TQ_ERR_INVALID;
    // a grid holds fewer than 2^32 threads: 512 per 16 features or per tile of 256 tokens and 128 features
    if (K > 131071 || cdiv(M, ET) > 65535 || cdiv(F, 16) > 0x7fffff || cdiv(M, 256) * cdiv(F, 128) > 0x7fffff)
        return TQ_ERR_UNSUPPORTED;
    if (!natural(sx, TQ_F32) || !natural(sw_gate, TQ_F32) || !natural(sw_up, TQ_F32) ||
        (bias_gate && !natural(bias_gate, bias_dtype)) || (bias_up && !natural(bias_up, bias_dtype)) ||
        !natural(y, y_dtype) || !natural(preact, y_dtype))
        return TQ_ERR_ALIGN;
    const Gate e = {sx, {sw_gate, sw_up}, {bias_gate, bias_up}, bias_dtype, act, y, preact, M, F};
    TQ_LLM_FT_SWITCH(y_dtype, gate_launch<FTV>(qx, qw_gate, qw_up, K, e, as_stream(stream)));
    return launch_status();
}

tq_status tq_gated_act(const void* z, int dtype, int64_t M, int64_t F, int act, void* y, void* stream)
{
    if (!valid_ftype(dtype) || !valid_act(act) || M < 0 || F < 0) return TQ_ERR_INVALID;
    if (M == 0 || F == 0) return TQ_OK;
    if (!z || !y) return TQ_ERR_INVALID;
    if (F > 0x7ffffff0) return TQ_ERR_UNSUPPORTED;
    if (!natural(z, dtype) || !natural(y, dtype)) return TQ_ERR_ALIGN;
    const int64_t per = F < 8 ? F : cdiv(F, 8), most = std::max<int64_t>(1, 0xff000000u / per);
    for (int64_t r = 0; r < M; r += most) {      // a grid holds fewer than 2^32 threads
        const int64_t rows = std::min(M - r, most);
        TQ_LLM_FT_SWITCH(dtype, hipLaunchKernelGGL((k_gate_act<FTV>), dim3((unsigned)cdiv(rows * per, 256)), dim3(256),
                                                   0, as_stream(stream), forward_by(z, r * 2 * F * ftype_size(dtype)),
                                                   (uint32_t)rows, F, (uint32_t)per, act,
                                                   forward_by(y, r * F * ftype_size(dtype))));
    }
    return launch_status();
}

size_t tq_gated_act_backward_workspace_bytes(int64_t M, int64_t F)
{
    if (M <= GATE_ONE || F <= 0) return 0;
    return (size_t)cdiv(M, gate_chunk(M, F)) * (size_t)colsum_ld(2 * F) * sizeof(float);
}

tq_status tq_gated_act_backward(const void* dy, const void* z, int dtype, int64_t M, int64_t F, int act, void* dz,
                                float* dbias, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!valid_ftype(dtype) || !valid_act(act) || M < 0 || F < 0) return TQ_ERR_INVALID;
    if (F == 0) return TQ_OK;
    if (!natural(dbias, TQ_F32)) return TQ_ERR_ALIGN;
    hipStream_t st = as_stream(stream);
    if (F > 0x7ffffff0) return TQ_ERR_UNSUPPORTED;
    if (M == 0) {                        // no rows: the sums are empty, not unwritten
        zero_vec_launch(dbias, TQ_F32, 2 * F, st);
        return launch_status();
    }
    if (!dy || !z || !dz) return TQ_ERR_INVALID;
    if (!natural(dy, dtype) || !natural(z, dtype) || !natural(dz, dtype)) return TQ_ERR_ALIGN;
    const int64_t chunk = gate_chunk(M, F), chunks = cdiv(M, chunk), ld = colsum_ld(2 * F);
    if (dbias && chunks > 1) {
        if (!workspace || workspace_bytes < tq_gated_act_backward_workspace_bytes(M, F)) return TQ_ERR_INVALID;
        if (!aligned16(workspace)) return TQ_ERR_ALIGN;
    }
    float* part = dbias && chunks > 1 ? static_cast<float*>(workspace) : dbias;
    const dim3 grid((unsigned)cdiv(F, 512), (unsigned)chunks);
    TQ_LLM_FT_SWITCH(dtype, {
        if (F < 8)
            hipLaunchKernelGGL((k_gate_bwd_thin<FTV>), grid, dim3(256), 0, st, dy, z, M, F, chunk, act, dz, part, ld);
        else
            hipLaunchKernelGGL((k_gate_bwd<FTV>), grid, dim3(256), 0, st, dy, z, M, F, chunk, act, dz, part, ld);
    });
    if (dbias && chunks > 1) colsum_launch(part, chunks, 1, ld, 2 * F, dbias, nullptr, TQ_F32, st);
    return launch_status();
}

}  // extern "C"
