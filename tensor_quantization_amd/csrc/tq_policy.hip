// tq_policy.hip -- a token's log-probability from the logits, and the clipped
// policy loss with its KL term on it: forwards, back, and both in one call.
//
//   s = 1 / T, y = token[row];   l = s z_y - lse(s z)
//   rho = exp(l - old);   d = ref - l
//   L = -min(rho A, clip(rho, 1 - lo, 1 + hi) A) + beta (exp(d) - 1 - d)
//   dL/dl = -rho A where rho A <= clip(rho) A, else 0;   + beta (1 - exp(d))
//   dL/dz_j = s dL/dl (1[j = y] - q_j),   q_j = exp(s z_j - lse(s z))
//
// A row whose token lies outside [0, V) counts nowhere: loss, log-probability and
// gradient 0.  Everything here is bound by HBM: the forward pass reads the logits
// once, the gradient reads them and writes as much; in one call the row is held in
// registers between the two.  All sums are binary32, relative to the largest of
// what they add; c = s log2 e.
#include "tq_llm.h"

namespace tq {

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }
__device__ __forceinline__ float base_of(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// The sum of 2^((z - m) c) over some columns, m the largest z of them.
struct Sum {
    float m, sum;
};
__device__ __forceinline__ float sum_at(const Sum& a, float base, float c)
{
    return a.sum * ex2((a.m - base) * c);    // m = -inf: 0
}
__device__ __forceinline__ Sum wave_join(const Sum& a, float c)
{
    const float m = wave_max(a.m);
    return Sum{m, wave_sum(sum_at(a, base_of(m), c))};
}

struct Tokens {
    const void* idx;
    int idx64;
};
__device__ __forceinline__ int token_of(const Tokens& k, int64_t row, int V)
{
    const int64_t i = k.idx64 ? static_cast<const int64_t*>(k.idx)[row] : static_cast<const int32_t*>(k.idx)[row];
    return i >= 0 && i < V ? (int)i : -1;
}

// What the loss takes besides the logits, by row.  Without advantages there is no
// loss, and the gradient's coefficient is dloss itself.
struct Policy {
    const float* adv;
    const float* old;                    // null: the present policy's own, rho = 1
    const float* ref;                    // null: no KL term
    float lo, hi, beta;
};

// The loss of a row's log-probability l, and its slope dL/dl.  Where l is -inf, what
// the other policies say of the token does not matter (but a NaN stays): rho = 0, and d =
// +inf.
__device__ __forceinline__ float policy_loss(const Policy& p, int64_t row, float l, float* slope)
{
    constexpr float INF = __builtin_inff();
    const float A = p.adv[row], old = p.old ? p.old[row] : l;
    const float rho = l == -INF && old == old ? 0.0f : ex2((l - old) * LOG2E);
    const float held = __builtin_fminf(__builtin_fmaxf(rho, 1.0f - p.lo), 1.0f + p.hi);
    const float u = A == 0.0f && rho == INF ? A : rho * A, v = held * A;     // no advantage, however far rho overflows
    float loss = u <= v || u != u ? -u : -v, g = u <= v || u != u ? -u : 0.0f;
    if (p.ref) {
        const float ref = p.ref[row], d = l == -INF && ref == ref ? INF : ref - l, x = expm1f(d);
        loss += p.beta * (x == INF ? x : x - d);
        g -= p.beta * x;
    }
    *slope = g;
    return loss;
}

// l from the row's largest logit m and its sum S relative to it.  Nothing can be
// drawn from a row of nothing but -inf: l = -inf.
__device__ __forceinline__ float logp_of(float z, float m, float S, float s)
{
    return S == 0.0f ? -__builtin_inff() : (z - base_of(m)) * s - lg2(S) * LN2;
}

// --------------------------------------------------------------- statistics
// Adds the vector's elements lo .. 7 to a running maximum and sum.
__device__ __forceinline__ void add8(Sum& a, const float v[8], int lo, float c)
{
    float top = v[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, v[i]);
    if (top > a.m) {
        a.sum *= ex2((a.m - top) * c);       // m = -inf: 0
        a.m = top;
    }
    const float b = base_of(a.m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = ex2((v[i] - b) * c);
        sum += i >= lo ? x : 0.0f;
    }
    a.sum += sum;
}

// The sum over n columns from `base` on by the NT threads of a workgroup, in wave 0
// (every lane) after the call.
template <int FT, int NT>
__device__ __forceinline__ Sum columns_sum(const void* z, int64_t base, int n, float c, Sum (&red)[NT / 64])
{
    constexpr int U = 4;
    const int t = threadIdx.x, lane = t & 63, nvec = (n + 7) / 8;
    Sum a = {-__builtin_inff(), 0.0f};
    if (n >= 8) {
        for (int v0 = t; v0 < nvec; v0 += NT * U) {
            Raw8<FT> raw[U];
            Vec8 at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                at[u] = vec8(v0 + NT * u, n);
                raw[u] = load8_any<FT>(z, base + at[u].at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (at[u].lo == 8) continue;
                float v[8];
                widen8<FT>(raw[u], v);
                add8(a, v, at[u].lo, c);
            }
        }
    } else if (t < n) {
        float v[8];
        v[0] = load1<FT>(z, base + t);
#pragma unroll
        for (int i = 1; i < 8; ++i) v[i] = -__builtin_inff();
        add8(a, v, 0, c);
    }
    a = wave_join(a, c);
    if (lane == 0) red[t >> 6] = a;
    __syncthreads();
    return wave_join(lane < NT / 64 ? red[lane] : Sum{-__builtin_inff(), 0.0f}, c);
}

// Writes what the forward pass leaves of a row; `a` of a row that counts nowhere is
// the sum of no columns.
__device__ __forceinline__ void row_out(const Policy& p, int64_t row, int tok, float zy, const Sum& a, float s,
                                        float* loss, float* logp, float* stats)
{
    const float l = tok >= 0 ? logp_of(zy, a.m, a.sum, s) : 0.0f;
    float slope;
    if (loss) loss[row] = tok >= 0 ? policy_loss(p, row, l, &slope) : 0.0f;
    logp[row] = l;
    if (stats) {
        stats[2 * row] = a.m;
        stats[2 * row + 1] = a.sum;
    }
}

// k_logp_rows: a workgroup per row.  512 x 32000 binary32 13.3 us (65.5 MB, 4.9 TB/s).
template <int FT, int NT>
__global__ __launch_bounds__(NT) void k_logp_rows(const void* __restrict__ z, int64_t ldz, int V, Tokens tok, Policy p,
                                                  float s, float c, float* __restrict__ loss, float* __restrict__ logp,
                                                  float* __restrict__ stats)
{
    __shared__ Sum red[NT / 64];
    const int64_t row = blockIdx.x;
    const int y = token_of(tok, row, V);
    Sum a = {-__builtin_inff(), 0.0f};
    float zy = 0.0f;
    if (y >= 0) {                        // uniform
        zy = load1<FT>(z, row * ldz + y);
        a = columns_sum<FT, NT>(z, row * ldz, V, c, red);
    }
    if (threadIdx.x == 0) row_out(p, row, y, zy, a, s, loss, logp, stats);
}

// k_logp_parts: a workgroup per row and part of it (`len` columns), whose sum it
// leaves, and the logit at the row's token where that lies in it (for whoever writes
// the loss when the gradient may have overwritten the logits).  k_logp_join: a wave
// per row joins its parts.  64 x 131072 bf16 6.9 and 3.0 us, 9 x 131001 f16 3.8: some 2-3
// us of each are a launch's beginning and end, which so few rows do not cover.
template <int FT>
__global__ __launch_bounds__(256) void k_logp_parts(const void* __restrict__ z, int64_t ldz, int V, int parts, int len,
                                                    Tokens tok, float c, Sum* __restrict__ part,
                                                    float* __restrict__ zy)
{
    __shared__ Sum red[4];
    const int64_t row = blockIdx.x / (unsigned)parts;
    const int p = (int)(blockIdx.x % (unsigned)parts), c0 = p * len, n = V - c0 < len ? V - c0 : len;
    const int y = token_of(tok, row, V);
    if (y < 0) return;                   // uniform; nobody reads this row's
    if (threadIdx.x == 0 && y >= c0 && y - c0 < n) zy[row] = load1<FT>(z, row * ldz + y);
    const Sum a = columns_sum<FT, 256>(z, row * ldz + c0, n, c, red);
    if (threadIdx.x == 0) part[row * parts + p] = a;
}

__device__ __forceinline__ Sum join_parts(const Sum* part, int parts, float c)
{
    Sum a = {-__builtin_inff(), 0.0f};
    for (int i = threadIdx.x & 63; i < parts; i += 64) {
        const Sum b = part[i];
        const float m = __builtin_fmaxf(a.m, b.m), base = base_of(m);
        a = Sum{m, sum_at(a, base, c) + sum_at(b, base, c)};
    }
    return wave_join(a, c);
}

__global__ __launch_bounds__(256) void k_logp_join(int64_t rows, int V, Tokens tok, Policy p, float s, float c,
                                                   const Sum* __restrict__ part, const float* __restrict__ zy,
                                                   int parts, float* __restrict__ loss, float* __restrict__ logp,
                                                   float* __restrict__ stats)
{
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= rows) return;
    const int y = token_of(tok, row, V);
    const Sum a = y >= 0 ? join_parts(part + row * parts, parts, c) : Sum{-__builtin_inff(), 0.0f};
    if ((threadIdx.x & 63) == 0) row_out(p, row, y, y >= 0 ? zy[row] : 0.0f, a, s, loss, logp, stats);
}

// ---------------------------------------------------------------- gradient
// dL/dz_j = k (1[j = y] - q_j): `at` of the token, `all` = k / S for every column.
struct Grad {
    float at, all;
};
__device__ __forceinline__ Grad grad_of(float slope, float g, float s, float S)
{
    const float k = slope * g * s;
    return S == 0.0f ? Grad{0.0f, 0.0f} : Grad{k, k / S};     // a row of -inf logits has no gradient
}

// k_logp_grad: a workgroup per row and part of it.  FROM_PARTS: the row's sum from
// its parts, and the row's first workgroup writes loss and log-probability; otherwise
// from the saved ones.  512 x 32000 binary32 21.2 us (131 MB, 6.2 TB/s).
template <int FT, bool FROM_PARTS>
__global__ __launch_bounds__(256) void k_logp_grad(const void* z, int64_t ldz, int V, int parts, int len, Tokens tok,
                                                   Policy p, float s, float c, const Sum* __restrict__ part,
                                                   const float* __restrict__ zy, const float* __restrict__ stats,
                                                   const float* __restrict__ dloss, float* __restrict__ loss,
                                                   float* __restrict__ logp, void* dz, int64_t lddz)
{
    constexpr int U = 2;
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x / (unsigned)parts;
    const int q = (int)(blockIdx.x % (unsigned)parts), c0 = q * len;
    const int n = V - c0 < len ? V - c0 : len, nvec = (n + 7) / 8;
    const int64_t from = row * ldz + c0, to = row * lddz + c0;
    const int y = token_of(tok, row, V);
    Raw8<FT> raw[U];
    auto fetch = [&](int v0) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load8_any<FT>(z, from + vec8(v0 + 256 * u, n).at);
    };
    if (n >= 8 && y >= 0) fetch(t);
    const float g = dloss ? dloss[row] : 1.0f;
    Sum a;
    float l;
    if constexpr (FROM_PARTS) {
        a = y >= 0 ? join_parts(part + row * parts, parts, c) : Sum{-__builtin_inff(), 0.0f};
        l = y >= 0 ? logp_of(zy[row], a.m, a.sum, s) : 0.0f;
    } else {
        a = Sum{stats[2 * row], stats[2 * row + 1]};
        l = logp ? logp[row] : 0.0f;
    }
    float slope = 1.0f, L = 0.0f;
    if (p.adv && y >= 0) L = policy_loss(p, row, l, &slope);
    if (FROM_PARTS && q == 0 && t == 0) {
        loss[row] = L;
        logp[row] = l;
    }
    const Grad k = grad_of(y >= 0 ? slope : 0.0f, g, s, a.sum);
    const float b = base_of(a.m);
    const int mine = y - c0;             // the token's place in this part, or outside it
    auto grad = [&](float v, int j) { return (j == mine ? k.at : 0.0f) - ex2((v - b) * c) * k.all; };
    if (y < 0 || a.sum == 0.0f) {        // uniform: no gradient, whatever the logits hold
        for (int j = t; j < n; j += 256) store1<FT>(dz, to + j, 0.0f);
        return;
    }
    if (n < 8) {
        if (t < n) store1<FT>(dz, to + t, grad(load1<FT>(z, from + t), t));
        return;
    }
    for (int v0 = t; v0 < nvec; v0 += 256 * U) {
        Raw8<FT> now[U];
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = raw[u];
        if (v0 + 256 * U < nvec) fetch(v0 + 256 * U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const Vec8 at = vec8(v0 + 256 * u, n);
            if (at.lo == 8) continue;
            float v[8];
            widen8<FT>(now[u], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = grad(v[i], at.at + i);
            store8_own<FT>(dz, to, at, v);
        }
    }
}

// k_policy_held: loss and gradient of a row in one read: NT threads hold the row (8
// <= V <= 8 NT W) in registers in its own type, and every vector's exponentials are
// summed as it arrives.  For that a wave takes them relative to the largest logit m of
// its first vector instead of the row's, as 2^(z c - mc) with one rounding, mc being
// m c rounded; whatever meets these sums knows that rounding: the waves are joined by
// 2^(mc - mc'), the gradient's exponentials take the same mc, and the loss, which needs
// log2 S relative to m itself, takes m c - mc out again.  A factor 2^(mc - mc') below
// 2^-126 comes out as 0, which a wave's sum survives only while it is small: one of 2^96
// or more counts as infinite.  Then the sums lose nothing (a share of 2^-30, one in 2^26 of
// the row's at most, over sixteen waves) unless they overflow or come out below 1/2 (no logit
// near the row's largest where a wave looks first); in both cases the row is summed again
// around its own maximum.
//
// A workgroup walks the rows blockIdx + k gridDim: as soon as a vector's gradient is
// computed its registers take the next row's vector, so that the reads go on under the
// gradient's arithmetic and stores.  Of a row whose token counts nowhere one address is
// read, and not used.
// Loads and stores are non-temporal: a row is not met again.  4096 x 131072 bf16 410 us
// (2148 MB, 5.2 TB/s, a large copy 5.0; a pass for the sums and one for the gradient
// would read 1074 MB more).
template <int FT, int NT, int W>
__global__ __launch_bounds__(NT, FT != F32 && W == 4 ? 8 : 1) void k_policy_held(
    const void* z, int64_t ldz, uint32_t rows, int V, Tokens tok, Policy p, float s, float c,
    const float* __restrict__ dloss, float* __restrict__ loss, float* __restrict__ logp, void* dz, int64_t lddz)
{
    constexpr int NW = NT / 64, ES = FT == F32 ? 4 : 2;
    __shared__ float red[2][NW];
    // V / 8 whole vectors (absent ones read the last again), and an element more for the first V % 8 threads
    const int nvec = V >> 3, ntail = V & 7;
    Raw8<FT> raw[W];
    const uint32_t step = gridDim.x;
    // a row that counts nowhere reads one address
    auto at_of = [&](int at, bool counts) { return counts ? (uint32_t)(at < nvec ? at : nvec - 1) * (8 * ES) : 0u; };
    const char* from = static_cast<const char*>(z) + blockIdx.x * ldz * ES;
    int y = blockIdx.x < rows ? token_of(tok, blockIdx.x, V) : -1;
#pragma unroll
    for (int w = 0; w < W; ++w) raw[w] = load8_off<FT, true>(from, at_of(w * NT + (int)threadIdx.x, y >= 0));
    for (uint32_t r = blockIdx.x; r < rows; r += step) {
        // opaque, so that nothing computed from them is kept in registers over the rows
        const int64_t row = afresh_uniform((int)r);
        const int t = afresh((int)threadIdx.x), wave = t >> 6, lane = t & 63;
        char* to = static_cast<char*>(dz) + row * lddz * ES;
        from = static_cast<const char*>(z) + row * ldz * ES;
        const bool more = r + step < rows;
        const char* next = from + (more ? step * ldz * ES : 0);
        const int ynext = more ? token_of(tok, row + step, V) : -1;
        // vector w of the next row
        auto ahead = [&](int w) { raw[w] = load8_off<FT, true>(next, at_of(afresh(afresh(t) + w * NT), ynext >= 0)); };
        if (y < 0) {                     // uniform: nothing of this row is used
#pragma unroll
            for (int w = 0; w < W; ++w) {
                ahead(w);
                const int at = afresh(afresh(t) + w * NT);
                const float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (at < nvec) store8_off<FT, true>(to, (uint32_t)at * (8 * ES), v);
            }
            if (t < ntail) store1<FT>(to, 8 * nvec + t, 0.0f);
            if (t == 0) {
                loss[row] = 0.0f;
                logp[row] = 0.0f;
            }
            y = ynext;
            continue;
        }
        const float tail = t < ntail ? load1<FT>(from, 8 * nvec + t) : -__builtin_inff();
        float zy = load1<FT>(from, y);
        const float g = dloss ? dloss[row] : 1.0f;
        float m, S;
        // x(z) added up over this thread's vectors
        auto sum = [&](auto x) {
            S = t < ntail ? x(tail) : 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int at = afresh(afresh(t) + w * NT);
                float v[8], part = 0.0f;
                keep_raw<FT>(raw[w]);
                widen8<FT>(raw[w], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) part += x(v[i]);
                S += at < nvec ? part : 0.0f;
                __builtin_amdgcn_sched_barrier(0);   // one vector at a time, in the order they arrive
            }
            S = wave_sum(S);
        };
        auto top = [&](float v) {
#pragma unroll
            for (int w = 0; w < W; ++w) {            // repeated elements do not change a maximum
                float x[8];
                keep_raw<FT>(raw[w]);
                widen8<FT>(raw[w], x);
#pragma unroll
                for (int i = 0; i < 8; ++i) v = __builtin_fmaxf(v, x[i]);
                __builtin_amdgcn_sched_barrier(0);
            }
            return wave_max(v);
        };
        {
            float v[8];
            widen8<FT>(raw[0], v);
            m = v[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = __builtin_fmaxf(m, v[i]);
            m = base_of(wave_max(m));
            const float mc = m * c;
            sum([&](float v) { return ex2(__builtin_fmaf(v, c, -mc)); });
        }
        asm volatile("" : "+v"(zy));         // here ahead of the barrier, and so of any store: dz may be z
        __syncthreads();                     // the row before is done with `red`
        if (lane == 0) {
            red[0][wave] = m;
            red[1][wave] = S < 0x1p96f ? S : __builtin_inff();    // 0 times it is NaN, which is not near
        }
        __syncthreads();
        m = wave_max(lane < NW ? red[0][lane] : -__builtin_inff());
        S = wave_sum(lane < NW ? red[1][lane] * ex2(red[0][lane] * c - m * c) : 0.0f);   // products rounded as the waves' own
        const bool near = S >= 0.5f && S < 0x1p100f;
        const float off = near ? __builtin_fmaf(m, c, -(m * c)) : 0.0f;
        if (!near) {                         // uniform: around the row's own maximum
            m = top(tail);
            __syncthreads();
            if (lane == 0) red[0][wave] = m;
            __syncthreads();
            m = wave_max(lane < NW ? red[0][lane] : -__builtin_inff());
            const float b = base_of(m);
            sum([&](float v) { return ex2((v - b) * c); });
            if (lane == 0) red[1][wave] = S;
            __syncthreads();
            S = wave_sum(lane < NW ? red[1][lane] : 0.0f);
        }
        const float l = logp_of(zy, m, S, s) + off * LN2;
        float slope;
        const float L = policy_loss(p, row, l, &slope);
        if (t == 0) {
            loss[row] = L;
            logp[row] = l;
        }
        const Grad k = grad_of(slope, g, s, S);
        // 2^(z c - mc) or 2^((z - m) c)
        const float b = near ? 0.0f : base_of(m), mc = near ? m * c : 0.0f;
        auto grad = [&](float v, bool token) {
            const float q = ex2(__builtin_fmaf(v - b, c, -mc)) * k.all;
            return (token ? k.at : 0.0f) - q;
        };
        const bool none = S == 0.0f;         // uniform
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int at = afresh(afresh(t) + w * NT);
            float v[8];
            keep_raw<FT>(raw[w]);
            widen8<FT>(raw[w], v);
            // the old vector's registers are free before the new one's load is issued: it goes into the same ones,
            // and no copy at the loop's end waits for it
#pragma unroll
            for (int i = 0; i < 8; ++i) asm volatile("" : "+v"(v[i]));
            __builtin_amdgcn_sched_barrier(0);
            ahead(w);
            if (at < nvec) {
                const int mine = y - 8 * at;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = none ? 0.0f : grad(v[i], i == mine);
                store8_off<FT, true>(to, (uint32_t)at * (8 * ES), v);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (t < ntail) store1<FT>(to, 8 * nvec + t, none ? 0.0f : grad(tail, 8 * nvec + t == y));
        y = ynext;
    }
}

// ---------------------------------------------------------------- launches
// Most columns per part: 8192, or 4096 where that would not give the chip LP_GROUPS
// workgroups.  The parts of a row have one length, a multiple of 8 (the last may be
// shorter).
constexpr int64_t LP_GROUPS = 2048;
struct Split {
    int len, parts;
};
inline Split logp_split(int64_t rows, int64_t V)
{
    const int64_t most = rows * cdiv(V, 8192) >= LP_GROUPS ? 8192 : 4096;
    Split q;
    q.len = (int)cdiv(cdiv(V, cdiv(V, most)), 8) * 8;
    q.parts = (int)cdiv(V, q.len);
    return q;
}

// Whether a workgroup takes a whole row forwards, in one launch: from LP_ROWS rows on,
// and where a row is so short (LP_BYTES) that the second launch costs more than its
// reading by one CU.  Longer rows go by what the GPU takes in a replayed graph, where no host
// stands between the launches.  Whole rows / parts and their join, us, bf16, called one after
// another and, where two pairs are given, replayed:
//   64 x 32000   11.5 / 14.6     16 x 131072   12.0 / 14.0, 11.4 / 6.1
//   256 x 32000  11.5 / 14.5     64 x 131072   12.8 / 13.7, 12.7 / 9.1
//   2048 x 32000 30.5 / 33.2     128 x 131072  13.2 / 13.9, 12.9 / 12.0
//   64 x 66000   10.8 / 13.9, 8.0 / 7.5     192 x 131072  13.6 / 15.0, 13.4 / 14.6
//   64 x 100000  11.0 / 14.2, 10.6 / 8.4    255 x 131072  14.5 / 17.4, 14.5 / 17.4
//                                           512 x 131072  30.2 / 30.0
// (between some 150 and LP_ROWS long rows whole ones would be faster by up to a sixth).
constexpr int64_t LP_ROWS = 256, LP_BYTES = 131072;
inline bool whole_rows(int64_t rows, int64_t V, int FT) { return rows >= LP_ROWS || V * ftype_size(FT) <= LP_BYTES; }
constexpr int64_t LP_NO_WORKSPACE = 8192;    // whole rows forwards and held in one call, in every type

// Most workgroups per launch: a grid holds fewer than 2^32 threads.  Further rows
// are further launches.
constexpr int64_t LP_LAUNCH = 1 << 22;

struct Logp {
    const void* z;
    int64_t ldz, rows;
    int V;
    Tokens tok;
    Policy p;
    float s, c;
};

// The same for the rows from `first` on, at most `most` of them.
static Logp rows_from(const Logp& d, int FT, int64_t first, int64_t most)
{
    Logp r = d;
    r.z = forward_by(d.z, first * d.ldz * ftype_size(FT));
    r.tok.idx = forward_by(d.tok.idx, first * (d.tok.idx64 ? 8 : 4));
    r.p.adv = forward_by(d.p.adv, 4 * first);
    r.p.old = forward_by(d.p.old, 4 * first);
    r.p.ref = forward_by(d.p.ref, 4 * first);
    r.rows = std::min(d.rows - first, most);
    return r;
}

// Workspace: the parts' sums, then the logits at the tokens.
inline size_t logp_part_floats(int64_t rows, int64_t V)
{
    return 2 * (size_t)rows * (size_t)logp_split(rows, V).parts;
}

template <int FT>
static void parts_launch(const Logp& all, float* ws, hipStream_t st)
{
    const Split q = logp_split(all.rows, all.V);
    Sum* part = reinterpret_cast<Sum*>(ws);
    float* zy = ws + logp_part_floats(all.rows, all.V);
    const int64_t most = std::max<int64_t>(1, LP_LAUNCH / q.parts);
    for (int64_t r = 0; r < all.rows; r += most) {
        const Logp d = rows_from(all, FT, r, most);
        hipLaunchKernelGGL((k_logp_parts<FT>), dim3((unsigned)(d.rows * q.parts)), dim3(256), 0, st, d.z, d.ldz, d.V,
                           q.parts, q.len, d.tok, d.c, part + r * q.parts, zy + r);
    }
}

template <int FT>
static void forward_launch(const Logp& all, float* ws, float* loss, float* logp, float* stats, hipStream_t st)
{
    if (whole_rows(all.rows, all.V, FT)) {
        for (int64_t r = 0; r < all.rows; r += LP_LAUNCH / 4) {
            const Logp d = rows_from(all, FT, r, LP_LAUNCH / 4);
#define TQ_ROWS(NT)                                                                                                  \
    hipLaunchKernelGGL((k_logp_rows<FT, NT>), dim3((unsigned)d.rows), dim3(NT), 0, st, d.z, d.ldz, d.V, d.tok, d.p,   \
                       d.s, d.c, forward_by(loss, 4 * r), logp + r, forward_by(stats, 8 * r))
            if (d.V <= 8192) TQ_ROWS(256);
            else TQ_ROWS(1024);
#undef TQ_ROWS
        }
        return;
    }
    parts_launch<FT>(all, ws, st);
    hipLaunchKernelGGL(k_logp_join, dim3((unsigned)cdiv(all.rows, 4)), dim3(256), 0, st, all.rows, all.V, all.tok, all.p,
                       all.s, all.c, reinterpret_cast<const Sum*>(ws), ws + logp_part_floats(all.rows, all.V),
                       logp_split(all.rows, all.V).parts, loss, logp, stats);
}

template <int FT, bool FROM_PARTS>
static void grad_launch(const Logp& all, const float* ws, const float* stats, const float* dloss, float* loss,
                        float* logp, void* dz, int64_t lddz, hipStream_t st)
{
    const Split q = logp_split(all.rows, all.V);
    const Sum* part = reinterpret_cast<const Sum*>(ws);
    const float* zy = FROM_PARTS ? ws + logp_part_floats(all.rows, all.V) : nullptr;
    const int64_t most = std::max<int64_t>(1, LP_LAUNCH / q.parts);
    for (int64_t r = 0; r < all.rows; r += most) {
        const Logp d = rows_from(all, FT, r, most);
        hipLaunchKernelGGL((k_logp_grad<FT, FROM_PARTS>), dim3((unsigned)(d.rows * q.parts)), dim3(256), 0, st, d.z,
                           d.ldz, d.V, q.parts, q.len, d.tok, d.p, d.s, d.c, FROM_PARTS ? part + r * q.parts : nullptr,
                           forward_by(zy, 4 * r), forward_by(stats, 8 * r), forward_by(dloss, 4 * r),
                           forward_by(loss, 4 * r), forward_by(logp, 4 * r),
                           forward_by(dz, r * lddz * ftype_size(FT)), lddz);
    }
}

// Whether the joint call holds its rows in registers (see distillation, whose rows
// cost the same): of 64 KB at any number of them; of 128 KB from LP_HELD_ROWS of them
// on; of 256 KB, which take a CU each, where they fill at least 5/8 of their rounds
// over the CUs (binary32 7/8 of at least two rounds).
constexpr int64_t LP_HELD_ROWS = 128;
template <int FT>
static bool held_launch(const Logp& d, const float* dloss, float* loss, float* logp, void* dz, int64_t lddz,
                        hipStream_t st)
{
    constexpr int H = FT == F32 ? 2 : 1;  // binary32 rows hold half as many elements
    if (d.V < 8 || d.V > 131072 / H) return false;
    if (d.V > 65536 / H) {
        const int64_t rounds = std::max<int64_t>(H, cdiv(d.rows, 256));
        if (8 * d.rows < (H == 2 ? 7 : 5) * 256 * rounds) return false;
    } else if (d.V > 32768 / H && d.rows < LP_HELD_ROWS) {
        return false;
    }
    // as many workgroups as fit on the chip by their registers
#define TQ_HELD(NT, W)                                                                                             \
    hipLaunchKernelGGL((k_policy_held<FT, NT, W>), dim3((unsigned)std::min<int64_t>(d.rows, 256 * (1024 / NT) *    \
                       (W * (FT == F32 ? 2 : 1) <= 8 ? 2 : 1))), dim3(NT), 0, st, d.z, d.ldz, (uint32_t)d.rows, d.V,  \
                       d.tok, d.p, d.s, d.c, dloss, loss, logp, dz, lddz)
    if (d.V <= 8192) TQ_HELD(256, 4);
    else if (d.V <= 32768 / H) TQ_HELD(256, 16 / H);
    else if (d.V <= 65536 / H) TQ_HELD(512, 16 / H);
    else TQ_HELD(1024, 16 / H);
#undef TQ_HELD
    return true;
}

static bool natural(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Checks what the calls share and fills `d`; *work is false where there is nothing
// to do.
static tq_status logp_check(const void* logits, int dt, int64_t rows, int64_t vocab, int64_t ldz, const void* token,
                            int idx_bits, float temperature, Logp* d, bool* work)
{
    *work = false;
    if (!valid_ftype(dt) || (idx_bits != 32 && idx_bits != 64) || rows < 0 || vocab < 0) return TQ_ERR_INVALID;
    if (!(temperature >= 1e-38f) || temperature > 3.0e38f) return TQ_ERR_INVALID;    // s and c are finite
    if (rows == 0) return TQ_OK;
    if (vocab == 0 || !logits || ldz < vocab || !token) return TQ_ERR_INVALID;
    if (vocab > 0x7fffff00 || rows > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    if (!natural(logits, ftype_size(dt)) || !natural(token, idx_bits / 8)) return TQ_ERR_ALIGN;
    *d = Logp{logits, ldz, rows, (int)vocab, {token, idx_bits == 64}, {}, (float)(1.0 / (double)temperature),
              (float)(1.4426950408889634 / (double)temperature)};
    *work = true;
    return TQ_OK;
}

static tq_status policy_check(const float* advantage, const float* old_logp, const float* ref_logp, float clip_low,
                              float clip_high, float kl_coef, Logp* d, bool work)
{
    if (!(clip_low >= 0.0f && clip_low <= 1.0f) || !(clip_high >= 0.0f) || !(kl_coef >= 0.0f) || kl_coef > 3.0e38f)
        return TQ_ERR_INVALID;
    if (!work) return TQ_OK;
    if (!advantage) return TQ_ERR_INVALID;
    if (!natural(advantage, 4) || !natural(old_logp, 4) || !natural(ref_logp, 4)) return TQ_ERR_ALIGN;
    d->p = Policy{advantage, old_logp, kl_coef > 0.0f ? ref_logp : nullptr, clip_low, clip_high, kl_coef};
    return TQ_OK;
}

static tq_status workspace_check(const void* ws, size_t have, int64_t rows, int64_t vocab)
{
    const size_t need = tq_policy_loss_workspace_bytes(rows, vocab);
    if (need == 0) return TQ_OK;
    if (!ws || have < need) return TQ_ERR_INVALID;
    return aligned16(ws) ? TQ_OK : TQ_ERR_ALIGN;
}

}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_policy_loss_workspace_bytes(int64_t rows, int64_t vocab)
{
    if (rows <= 0 || vocab <= 0 || (vocab <= LP_NO_WORKSPACE && vocab >= 8)) return 0;
    return (logp_part_floats(rows, vocab) + (size_t)rows) * sizeof(float);
}

tq_status tq_token_logp(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                        const void* token, int idx_bits, float temperature, float* logp, float* stats, void* workspace,
                        size_t workspace_bytes, void* stream)
{
    Logp d;
    bool work;
    tq_status r = logp_check(logits, dtype, rows, vocab, row_stride, token, idx_bits, temperature, &d, &work);
    if (r != TQ_OK || !work) return r;
    if (!logp) return TQ_ERR_INVALID;
    if (!natural(logp, 4) || !natural(stats, 4)) return TQ_ERR_ALIGN;
    if ((r = workspace_check(workspace, workspace_bytes, rows, vocab)) != TQ_OK) return r;
    TQ_LLM_FT_SWITCH(dtype, forward_launch<FTV>(d, static_cast<float*>(workspace), nullptr, logp, stats,
                                                as_stream(stream)));
    return launch_status();
}

tq_status tq_token_logp_backward(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                 const void* token, int idx_bits, float temperature, const float* stats,
                                 const float* dlogp, void* dlogits, int64_t d_row_stride, void* stream)
{
    Logp d;
    bool work;
    const tq_status r = logp_check(logits, dtype, rows, vocab, row_stride, token, idx_bits, temperature, &d, &work);
    if (r != TQ_OK || !work) return r;
    if (!stats || !dlogits || d_row_stride < vocab) return TQ_ERR_INVALID;
    if (!natural(stats, 4) || !natural(dlogp, 4) || !natural(dlogits, ftype_size(dtype))) return TQ_ERR_ALIGN;
    TQ_LLM_FT_SWITCH(dtype, (grad_launch<FTV, false>(d, nullptr, stats, dlogp, nullptr, nullptr, dlogits, d_row_stride,
                                                     as_stream(stream))));
    return launch_status();
}

tq_status tq_policy_loss(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                         const void* token, int idx_bits, const float* advantage, const float* old_logp,
                         const float* ref_logp, float clip_low, float clip_high, float kl_coef, float temperature,
                         float* loss, float* logp, float* stats, void* workspace, size_t workspace_bytes, void* stream)
{
    Logp d;
    bool work;
    tq_status r = logp_check(logits, dtype, rows, vocab, row_stride, token, idx_bits, temperature, &d, &work);
    if (r == TQ_OK) r = policy_check(advantage, old_logp, ref_logp, clip_low, clip_high, kl_coef, &d, work);
    if (r != TQ_OK || !work) return r;
    if (!loss || !logp) return TQ_ERR_INVALID;
    if (!natural(loss, 4) || !natural(logp, 4) || !natural(stats, 4)) return TQ_ERR_ALIGN;
    if ((r = workspace_check(workspace, workspace_bytes, rows, vocab)) != TQ_OK) return r;
    TQ_LLM_FT_SWITCH(dtype, forward_launch<FTV>(d, static_cast<float*>(workspace), loss, logp, stats,
                                                as_stream(stream)));
    return launch_status();
}

tq_status tq_policy_loss_backward(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                  const void* token, int idx_bits, const float* advantage, const float* old_logp,
                                  const float* ref_logp, float clip_low, float clip_high, float kl_coef,
                                  float temperature, const float* logp, const float* stats, const float* dloss,
                                  void* dlogits, int64_t d_row_stride, void* stream)
{
    Logp d;
    bool work;
    tq_status r = logp_check(logits, dtype, rows, vocab, row_stride, token, idx_bits, temperature, &d, &work);
    if (r == TQ_OK) r = policy_check(advantage, old_logp, ref_logp, clip_low, clip_high, kl_coef, &d, work);
    if (r != TQ_OK || !work) return r;
    if (!logp || !stats || !dlogits || d_row_stride < vocab) return TQ_ERR_INVALID;
    if (!natural(logp, 4) || !natural(stats, 4) || !natural(dloss, 4) || !natural(dlogits, ftype_size(dtype)))
        return TQ_ERR_ALIGN;
    TQ_LLM_FT_SWITCH(dtype, (grad_launch<FTV, false>(d, nullptr, stats, dloss, nullptr, const_cast<float*>(logp),
                                                     dlogits, d_row_stride, as_stream(stream))));
    return launch_status();
}

tq_status tq_policy_loss_grad(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                              const void* token, int idx_bits, const float* advantage, const float* old_logp,
                              const float* ref_logp, float clip_low, float clip_high, float kl_coef, float temperature,
                              const float* dloss, float* loss, float* logp, void* dlogits, int64_t d_row_stride,
                              void* workspace, size_t workspace_bytes, void* stream)
{
    Logp d;
    bool work;
    tq_status r = logp_check(logits, dtype, rows, vocab, row_stride, token, idx_bits, temperature, &d, &work);
    if (r == TQ_OK) r = policy_check(advantage, old_logp, ref_logp, clip_low, clip_high, kl_coef, &d, work);
    if (r != TQ_OK || !work) return r;
    if (!loss || !logp || !dlogits || d_row_stride < vocab) return TQ_ERR_INVALID;
    if (!natural(loss, 4) || !natural(logp, 4) || !natural(dloss, 4) || !natural(dlogits, ftype_size(dtype)))
        return TQ_ERR_ALIGN;
    if ((r = workspace_check(workspace, workspace_bytes, rows, vocab)) != TQ_OK) return r;
    float* ws = static_cast<float*>(workspace);
    hipStream_t st = as_stream(stream);
    TQ_LLM_FT_SWITCH(dtype, {
        if (!held_launch<FTV>(d, dloss, loss, logp, dlogits, d_row_stride, st)) {
            parts_launch<FTV>(d, ws, st);
            grad_launch<FTV, true>(d, ws, nullptr, dloss, loss, logp, dlogits, d_row_stride, st);
        }
    });
    return launch_status();
}

}  // extern "C"
