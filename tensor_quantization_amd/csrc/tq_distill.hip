// tq_distill.hip -- distillation of a student from its teacher's top logits:
// the loss of every row, its gradient, and both in one call.
//
//   s = 1 / T;  entry k of a row is (i_k, t_k), a padding entry when i_k lies
//   outside [0, V);  log q_j = s z_j - lse(s z)
//   without the teacher's normaliser: p = softmax(s t) over the row's entries,
//     L = sum_k p_k (log p_k - log q_{i_k}),  dL/dz_j = s (q_j - sum_{i_k = j} p_k)
//   with it (log-sum-exp of all the teacher's s t): p_k = exp(s t_k - teacher_lse),
//     p_r = max(0, 1 - sum p), q_r = the student's mass outside the entries,
//     L gains p_r (log p_r - log q_r), and with Z = sum p + p_r
//     dL/dz_j = s (q_j Z - p_j) for an entry's j, s q_j (Z - p_r / q_r) elsewhere.
//   A row without entries has loss 0 and gradient 0.
//
// q_r is summed over the entries' complement, not taken as 1 - sum q, which
// would lose it where the student agrees with the teacher, and relative to the
// complement's own largest logit m_r: relative to the row's it would vanish
// where every other logit lies 87 T below an entry's (a confident student, a
// mask of large finite values).  So the row's sum S, relative to its largest
// logit m, is joined from the complement's R and the entries' own, and
//   log q_r = s (m_r - m) + log R - log S,
//   dL/dz_j = s e_j (Z 2^((m_r - m) c) / S - p_r / R), e_j = 2^((z_j - m_r) c)
// outside the entries (c = s log2 e).  To know which
// columns are entries, a workgroup keeps one bit per column of its part of the
// row in LDS; the gradient finds an entry's probability by the rank of its bit
// (a prefix count per 32-column word, then the bits below it), so each element
// is written once, in order, with no scatter afterwards.
//
// All sums are binary32, relative to the largest of what they add.  Every kernel is
// bound by HBM: the loss reads the logits once, the gradient reads them and
// writes as much; in one call the row is held in registers between the two.
#include "tq_llm.h"

namespace tq {

constexpr int DT_K = 1024;               // most entries per row

struct Entries {
    const void* idx;
    int idx64;
    const void* val;
    int val_dt;
    int K;
    const float* tlse;                   // null: the probabilities are normalised over the entries
};

// Entry k's column, or -1 for a padding entry.
__device__ __forceinline__ int entry_col(const Entries& e, int64_t row, int k, int V)
{
    const int64_t at = row * e.K + k;
    const int64_t i = e.idx64 ? static_cast<const int64_t*>(e.idx)[at] : static_cast<const int32_t*>(e.idx)[at];
    return i >= 0 && i < V ? (int)i : -1;
}
__device__ __forceinline__ float entry_val(const Entries& e, int64_t row, int k)
{
    return load1_rt(e.val, e.val_dt, row * e.K + k, 0.0f);
}

// A row's entries, read once into LDS by the NT threads of a workgroup.
struct EntryList {
    int col[DT_K];
    float val[DT_K];
};
template <int NT>
__device__ __forceinline__ void load_entries(EntryList& l, const Entries& e, int64_t row, int V)
{
#pragma unroll 1
    for (int i = threadIdx.x; i < e.K; i += NT) {
        l.col[i] = entry_col(e, row, i, V);
        l.val[i] = entry_val(e, row, i);
    }
}

// 2^x by the exponential unit (x of a probability, at most 0 up to rounding;
// results below 2^-126 are flushed, far under any sum they join: each sum's
// largest term is about 1).
__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float lg2(float x) { return __builtin_amdgcn_logf(x); }

// The logit that a row's exponentials are taken relative to.
__device__ __forceinline__ float base_of(float m) { return m == -__builtin_inff() ? 0.0f : m; }

// What a row's gradient needs: dL/dz_j = e_j in - sg p_j at entries, e_j out
// elsewhere, e_j the exponential relative to the row's and to the complement's
// base; the sums' reciprocals are folded into `in` and `out`.
struct Coef {
    float in, out, sg, tm, ti;
    bool some;
};

__device__ __forceinline__ float entry_p(const Entries& e, const Coef& q, float t, float s, float c)
{
    return e.tlse ? ex2((t * s - q.tm) * LOG2E) : ex2((t - q.tm) * c) * q.ti;
}

// The coefficients from the student's sums S and R, the ratio of their bases
// up = 2^((m_r - m) c) (without the normaliser 1, and R unused), the teacher's base
// tm and sum (`tsum`: of 2^((t - tm) c) without, of p with the normaliser) and
// whether the row has entries at all.
__device__ __forceinline__ Coef make_coef(bool rest, bool some, float S, float R, float up, float tm, float tsum,
                                          float s, float g, float* p_rest)
{
    Coef q;
    q.some = some;
    q.sg = s * g;
    q.tm = tm;
    q.ti = rest ? 1.0f : 1.0f / tsum;
    const float pr = rest && some ? __builtin_fmaxf(0.0f, 1.0f - tsum) : 0.0f;
    const float Z = rest ? tsum + pr : 1.0f;
    const float is = S == 0.0f ? 0.0f : 1.0f / S;    // a row of -inf logits has no gradient
    q.in = q.sg * Z * is;
    q.out = rest ? q.sg * (Z * is * up - (R == 0.0f ? 0.0f : pr / R)) : q.in;    // R = 0: no such exponential
    if (S == 0.0f) {
        q.out = 0.0f;
        q.sg = 0.0f;
    }
    *p_rest = pr;
    return q;
}

// Entry k's part of the loss; lgS is log2 of the student's sum relative to m.
__device__ __forceinline__ float entry_loss(const Entries& e, float t, float z, float s, float c, float tm, float tsum,
                                            float m, float S, float lgS)
{
    const float logp = e.tlse ? (t * s - tm) : ((t - tm) * s - lg2(tsum) * LN2);
    const float p = e.tlse ? ex2(logp * LOG2E) : ex2((t - tm) * c) / tsum;
    if (p == 0.0f) return 0.0f;
    if (S == 0.0f) return __builtin_inff();
    return p * (logp - ((z - base_of(m)) * s - lgS * LN2));
}
// The rest's, `above` = s (m_r - m).
__device__ __forceinline__ float rest_loss(float pr, float R, float S, float above)
{
    if (pr == 0.0f) return 0.0f;
    return S == 0.0f ? __builtin_inff() : pr * ((lg2(pr) - (lg2(R) - lg2(S))) * LN2 - above);
}

// The sum of 2^((z - m) c) over some columns, m the largest z of them (or of more).
struct Part {
    float m, sum;
};
__device__ __forceinline__ float part_at(const Part& a, float base, float c)
{
    return a.sum * ex2((a.m - base) * c);    // m = -inf: 0
}
__device__ __forceinline__ Part join(const Part& a, const Part& b, float c)
{
    const float m = __builtin_fmaxf(a.m, b.m), base = base_of(m);
    return Part{m, part_at(a, base, c) + part_at(b, base, c)};
}
__device__ __forceinline__ Part wave_join(const Part& a, float c)
{
    const float m = wave_max(a.m);
    return Part{m, wave_sum(part_at(a, base_of(m), c))};
}

// ------------------------------------------------------------ entry columns
// One bit per column of the workgroup's part of the row, a count of the bits
// before each word, and the entries' values by rank.
template <int NT, int WORDS>
struct Marks {
    uint32_t bits[WORDS];
    uint16_t before[WORDS];
    float value[DT_K];
    int waves[NT / 64];
    int twice;
};

template <int NT, int WORDS>
__device__ __forceinline__ void marks_clear(Marks<NT, WORDS>& k)
{
    for (int i = threadIdx.x; i < WORDS; i += NT) k.bits[i] = 0;
    if (threadIdx.x == 0) k.twice = 0;
}

// Marks column `at` (relative to the part).
template <int NT, int WORDS>
__device__ __forceinline__ void mark(Marks<NT, WORDS>& k, int at)
{
    const uint32_t bit = 1u << (at & 31);
    if (atomicOr(&k.bits[at >> 5], bit) & bit) k.twice = 1;
}

// The eight bits of columns at .. at + 7.
template <int NT, int WORDS>
__device__ __forceinline__ uint32_t marks8(const Marks<NT, WORDS>& k, int at)
{
    const uint8_t* b = reinterpret_cast<const uint8_t*>(k.bits);
    uint32_t m = b[at >> 3];
    if (at & 7) m = (m | (uint32_t)b[(at >> 3) + 1] << 8) >> (at & 7) & 0xffu;
    return m;
}

template <int NT, int WORDS>
__device__ __forceinline__ int rank_of(const Marks<NT, WORDS>& k, int at)
{
    return k.before[at >> 5] + __popc(k.bits[at >> 5] & ((1u << (at & 31)) - 1));
}

// Counts the bits before every word (after a barrier behind the marking;
// contains one barrier, and needs one before the ranks are used).
template <int NT, int WORDS>
__device__ __forceinline__ void marks_count(Marks<NT, WORDS>& k)
{
    constexpr int PER = (WORDS + NT - 1) / NT;
    const int t = afresh((int)threadIdx.x), first = t * PER;
    int n = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (first + i < WORDS) n += __popc(k.bits[first + i]);
    int upto = n;                        // over this lane and those before it
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __builtin_amdgcn_ds_bpermute((t - d) << 2, upto);
        if ((t & 63) >= d) upto += o;
    }
    if ((t & 63) == 63) k.waves[t >> 6] = upto;
    __syncthreads();
    int at = upto - n;
#pragma unroll 1
    for (int w = 0; w < (t >> 6); ++w) at += k.waves[w];
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (first + i < WORDS) {
            k.before[first + i] = (uint16_t)at;
            at += __popc(k.bits[first + i]);
        }
}

// Writes every entry's sg p to its rank.  Entries of one column (a row should
// not have any) are added in entry order by one thread.
template <int NT, int WORDS>
__device__ __forceinline__ void marks_fill(Marks<NT, WORDS>& k, const EntryList& l, const Entries& e, const Coef& q,
                                           int c0, int n, float s, float c)
{
    const int t = threadIdx.x;
    if (!k.twice) {
#pragma unroll 1
        for (int i = t; i < e.K; i += NT) {
            const int col = l.col[i] - c0;
            if (l.col[i] >= 0 && col >= 0 && col < n) k.value[rank_of(k, col)] = q.sg * entry_p(e, q, l.val[i], s, c);
        }
    } else {
#pragma unroll 1
        for (int r = t; r < e.K; r += NT) {
            float v = 0.0f;
#pragma unroll 1
            for (int i = 0; i < e.K; ++i) {
                const int col = l.col[i] - c0;
                if (l.col[i] >= 0 && col >= 0 && col < n && rank_of(k, col) == r)
                    v += q.sg * entry_p(e, q, l.val[i], s, c);
            }
            k.value[r] = v;
        }
    }
}

// The gradient of eight elements, out(z) and in(z) the exponentials outside and
// at entries.  Entries are few: the loop over their bits is rolled, and picks its
// element by selects.
template <int NT, int WORDS, class X, class Y>
__device__ __forceinline__ void grad8(const Marks<NT, WORDS>& k, const Coef& q, int at, float v[8], X out, Y in)
{
    uint32_t m = marks8(k, at);
    float z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        z[i] = v[i];
        v[i] = out(v[i]) * q.out;
    }
#pragma unroll 1
    while (m) {
        const int b = __ffs(m) - 1;
        m &= m - 1;
        float g = z[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) g = b == i ? z[i] : g;
        g = in(g) * q.in - k.value[rank_of(k, at + b)];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = b == i ? g : v[i];
    }
}

// --------------------------------------------------------------- statistics
// k_distill_stats: a workgroup per row and part of the row (`len` columns, at
// most CH): the largest logit m of the part's columns and the sum of 2^((z - m) c)
// over them, with REST one pair over the columns that are no entries and one over
// those that are, and the logits at its entries, zk [rows, K] (for the loss,
// which may be taken after the gradient has overwritten the logits).  A thread
// keeps its own running maximum and sum, rescaled when a vector of eight exceeds
// it, so a part is one pass with no barrier before the end; the entries' pair
// comes from zk.  Bound by HBM: [512, 32000] f32 12.9 us (5.1 TB/s).
template <int FT, bool REST, int CH>
__global__ __launch_bounds__(256) void k_distill_stats(const void* __restrict__ z, int64_t ldz, int V, int parts,
                                                       int len, Entries ent, float c, float4* __restrict__ part,
                                                       float* __restrict__ zk)
{
    constexpr int U = 4;
    __shared__ uint32_t bits[REST ? CH / 32 + 1 : 1];
    __shared__ Part red[4][2];
    __shared__ int twice;
    const int t = threadIdx.x;
    const int64_t row = blockIdx.x / (unsigned)parts;
    const int p = (int)(blockIdx.x % (unsigned)parts), c0 = p * len;
    const int n = V - c0 < len ? V - c0 : len, nvec = (n + 7) / 8;
    const int64_t base = row * ldz + c0;
    if constexpr (REST) {
        for (int i = t; i < CH / 32 + 1; i += 256) bits[i] = 0;
        if (t == 0) twice = 0;
        __syncthreads();
    }
    constexpr int KT = DT_K / 256;
    float ze[KT];                        // the logits at this thread's entries t, t + 256, ...
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        ze[i] = -__builtin_inff();
        const int k = t + 256 * i;
        if (k >= ent.K) continue;
        const int all = entry_col(ent, row, k, V), col = all - c0;
        if (all >= 0 && col >= 0 && col < n) {
            ze[i] = load1<FT>(z, base + col);
            zk[row * ent.K + k] = ze[i];
            if constexpr (REST)
                if (atomicOr(&bits[col >> 5], 1u << (col & 31)) >> (col & 31) & 1) twice = 1;
        }
    }
    if constexpr (REST) __syncthreads();
    Part out = {-__builtin_inff(), 0.0f}, in = out;
    // adds a vector's own elements, with REST those that are no entries
    auto add = [&](float v[8], int lo, uint32_t mask) {
        if constexpr (REST) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = mask >> i & 1 ? -__builtin_inff() : v[i];
        }
        float top = v[0];
#pragma unroll
        for (int i = 1; i < 8; ++i) top = __builtin_fmaxf(top, v[i]);
        if (top > out.m) {
            out.sum *= ex2((out.m - top) * c);    // m = -inf: 0
            out.m = top;
        }
        const float b = base_of(out.m);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float x = ex2((v[i] - b) * c);
            sum += i >= lo ? x : 0.0f;
        }
        out.sum += sum;
    };
    if (n >= 8) {
        for (int v0 = t; v0 < nvec; v0 += 256 * U) {
            Raw8<FT> raw[U];
            Vec8 at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                at[u] = vec8(v0 + 256 * u, n);
                raw[u] = load8_any<FT>(z, base + at[u].at);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (at[u].lo == 8) continue;
                float v[8];
                widen8<FT>(raw[u], v);
                uint32_t mask = 0;
                if constexpr (REST) {
                    const uint8_t* b = reinterpret_cast<const uint8_t*>(bits);
                    mask = b[at[u].at >> 3];
                    if (at[u].at & 7) mask = (mask | (uint32_t)b[(at[u].at >> 3) + 1] << 8) >> (at[u].at & 7) & 0xffu;
                }
                add(v, at[u].lo, mask);
            }
        }
    } else if (t < n) {
        float v[8];
        v[0] = load1<FT>(z, base + t);
#pragma unroll
        for (int i = 1; i < 8; ++i) v[i] = -__builtin_inff();
        // the seven other places hold nothing: their exponentials are zeros
        add(v, 0, REST ? bits[0] >> t & 1 : 0);
    }
    if constexpr (REST) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int k = t + 256 * i;
            bool count = k < ent.K;
            if (twice && count)          // a column counts once, by the first of its entries
                for (int j = 0; j < k; ++j) count = count && entry_col(ent, row, j, V) != entry_col(ent, row, k, V);
            if (count) in = join(in, Part{ze[i], 1.0f}, c);
        }
        in = wave_join(in, c);
    }
    out = wave_join(out, c);
    if ((t & 63) == 0) {
        red[t >> 6][0] = out;
        red[t >> 6][1] = in;
    }
    __syncthreads();
    if (t != 0) return;
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        if (o && !REST) continue;
        Part& all = o ? in : out;
        const float m = __builtin_fmaxf(__builtin_fmaxf(red[0][o].m, red[1][o].m),
                                        __builtin_fmaxf(red[2][o].m, red[3][o].m));
        all = Part{m, 0.0f};
#pragma unroll
        for (int w = 0; w < 4; ++w) all.sum += part_at(red[w][o], base_of(m), c);
    }
    part[row * parts + p] = make_float4(out.m, out.sum, in.m, in.sum);
}

// k_distill_rows: a wave per row joins the row's parts and writes the loss and
// the row's statistics: stats[row] = {largest logit, sum of exp(s (z - it))},
// rest_sum[row] the same pair over the columns outside the entries.  A launch's
// latency (4.3 us), whatever the rows.
__global__ __launch_bounds__(256) void k_distill_rows(int64_t rows, int V, Entries ent, float s, float c,
                                                      const float4* __restrict__ part, const float* __restrict__ zk,
                                                      int parts, float* __restrict__ loss, float* __restrict__ stats,
                                                      float* __restrict__ rest_sum)
{
    const int lane = threadIdx.x & 63;
    const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (row >= rows) return;
    const bool rest = ent.tlse != nullptr;
    Part out = {-__builtin_inff(), 0.0f}, in = out;
    for (int i = lane; i < parts; i += 64) {
        const float4 of = part[row * parts + i];
        out = join(out, Part{of.x, of.y}, c);
        in = join(in, Part{of.z, of.w}, c);
    }
    // the teacher
    float tm = -__builtin_inff(), tsum = 0.0f;
    bool some = false;
    for (int k = lane; k < ent.K; k += 64)
        if (entry_col(ent, row, k, V) >= 0) {
            some = true;
            tm = __builtin_fmaxf(tm, entry_val(ent, row, k));
        }
    out = wave_join(out, c);
    in = wave_join(in, c);
    const Part all = join(out, in, c);
    const float m = all.m, S = all.sum, R = out.sum;
    some = __any(some);
    tm = rest ? ent.tlse[row] : base_of(wave_max(tm));
    for (int k = lane; k < ent.K; k += 64)
        if (entry_col(ent, row, k, V) >= 0) {
            const float t = entry_val(ent, row, k);
            tsum += rest ? ex2((t * s - tm) * LOG2E) : ex2((t - tm) * c);
        }
    tsum = wave_sum(tsum);
    if (!rest && tsum == 0.0f) some = false;      // every entry at -inf
    float l = 0.0f;
    if (some)
        for (int k = lane; k < ent.K; k += 64)
            if (entry_col(ent, row, k, V) >= 0)
                l += entry_loss(ent, entry_val(ent, row, k), zk[row * ent.K + k], s, c, tm, tsum, m, S, lg2(S));
    l = wave_sum(l);
    if (lane != 0) return;
    float pr;
    make_coef(rest, some, S, R, 1.0f, tm, tsum, s, 1.0f, &pr);
    loss[row] = some ? l + rest_loss(pr, R, S, (out.m - base_of(m)) * s) : 0.0f;
    if (stats) {
        stats[2 * row] = m;
        stats[2 * row + 1] = S;
    }
    if (rest_sum) {
        rest_sum[2 * row] = out.m;
        rest_sum[2 * row + 1] = R;
    }
}

// k_distill_grad: a workgroup per row and part of the row.  Every workgroup
// derives the row's coefficients itself, from the parts' statistics
// (FROM_PARTS; the row's first workgroup writes the loss too) or from saved
// ones, while its first vectors are under way: that costs a few hundred
// operations per workgroup and saves a launch (9 rows of 131001 f16 loss and
// gradient 15.8 us, 18.6 with one; 40 / 43 for [512, 32000] f32 forwards and
// back).  Bound by HBM: [512, 32000] f32 23.4 us (5.6 TB/s).
template <int FT, int CH, bool FROM_PARTS>
__global__ __launch_bounds__(256) void k_distill_grad(const void* z, int64_t ldz, int V, int parts, int len,
                                                      Entries ent, float s, float c, const float4* __restrict__ part,
                                                      const float* __restrict__ zk, const float* __restrict__ stats,
                                                      const float* __restrict__ rest_sum,
                                                      const float* __restrict__ dloss, float* __restrict__ loss,
                                                      void* dz, int64_t lddz)
{
    constexpr int U = 2;
    __shared__ Marks<256, CH / 32 + 1> k;
    __shared__ EntryList list;
    __shared__ float red[7][4];
    __shared__ int any;
    const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
    const int64_t row = blockIdx.x / (unsigned)parts;
    const int p = (int)(blockIdx.x % (unsigned)parts), c0 = p * len;
    const int n = V - c0 < len ? V - c0 : len, nvec = (n + 7) / 8;
    const int64_t from = row * ldz + c0, to = row * lddz + c0;
    const bool rest = ent.tlse != nullptr;
    Raw8<FT> raw[U];
    auto fetch = [&](int v0) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u] = load8_any<FT>(z, from + vec8(v0 + 256 * u, n).at);
    };
    if (n >= 8) fetch(t);

    // everything from memory is asked for ahead of the first barrier
    if (t == 0) any = 0;
    marks_clear(k);
    load_entries<256>(list, ent, row, V);
    const float lse = rest ? ent.tlse[row] : 0.0f, g = dloss ? dloss[row] : 1.0f;
    Part out = {-__builtin_inff(), 0.0f}, in = out, all = out;   // columns outside the entries, entries, the row
    if constexpr (FROM_PARTS) {
        for (int i = t; i < parts; i += 256) {
            const float4 of = part[row * parts + i];
            out = join(out, Part{of.x, of.y}, c);
            in = join(in, Part{of.z, of.w}, c);
        }
    } else {
        all = Part{stats[2 * row], stats[2 * row + 1]};
        out = rest ? Part{rest_sum[2 * row], rest_sum[2 * row + 1]} : all;
    }
    const float zk0 = FROM_PARTS && p == 0 && t < ent.K ? zk[row * ent.K + t] : 0.0f;
    __syncthreads();
    float tm = -__builtin_inff();
    for (int i = t; i < ent.K; i += 256) {
        if (list.col[i] < 0) continue;
        any = 1;
        tm = __builtin_fmaxf(tm, list.val[i]);
        const int col = list.col[i] - c0;
        if (col >= 0 && col < n) mark(k, col);
    }
    auto four = [&](int i) { return lane < 4 ? red[i][lane] : 0.0f; };
    auto top = [&](int i) { return wave_max(lane < 4 ? red[i][lane] : -__builtin_inff()); };
    tm = wave_max(tm);
    if constexpr (FROM_PARTS) {
        const float mo = wave_max(out.m), mi = wave_max(in.m);
        if (lane == 0) {
            red[1][wave] = mo;
            red[6][wave] = mi;
        }
    }
    if (lane == 0) red[0][wave] = tm;
    __syncthreads();
    tm = rest ? lse : base_of(top(0));
    float tsum = 0.0f;
    if constexpr (FROM_PARTS) {
        const float mo = top(1), mi = top(6);
        out = Part{mo, wave_sum(part_at(out, base_of(mo), c))};
        in = Part{mi, wave_sum(part_at(in, base_of(mi), c))};
    }
    for (int i = t; i < ent.K; i += 256)
        if (list.col[i] >= 0) tsum += rest ? ex2((list.val[i] * s - tm) * LOG2E) : ex2((list.val[i] - tm) * c);
    tsum = wave_sum(tsum);
    if (lane == 0) {
        red[2][wave] = tsum;
        red[3][wave] = out.sum;
        red[4][wave] = in.sum;
    }
    marks_count(k);                      // its barrier also publishes the sums
    __syncthreads();
    tsum = wave_sum(four(2));
    if constexpr (FROM_PARTS) {
        out.sum = wave_sum(four(3));
        in.sum = wave_sum(four(4));
        all = join(out, in, c);
    }
    const float S = all.sum, R = out.sum, mi = base_of(all.m), mo = base_of(out.m);
    const bool some = any && (rest || tsum != 0.0f);
    float pr;
    const Coef q = make_coef(rest, some, S, R, rest ? ex2((out.m - mi) * c) : 1.0f, tm, tsum, s, g, &pr);
    if (FROM_PARTS && p == 0) {          // uniform
        float l = 0.0f;
        for (int i = t; i < (some ? ent.K : 0); i += 256)
            if (list.col[i] >= 0)
                l += entry_loss(ent, list.val[i], i < 256 ? zk0 : zk[row * ent.K + i], s, c, tm, tsum, all.m, S, lg2(S));
        l = wave_sum(l);
        if (lane == 0) red[5][wave] = l;
        __syncthreads();
        l = wave_sum(four(5));
        if (t == 0) loss[row] = some ? l + rest_loss(pr, R, S, (out.m - mi) * s) : 0.0f;
    }
    if (!some) {                         // uniform: no entries, no gradient
        for (int j = t; j < n; j += 256) store1<FT>(dz, to + j, 0.0f);
        return;
    }
    marks_fill(k, list, ent, q, c0, n, s, c);
    __syncthreads();
    auto xo = [&](float v) { return ex2((v - mo) * c); };
    auto xi = [&](float v) { return ex2((v - mi) * c); };
    if (n < 8) {
        if (t < n) {
            float v[8] = {load1<FT>(z, from + t), 0, 0, 0, 0, 0, 0, 0};
            grad8(k, q, t, v, xo, xi);
            store1<FT>(dz, to + t, v[0]);
        }
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
            grad8(k, q, at.at, v, xo, xi);
            store8_own<FT>(dz, to, at, v);
        }
    }
}

// k_distill_held: loss and gradient of a row in one read: NT threads hold the
// row (8 <= V <= 8 NT W) in registers in its own type.  The entries are marked
// while the loads are under way, and every vector's exponentials are summed as
// it arrives, so that only the gradient's own arithmetic follows the last load.
// For that a wave takes its exponentials relative to the largest logit m outside
// the entries in its first vector instead of the row's, as 2^(z c - mc) with one
// rounding, where mc is m c rounded.  That rounding grows with |m| and differs
// from wave to wave, so whatever meets these sums knows it: the waves are joined
// by 2^(mc - mc'), the gradient's exponentials take the same mc, and the loss,
// which needs log2 S relative to m itself, subtracts m c - mc.  A factor
// 2^(mc - mc') below 2^-126 comes out as 0, which a wave's sum survives only while
// it is small: one of 2^96 or more counts as infinite.  Then such sums lose nothing
// (a share of 2^-30, one in 2^26 of the row's at most, over sixteen waves) unless they
// overflow (a logit more than 66 / s above a wave's m), m c does, or the complement's
// comes out below its largest term's 1 (no logit above -inf where a wave looks first);
// then the complement and the entries are each summed again around their own maximum,
// the products taken after the difference.
//
// A workgroup walks the rows blockIdx + k gridDim: as soon as a vector's
// gradient is computed its registers take the next row's vector, so that the
// reads go on under the gradient's arithmetic and stores.  Loads and stores are
// non-temporal: a row is not met again.
//
// Bound by HBM and by how far reads and writes overlap with one row per CU:
// [4096, 131072] bf16 482 us (4.45 TB/s; a large copy reaches 5.0, and the same
// kernel without its stores takes 406).  Two passes with the parts' kernels
// take 640, a workgroup per row without the next row's loads 516, temporal
// stores 506 and temporal loads 496.
//
// 16-bit rows of up to 8192 stand eight to a CU, as the launch counts on, where
// the registers are held to eight waves per SIMD (4096 rows of 8000 42.4 -> 38.8).
template <int FT, int NT, int W>
__global__ __launch_bounds__(NT, FT != F32 && W == 4 ? 8 : 1) void k_distill_held(
    const void* z, int64_t ldz, uint32_t rows, int V, Entries ent, float s, float c, const float* __restrict__ dloss,
    float* __restrict__ loss, void* dz, int64_t lddz)
{
    constexpr int NW = NT / 64, ES = FT == F32 ? 4 : 2;
    __shared__ Marks<NT, NT * W / 4 + 1> k;
    __shared__ float red[7][NW], tails[8];
    __shared__ EntryList list;
    __shared__ int any;
    const bool rest = ent.tlse != nullptr;
    // V / 8 whole vectors (absent ones read the last again), and an element more for the first V % 8 threads
    const int nvec = V >> 3, ntail = V & 7;
    Raw8<FT> raw[W];
    const char* from = static_cast<const char*>(z) + blockIdx.x * ldz * ES;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        const int v = w * NT + (int)threadIdx.x;
        raw[w] = load8_off<FT, true>(from, (uint32_t)(v < nvec ? v : nvec - 1) * (8 * ES));
    }
    const uint32_t step = gridDim.x;
    for (uint32_t r = blockIdx.x; r < rows; r += step) {
        // opaque, so that nothing computed from them is kept in registers over the rows
        const int64_t row = afresh_uniform((int)r);
        const int t = afresh((int)threadIdx.x), wave = t >> 6;
        char* to = static_cast<char*>(dz) + row * lddz * ES;
        from = static_cast<const char*>(z) + row * ldz * ES;
        const bool more = r + step < rows;
        const char* next = from + (more ? step * ldz * ES : 0);
        // vector w of the next row (after the last row, one address of this one again)
        auto ahead = [&](int w) {
            const int at = afresh(afresh(t) + w * NT);
            raw[w] = load8_off<FT, true>(next, more ? (uint32_t)(at < nvec ? at : nvec - 1) * (8 * ES) : 0u);
        };
        const float tail = t < ntail ? load1<FT>(from, 8 * nvec + t) : -__builtin_inff();
        __syncthreads();                     // the row before is done with the marks
        if (t < 8) tails[t] = tail;          // read by the same threads
        if (t == 0) any = 0;
        marks_clear(k);
        load_entries<NT>(list, ent, row, V);
        __syncthreads();
        float tm = -__builtin_inff();
#pragma unroll 1
        for (int i = t; i < ent.K; i += NT) {
            const int col = list.col[i];
            if (col >= 0) {
                any = 1;
                mark(k, col);
                tm = __builtin_fmaxf(tm, list.val[i]);
            }
        }
        tm = wave_max(tm);
        if ((t & 63) == 0) red[0][wave] = tm;
        __syncthreads();
        bool some = any != 0;
        marks_count(k);
        // one value per wave, joined across the lanes
        const int lane = t & 63;
        auto top = [&](int i) { return wave_max(lane < NW ? red[i][lane] : -__builtin_inff()); };
        auto total = [&](int i) { return wave_sum(lane < NW ? red[i][lane] : 0.0f); };
        tm = top(0);
        tm = rest ? ent.tlse[row] : base_of(tm);
        float tsum = 0.0f;
#pragma unroll 1
        for (int i = t; i < ent.K; i += NT)
            if (list.col[i] >= 0) {
                const float x = list.val[i];
                tsum += rest ? ex2((x * s - tm) * LOG2E) : ex2((x - tm) * c);
            }

        // the entries among the eight columns of vector v (or the last); none without the normaliser
        auto entries8 = [&](int v) { return rest ? marks8(k, 8 * (v < nvec ? v : nvec - 1)) : 0u; };
        const bool tail_in = rest && t < ntail && (marks8(k, 8 * nvec) >> t & 1);
        float m, S, R;
        // over this thread's vectors x(z) added up in S and, with the normaliser, what lies outside the entries in R
        auto sum = [&](auto x) {
            S = t < ntail ? x(tails[t]) : 0.0f;
            R = rest && !tail_in ? S : 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const int at = afresh(afresh(t) + w * NT);
                float v[8], part = 0.0f;
                keep_raw<FT>(raw[w]);
                widen8<FT>(raw[w], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[i] = x(v[i]);
                    part += v[i];
                }
                const bool here = at < nvec;
                S += here ? part : 0.0f;
                if (rest) {
                    const uint32_t mask = here ? marks8(k, 8 * at) : 0;
                    if (mask) {
                        part = 0.0f;
#pragma unroll
                        for (int i = 0; i < 8; ++i) part += mask >> i & 1 ? 0.0f : v[i];
                    }
                    R += here ? part : 0.0f;
                }
                __builtin_amdgcn_sched_barrier(0);   // one vector at a time, in the order they arrive
            }
        };
        {
            float v[8];
            widen8<FT>(raw[0], v);
            const uint32_t mask = entries8(t);
            m = -__builtin_inff();
#pragma unroll
            for (int i = 0; i < 8; ++i) m = __builtin_fmaxf(m, mask >> i & 1 ? -__builtin_inff() : v[i]);
            m = base_of(wave_max(m));
            const float mc = m * c;
            sum([&](float v) { return ex2(__builtin_fmaf(v, c, -mc)); });
        }
        S = wave_sum(S);
        R = wave_sum(R);
        tsum = wave_sum(tsum);
        if ((t & 63) == 0) {
            red[1][wave] = m;
            red[2][wave] = S < 0x1p96f ? S : __builtin_inff();   // 0 times it is NaN, which is not near
            red[3][wave] = R;
            red[4][wave] = tsum;
        }
        __syncthreads();
        m = top(1);
        const float f = lane < NW ? ex2(red[1][lane] * c - m * c) : 0.0f;   // products rounded as the waves' own
        S = wave_sum(lane < NW ? red[2][lane] * f : 0.0f);
        R = wave_sum(lane < NW ? red[3][lane] * f : 0.0f);
        tsum = total(4);
        const bool near = (rest ? R : S) >= 0.5f && S < 0x1p100f;
        const float off = near ? __builtin_fmaf(m, c, -(m * c)) : 0.0f;
        float mr = m;                        // the complement's base
        if (!near) {                         // uniform: the complement and the entries around their own maxima
            // f(logit) for this thread's entries, a column by the first of its entries
            auto columns = [&](auto f) {
#pragma unroll 1
                for (int i = t; i < (rest ? ent.K : 0); i += NT) {
                    bool first = list.col[i] >= 0;
                    if (k.twice)
#pragma unroll 1
                        for (int j = 0; j < i; ++j) first = first && list.col[j] != list.col[i];
                    if (first) f(load1<FT>(from, list.col[i]));
                }
            };
            float me = -__builtin_inff(), E = 0.0f;
            columns([&](float z) { me = __builtin_fmaxf(me, z); });
            mr = t < ntail && !tail_in ? tails[t] : -__builtin_inff();
#pragma unroll
            for (int w = 0; w < W; ++w) {    // repeated elements do not change a maximum
                const uint32_t mask = entries8(afresh(afresh(t) + w * NT));
                float v[8], most = -__builtin_inff();
                keep_raw<FT>(raw[w]);
                widen8<FT>(raw[w], v);
#pragma unroll
                for (int i = 0; i < 8; ++i) most = __builtin_fmaxf(most, v[i]);
                if (mask) {
                    most = -__builtin_inff();
#pragma unroll
                    for (int i = 0; i < 8; ++i) most = __builtin_fmaxf(most, mask >> i & 1 ? -__builtin_inff() : v[i]);
                }
                mr = __builtin_fmaxf(mr, most);
                __builtin_amdgcn_sched_barrier(0);
            }
            mr = wave_max(mr);
            me = wave_max(me);
            __syncthreads();
            if ((t & 63) == 0) {
                red[1][wave] = mr;
                red[6][wave] = me;
            }
            __syncthreads();
            mr = top(1);
            me = top(6);
            const float br = base_of(mr), be = base_of(me);
            sum([&](float v) { return ex2((v - br) * c); });
            R = rest ? R : S;
            columns([&](float z) { E += ex2((z - be) * c); });
            R = wave_sum(R);
            E = wave_sum(E);
            __syncthreads();
            if ((t & 63) == 0) {
                red[2][wave] = R;
                red[3][wave] = E;
            }
            __syncthreads();
            R = total(2);
            const Part all = join(Part{mr, R}, Part{me, total(3)}, c);
            m = all.m;
            S = all.sum;
        }
        if (!rest && tsum == 0.0f) some = false;
        float pr;
        const Coef q = make_coef(rest, some, S, R, rest && !near ? ex2((mr - base_of(m)) * c) : 1.0f, tm, tsum, s,
                                 dloss ? dloss[row] : 1.0f, &pr);
        if (q.some) marks_fill(k, list, ent, q, 0, V, s, c);
        float l = 0.0f;
#pragma unroll 1
        for (int i = t; i < (q.some ? ent.K : 0); i += NT) {
            const int col = list.col[i];
            if (col >= 0)
                l += entry_loss(ent, list.val[i], load1<FT>(from, col), s, c, tm, tsum, m, S, lg2(S) - off);
        }
        l = wave_sum(l);
        if ((t & 63) == 0) red[5][wave] = l;
        __syncthreads();                     // also before the first store: dz may be z
        if (wave == 0) {
            l = total(5) + rest_loss(pr, R, S, (mr - base_of(m)) * s);
            if (t == 0) loss[row] = q.some ? l : 0.0f;
        }
        // 2^(z c - mc) or 2^((z - m) c), outside the entries (z - m_r)
        const float si = near ? 0.0f : base_of(m), so = near ? 0.0f : base_of(mr), mc = near ? m * c : 0.0f;
        auto xo = [&](float v) { return ex2(__builtin_fmaf(v - so, c, -mc)); };
        auto xi = [&](float v) { return ex2(__builtin_fmaf(v - si, c, -mc)); };
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
                if (q.some) grad8(k, q, 8 * at, v, xo, xi);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.0f;
                store8_off<FT, true>(to, (uint32_t)at * (8 * ES), v);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (t < ntail) {
            const int at = 8 * nvec + t;
            const bool entry = marks8(k, 8 * nvec) >> t & 1;
            store1<FT>(to, at, !q.some ? 0.0f : entry ? xi(tails[t]) * q.in - k.value[rank_of(k, at)]
                                                      : xo(tails[t]) * q.out);
        }
    }
}

// ---------------------------------------------------------------- launches
// Most columns per part: 8192, or 4096 where that would not give the chip
// DT_GROUPS workgroups.  Measured, forwards and back, us, parts of 4096 / 8192 /
// longer: [512, 32000] f32 44 / 37.7 / 41.5, [128, 131072] bf16 30.9 / 25.4 /
// 28.8, [2048, 32000] bf16 - / 84 / 92, [2048, 131072] bf16 - / 297 / 324.
constexpr int64_t DT_GROUPS = 2048;
// The parts of a row have one length, a multiple of 8 (the last may be shorter):
// [1700, 41410] f32 234 -> 187 us against full parts and a rest.
struct Split {
    int ch, len, parts;
};
inline Split distill_split(int64_t rows, int64_t V)
{
    Split q;
    q.ch = rows * cdiv(V, 8192) >= DT_GROUPS ? 8192 : 4096;
    q.len = (int)cdiv(cdiv(V, cdiv(V, q.ch)), 8) * 8;
    q.parts = (int)cdiv(V, q.len);
    return q;
}

#define TQ_CH_SWITCH(ch, ...)                                    \
    do {                                                         \
        if ((ch) == 8192) { constexpr int CHV = 8192; __VA_ARGS__; } \
        else { constexpr int CHV = 4096; __VA_ARGS__; }          \
    } while (0)

struct Distill {
    const void* z;
    int64_t ldz, rows;
    int V;
    Entries ent;
    float s, c;
};

// Most workgroups per launch: a grid holds fewer than 2^32 threads.  Further rows
// are further launches.
constexpr int64_t DT_LAUNCH = 1 << 23;

// The same for the rows from `first` on, at most `most` of them.
static Distill rows_from(const Distill& d, int FT, int64_t first, int64_t most)
{
    Distill r = d;
    r.z = forward_by(d.z, first * d.ldz * ftype_size(FT));
    r.ent.idx = forward_by(d.ent.idx, first * d.ent.K * (d.ent.idx64 ? 8 : 4));
    r.ent.val = forward_by(d.ent.val, first * d.ent.K * ftype_size(d.ent.val_dt));
    r.ent.tlse = forward_by(d.ent.tlse, 4 * first);
    r.rows = std::min(d.rows - first, most);
    return r;
}

// Workspace: the parts' statistics, then the logits at the entries.
inline size_t distill_part_floats(int64_t rows, int64_t V)
{
    return 4 * (size_t)rows * (size_t)distill_split(rows, V).parts;
}

template <int FT>
static void stats_launch(const Distill& all, float* ws, hipStream_t st)
{
    const Split q = distill_split(all.rows, all.V);
    float4* part = reinterpret_cast<float4*>(ws);
    float* zk = ws + distill_part_floats(all.rows, all.V);
    const int64_t most = std::max<int64_t>(1, DT_LAUNCH / q.parts);
    for (int64_t r = 0; r < all.rows; r += most) {
        const Distill d = rows_from(all, FT, r, most);
        const dim3 grid((unsigned)(d.rows * q.parts));
        if (d.ent.tlse)
            TQ_CH_SWITCH(q.ch, hipLaunchKernelGGL((k_distill_stats<FT, true, CHV>), grid, dim3(256), 0, st, d.z, d.ldz,
                                                d.V, q.parts, q.len, d.ent, d.c, part + r * q.parts,
                                                zk + r * d.ent.K));
        else
            TQ_CH_SWITCH(q.ch, hipLaunchKernelGGL((k_distill_stats<FT, false, CHV>), grid, dim3(256), 0, st, d.z, d.ldz,
                                                d.V, q.parts, q.len, d.ent, d.c, part + r * q.parts,
                                                zk + r * d.ent.K));
    }
}

static void rows_launch(const Distill& all, const float* ws, float* loss, float* stats, float* rest_sum,
                        hipStream_t st)
{
    const int parts = distill_split(all.rows, all.V).parts;
    const float4* part = reinterpret_cast<const float4*>(ws);
    const float* zk = ws + distill_part_floats(all.rows, all.V);
    for (int64_t r = 0; r < all.rows; r += DT_LAUNCH) {
        const Distill d = rows_from(all, TQ_F32, r, DT_LAUNCH);       // the logits are not read
        hipLaunchKernelGGL(k_distill_rows, dim3((unsigned)cdiv(d.rows, 4)), dim3(256), 0, st, d.rows, d.V, d.ent, d.s,
                           d.c, part + r * parts, zk + r * d.ent.K, parts, loss + r, forward_by(stats, 8 * r),
                           forward_by(rest_sum, 8 * r));
    }
}

template <int FT, bool FROM_PARTS>
static void grad_launch(const Distill& all, const float* ws, const float* stats, const float* rest_sum,
                        const float* dloss, float* loss, void* dz, int64_t lddz, hipStream_t st)
{
    const Split q = distill_split(all.rows, all.V);
    const float4* part = reinterpret_cast<const float4*>(ws);
    const float* zk = FROM_PARTS ? ws + distill_part_floats(all.rows, all.V) : nullptr;
    const int64_t most = std::max<int64_t>(1, DT_LAUNCH / q.parts);
    for (int64_t r = 0; r < all.rows; r += most) {
        const Distill d = rows_from(all, FT, r, most);
        TQ_CH_SWITCH(q.ch, hipLaunchKernelGGL((k_distill_grad<FT, CHV, FROM_PARTS>),
                                            dim3((unsigned)(d.rows * q.parts)), dim3(256), 0, st, d.z, d.ldz, d.V,
                                            q.parts, q.len, d.ent, d.s, d.c, forward_by(part, 16 * r * q.parts),
                                            forward_by(zk, 4 * r * d.ent.K), forward_by(stats, 8 * r),
                                            forward_by(rest_sum, 8 * r), forward_by(dloss, 4 * r),
                                            forward_by(loss, 4 * r), forward_by(dz, r * lddz * ftype_size(FT)), lddz));
    }
}

// Whether the joint call holds its rows in registers.  A row in registers costs
// one read instead of two, and spreads over no more than one workgroup: rows of
// 64 KB (a workgroup of 256 threads) are held at any number of them; of 128 KB
// from DT_HELD_ROWS of them on; of 256 KB, which take a CU each, where they
// fill at least 5/8 of their rounds over the CUs (binary32, which takes more
// instructions per byte, 7/8 of at least two rounds).  Measured, us, held / in
// parts:   1 row of 32000 bf16 12.1 / 14.7, 256 rows 13.0 / 17.8, 2048 rows 56 /
// 83;   64 rows of 65536 bf16 15.6 / 14.6, 128 rows 15.8 / 17.8;   rows of
// 131072 bf16: 128 of them 26.4 / 22.7, 160 28.2 / 29.3, 300 57 / 48, 512 66 /
// 80, 4096 482 / 643;   of 65536 f32: 256 43 / 36, 512 76 / 79, 2048 278 / 306.
constexpr int64_t DT_HELD_ROWS = 128;
template <int FT>
static bool held_launch(const Distill& d, const float* dloss, float* loss, void* dz, int64_t lddz, hipStream_t st)
{
    constexpr int H = FT == F32 ? 2 : 1;  // binary32 rows hold half as many elements
    if (d.V < 8 || d.V > 131072 / H) return false;
    if (d.V > 65536 / H) {
        const int64_t rounds = std::max<int64_t>(H, cdiv(d.rows, 256));
        if (8 * d.rows < (H == 2 ? 7 : 5) * 256 * rounds) return false;
    } else if (d.V > 32768 / H && d.rows < DT_HELD_ROWS) {
        return false;
    }
    // as many workgroups as fit on the chip by their registers
#define TQ_HELD(NT, W)                                                                                            \
    hipLaunchKernelGGL((k_distill_held<FT, NT, W>), dim3((unsigned)std::min<int64_t>(d.rows, 256 * (1024 / NT) * \
                       (W * (FT == F32 ? 2 : 1) <= 8 ? 2 : 1))), dim3(NT), 0, st, d.z, d.ldz, (uint32_t)d.rows, d.V, \
                       d.ent, d.s, d.c, dloss, loss, dz, lddz)
    if (d.V <= 8192) TQ_HELD(256, 4);
    else if (d.V <= 32768 / H) TQ_HELD(256, 16 / H);
    else if (d.V <= 65536 / H) TQ_HELD(512, 16 / H);
    else TQ_HELD(1024, 16 / H);
#undef TQ_HELD
    return true;
}

static bool natural(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// Checks what the three calls share and fills `d`; *work is false where there
// is nothing to do.
static tq_status distill_check(const void* logits, int dt, int64_t rows, int64_t vocab, int64_t ldz, const void* idx,
                               int idx_bits, const void* val, int val_dt, int64_t K, const float* teacher_lse,
                               float temperature, Distill* d, bool* work)
{
    *work = false;
    if (!valid_ftype(dt) || !valid_ftype(val_dt) || (idx_bits != 32 && idx_bits != 64)) return TQ_ERR_INVALID;
    if (rows < 0 || vocab < 0 || K < 1) return TQ_ERR_INVALID;
    if (!(temperature >= 1e-38f) || temperature > 3.0e38f) return TQ_ERR_INVALID;    // s and c are finite
    if (rows == 0) return TQ_OK;
    if (vocab == 0 || !logits || ldz < vocab || !idx || !val) return TQ_ERR_INVALID;
    if (K > DT_K || vocab > 0x7fffff00 || rows > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
    if (!natural(logits, ftype_size(dt)) || !natural(idx, idx_bits / 8) || !natural(val, ftype_size(val_dt)) ||
        !natural(teacher_lse, 4))
        return TQ_ERR_ALIGN;
    d->z = logits;
    d->ldz = ldz;
    d->rows = rows;
    d->V = (int)vocab;
    d->ent = Entries{idx, idx_bits == 64, val, val_dt, (int)K, teacher_lse};
    d->s = (float)(1.0 / (double)temperature);
    d->c = (float)(1.4426950408889634 / (double)temperature);
    *work = true;
    return TQ_OK;
}

static tq_status workspace_check(const void* ws, size_t have, int64_t rows, int64_t vocab, int64_t k)
{
    if (!ws || have < tq_topk_distill_workspace_bytes(rows, vocab, k)) return TQ_ERR_INVALID;
    return aligned16(ws) ? TQ_OK : TQ_ERR_ALIGN;
}

}  // namespace tq

using namespace tq;

extern "C" {

size_t tq_topk_distill_workspace_bytes(int64_t rows, int64_t vocab, int64_t k)
{
    if (rows <= 0 || vocab <= 0 || k <= 0) return 0;
    return (distill_part_floats(rows, vocab) + (size_t)rows * (size_t)k) * sizeof(float);
}

tq_status tq_topk_distill(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                          const void* top_idx, int idx_bits, const void* top_val, int val_dtype, int64_t k,
                          const float* teacher_lse, float temperature, float* loss, float* stats, float* rest_sum,
                          void* workspace, size_t workspace_bytes, void* stream)
{
    Distill d;
    bool work;
    tq_status r = distill_check(logits, dtype, rows, vocab, row_stride, top_idx, idx_bits, top_val, val_dtype, k,
                                teacher_lse, temperature, &d, &work);
    if (r != TQ_OK || !work) return r;
    if (!loss) return TQ_ERR_INVALID;
    if (!natural(loss, 4) || !natural(stats, 4) || !natural(rest_sum, 4)) return TQ_ERR_ALIGN;
    if ((r = workspace_check(workspace, workspace_bytes, rows, vocab, k)) != TQ_OK) return r;
    float* ws = static_cast<float*>(workspace);
    hipStream_t st = as_stream(stream);
    TQ_LLM_FT_SWITCH(dtype, stats_launch<FTV>(d, ws, st));
    rows_launch(d, ws, loss, stats, teacher_lse ? rest_sum : nullptr, st);
    return launch_status();
}

tq_status tq_topk_distill_backward(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                                   const void* top_idx, int idx_bits, const void* top_val, int val_dtype, int64_t k,
                                   const float* teacher_lse, float temperature, const float* stats,
                                   const float* rest_sum, const float* dloss, void* dlogits, int64_t d_row_stride,
                                   void* stream)
{
    Distill d;
    bool work;
    const tq_status r = distill_check(logits, dtype, rows, vocab, row_stride, top_idx, idx_bits, top_val, val_dtype, k,
                                      teacher_lse, temperature, &d, &work);
    if (r != TQ_OK || !work) return r;
    if (!stats || (teacher_lse && !rest_sum) || !dlogits || d_row_stride < vocab) return TQ_ERR_INVALID;
    if (!natural(stats, 4) || !natural(rest_sum, 4) || !natural(dloss, 4) || !natural(dlogits, ftype_size(dtype)))
        return TQ_ERR_ALIGN;
    TQ_LLM_FT_SWITCH(dtype, (grad_launch<FTV, false>(d, nullptr, stats, rest_sum, dloss, nullptr, dlogits, d_row_stride,
                                                     as_stream(stream))));
    return launch_status();
}

tq_status tq_topk_distill_grad(const void* logits, int dtype, int64_t rows, int64_t vocab, int64_t row_stride,
                               const void* top_idx, int idx_bits, const void* top_val, int val_dtype, int64_t k,
                               const float* teacher_lse, float temperature, const float* dloss, float* loss,
                               void* dlogits, int64_t d_row_stride, void* workspace, size_t workspace_bytes,
                               void* stream)
{
    Distill d;
    bool work;
    tq_status r = distill_check(logits, dtype, rows, vocab, row_stride, top_idx, idx_bits, top_val, val_dtype, k,
                                teacher_lse, temperature, &d, &work);
    if (r != TQ_OK || !work) return r;
    if (!loss || !dlogits || d_row_stride < vocab) return TQ_ERR_INVALID;
    if (!natural(loss, 4) || !natural(dloss, 4) || !natural(dlogits, ftype_size(dtype))) return TQ_ERR_ALIGN;
    if ((r = workspace_check(workspace, workspace_bytes, rows, vocab, k)) != TQ_OK) return r;
    float* ws = static_cast<float*>(workspace);
    hipStream_t st = as_stream(stream);
    TQ_LLM_FT_SWITCH(dtype, {
        if (!held_launch<FTV>(d, dloss, loss, dlogits, d_row_stride, st)) {
            stats_launch<FTV>(d, ws, st);
            grad_launch<FTV, true>(d, ws, nullptr, nullptr, dloss, loss, dlogits, d_row_stride, st);
        }
    });
    return launch_status();
}

}  // extern "C"
