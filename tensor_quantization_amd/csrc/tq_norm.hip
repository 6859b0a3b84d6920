// tq_norm.hip -- layer norm over the last dimension: the forward pass, the
// forward pass fused with the per-token s8 quantizer that feeds the W8A8
// product, and the backward pass with the reduction of the weight's and the
// bias's gradient.
//
//   mu = sum_j x_j / C,  v = sum_j (x_j - mu)^2 / C,  r = 1 / sqrt(v + eps)
//   y_j = (x_j - mu) r w_j + b_j
//   backward, with g = dy w and h = (x - mu) r:
//   dx = r (g - sum(g)/C - h sum(g h)/C),  dw_j = sum_rows dy h,  db_j = sum_rows dy
//
// All statistics and sums are binary32; the variance is taken around the mean
// from the values held in registers (one read of the row, no E[x^2] - mu^2
// cancellation).  Outputs are rounded once to their type.  The fused form
// rounds y to x's type before it takes the row's maximum, so that its codes
// and scales are those of tq_layer_norm followed by tq_quant_per_token.
//
// Every kernel is bound by HBM: 2 bytes in and 2 out per bf16 element
// forwards, 4 in and 2 out backwards.
#include "tq_llm.h"

namespace tq {

enum { OUT_Y = 0, OUT_S8 = 1 };

// One sum over the NT threads of a row (a wave's own when NT is 64).  `slot`
// alternates so that a row's second sum needs no barrier before it.
template <int NT>
__device__ __forceinline__ float row_sum(float v, float* slot)
{
    v = wave_sum(v);
    if constexpr (NT > 64) {
        const int t = threadIdx.x;
        if ((t & 63) == 0) slot[t >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < NT / 64; ++k) v += slot[k];
    }
    return v;
}
// The largest magnitude.  Magnitudes are compared as bit patterns: a NaN's lies
// above an infinity's, so a row that holds one has it for its maximum (a float
// maximum would drop it).
__device__ __forceinline__ float larger(float a, float b) { return as_f(max(as_u(a), as_u(b))); }
template <int NT>
__device__ __forceinline__ float row_max(float v, float* slot)
{
    v = team_max<64>(v);
    if constexpr (NT > 64) {
        const int t = threadIdx.x;
        if ((t & 63) == 0) slot[t >> 6] = v;
        __syncthreads();
        v = slot[0];
#pragma unroll
        for (int k = 1; k < NT / 64; ++k) v = larger(v, slot[k]);
    }
    return v;
}

// The value as x's type holds it.
template <int FT>
__device__ __forceinline__ float as_stored(float v)
{
    if constexpr (FT == F32) return v;
    else if constexpr (FT == BF16) return as_f((uint32_t)to_bf16_bits(v) << 16);
    else return (float)__builtin_bit_cast(_Float16, to_f16_bits(v));
}

// Symmetric s8 codes of a row: scale = amax / 127 (1 if that is 0), code =
// clamp(rne(v / scale)), both divisions correctly rounded.  A row with a NaN has
// the scale NaN, whose codes say nothing.
struct S8Row {
    float s, y;
    bool fast;
};
__device__ __forceinline__ S8Row s8_row(float amax)
{
    S8Row r;
    r.s = amax / 127.0f;
    r.s = r.s == 0.0f ? 1.0f : r.s;
    r.fast = scale_in_fast_range(r.s);
    r.y = r.fast ? rcp_rn(r.s) : 0.0f;
    return r;
}
template <int FT>
__device__ __forceinline__ float s8_code(float v, const S8Row& r)
{
    const float q = r.fast && __builtin_fabsf(v) <= 0x1p86f ? div_q<FT>(v, r.s, r.y) : v / r.s;
    return int_code_f(q, 0.0f, MAGIC - 127.0f, MAGIC + 127.0f);
}

// Stores the codes of the vector's own elements, v as x's type holds them.
template <int FT>
__device__ __forceinline__ void store_codes(uint8_t* q, Vec8 at, const float v[8], const S8Row& p)
{
    float c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = s8_code<FT>(v[i], p);
    if (at.lo == 0) {
        const u32x2_any o = {pack_bytes4(c[0], c[1], c[2], c[3]), pack_bytes4(c[4], c[5], c[6], c[7])};
        *reinterpret_cast<u32x2_any*>(q + at.at) = o;
    } else {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (i >= at.lo) q[at.at + i] = (uint8_t)as_u(c[i]);
    }
}

// k_ln_rows: NT threads per row, W vectors of eight elements per thread, the
// row held in registers (8 <= cols <= 8 * NT * W): one read of x, the two sums
// in turn from the registers, one write.  NT = 64 puts four rows in a workgroup
// and needs no barrier.  The parameters are loaded between the two sums: later
// (24.9 us instead of 25.6 at the size below) a single token waits for them.
// Bound by HBM: [8192, 4096] bf16 24.9 us (5.4 TB/s; a large copy
// reaches 5.0), its codes 28 (two calls 43), one row of 4096 3.2 us, latency.  Stores
// are plain: what follows reads y, and non-temporal loads, which skip the last-level
// cache that x comes from, take 32 us.
template <int FT, int NT, int W, int OUT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void k_ln_rows(
    const void* __restrict__ x, int64_t ldx, int64_t rows, int64_t cols, const void* __restrict__ weight,
    const void* __restrict__ bias, int wdt, float eps, void* __restrict__ y, float* __restrict__ scale,
    float* __restrict__ mean, float* __restrict__ rstd)
{
    constexpr int RPB = NT < 256 ? 256 / NT : 1;
    __shared__ float slots[3][NT / 64];
    const int t = threadIdx.x % NT;
    const int64_t row = (int64_t)blockIdx.x * RPB + __builtin_amdgcn_readfirstlane(threadIdx.x / NT);
    if (row >= rows) return;     // only with NT == 64, whose rows meet no barrier

    Vec8 at[W];
    Raw8<FT> raw[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        at[w] = vec8(w * NT + t, (int)cols);
        raw[w] = load8_any<FT>(x, row * ldx + at[w].at);
    }
    float v[W][8];
    float s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        widen8<FT>(raw[w], v[w]);
#pragma unroll
        for (int i = 0; i < 8; ++i) s += i >= at[w].lo ? v[w][i] : 0.0f;
    }
    const float mu = row_sum<NT>(s, slots[0]) / (float)cols;
    RawAny rw[W], rb[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
        rw[w] = load8_rt(weight, wdt, at[w].at);
        rb[w] = load8_rt(bias, wdt, at[w].at);
    }
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[w][i] -= mu;
            const float d = i >= at[w].lo ? v[w][i] : 0.0f;
            s = __builtin_fmaf(d, d, s);
        }
    const float r = 1.0f / __builtin_sqrtf(row_sum<NT>(s, slots[1]) / (float)cols + eps);
    if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
    float amax = 0.0f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        float ww[8], bb[8];
        widen8_rt(rw[w], weight, wdt, 1.0f, ww);
        widen8_rt(rb[w], bias, wdt, 0.0f, bb);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[w][i] = __builtin_fmaf(v[w][i] * r, ww[i], bb[i]);
        if constexpr (OUT == OUT_Y) {
            if (at[w].lo < 8) store8_own<FT>(y, row * cols, at[w], v[w]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                v[w][i] = as_stored<FT>(v[w][i]);
                amax = larger(amax, i >= at[w].lo ? __builtin_fabsf(v[w][i]) : 0.0f);
            }
        }
    }
    if constexpr (OUT == OUT_S8) {
        amax = row_max<NT>(amax, slots[2]);
        const S8Row p = s8_row(amax);
        if (t == 0) scale[row] = p.s;
        uint8_t* q = static_cast<uint8_t*>(y) + row * cols;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (at[w].lo < 8) store_codes<FT>(q, at[w], v[w], p);
        }
    }
}

// k_ln_long: rows longer than a workgroup holds: a workgroup per row reads it
// once for the mean, once around the mean and once for the output (the later
// reads meet the caches), and once more for the codes.  [4096, 20000] bf16 84-95 us
// (3.4-3.9 TB/s of what it must read and write); an element per load took 245.
constexpr int LN_LT = 1024;              // threads per long row
template <int FT, int OUT>
__global__ __launch_bounds__(LN_LT) void k_ln_long(const void* __restrict__ x, int64_t ldx, int cols,
                                                   const void* __restrict__ weight, const void* __restrict__ bias,
                                                   int wdt, float eps, void* __restrict__ y, float* __restrict__ scale,
                                                   float* __restrict__ mean, float* __restrict__ rstd)
{
    __shared__ float slots[3][LN_LT / 64];
    const int t = threadIdx.x, nvec = (cols + 7) / 8;
    const int64_t row = blockIdx.x, base = row * ldx;
    // f(a vector's eight elements, which of them are its own)
    auto each = [&](auto f) {
        for (int k = t; k < nvec; k += LN_LT) {
            const Vec8 at = vec8(k, cols);
            float v[8];
            widen8<FT>(load8_any<FT>(x, base + at.at), v);
            f(v, at);
        }
    };
    float s = 0.0f;
    each([&](const float v[8], Vec8 at) {
#pragma unroll
        for (int i = 0; i < 8; ++i) s += i >= at.lo ? v[i] : 0.0f;
    });
    const float mu = row_sum<LN_LT>(s, slots[0]) / (float)cols;
    s = 0.0f;
    each([&](const float v[8], Vec8 at) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float d = i >= at.lo ? v[i] - mu : 0.0f;
            s = __builtin_fmaf(d, d, s);
        }
    });
    const float r = 1.0f / __builtin_sqrtf(row_sum<LN_LT>(s, slots[1]) / (float)cols + eps);
    if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = r;
    }
    auto values = [&](float v[8], Vec8 at) {
        float w[8], b[8];
        widen8_rt(load8_rt(weight, wdt, at.at), weight, wdt, 1.0f, w);
        widen8_rt(load8_rt(bias, wdt, at.at), bias, wdt, 0.0f, b);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf((v[i] - mu) * r, w[i], b[i]);
    };
    if constexpr (OUT == OUT_Y) {
        each([&](float v[8], Vec8 at) {
            values(v, at);
            store8_own<FT>(y, row * cols, at, v);
        });
    } else {
        float amax = 0.0f;
        each([&](float v[8], Vec8 at) {
            values(v, at);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                amax = larger(amax, i >= at.lo ? __builtin_fabsf(as_stored<FT>(v[i])) : 0.0f);
        });
        const S8Row p = s8_row(row_max<LN_LT>(amax, slots[2]));
        if (t == 0) scale[row] = p.s;
        each([&](float v[8], Vec8 at) {
            values(v, at);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = as_stored<FT>(v[i]);
            store_codes<FT>(static_cast<uint8_t*>(y) + row * cols, at, v, p);
        });
    }
}

// k_ln_thin: rows of fewer than 8 elements, a thread each: [1000000, 7] bf16
// 16.8 us (a workgroup per row: 3130).
template <int FT, int OUT>
__global__ __launch_bounds__(256) void k_ln_thin(const void* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                 const void* __restrict__ weight, const void* __restrict__ bias,
                                                 int wdt, float eps, void* __restrict__ y, float* __restrict__ scale,
                                                 float* __restrict__ mean, float* __restrict__ rstd)
{
    const int64_t row = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (row >= rows) return;
    float v[7], s = 0.0f, amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        v[j] = j < cols ? load1<FT>(x, row * ldx + j) : 0.0f;
        s += v[j];
    }
    const float mu = s / (float)cols;
    s = 0.0f;
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        v[j] = j < cols ? v[j] - mu : 0.0f;
        s = __builtin_fmaf(v[j], v[j], s);
    }
    const float r = 1.0f / __builtin_sqrtf(s / (float)cols + eps);
    if (mean) mean[row] = mu;
    if (rstd) rstd[row] = r;
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        if (j >= cols) break;
        v[j] = __builtin_fmaf(v[j] * r, load1_rt(weight, wdt, j, 1.0f), load1_rt(bias, wdt, j, 0.0f));
        if constexpr (OUT == OUT_Y) {
            store1<FT>(y, row * cols + j, v[j]);
        } else {
            v[j] = as_stored<FT>(v[j]);
            amax = larger(amax, __builtin_fabsf(v[j]));
        }
    }
    if constexpr (OUT == OUT_S8) {
        const S8Row p = s8_row(amax);
        scale[row] = p.s;
#pragma unroll
        for (int j = 0; j < 7; ++j)
            if (j < cols) static_cast<uint8_t*>(y)[row * cols + j] = (uint8_t)as_u(s8_code<FT>(v[j], p));
    }
}

// ---------------------------------------------------------------- backward
// k_ln_bwd: teams of NT threads, a team per row at a time, W vectors per
// thread.  A workgroup of BT threads walks the rows blockIdx + k gridDim (in
// units of its BT / NT teams); each thread keeps the sums of dy h and dy of
// its own columns in registers over all its rows, the teams add theirs in LDS
// in a fixed order at the end, and the workgroup leaves one row of partial
// sums.  The rows of the next step are loaded before the sums of the present
// one are taken.  Bound by HBM: [8192, 4096] bf16 35.6 us (5.7 TB/s) and 4.7 us
// for the column sums; [1021, 5003] f32 15.4 and 4.8 us, where four rows per
// workgroup leave the ends of the pipeline uncovered and 10 MB of partial sums
// join 61 MB of tensors.  256 workgroups, one per CU: more would write more
// partials.  Rows of more than 8192 columns keep the sums in LDS, each
// thread its own, where registers would not hold them beside two rows.
template <int FT, int NT, int W, int BT>
__global__ __launch_bounds__(BT) void k_ln_bwd(const void* __restrict__ dy, int64_t lddy, const void* __restrict__ x,
                                               int64_t ldx, int64_t rows, int64_t cols,
                                               const void* __restrict__ weight, int wdt,
                                               const float* __restrict__ mean, const float* __restrict__ rstd,
                                               void* __restrict__ dx, float* __restrict__ part, int64_t ldp)
{
    constexpr int TEAMS = BT / NT, NW = NT / 64;
    constexpr bool IN_LDS = 8 * NT * W > 8192;
    __shared__ float slots[2][TEAMS][NW][2];
    __shared__ float fold[TEAMS > 1 ? 8 * NT * W : 1];
    __shared__ float4 sums[IN_LDS ? 4 * NT * W : 1];     // [w][dw 0 .. 3, 4 .. 7, db 0 .. 3, 4 .. 7][t]
    const int t = threadIdx.x % NT, team = __builtin_amdgcn_readfirstlane(threadIdx.x / NT);

    Vec8 at[W];
    float ww[W][8], dw[W][8], db[W][8];           // the sums unused with IN_LDS
#pragma unroll
    for (int w = 0; w < W; ++w) {
        at[w] = vec8(w * NT + t, (int)cols);
        widen8_rt(load8_rt(weight, wdt, at[w].at), weight, wdt, 1.0f, ww[w]);
        if constexpr (IN_LDS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) sums[(4 * w + i) * NT + t] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[w][i] = 0.0f;
                db[w][i] = 0.0f;
            }
        }
    }
    const int64_t step = (int64_t)gridDim.x * TEAMS;
    const int64_t first = (int64_t)blockIdx.x * TEAMS;
    const float rc = 1.0f / (float)cols;
    Raw8<FT> nx[W], ny[W];
    float nmu = 0.0f, nr = 0.0f;
    // a team past the last row reads the last row again; its sums stay out
    auto fetch = [&](int64_t row) {
        row = row < rows ? row : rows - 1;
        nmu = mean[row];
        nr = rstd[row];
#pragma unroll
        for (int w = 0; w < W; ++w) {
            nx[w] = load8_any<FT>(x, row * ldx + at[w].at);
            ny[w] = load8_any<FT>(dy, row * lddy + at[w].at);
        }
    };
    fetch(first + team);
    int turn = 0;
    for (int64_t base = first; base < rows; base += step, turn ^= 1) {
        const int64_t row = base + team;
        const bool mine = row < rows;
        Raw8<FT> cx[W], cy[W];
        const float mu = nmu, r = nr;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            cx[w] = nx[w];
            cy[w] = ny[w];
        }
        if (base + step < rows) fetch(row + step);
        float sg = 0.0f, sgh = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float h[8], d[8];
            widen8<FT>(cx[w], h);
            widen8<FT>(cy[w], d);
            auto add = [&](int i, float& to_dw, float& to_db) {
                const bool own = mine && i >= at[w].lo;
                const float dd = own ? d[i] : 0.0f, hh = own ? (h[i] - mu) * r : 0.0f;
                const float g = dd * ww[w][i];
                sg += g;
                sgh = __builtin_fmaf(g, hh, sgh);
                to_dw = __builtin_fmaf(dd, hh, to_dw);
                to_db += dd;
            };
            if constexpr (IN_LDS) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float4* s = sums + (4 * w + k) * NT + t;
                    float4 a = s[0], b = s[2 * NT];
                    add(4 * k, a.x, b.x);
                    add(4 * k + 1, a.y, b.y);
                    add(4 * k + 2, a.z, b.z);
                    add(4 * k + 3, a.w, b.w);
                    s[0] = a;
                    s[2 * NT] = b;
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) add(i, dw[w][i], db[w][i]);
            }
        }
        sg = wave_sum(sg);
        sgh = wave_sum(sgh);
        if constexpr (NW > 1) {
            if ((t & 63) == 0) {
                slots[turn][team][t >> 6][0] = sg;
                slots[turn][team][t >> 6][1] = sgh;
            }
            __syncthreads();
            sg = 0.0f;
            sgh = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                sg += slots[turn][team][k][0];
                sgh += slots[turn][team][k][1];
            }
        }
        if (!mine || !dx) continue;
        const float c1 = sg * rc, c2 = sgh * rc;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            float h[8], d[8];
            if constexpr (IN_LDS) {      // nothing held from the first pass over the row
                keep_raw<FT>(cx[w]);
                keep_raw<FT>(cy[w]);
                __builtin_amdgcn_sched_barrier(0);
            }
            widen8<FT>(cx[w], h);
            widen8<FT>(cy[w], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = (h[i] - mu) * r;
                d[i] = (d[i] * ww[w][i] - c1 - h[i] * c2) * r;
            }
            if (at[w].lo < 8) store8_own<FT>(dx, row * cols, at[w], d);
        }
    }
    if (!part) return;
    // the teams' sums, added in team order, first those of dw, then of db
    float* to = part + (int64_t)blockIdx.x * 2 * ldp;
    if constexpr (IN_LDS) {
#pragma unroll
        for (int w = 0; w < W; ++w)
            if (at[w].lo < 8) {
#pragma unroll
                for (int o = 0; o < 2; ++o) {
                    const float4 a = sums[(4 * w + 2 * o) * NT + t], b = sums[(4 * w + 2 * o + 1) * NT + t];
                    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
                    store8_own<F32>(to + o * ldp, 0, at[w], v);
                }
            }
        return;
    }
#pragma unroll
    for (int o = 0; o < 2; ++o) {
        if constexpr (TEAMS > 1) {
            for (int k = 1; k < TEAMS; ++k) {
                __syncthreads();
                if (team == k) {
#pragma unroll
                    for (int w = 0; w < W; ++w)
#pragma unroll
                        for (int i = 0; i < 8; ++i) fold[(w * 8 + i) * NT + t] = o ? db[w][i] : dw[w][i];
                }
                __syncthreads();
                if (team == 0) {
#pragma unroll
                    for (int w = 0; w < W; ++w)
#pragma unroll
                        for (int i = 0; i < 8; ++i) (o ? db : dw)[w][i] += fold[(w * 8 + i) * NT + t];
                }
            }
        }
        if (team == 0) {
#pragma unroll
            for (int w = 0; w < W; ++w)
                if (at[w].lo < 8) store8_own<F32>(to + o * ldp, 0, at[w], o ? db[w] : dw[w]);
        }
    }
}

// Rows longer than that: a workgroup per row for dx (two reads), and a second
// kernel for the column sums (one more): a wave owns 512 columns, a workgroup's
// four waves take a chunk of the rows in turn, U rows in flight each, and their
// sums meet in LDS in wave order.  [4096, 20000] bf16 190-198 us (2.5 TB/s: x and dy
// cross three times), [4096, 16384] f32 305; an element per load took 328.
template <int FT>
__global__ __launch_bounds__(LN_LT) void k_ln_bwd_long(const void* __restrict__ dy, int64_t lddy,
                                                       const void* __restrict__ x, int64_t ldx, int cols,
                                                       const void* __restrict__ weight, int wdt,
                                                       const float* __restrict__ mean, const float* __restrict__ rstd,
                                                       void* __restrict__ dx)
{
    __shared__ float slots[2][LN_LT / 64];
    const int t = threadIdx.x, nvec = (cols + 7) / 8;
    const int64_t row = blockIdx.x;
    const float mu = mean[row], r = rstd[row];
    // f(h, g, which of the eight are the vector's own)
    auto each = [&](auto f) {
        for (int k = t; k < nvec; k += LN_LT) {
            const Vec8 at = vec8(k, cols);
            const Raw8<FT> a = load8_any<FT>(x, row * ldx + at.at), b = load8_any<FT>(dy, row * lddy + at.at);
            float h[8], g[8], w[8];
            widen8_rt(load8_rt(weight, wdt, at.at), weight, wdt, 1.0f, w);
            widen8<FT>(a, h);
            widen8<FT>(b, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                h[i] = (h[i] - mu) * r;
                g[i] *= w[i];
            }
            f(h, g, at);
        }
    };
    float sg = 0.0f, sgh = 0.0f;
    each([&](const float h[8], const float g[8], Vec8 at) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float gg = i >= at.lo ? g[i] : 0.0f;
            sg += gg;
            sgh = __builtin_fmaf(gg, i >= at.lo ? h[i] : 0.0f, sgh);
        }
    });
    const float c1 = row_sum<LN_LT>(sg, slots[0]) / (float)cols, c2 = row_sum<LN_LT>(sgh, slots[1]) / (float)cols;
    each([&](const float h[8], float g[8], Vec8 at) {
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] = (g[i] - c1 - h[i] * c2) * r;
        store8_own<FT>(dx, row * cols, at, g);
    });
}

template <int FT>
__global__ __launch_bounds__(256) void k_ln_bwd_cols(const void* __restrict__ dy, int64_t lddy,
                                                     const void* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                     int64_t chunk, const float* __restrict__ mean,
                                                     const float* __restrict__ rstd, float* __restrict__ part,
                                                     int64_t ldp)
{
    constexpr int U = 4;
    __shared__ float fold[3][2][8][64];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const Vec8 at = vec8((int)blockIdx.x * 64 + lane, cols);
    const int64_t r0 = blockIdx.y * chunk, r1 = r0 + chunk < rows ? r0 + chunk : rows;
    float dw[8], db[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        dw[i] = 0.0f;
        db[i] = 0.0f;
    }
    for (int64_t r = r0 + w; r < r1; r += 4 * U) {
        Raw8<FT> a[U], b[U];
        float mu[U], rs[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t row = r + 4 * u < r1 ? r + 4 * u : r1 - 1;
            mu[u] = mean[row];
            rs[u] = rstd[row];
            a[u] = load8_any<FT>(x, row * ldx + at.at);
            b[u] = load8_any<FT>(dy, row * lddy + at.at);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (r + 4 * u >= r1) break;
            float h[8], d[8];
            widen8<FT>(a[u], h);
            widen8<FT>(b[u], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                dw[i] = __builtin_fmaf(d[i], (h[i] - mu[u]) * rs[u], dw[i]);
                db[i] += d[i];
            }
        }
    }
    if (w > 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            fold[w - 1][0][i][lane] = dw[i];
            fold[w - 1][1][i][lane] = db[i];
        }
    }
    __syncthreads();
    if (w > 0 || at.lo == 8) return;
#pragma unroll
    for (int k = 0; k < 3; ++k)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            dw[i] += fold[k][0][i][lane];
            db[i] += fold[k][1][i][lane];
        }
    float* to = part + (int64_t)blockIdx.y * 2 * ldp;
    store8_own<F32>(to, 0, at, dw);
    store8_own<F32>(to + ldp, 0, at, db);
}

// Rows of fewer than 8 elements: a thread per row and step, [1000000, 7] bf16
// 45.5 us (a workgroup per row and column sums by single elements: 4640).
template <int FT>
__global__ __launch_bounds__(256) void k_ln_bwd_thin(const void* __restrict__ dy, int64_t lddy,
                                                     const void* __restrict__ x, int64_t ldx, int64_t rows, int cols,
                                                     int64_t chunk, const void* __restrict__ weight, int wdt,
                                                     const float* __restrict__ mean, const float* __restrict__ rstd,
                                                     void* __restrict__ dx, float* __restrict__ part, int64_t ldp)
{
    __shared__ float fold[4][2][7];
    const int t = threadIdx.x;
    const int64_t r0 = (int64_t)blockIdx.x * chunk, r1 = r0 + chunk < rows ? r0 + chunk : rows;
    float ww[7], dw[7], db[7];
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        ww[j] = j < cols ? load1_rt(weight, wdt, j, 1.0f) : 0.0f;
        dw[j] = 0.0f;
        db[j] = 0.0f;
    }
    for (int64_t r = r0 + t; r < r1; r += 256) {
        const float mu = mean[r], rs = rstd[r];
        float h[7], d[7], sg = 0.0f, sgh = 0.0f;
#pragma unroll
        for (int j = 0; j < 7; ++j) {
            h[j] = j < cols ? (load1<FT>(x, r * ldx + j) - mu) * rs : 0.0f;
            d[j] = j < cols ? load1<FT>(dy, r * lddy + j) : 0.0f;
            dw[j] = __builtin_fmaf(d[j], h[j], dw[j]);
            db[j] += d[j];
            sg = __builtin_fmaf(d[j], ww[j], sg);
            sgh = __builtin_fmaf(d[j] * ww[j], h[j], sgh);
        }
        const float c1 = sg / (float)cols, c2 = sgh / (float)cols;
        if (dx) {
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < cols) store1<FT>(dx, r * cols + j, (d[j] * ww[j] - c1 - h[j] * c2) * rs);
        }
    }
    if (!part) return;
#pragma unroll
    for (int j = 0; j < 7; ++j) {
        const float a = wave_sum(dw[j]), b = wave_sum(db[j]);
        if ((t & 63) == 0) {
            fold[t >> 6][0][j] = a;
            fold[t >> 6][1][j] = b;
        }
    }
    __syncthreads();
    if (t >= cols) return;
    float* to = part + (int64_t)blockIdx.x * 2 * ldp + t;
#pragma unroll
    for (int o = 0; o < 2; ++o) to[o * ldp] = fold[0][o][t] + fold[1][o][t] + fold[2][o][t] + fold[3][o][t];
}

// ------------------------------------------------------------- column sums
// k_colsum: a workgroup takes 32 columns of one output: 8 lanes of four columns by 32
// rows of partials at a time, U such loads under way per thread, then the
// 32 row sums in order through LDS.  Bound by latency: 8 MB of partials (256
// rows of 2 x 4096) take 4.7 us; slices of 256 columns, which leave most CUs
// without one, made the backward pass 45 us instead of 40.
__global__ __launch_bounds__(256) void k_colsum(const float* __restrict__ part, int64_t parts, int outs, int64_t ld,
                                                int64_t cols, void* __restrict__ out0, void* __restrict__ out1, int dt)
{
    constexpr int U = 8;
    __shared__ float4 sums[32][8];
    const int o = blockIdx.y;
    void* out = o ? out1 : out0;
    if (!out) return;            // uniform in the workgroup
    const int c4 = threadIdx.x & 7, rl = threadIdx.x >> 3;
    const int64_t col = (int64_t)blockIdx.x * 32 + 4 * c4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (col < cols) {
        for (int64_t p = rl; p < parts; p += 32 * U) {
            float4 a[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int64_t q = p + 32 * k < parts ? p + 32 * k : p;
                a[k] = *reinterpret_cast<const float4*>(part + (q * outs + o) * ld + col);
            }
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (p + 32 * k < parts) {
                    s.x += a[k].x;
                    s.y += a[k].y;
                    s.z += a[k].z;
                    s.w += a[k].w;
                }
        }
    }
    sums[rl][c4] = s;
    __syncthreads();
    const int c = threadIdx.x;
    const int64_t j = (int64_t)blockIdx.x * 32 + c;
    if (c >= 32 || j >= cols) return;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) v += reinterpret_cast<const float*>(&sums[k][c >> 2])[c & 3];
    store1_rt(out, dt, j, v);
}

void colsum_launch(const float* part, int64_t parts, int outs, int64_t ld, int64_t cols, void* out0, void* out1,
                   int dt, hipStream_t st)
{
    constexpr int64_t MOST = 1 << 28;    // columns per launch: 2^31 threads
    for (int64_t c = 0; c < cols; c += MOST) {
        const int64_t n = std::min(cols - c, MOST);
        const dim3 grid((unsigned)cdiv(n, 32), out1 ? 2u : 1u);
        hipLaunchKernelGGL(k_colsum, grid, dim3(256), 0, st, part + c, parts, outs, ld, n,
                           forward_by(out0, c * ftype_size(dt)), forward_by(out1, c * ftype_size(dt)), dt);
    }
}

// ---------------------------------------------------------------- launches
constexpr int64_t LN_HELD = 16384;       // longest row that a workgroup holds in registers
constexpr int64_t LN_BWD_HELD = 16384;   // and that of dy beside it; half as many in binary32
constexpr int64_t LN_PARTS = 256;        // workgroups of the backward pass, one row of partials each
constexpr int64_t LN_COL_CHUNKS = 64;    // row chunks of the column kernel of longer rows
// Most rows per launch of the kernels that give every row its own threads, up to
// 1024: a grid holds fewer than 2^32 threads.  Further rows are further launches.
constexpr int64_t LN_LAUNCH = 1 << 21;

// Threads and vectors per row, measured on 8192 rows (us, taken / next best):
//   1024 bf16  64 x 2  11.0 / 13.3 (256 x 1)     4096 bf16  256 x 2  23.5 / 25.5 (512 x 1)
//   2048 bf16  256 x 1 14.6 / 16.1 (64 x 4)      8192 bf16  512 x 2  54.3 / 53.6 (1024 x 1)
//   2048 f32   256 x 1 24.0 / 27.4 (64 x 4)     16384 bf16 1024 x 2  66.5 (4096 rows)
// A wave per row needs no barrier while its registers hold the row lightly;
// beyond that two vectors per thread keep enough loads under way.
template <int FT, int OUT>
static void ln_launch(const void* x, int64_t ldx, int64_t rows, int64_t cols, const void* w, const void* b, int wdt,
                      float eps, void* y, float* scale, float* mean, float* rstd, hipStream_t st)
{
    for (; rows > LN_LAUNCH; rows -= LN_LAUNCH) {
        ln_launch<FT, OUT>(x, ldx, LN_LAUNCH, cols, w, b, wdt, eps, y, scale, mean, rstd, st);
        x = forward_by(x, LN_LAUNCH * ldx * ftype_size(FT));
        y = forward_by(y, LN_LAUNCH * cols * (OUT == OUT_Y ? ftype_size(FT) : 1));
        scale = forward_by(scale, 4 * LN_LAUNCH);
        mean = forward_by(mean, 4 * LN_LAUNCH);
        rstd = forward_by(rstd, 4 * LN_LAUNCH);
    }
#define TQ_LN(NT, W)                                                                                              \
    hipLaunchKernelGGL((k_ln_rows<FT, NT, W, OUT>), dim3((unsigned)cdiv(rows, NT < 256 ? 256 / NT : 1)),          \
                       dim3(NT < 256 ? 256 : NT), 0, st, x, ldx, rows, cols, w, b, wdt, eps, y, scale, mean, rstd)
    if (cols < 8)
        hipLaunchKernelGGL((k_ln_thin<FT, OUT>), dim3((unsigned)cdiv(rows, 256)), dim3(256), 0, st, x, ldx, rows,
                           (int)cols, w, b, wdt, eps, y, scale, mean, rstd);
    else if (cols > LN_HELD)
        hipLaunchKernelGGL((k_ln_long<FT, OUT>), dim3((unsigned)rows), dim3(LN_LT), 0, st, x, ldx, (int)cols, w, b, wdt,
                           eps, y, scale, mean, rstd);
    else if (cols <= 512) TQ_LN(64, 1);
    else if (cols <= 1024) TQ_LN(64, 2);
    else if (cols <= 2048) TQ_LN(256, 1);
    else if (cols <= 4096) TQ_LN(256, 2);
    else if (cols <= 8192) TQ_LN(512, 2);
    else TQ_LN(1024, 2);
#undef TQ_LN
}

// Workgroup count of the backward pass: the rows are dealt out evenly.
inline int64_t ln_bwd_groups(int64_t rows, int teams)
{
    const int64_t want = cdiv(rows, teams);
    return want < LN_PARTS ? want : LN_PARTS;
}

// Threads and vectors per row, 8192 rows (us, taken / next best): 1024 f32
// 128 x 1 21.4 / 22.9 (64 x 2), 2048 f32 256 x 1 38.0 / 39.4 (128 x 2), 4096
// bf16 256 x 2 40.2 / 42.5 (512 x 1), 8192 bf16 512 x 2 81 / 80 (1024 x 1).
template <int FT>
static void ln_bwd_launch(const void* dy, int64_t lddy, const void* x, int64_t ldx, int64_t rows, int64_t cols,
                          const void* w, int wdt, const float* mean, const float* rstd, void* dx, void* dw, void* db,
                          float* ws, hipStream_t st)
{
    const int64_t ld = colsum_ld(cols);
    float* part = dw || db ? ws : nullptr;
    int64_t parts = 0;
#define TQ_LNB(NT, W, BT)                                                                                         \
    do {                                                                                                          \
        parts = ln_bwd_groups(rows, BT / NT);                                                                     \
        hipLaunchKernelGGL((k_ln_bwd<FT, NT, W, BT>), dim3((unsigned)parts), dim3(BT), 0, st, dy, lddy, x, ldx,   \
                           rows, cols, w, wdt, mean, rstd, dx, part, ld);                                         \
    } while (0)
    if (cols < 8) {
        const int64_t chunk = cdiv(cdiv(rows, LN_PARTS), 256) * 256;
        parts = cdiv(rows, chunk);
        hipLaunchKernelGGL((k_ln_bwd_thin<FT>), dim3((unsigned)parts), dim3(256), 0, st, dy, lddy, x, ldx, rows,
                           (int)cols, chunk, w, wdt, mean, rstd, dx, part, ld);
    } else if (cols > (FT == F32 ? LN_BWD_HELD / 2 : LN_BWD_HELD)) {
        if (part) {
            const int64_t chunk = cdiv(cdiv(rows, LN_COL_CHUNKS), 16) * 16;
            parts = cdiv(rows, chunk);
            hipLaunchKernelGGL((k_ln_bwd_cols<FT>), dim3((unsigned)cdiv(cols, 512), (unsigned)parts), dim3(256), 0, st,
                               dy, lddy, x, ldx, rows, (int)cols, chunk, mean, rstd, part, ld);
        }
        for (int64_t r = 0; dx && r < rows; r += LN_LAUNCH)
            hipLaunchKernelGGL((k_ln_bwd_long<FT>), dim3((unsigned)std::min(rows - r, LN_LAUNCH)), dim3(LN_LT), 0, st,
                               forward_by(dy, r * lddy * ftype_size(FT)), lddy,
                               forward_by(x, r * ldx * ftype_size(FT)), ldx, (int)cols, w, wdt, mean + r, rstd + r,
                               forward_by(dx, r * cols * ftype_size(FT)));
    }
    else if (cols <= 512) TQ_LNB(64, 1, 512);
    else if (cols <= 1024) TQ_LNB(128, 1, 512);
    else if (cols <= 2048) TQ_LNB(256, 1, 512);
    else if (cols <= 4096) TQ_LNB(256, 2, 512);
    else if (cols <= 8192) TQ_LNB(512, 2, 512);
    else if constexpr (FT != F32) TQ_LNB(1024, 2, 1024);
#undef TQ_LNB
    if (part) colsum_launch(part, parts, 2, ld, cols, dw, db, wdt, st);
}

__global__ __launch_bounds__(256) void k_zero_vec(void* __restrict__ p, int dt, int64_t n)
{
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += 256 * (int64_t)gridDim.x)
        store1_rt(p, dt, i, 0.0f);
}

void zero_vec_launch(void* p, int dt, int64_t n, hipStream_t st)
{
    if (p && n > 0) hipLaunchKernelGGL(k_zero_vec, dim3(grid_for(n, 256)), dim3(256), 0, st, p, dt, n);
}

static bool natural(const void* p, int dt) { return ((uintptr_t)p & (uintptr_t)(ftype_size(dt) - 1)) == 0; }

// Columns are counted in 32 bits, a slab past their end.
static bool ln_fits(int64_t rows, int64_t cols)
{
    return rows <= 0x7fffffff && cols <= 0x7fffffff - 1024;
}

static tq_status ln_check(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t ldx, const void* w,
                          const void* b, int wdt, float eps)
{
    if (!valid_ftype(x_dtype) || rows < 0 || cols < 0 || !(eps >= 0.0f)) return TQ_ERR_INVALID;
    if ((w || b) && !valid_ftype(wdt)) return TQ_ERR_INVALID;
    if (rows == 0 || cols == 0) return TQ_OK;
    if (!x || ldx < cols) return TQ_ERR_INVALID;
    if (!ln_fits(rows, cols)) return TQ_ERR_UNSUPPORTED;
    if (!natural(x, x_dtype) || (w && !natural(w, wdt)) || (b && !natural(b, wdt))) return TQ_ERR_ALIGN;
    return TQ_OK;
}

}  // namespace tq

using namespace tq;

extern "C" {

tq_status tq_layer_norm(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t x_row_stride,
                        const void* weight, const void* bias, int w_dtype, float eps, void* y, float* mean,
                        float* rstd, void* stream)
{
    const tq_status s = ln_check(x, x_dtype, rows, cols, x_row_stride, weight, bias, w_dtype, eps);
    if (s != TQ_OK || rows == 0 || cols == 0) return s;
    if (!y) return TQ_ERR_INVALID;
    if (!natural(y, x_dtype) || !natural(mean, TQ_F32) || !natural(rstd, TQ_F32)) return TQ_ERR_ALIGN;
    TQ_LLM_FT_SWITCH(x_dtype, (ln_launch<FTV, OUT_Y>(x, x_row_stride, rows, cols, weight, bias, w_dtype, eps, y,
                                                     nullptr, mean, rstd, as_stream(stream))));
    return launch_status();
}

tq_status tq_layer_norm_quant_per_token(const void* x, int x_dtype, int64_t rows, int64_t cols, int64_t x_row_stride,
                                        const void* weight, const void* bias, int w_dtype, float eps, int8_t* q,
                                        float* scale, float* mean, float* rstd, void* stream)
{
    const tq_status s = ln_check(x, x_dtype, rows, cols, x_row_stride, weight, bias, w_dtype, eps);
    if (s != TQ_OK || rows == 0 || cols == 0) return s;
    if (!q || !scale) return TQ_ERR_INVALID;
    if (!natural(scale, TQ_F32) || !natural(mean, TQ_F32) || !natural(rstd, TQ_F32)) return TQ_ERR_ALIGN;
    TQ_LLM_FT_SWITCH(x_dtype, (ln_launch<FTV, OUT_S8>(x, x_row_stride, rows, cols, weight, bias, w_dtype, eps, q,
                                                      scale, mean, rstd, as_stream(stream))));
    return launch_status();
}

size_t tq_layer_norm_backward_workspace_bytes(int64_t rows, int64_t cols)
{
    if (rows <= 0 || cols <= 0) return 0;
    const int64_t parts = cols > LN_BWD_HELD ? LN_COL_CHUNKS : LN_PARTS;
    return (size_t)(rows < parts ? rows : parts) * 2 * (size_t)colsum_ld(cols) * sizeof(float);
}

tq_status tq_layer_norm_backward(const void* dy, const void* x, int x_dtype, int64_t rows, int64_t cols,
                                 int64_t dy_row_stride, int64_t x_row_stride, const void* weight, int w_dtype,
                                 const float* mean, const float* rstd, void* dx, void* dweight, void* dbias,
                                 void* workspace, size_t workspace_bytes, void* stream)
{
    if ((dweight || dbias) && !valid_ftype(w_dtype)) return TQ_ERR_INVALID;
    const tq_status s = ln_check(x, x_dtype, rows, cols, x_row_stride, weight, nullptr, w_dtype, 0.0f);
    if (s != TQ_OK || cols == 0) return s;
    if ((dweight && !natural(dweight, w_dtype)) || (dbias && !natural(dbias, w_dtype))) return TQ_ERR_ALIGN;
    hipStream_t st = as_stream(stream);
    if (rows == 0) {             // no rows: the sums are empty, not unwritten
        zero_vec_launch(dweight, w_dtype, cols, st);
        zero_vec_launch(dbias, w_dtype, cols, st);
        return launch_status();
    }
    if (!dy || !mean || !rstd || dy_row_stride < cols) return TQ_ERR_INVALID;
    if (!dx && !dweight && !dbias) return TQ_OK;
    if (!natural(dy, x_dtype) || !natural(dx, x_dtype) || !natural(mean, TQ_F32) || !natural(rstd, TQ_F32))
        return TQ_ERR_ALIGN;
    if (dweight || dbias) {
        if (!workspace || workspace_bytes < tq_layer_norm_backward_workspace_bytes(rows, cols)) return TQ_ERR_INVALID;
        if (!aligned16(workspace)) return TQ_ERR_ALIGN;
    }
    TQ_LLM_FT_SWITCH(x_dtype, (ln_bwd_launch<FTV>(dy, dy_row_stride, x, x_row_stride, rows, cols, weight, w_dtype, mean,
                                                  rstd, dx, dweight, dbias, static_cast<float*>(workspace), st)));
    return launch_status();
}

}  // extern "C"
