// tq_llm.h -- device helpers of the operators around a quantized layer
// (layer norm, the W8A8 product's epilogue, distillation): lane sums, vectors
// of eight elements at any element alignment, parameters whose type is known
// at run time, and the column sums that finish a weight's or a bias's gradient.
#pragma once

#include <type_traits>

#include "tq_device.h"
#include "tq_host.h"

namespace tq {

constexpr float LOG2E = 1.44269504088896340736f;
constexpr float LN2 = 0.69314718055994530942f;

// ------------------------------------------------------------------ lanes
__device__ __forceinline__ float lane_get(float v, int ctrl_xor)
{
    return __shfl_xor(v, ctrl_xor, 64);
}

// Sum / maximum over the wave's 64 lanes, the same bits in every lane (the
// tree is symmetric, so each lane adds the same pairs).
__device__ __forceinline__ float wave_sum(float v)
{
    v += as_f(dpp<DPP_XOR1>(as_u(v)));
    v += as_f(dpp<DPP_XOR2>(as_u(v)));
    v += as_f(dpp<DPP_HALF_MIRROR>(as_u(v)));
    v += as_f(dpp<DPP_MIRROR>(as_u(v)));
    v += lane_get(v, 16);
    v += lane_get(v, 32);
    return v;
}

__device__ __forceinline__ float wave_max(float v)
{
    v = __builtin_fmaxf(v, as_f(dpp<DPP_XOR1>(as_u(v))));
    v = __builtin_fmaxf(v, as_f(dpp<DPP_XOR2>(as_u(v))));
    v = __builtin_fmaxf(v, as_f(dpp<DPP_HALF_MIRROR>(as_u(v))));
    v = __builtin_fmaxf(v, as_f(dpp<DPP_MIRROR>(as_u(v))));
    v = __builtin_fmaxf(v, lane_get(v, 16));
    v = __builtin_fmaxf(v, lane_get(v, 32));
    return v;
}

// ---------------------------------------------------------------- vectors
// Eight consecutive elements at any element-aligned address.  The global
// memory instructions take 16-byte accesses at any 2-byte address, so rows of
// an odd width or a sliced tensor need no scalar path; an access that crosses
// a cache line costs one more line.
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(1)));

template <bool NT = false>
__device__ __forceinline__ uint4 ld16_any(const void* p)
{
    u32x4_any v;
    if constexpr (NT) v = __builtin_nontemporal_load(static_cast<const u32x4_any*>(p));
    else v = *static_cast<const u32x4_any*>(p);
    return make_uint4(v.x, v.y, v.z, v.w);
}

template <bool NT = false>
__device__ __forceinline__ void st16_any(void* p, uint4 w)
{
    const u32x4_any v = {w.x, w.y, w.z, w.w};
    if constexpr (NT) __builtin_nontemporal_store(v, static_cast<u32x4_any*>(p));
    else *static_cast<u32x4_any*>(p) = v;
}

template <int FT, bool NT = false>
__device__ __forceinline__ Raw8<FT> load8_any(const void* base, int64_t e)
{
    Raw8<FT> r;
    if constexpr (FT == F32) {
        const float* p = static_cast<const float*>(base) + e;
        r.w[0] = ld16_any<NT>(p);
        r.w[1] = ld16_any<NT>(p + 4);
    } else {
        r.w[0] = ld16_any<NT>(static_cast<const uint16_t*>(base) + e);
    }
    return r;
}

template <int FT, bool NT = false>
__device__ __forceinline__ void store8_any(void* base, int64_t e, const float v[8])
{
    if constexpr (FT == F32) {
        float* p = static_cast<float*>(base) + e;
        st16_any<NT>(p, make_uint4(as_u(v[0]), as_u(v[1]), as_u(v[2]), as_u(v[3])));
        st16_any<NT>(p + 4, make_uint4(as_u(v[4]), as_u(v[5]), as_u(v[6]), as_u(v[7])));
    } else {
        st16_any<NT>(static_cast<uint16_t*>(base) + e,
                     make_uint4(narrow2<FT>(v[0], v[1]), narrow2<FT>(v[2], v[3]), narrow2<FT>(v[4], v[5]),
                                narrow2<FT>(v[6], v[7])));
    }
}

// The same from a uniform row address and a 32-bit byte offset per lane, which
// costs one register per vector instead of two.
template <int FT, bool NT = false>
__device__ __forceinline__ Raw8<FT> load8_off(const void* row, uint32_t off)
{
    const char* p = static_cast<const char*>(row) + off;
    Raw8<FT> r;
    r.w[0] = ld16_any<NT>(p);
    if constexpr (FT == F32) r.w[1] = ld16_any<NT>(p + 16);
    return r;
}
template <int FT, bool NT = false>
__device__ __forceinline__ void store8_off(void* row, uint32_t off, const float v[8])
{
    store8_any<FT, NT>(static_cast<char*>(row) + off, 0, v);
}

// Makes a raw vector opaque, so that values widened from it before are widened
// again after, instead of being held in twice the registers.
template <int FT>
__device__ __forceinline__ void keep_raw(Raw8<FT>& r)
{
#pragma unroll
    for (int i = 0; i < (FT == F32 ? 2 : 1); ++i) {
        u32x4 v = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
        asm("" : "+v"(v));
        r.w[i] = make_uint4(v.x, v.y, v.z, v.w);
    }
}

// The same for an index: what is computed from it is computed again.
__device__ __forceinline__ int afresh(int v)
{
    asm volatile("" : "+v"(v));
    return v;
}

__device__ __forceinline__ int afresh_uniform(int v)
{
    asm volatile("" : "+s"(v));
    return v;
}

// Vector v of a row of n >= 8 elements: it starts at element `at`, and its
// elements lo .. 7 are its own.  Only the last vector of a row whose length is
// no multiple of 8 has lo > 0: it is moved back to end with the row, so every
// load stays inside the row and none needs a branch.  Past the row lo is 8.
struct Vec8 {
    int at, lo;
};
__device__ __forceinline__ Vec8 vec8(int v, int n)
{
    const int e = 8 * v;
    Vec8 r;
    r.at = e < n - 8 ? e : n - 8;
    r.lo = e - r.at < 8 ? e - r.at : 8;
    return r;
}

// Stores the vector's own elements.
template <int FT, bool NT = false>
__device__ __forceinline__ void store8_own(void* base, int64_t row, Vec8 q, const float v[8])
{
    if (__builtin_expect(q.lo == 0, 1)) {
        store8_any<FT, NT>(base, row + q.at, v);
    } else {
#pragma unroll
        for (int i = 1; i < 8; ++i)
            if (i >= q.lo) store1<FT>(base, row + q.at + i, v[i]);
    }
}

// ------------------------------------------------- parameters of a layer
// A weight, bias or gradient vector in a type known at run time (the branch
// is uniform); null reads as `none`.  Raw and widened apart, so that the loads
// can be issued long before their use.
struct RawAny {
    uint4 w[2];
};
__device__ __forceinline__ RawAny load8_rt(const void* p, int dt, int64_t e)
{
    RawAny r;
    r.w[0] = make_uint4(0, 0, 0, 0);
    r.w[1] = make_uint4(0, 0, 0, 0);
    if (p) {
        if (dt == F32) {
            r.w[0] = ld16_any(static_cast<const float*>(p) + e);
            r.w[1] = ld16_any(static_cast<const float*>(p) + e + 4);
        } else {
            r.w[0] = ld16_any(static_cast<const uint16_t*>(p) + e);
        }
    }
    return r;
}
__device__ __forceinline__ void widen8_rt(const RawAny& r, const void* p, int dt, float none, float v[8])
{
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = none;
    } else if (dt == F32) {
        Raw8<F32> q;
        q.w[0] = r.w[0];
        q.w[1] = r.w[1];
        widen8<F32>(q, v);
    } else if (dt == BF16) {
        Raw8<BF16> q;
        q.w[0] = r.w[0];
        widen8<BF16>(q, v);
    } else {
        Raw8<F16> q;
        q.w[0] = r.w[0];
        widen8<F16>(q, v);
    }
}
__device__ __forceinline__ float load1_rt(const void* p, int dt, int64_t e, float none)
{
    if (!p) return none;
    return dt == F32 ? load1<F32>(p, e) : dt == BF16 ? load1<BF16>(p, e) : load1<F16>(p, e);
}
__device__ __forceinline__ void store1_rt(void* p, int dt, int64_t e, float v)
{
    if (dt == F32) store1<F32>(p, e, v);
    else if (dt == BF16) store1<BF16>(p, e, v);
    else store1<F16>(p, e, v);
}

// ------------------------------------------------------------ column sums
// The second half of a sum down the rows of a matrix: the first half left
// `parts` rows of partial sums (binary32), part p's output o at
// part[(p * outs + o) * ld + col].  Adds them in a fixed order and writes
// output o in type dt to out[o] (null outputs are skipped).  ld is a multiple
// of 4.  Defined in tq_norm.hip.
void colsum_launch(const float* part, int64_t parts, int outs, int64_t ld, int64_t cols, void* out0, void* out1,
                   int dt, hipStream_t st);
// Zeros of a vector of n elements of type dt (null: nothing).
void zero_vec_launch(void* p, int dt, int64_t n, hipStream_t st);
inline int64_t colsum_ld(int64_t cols) { return (cols + 3) / 4 * 4; }

// The address `bytes` further on; null stays null.
template <class T>
inline T* forward_by(T* p, int64_t bytes)
{
    typedef std::conditional_t<std::is_const_v<T>, const char, char> byte;
    return p ? reinterpret_cast<T*>(reinterpret_cast<byte*>(p) + bytes) : p;
}

#define TQ_LLM_FT_SWITCH(ft, ...)                              \
    do {                                                       \
        if ((ft) == TQ_F32) { constexpr int FTV = F32; __VA_ARGS__; }        \
        else if ((ft) == TQ_F16) { constexpr int FTV = F16; __VA_ARGS__; }   \
        else { constexpr int FTV = BF16; __VA_ARGS__; }                      \
    } while (0)

}  // namespace tq
