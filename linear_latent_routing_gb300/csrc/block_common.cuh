// block_common.cuh -- what the kernels behind gma_block.h share: rows with strides, eight channels
// at a time, packed fp32 pairs, and the host-side checks of gma_rows_t.
#pragma once

#include "gma_block.h"
#include "gma_internal.cuh"

namespace gma {
namespace blk {

constexpr float LOG2E = 1.4426950408889634f;

// ------------------------------------------------------------------ rows
template <typename T> struct Rows {
    T *p;
    long long sb, st;   // element strides between batch rows and tokens
    __device__ __forceinline__ T *at(int b, int t) const { return p + (long long)b * sb + (long long)t * st; }
};

template <typename T> inline Rows<T> rows_of(const gma_rows_t &r)
{
    return Rows<T>{(T *)r.ptr, (long long)r.batch, (long long)r.token};
}

// Eight neighbouring channels as fp32: 16-byte accesses (the caller has checked alignment and that
// all eight exist), or the first n of them one by one.
template <bool VEC> __device__ __forceinline__ void load8(const __nv_bfloat16 *p, int n, float (&v)[8])
{
    if (VEC) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}

template <bool VEC> __device__ __forceinline__ void load8(const float *p, int n, float (&v)[8])
{
    if (VEC) {
        const float4 a = reinterpret_cast<const float4 *>(p)[0];
        const float4 b = reinterpret_cast<const float4 *>(p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}

template <bool VEC> __device__ __forceinline__ void store8(__nv_bfloat16 *p, int n, const float (&v)[8])
{
    if (VEC) {
        uint4 q;
        __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&q);
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        *reinterpret_cast<uint4 *>(p) = q;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}

template <bool VEC> __device__ __forceinline__ void store8(float *p, int n, const float (&v)[8])
{
    if (VEC) {
        reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}

// ------------------------------------------------------------------ packed fp32 pairs
// Two fp32 values in one 64-bit register pair: one instruction works on both (each half rounds as
// the scalar instruction does).
typedef unsigned long long f2;

__device__ __forceinline__ f2 pack2(float lo, float hi)
{
    f2 d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ float2 unpack2(f2 v)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c)
{
    f2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b)
{
    f2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b)
{
    f2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// ------------------------------------------------------------------ functions
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ f2 ex2_2(f2 v)
{
    const float2 x = unpack2(v);
    return pack2(ex2(x.x), ex2(x.y));
}
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }
__device__ __forceinline__ float silu(float x) { return __fdividef(x, 1.f + __expf(-x)); }
// silu'(x) = s (1 + x (1 - s)), s = sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * (1.f + x * (1.f - s)); }
__device__ __forceinline__ float softplus(float x) { return x > 20.f ? x : log1pf(__expf(x)); }

__device__ __forceinline__ int row_length(const int *lengths, int b, int N)
{
    return lengths ? min(max(lengths[b], 0), N) : N;
}

// ------------------------------------------------------------------ host-side checks
inline size_t elem_size(int dtype) { return dtype == GMA_BF16 ? 2 : 4; }

// Rows that can be used: aligned to their elements, strides that are not negative.  Output rows
// must not overlap one another either.
inline bool rows_ok(const gma_rows_t &r, int dtype, long long B, long long N, long long width, bool out)
{
    if (!r.ptr || ((uintptr_t)r.ptr & (elem_size(dtype) - 1)) || r.batch < 0 || r.token < 0) return false;
    if (!out) return true;
    if (N > 1 && r.token < width) return false;
    if (B > 1 && r.batch < width) return false;
    // token rows nested in batch rows, or batch rows nested in token rows
    return B == 1 || N == 1 || r.batch >= (N - 1) * r.token + width || r.token >= (B - 1) * r.batch + width;
}

// Whether 16-byte accesses at multiples of eight channels are aligned in every row.
inline bool rows_vec(const gma_rows_t &r, int dtype)
{
    const size_t e = elem_size(dtype);
    return (((uintptr_t)r.ptr | (uintptr_t)(r.batch * e) | (uintptr_t)(r.token * e)) & 15u) == 0;
}

inline bool ptr_ok(const void *p, size_t align) { return p && ((uintptr_t)p & (align - 1)) == 0; }
inline bool opt_ok(const void *p, size_t align) { return ((uintptr_t)p & (align - 1)) == 0; }

// Adds up the first K of `per_row` vectors of n fp32 values (vector stride pitch, row stride
// per_row * pitch) over `rows` rows in a fixed order: vector k's element i goes to out[k].p[i * out[k].stride].
struct SumOut {
    float *p;
    long long stride;
};
constexpr int MAX_SUMS = 5;
gma_status_t sum_rows(const float *part, long long rows, int K, int per_row, int n, int pitch, const SumOut *out,
                      cudaStream_t st);

inline bool ws_ok(const void *ws, size_t have, size_t need)
{
    return need == 0 || (ws && ((uintptr_t)ws & 255u) == 0 && have >= need);
}

}  // namespace blk
}  // namespace gma
