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

// The same eight values as they lie in memory, loaded ahead of their use (VEC rows only).
template <typename T> struct Raw8 {
    uint4 q[sizeof(T) / 2];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) q[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        if (sizeof(T) == 2) {
            const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < (int)sizeof(T) / 2; ++i) {
                v[4 * i] = __uint_as_float(q[i].x); v[4 * i + 1] = __uint_as_float(q[i].y);
                v[4 * i + 2] = __uint_as_float(q[i].z); v[4 * i + 3] = __uint_as_float(q[i].w);
            }
        }
    }
};

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
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// 1 / (1 + exp(-x)): 1 ulp from each of the three steps; exp(-x) may overflow, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid(float x) { return rcp(1.f + ex2(-LOG2E * x)); }
__device__ __forceinline__ float silu(float x) { return x * sigmoid(x); }
// silu'(x) = s (1 + x (1 - s)), s = sigmoid(x)
__device__ __forceinline__ float dsilu(float x, float s) { return s * (1.f + x * (1.f - s)); }
// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|) in [0, 1], without a branch, two at a time.
// log1p(e) / e is a polynomial of degree 8 fitted on [0, 1] at Chebyshev points (3e-8 relative, 2.8 U with its
// fp32 rounding); a small e keeps its relative accuracy.
__device__ __forceinline__ f2 softplus2(f2 x)
{
    const float2 v = unpack2(x);
    const float2 m = make_float2(fabsf(v.x) * -LOG2E, fabsf(v.y) * -LOG2E);
    const f2 e = pack2(ex2(m.x), ex2(m.y));
    const float c[9] = {1.0f, -0.49999502301216125f, 0.33319270610809326f, -0.24844369292259216f, 0.19111430644989014f,
                        -0.13674770295619965f, 0.07836166769266129f, -0.02958850748836994f, 0.005253457929939032f};
    f2 p = pack2(c[8], c[8]);
#pragma unroll
    for (int k = 7; k >= 0; --k) p = fma2(p, e, pack2(c[k], c[k]));
    return fma2(p, e, pack2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus(float x) { return unpack2(softplus2(pack2(x, 0.f))).x; }

// A log2(e) of A = -exp(a_log), kept finite: the decay of a delta of zero (the tokens behind a sequence's
// end) is one whatever the rate.  Not fmaxf, which would turn a NaN into a rate.
__device__ __forceinline__ float decay_rate(float a_log)
{
    const float r = -expf(a_log) * LOG2E;
    return r < -3e38f ? -3e38f : r;
}

__device__ __forceinline__ int row_length(const int *lengths, int b, int N)
{
    return lengths ? min(max(lengths[b], 0), N) : N;
}

// Launches of one call follow one another by programmatic dependent launch: a kernel lets the next one be
// scheduled when it starts, and waits for the one before it to finish where it first reads what that
// wrote, or before it returns.  A call's first launch is an ordinary one, which waits for all work
// before the call, and its last one lets nothing start early.
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

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

// Adds up rows of partial sums in a fixed order, up to MAX_SUMS vectors in one launch: element i of a
// vector is the sum over r < rows of part[r * row_stride + i], and goes to out[i * out_stride].
struct SumVec {
    const float *part;
    long long row_stride, n;
    float *out;
    long long out_stride;
};
constexpr int MAX_SUMS = 5;
struct SumList {
    SumVec v[MAX_SUMS];
    unsigned first[MAX_SUMS + 1];        // first block of each vector; [count]: how many there are
    int count;
    long long rows;
};
SumList sum_list(const SumVec *vecs, int count, long long rows);

// A block of 256 threads' share: 32 columns (one 128-byte line a row), eight warps of four independent sums each over
// every 32nd row, then the warps in order.  The partial rows were just written and come from L2.
__device__ __forceinline__ void sum_rows_block(const SumList &l, unsigned block)
{
    __shared__ float s[8][33];
    int k = 0;
#pragma unroll
    for (int j = 1; j < MAX_SUMS; ++j)
        if (j < l.count && block >= l.first[j]) k = j;
    const SumVec v = l.v[k];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long i = (long long)(block - l.first[k]) * 32 + lane;
    float a[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < v.n) {
        const float *p = v.part + i;
        long long r = warp;
        for (; r + 24 < l.rows; r += 32)
#pragma unroll
            for (int u = 0; u < 4; ++u) a[u] += p[(r + 8 * u) * v.row_stride];
        for (; r < l.rows; r += 8) a[0] += p[r * v.row_stride];
    }
    s[warp][lane] = (a[0] + a[1]) + (a[2] + a[3]);
    __syncthreads();
    if (warp == 0 && i < v.n) {
        float t = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += s[w][lane];
        v.out[i * v.out_stride] = t;
    }
}

gma_status_t sum_rows(const SumVec *vecs, int count, long long rows, cudaStream_t st);

inline bool ws_ok(const void *ws, size_t have, size_t need)
{
    return need == 0 || (ws && ((uintptr_t)ws & 255u) == 0 && have >= need);
}

}  // namespace blk
}  // namespace gma
