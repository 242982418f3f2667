// logits.cuh -- what the kernels on the language model's logits share: a row's
// layout, its loads, the pass that gives its softmax statistics, and the host
// side's choice of threads.
//
// A row is one position of one stream: V logits that start at any element. It
// is cut into 16-byte vectors on aligned addresses (the first and the last may
// be partly outside the row: their outside elements read as -inf and are never
// stored), and thread t of the TH that share a row takes vectors t, t + TH, ...
// Up to NV vectors per thread are kept in registers, so a gradient reads its
// row once; a longer part is walked in chunks of TH * NV vectors.
//
// Every statistic comes from m = max x, s = sum 2^t_i and w = sum 2^t_i t_i with
// t_i = log2(e) c (x_i - m), c = scale, all in float32:
//     lse = c m + ln s,  ln p_i = c (x_i - m) - ln s,  entropy = ln s - ln 2 w / s.
// Each warp sums against its own maximum (one hardware reduction), so a row
// needs one barrier, where the warps' triples are joined; a row split over a
// cluster needs one cluster barrier more.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mimi_rvq.h"
#include "../../include/mimi_rvq_streams.h"
#include "ptx.cuh"

namespace mimi {
namespace logits {

constexpr int kMaxTop = MIMI_RVQ_MAX_TOP;
constexpr int kMaxCluster = 8;  // CTAs that may share a row (the portable cluster size)
constexpr float kInf = INFINITY;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr uint32_t kFull = 0xffffffffu;

// The rows of a logits tensor [S][n][V]; strides in elements.
struct RowsIn {
    const void* x;
    int64_t ss, sn;
    int64_t rows;  // S * n
    int n, V;
    float c;       // scale
    int cluster;   // CTAs per row (1: a row is one CTA's or one warp's)
};

// ------------------------------------------------------------------ elements

template <typename T>
struct Elem;
template <>
struct Elem<float> {
    static constexpr int kPer = 4;  // elements of a 16-byte vector
    static constexpr uint32_t kFill = 0xFF800000u;
};
template <>
struct Elem<__nv_bfloat16> {
    static constexpr int kPer = 8;
    static constexpr uint32_t kFill = 0xFF80FF80u;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float* p) { *p = v; }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

// element j of a vector
template <typename T>
__device__ __forceinline__ float element(const uint32_t (&w)[4], int j) {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[j]);
    else return __uint_as_float((j & 1) ? (w[j / 2] & 0xFFFF0000u) : (w[j / 2] << 16));
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(kFull));
    return r;
}
template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
    return v;
}

// Two float32 values in a 64-bit register pair and the instructions that work on both.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
    Pair p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
    return p;
}
__device__ __forceinline__ void halves(Pair p, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
    Pair d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
    Pair d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
    Pair d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Pair ex2_pair(Pair t) {
    float a, b;
    halves(t, a, b);
    return pair_of(ex2(a), ex2(b));
}
// max that keeps NaN
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Exponents t = log2(e) c (x - m) of a row's or warp's logits, 2^t = e^{c (x - m)}.
// Near: t = x c2 - ref in one fused multiply-add per logit, ref = m c2 rounded; t is then off by
// the same `shift` = m c2 - ref for every logit, at most 2^-9, which is taken back from the sums.
// Far (logits or scales beyond that): the difference first, then the product. With kFinite, t is
// at least -236 (2^t is 0 there too), so that 0 t is 0 for a logit of -inf; bf16 logits are
// clamped as pairs before they are widened.
constexpr float kLow = -300.f;
struct Scale {
    float c2, m, ref, shift;
    uint32_t floor_bf16x2;
    bool far;

    __device__ Scale(float c2_, float m_) : c2(c2_), m(m_ == -kInf ? 0.f : m_) {
        ref = m * c2;
        far = !(fabsf(ref) < 32768.f && c2 > 1.0e-33f && c2 < 1.0e30f);
        shift = far ? 0.f : fmaf(m, c2, -ref);
        const float f = __fdividef(ref + kLow, c2);
        floor_bf16x2 = far ? 0xFF80FF80u : pack_bf16x2(f, f);  // far: no floor here
    }
};
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T, bool kFinite>
__device__ __forceinline__ void exponents(const uint32_t (&w)[4], const Scale& k,
                                          Pair (&t)[Elem<T>::kPer / 2]) {
    constexpr int kPairs = Elem<T>::kPer / 2;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        if constexpr (sizeof(T) == 4) {
            t[j] = pair_of(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        } else {
            const uint32_t u = kFinite ? max_nan_bf16x2(w[j], k.floor_bf16x2) : w[j];
            t[j] = pair_of(bf16_lo_to_f32(u), bf16_hi_to_f32(u));
        }
    }
    if (!k.far) {
        const Pair c = pair_of(k.c2, k.c2), r = pair_of(-k.ref, -k.ref);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[j] = fma2(t[j], c, r);
    } else {
        const Pair c = pair_of(k.c2, k.c2), m = pair_of(-k.m, -k.m);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[j] = mul2(add2(t[j], m), c);
    }
    if (kFinite && (sizeof(T) == 4 || k.far))
#pragma unroll
        for (int j = 0; j < kPairs; ++j) {
            float a, b;
            halves(t[j], a, b);
            t[j] = pair_of(max_nan(a, kLow), max_nan(b, kLow));
        }
}
// the same for one logit, without the near form
__device__ __forceinline__ float exponent(float x, float m, float c2) {
    return max_nan((x - (m == -kInf ? 0.f : m)) * c2, kLow);
}

// ln of a sum (0: -inf); the approximate logarithm is within 2^-22.
__device__ __forceinline__ float ln(float s) {
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
    return r * kLn2;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// ln p of a logit of the row. Logits of opposite sign near float32's limits, whose difference or
// product overflows, are taken in float64.
__device__ __forceinline__ float log_prob(float x, float c, float m, float ln_s) {
    const float d = c * (x - m);
    if (fabsf(d) < 1.0e38f) return fmaf(c, x - m, -ln_s);
    return (float)((double)c * ((double)x - (double)m) - (double)ln_s);
}

// ------------------------------------------------------------------ rows

// The rows r, r + step, ... of a group, as step s and stream j.
struct RowWalk {
    int64_t r, s, step, ds;
    int j, dj;
    __device__ __forceinline__ RowWalk(int64_t first, int64_t step_, int n) : r(first), step(step_) {
        split(r, n, s, j);
        split(step, n, ds, dj);
    }
    __device__ __forceinline__ static void split(int64_t v, int n, int64_t& q, int& rem) {
        q = n == 1 ? v : (v >> 32) == 0 ? (int64_t)((uint32_t)v / (uint32_t)n) : v / n;
        rem = (int)(v - q * n);
    }
    __device__ __forceinline__ void next(int n) {
        r += step;
        s += ds;
        j += dj;
        if (j >= n) {
            j -= n;
            ++s;
        }
    }
};

// One thread group's share of a row: vectors [v0, v1), of which [lo, hi) lie wholly in the row.
template <typename T>
struct Part {
    const T* x;
    int V;
    int a;  // elements between the 16-byte boundary at or below x and x
    int v0, v1, lo, hi;

    static constexpr int kPer = Elem<T>::kPer;

    __device__ Part(const T* row, int V_, int rank, int cluster) : x(row), V(V_) {
        a = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        const int all = (a + V + kPer - 1) / kPer;
        const int per = (all + cluster - 1) >> (31 - __clz(cluster));  // a power of two
        v0 = min(rank * per, all);
        v1 = min(v0 + per, all);
        lo = max(v0, a ? 1 : 0);
        hi = min(v1, (a + V) / kPer);
    }
    __device__ int size() const { return v1 - v0; }
    // element index of a vector's first element (below 0 or past V at the row's ends)
    __device__ int first(int vec) const { return vec * kPer - a; }
    // vector and place of an element
    __device__ int vector_of(int i) const { return (i + a) / kPer; }
    __device__ bool holds(int vec) const { return vec >= v0 && vec < v1; }
};

__device__ __forceinline__ void load16(const void* p, uint32_t (&w)[4]) {
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "l"(p));
}
__device__ __forceinline__ void store16(void* p, const uint32_t (&w)[4]) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}

// The vector at a row's end, element by element; -inf outside the row.
template <typename T>
__device__ __noinline__ uint4 load_edge(const T* x, int first, int V) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = Elem<T>::kFill;
#pragma unroll
    for (int j = 0; j < Elem<T>::kPer; ++j) {
        const int i = first + j;
        if (i >= 0 && i < V) {
            if constexpr (sizeof(T) == 4) {
                w[j] = __float_as_uint(x[i]);
            } else {
                const uint32_t b = __bfloat16_as_ushort(x[i]);
                w[j / 2] = (j & 1) ? ((w[j / 2] & 0xFFFFu) | (b << 16)) : ((w[j / 2] & 0xFFFF0000u) | b);
            }
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// A vector's gradients, rounded once: whole at an aligned place, or element by element (those of
// the row) where the row's ends or the gradient's own alignment want it.
template <typename T>
__device__ __forceinline__ void store_vector(T* row, int first, const float (&y)[4], bool whole,
                                             bool some, int V) {
    if (whole) {
        const uint32_t w[4] = {__float_as_uint(y[0]), __float_as_uint(y[1]), __float_as_uint(y[2]),
                               __float_as_uint(y[3])};
        store16(row + first, w);
    } else if (some) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (first + j >= 0 && first + j < V) narrow(y[j], row + first + j);
    }
}
template <typename T>
__device__ __forceinline__ void store_vector(T* row, int first, const float (&y)[8], bool whole,
                                             bool some, int V) {
    if (whole) {
        const uint32_t w[4] = {pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]),
                               pack_bf16x2(y[4], y[5]), pack_bf16x2(y[6], y[7])};
        store16(row + first, w);
    } else if (some) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (first + j >= 0 && first + j < V) narrow(y[j], row + first + j);
    }
}

// Loads vector `vec` of the row's ends into its place of the chunk, if it is this thread's.
template <int TH, int NV, typename T>
__device__ __forceinline__ void put_edge(const Part<T>& p, int vec, int base, int tid,
                                         uint32_t (&v)[NV][4]) {
    const int at = vec - base - tid;
    if (vec < p.v0 || vec >= p.v1 || at < 0 || at >= NV * TH || at % TH != 0) return;
    const uint4 w = load_edge(p.x, p.first(vec), p.V);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const bool here = at == i * TH;
        v[i][0] = here ? w.x : v[i][0];
        v[i][1] = here ? w.y : v[i][1];
        v[i][2] = here ? w.z : v[i][2];
        v[i][3] = here ? w.w : v[i][3];
    }
}

// The slots i < NV of a chunk in which a warp has vectors (base + i * TH + tid), and whether all
// of its vectors in the chunk lie wholly in the row (the same for a warp's lanes).
template <int TH, int NV, typename T>
struct Slots {
    int count;
    bool whole;
    __device__ __forceinline__ Slots(const Part<T>& p, int base, int tid) {
        const int first = base + (tid & ~31);
        if constexpr (TH == 32) count = min((p.v1 - first + 31) / 32, NV);
        else count = min((p.v1 - first + TH - 1) / TH, NV);
        whole = count == NV && first >= p.lo && first + (NV - 1) * TH + 32 <= p.hi;
    }
};

// A chunk's vectors: base + i * TH + tid, i < NV; -inf past the part's end.
template <int TH, int NV, typename T>
__device__ __forceinline__ void load_chunk(const Part<T>& p, int base, int tid,
                                           uint32_t (&v)[NV][4]) {
    const T* at = p.x + p.first(base + tid);
    const Slots<TH, NV, T> sl(p, base, tid);
    if (sl.whole) {
#pragma unroll
        for (int i = 0; i < NV; ++i) load16(at + i * TH * Elem<T>::kPer, v[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int vec = base + i * TH + tid;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = Elem<T>::kFill;
        if (vec >= p.lo && vec < p.hi) load16(at + i * TH * Elem<T>::kPer, v[i]);
    }
    // the row's ends, where they are not whole vectors (one of them if the row is that short)
    put_edge<TH, NV>(p, p.lo - 1, base, tid, v);
    if (p.hi >= p.lo) put_edge<TH, NV>(p, p.hi, base, tid, v);
}

// Puts -inf in the place of marked elements: mark[i] has a bit per element of vector i.
template <int NV, typename T>
__device__ __forceinline__ void hide(const uint8_t* mark, uint32_t (&v)[NV][4]) {
#pragma unroll
    for (int h = 0; h < NV / 4; ++h) {
        const uint32_t four = *reinterpret_cast<const uint32_t*>(mark + 4 * h);
        if (four == 0) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t b = (four >> (8 * i)) & 0xFFu;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t& w = v[4 * h + i][j];
                if constexpr (sizeof(T) == 4) {
                    if ((b >> j) & 1u) w = Elem<T>::kFill;
                } else {
                    if ((b >> (2 * j)) & 1u) w = (w & 0xFFFF0000u) | 0xFF80u;
                    if ((b >> (2 * j)) & 2u) w = (w & 0xFFFFu) | 0xFF800000u;
                }
            }
        }
    }
}

// f(i, registers) for the warp's slots.
template <int NV, typename F>
__device__ __forceinline__ void each_slot(uint32_t (&v)[NV][4], int count, F&& f) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (i >= count) break;
        f(i, v[i]);
    }
}

// Stores the gradients make(registers, y) of a chunk into the row d.
template <int TH, int NV, typename T, typename F>
__device__ __forceinline__ void store_chunk(const Part<T>& p, int base, int tid, T* d, bool wide,
                                            uint32_t (&v)[NV][4], F&& make) {
    constexpr int kPer = Elem<T>::kPer;
    const Slots<TH, NV, T> sl(p, base, tid);
    const int at = p.first(base + tid);
    const bool whole = sl.whole && wide;
    each_slot<NV>(v, sl.count, [&](int i, uint32_t (&w)[4]) {
        const int vec = base + i * TH + tid;
        float y[kPer];
        make(w, y);
        store_vector<T>(d, at + i * TH * kPer, y, whole || (wide && vec >= p.lo && vec < p.hi),
                        vec < p.v1, p.V);
    });
}

template <typename T>
__device__ __forceinline__ float vector_max(const uint32_t (&w)[4]) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1])),
                     fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
    } else {
        const uint32_t a = max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3]));
        return fmaxf(bf16_lo_to_f32(a), bf16_hi_to_f32(a));
    }
}

struct Stats {
    float m, s, w;  // m is -inf where no logit is above it
};

// Adds a chunk to a warp's running statistics: m is the warp's, s and w are the thread's.
// Returns the thread's own maximum in the chunk.
template <int TH, int NV, bool kW, typename T>
__device__ __forceinline__ float add_chunk(const Part<T>& p, int base, int tid,
                                           uint32_t (&v)[NV][4], float c2, Stats& st) {
    const int count = Slots<TH, NV, T>(p, base, tid).count;
    float mx;
    if constexpr (sizeof(T) == 4) {
        mx = -kInf;
        each_slot<NV>(v, count, [&](int, uint32_t (&w)[4]) {
            mx = fmaxf(fmaxf(mx, fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]))),
                       fmaxf(__uint_as_float(w[2]), __uint_as_float(w[3])));
        });
    } else {
        uint32_t a = Elem<T>::kFill;
        each_slot<NV>(v, count, [&](int, uint32_t (&w)[4]) {
            a = max_bf16x2(max_bf16x2(a, max_bf16x2(w[0], w[1])), max_bf16x2(w[2], w[3]));
        });
        mx = fmaxf(bf16_lo_to_f32(a), bf16_hi_to_f32(a));
    }
    const float m = fmaxf(st.m, warp_max(mx));
    const Scale k(c2, m);
    if (st.m != m && st.m != -kInf) {  // an earlier chunk's sums move to the new maximum
        const float t = exponent(st.m, m, c2), f = ex2(t);
        if constexpr (kW) st.w = f * fmaf(st.s, t, st.w);
        st.s *= f;
    }
    st.m = m;
    Pair s2 = 0, w2 = 0;  // (0, 0)
    each_slot<NV>(v, count, [&](int, uint32_t (&w)[4]) {
        Pair t[Elem<T>::kPer / 2];
        exponents<T, kW>(w, k, t);
#pragma unroll
        for (int j = 0; j < Elem<T>::kPer / 2; ++j) {
            const Pair e = ex2_pair(t[j]);
            s2 = add2(s2, e);
            if constexpr (kW) w2 = fma2(e, t[j], w2);
        }
    });
    float s, s1, w = 0.f, w1 = 0.f;
    halves(s2, s, s1);
    s += s1;
    if constexpr (kW) {
        halves(w2, w, w1);
        w += w1;
    }
    const float back = ex2(-k.shift);
    st.s = fmaf(s, back, st.s);
    if constexpr (kW) st.w = fmaf(fmaf(-k.shift, s, w), back, st.w);
    return mx;
}

// The triples of up to 32 lanes as one (the same in every lane).
template <bool kW>
__device__ __forceinline__ Stats join_lanes(float m, float s, float w, float c2) {
    const float M = warp_max(m);
    const float t = exponent(m, M, c2), f = ex2(t);
    Stats r{M, warp_sum(f * s), 0.f};
    if constexpr (kW) r.w = warp_sum(f * fmaf(s, t, w));
    return r;
}

template <int TH>
__device__ __forceinline__ void group_sync() {
    if constexpr (TH == 32) __syncwarp();
    else __syncthreads();
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster_u64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// Where a group's warps, and a cluster's CTAs, leave their triples. The CTAs' slots alternate
// between rows: a CTA may push its next row's triple while another still reads this row's.
template <int TH>
struct Joint {
    float warp[3][TH / 32];
    float cta[2][3][kMaxCluster];
};

// The group's statistics in every thread of it. Contains the group's barrier (before it, threads
// may leave what the others need after it in shared memory).
template <int TH, bool kW>
__device__ __forceinline__ Stats join_group(Joint<TH>& j, Stats st, int tid, float c2) {
    st.s = warp_sum(st.s);
    if constexpr (kW) st.w = warp_sum(st.w);
    if constexpr (TH == 32) {
        group_sync<TH>();
        return st;
    } else {
        const int lane = tid & 31;
        constexpr int NW = TH / 32;
        if (lane == 0) {
            j.warp[0][tid / 32] = st.m;
            j.warp[1][tid / 32] = st.s;
            if constexpr (kW) j.warp[2][tid / 32] = st.w;
        }
        group_sync<TH>();
        const bool in = lane < NW;
        return join_lanes<kW>(in ? j.warp[0][lane] : -kInf, in ? j.warp[1][lane] : 0.f,
                              kW && in ? j.warp[2][lane] : 0.f, c2);
    }
}

// Gives CTA `to` of the cluster this CTA's triple.
template <int TH, bool kW>
__device__ __forceinline__ void push_stats(Joint<TH>& j, const Stats& st, int rank, int to,
                                           int parity) {
    const uint32_t at = cluster_map(smem_u32(&j.cta[parity][0][rank]), to);
    st_cluster_f32(at, st.m);
    st_cluster_f32(at + 4 * kMaxCluster, st.s);
    if constexpr (kW) st_cluster_f32(at + 8 * kMaxCluster, st.w);
}
// The triples that the cluster's CTAs pushed, as one.
template <int TH, bool kW>
__device__ __forceinline__ Stats join_cluster(const Joint<TH>& j, int tid, int cluster, int parity,
                                              float c2) {
    const int lane = tid & 31;
    const bool in = lane < cluster;
    return join_lanes<kW>(in ? j.cta[parity][0][lane] : -kInf, in ? j.cta[parity][1][lane] : 0.f,
                          kW && in ? j.cta[parity][2][lane] : 0.f, c2);
}

// The row's statistics in every thread of every CTA that shares it.
template <int TH, bool kW>
__device__ __forceinline__ Stats join_row(Joint<TH>& j, Stats st, int tid, int cluster, int rank,
                                          int parity, float c2) {
    st = join_group<TH, kW>(j, st, tid, c2);
    if (cluster > 1) {
        if (tid < cluster) push_stats<TH, kW>(j, st, rank, tid, parity);
        cluster_sync();
        st = join_cluster<TH, kW>(j, tid, cluster, parity, c2);
    }
    return st;
}

// Registers for a row's vectors: 16 a thread where a warp has a float32 row, so that it holds
// the audio streams' 2048 logits like a bf16 row's; 8 otherwise.
template <typename T, int TH>
__host__ __device__ constexpr int vectors_of() { return TH == 32 && sizeof(T) == 4 ? 16 : 8; }

// CTAs per SM a kernel is compiled for: 64 registers a thread (128 where 64 hold the row).
template <typename T, int TH>
__host__ __device__ constexpr int blocks_of() {
    return TH == 32 ? (sizeof(T) == 4 ? 2 : 3) : 1024 / TH;
}

template <int TH>
__host__ __device__ constexpr int block_of() { return TH == 32 ? 256 : TH; }  // warps of short rows share a CTA

// ------------------------------------------------------------------ host side

struct Shape {
    int threads, cluster;
};

// Threads and CTAs for a row of V elements. hold: the row stays in registers between two passes,
// so it takes as many threads as that needs, then clusters of 512-thread CTAs; a row that is
// read once is walked in chunks by 256 threads, four CTAs a SM, so that some load while others
// join their sums. Rows of a small batch are spread over more CTAs.
inline Shape shape_of(int64_t rows, int V, int size, bool warp_ok, bool hold) {
    const int per = 16 / size;
    const int vecs = (V + per - 1) / per + 1;  // rows off a 16-byte boundary have one more
    if (warp_ok && (V + per - 1) / per <= 32 * (size == 4 ? 16 : 8)) return {32, 1};
    int cluster = 1;
    while (hold && cluster < kMaxCluster && vecs > cluster * 512 * 8) cluster *= 2;
    while (cluster < kMaxCluster && rows * cluster * 2 <= 148 && vecs >= cluster * 2 * 256)
        cluster *= 2;
    const int each = (vecs + cluster - 1) / cluster;
    if (each <= 128 * 8) return {128, cluster};
    return {each <= 256 * 8 || !hold ? 256 : 512, cluster};
}

inline bool on_device(const void* p, size_t align, int dev) {
    if (!p || (reinterpret_cast<uintptr_t>(p) % align) != 0) return false;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == dev);
}
inline bool maybe_on_device(const void* p, size_t align, int dev) {
    return p == nullptr || on_device(p, align, dev);
}

inline int status_of(cudaError_t e) {
    if (e == cudaSuccess) return MIMI_RVQ_OK;
    cudaGetLastError();
    return MIMI_RVQ_ECUDA;
}

inline bool rows_ok(int dtype, int64_t S, int n, int V, int64_t ss, int64_t sn, float scale) {
    if (dtype != MIMI_RVQ_F32 && dtype != MIMI_RVQ_BF16) return false;
    if (S < 0 || n < 0 || n > 65536 || S > (int64_t(1) << 40)) return false;
    if (V < 1 || V > MIMI_RVQ_MAX_VOCAB || ss < 0 || sn < 0) return false;
    if ((__int128)ss * S + (__int128)sn * n > ((__int128)1 << 58)) return false;  // no offset wraps
    return scale > 0.f && scale < kInf;
}

// Rows of a gradient must not share memory: the smaller stride holds a row, the larger one all
// rows of the smaller.
inline bool rows_apart(int64_t S, int n, int V, int64_t ss, int64_t sn) {
    if (S <= 1) return n <= 1 || sn >= V;
    if (n <= 1) return ss >= V;
    if (sn <= ss) return sn >= V && ss >= sn * (n - 1) + V;
    return ss >= V && sn >= ss * (S - 1) + V;
}

// The gradient may take the logits' own place (same pointer and strides) but may not overlap
// them in another way.
inline bool apart_or_same(const void* x, int64_t ss, int64_t sn, const void* d, int64_t dss,
                          int64_t dsn, int64_t S, int n, int V, int size) {
    if (x == d) return (S <= 1 || ss == dss) && (n <= 1 || sn == dsn);
    const char* a = static_cast<const char*>(x);
    const char* b = static_cast<const char*>(d);
    const char* a1 = a + (ss * (S - 1) + sn * (n - 1) + V) * size;
    const char* b1 = b + (dss * (S - 1) + dsn * (n - 1) + V) * size;
    return a1 <= b || b1 <= a;
}

// One launch over all rows: a CTA takes 256 / 32 rows of a warp each, one row, or a
// cluster's share of one.
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kernel)(KArgs...), int threads, const RowsIn& in, int smem,
                        cudaStream_t stream, Args... args) {
    const int block = threads == 32 ? 256 : threads;
    const int64_t groups = threads == 32 ? (in.rows + 7) / 8 : in.rows;
    int64_t most = int64_t(1) << 27;  // the kernels loop over the rest
    if (threads == 32) {              // as many CTAs as are resident: each sets up once
        int dev = 0, sms = 148, per_sm = 4;
        if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (groups > (int64_t)sms * 2)
            cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, block, smem);
        most = (int64_t)sms * (per_sm > 0 ? per_sm : 1);
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((groups < most ? groups : most) * in.cluster));
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = in.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = in.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace logits
}  // namespace mimi
