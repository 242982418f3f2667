// logits.cuh -- what the kernels on the language model's logits share: a row's
// layout, its way into shared memory, the passes that give its softmax
// statistics, and the host side's choice of threads.
//
// A row is one position of one stream: V logits that start at any element. Its
// whole 16-byte vectors (on aligned addresses) are copied into shared memory
// asynchronously, thread t of the TH that share the row taking vectors t, t + TH,
// ...; each thread works only on vectors that it copied, so a row needs no
// barrier before its passes. The up to 2 x 7 elements before the first and after
// the last whole vector are taken as single values by 16 lanes of the first warp.
// A group (half a warp or a warp for short rows, else a CTA, or a cluster of them
// that splits a row's vectors) goes through rows in a loop and sends for the next
// row as soon as it has read a row for the last time; several groups per SM overlap
// one's joining and output with the others' copies and passes. (Rows held in registers
// instead left room for half as many threads, and took bounds and fills on every
// vector: gradient of 3750 x 32000 bf16 rows 121 us, so 94 to 101.)
//
// Every statistic comes from m = max x, s = sum 2^t_i and w = sum 2^t_i t_i with
// t_i = log2(e) c (x_i - m), c = scale, all in float32:
//     lse = c m + ln s,  ln p_i = c (x_i - m) - ln s,  entropy = ln s - ln 2 w / s.
// Each warp sums against its own maximum (one hardware reduction); the warps'
// triples are joined behind one barrier, a cluster's behind one more.
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
    int log_cluster;  // CTAs per row: 1 << log_cluster (0: a row is one CTA's or one warp's)
    int slots;     // 16-byte places of a group's buffer
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

// A group of TH threads: half a warp, a warp or a CTA. Its lanes are those of a warp that work
// together: 16 of half a warp, else 32.
template <int TH>
__host__ __device__ constexpr int lanes_of() { return TH < 32 ? TH : 32; }
template <int TH>
__device__ __forceinline__ unsigned lane_mask() {
    return TH < 32 ? ((1u << (TH & 31)) - 1u) << (threadIdx.x & 31 & ~(TH - 1)) : kFull;
}
template <int TH>
__device__ __forceinline__ float lanes_max(float v) {
    if constexpr (TH < 32) {
#pragma unroll
        for (int o = TH / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(lane_mask<TH>(), v, o));
        return v;
    } else {
        float r;
        asm volatile("redux.sync.max.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "r"(kFull));
        return r;
    }
}
template <int TH, typename V>
__device__ __forceinline__ V lanes_sum(V v) {
#pragma unroll
    for (int o = lanes_of<TH>() / 2; o; o >>= 1) v += __shfl_xor_sync(lane_mask<TH>(), v, o);
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
        far = !(fabsf(ref) < 32768.f && c2 < 1.0e30f);
        shift = far ? 0.f : fmaf(m, c2, -ref);
        const float f = __fdividef(ref + kLow, c2);
        floor_bf16x2 = pack_bf16x2(f, f);
    }
};
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <typename T, bool kFinite, bool kFar>
__device__ __forceinline__ void exponents(const uint32_t (&w)[4], const Scale& k,
                                          Pair (&t)[Elem<T>::kPer / 2]) {
    constexpr int kPairs = Elem<T>::kPer / 2;
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
        if constexpr (sizeof(T) == 4) {
            t[j] = pair_of(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
        } else {
            const uint32_t u = kFinite && !kFar ? max_nan_bf16x2(w[j], k.floor_bf16x2) : w[j];
            t[j] = pair_of(bf16_lo_to_f32(u), bf16_hi_to_f32(u));
        }
    }
    if constexpr (!kFar) {
        const Pair c = pair_of(k.c2, k.c2), r = pair_of(-k.ref, -k.ref);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[j] = fma2(t[j], c, r);
    } else {
        const Pair c = pair_of(k.c2, k.c2), m = pair_of(-k.m, -k.m);
#pragma unroll
        for (int j = 0; j < kPairs; ++j) t[j] = mul2(add2(t[j], m), c);
    }
    if constexpr (kFinite && (sizeof(T) == 4 || kFar))
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

// ln of a sum (0: -inf) for gradients, within 2^-22 absolutely near 1; values take logf, as the
// logarithm of a token that is nearly certain is its log probability.
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

// One group's share of a row.
template <typename T>
struct Part {
    static constexpr int kPer = Elem<T>::kPer;
    const T* x;
    int V;
    int head;    // elements before the row's first whole vector
    int tail;    // first element after its last one
    int first;   // first element of this share's vectors
    int nv;      // vectors of this share

    __device__ __forceinline__ Part(const T* row, int V_, int rank, int log_cluster) : x(row), V(V_) {
        const int a = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
        head = min(V, (kPer - a) & (kPer - 1));
        const int whole = (V - head) / kPer;
        tail = head + whole * kPer;
        const int per = (whole + (1 << log_cluster) - 1) >> log_cluster;
        const int v0 = min(rank * per, whole);
        nv = min(per, whole - v0);
        first = head + v0 * kPer;
    }
    // place of element i in the share's buffer, -1 if it has none
    __device__ __forceinline__ int place(int i) const {
        const int q = i - first;
        return q >= 0 && q < nv * kPer ? q : -1;
    }
    // element that lane l < 16 of the row's first warp has beside the vectors, -1 for none
    __device__ __forceinline__ int edge(int l) const {
        if (l < 8) return l < head ? l : -1;
        return l < 16 && tail + l - 8 < V ? tail + l - 8 : -1;
    }
    // that lane's place for an element beside the vectors
    __device__ __forceinline__ int edge_lane(int i) const { return i < head ? i : 8 + i - tail; }
    __device__ __forceinline__ bool in_edges(int i) const { return i < head || i >= tail; }
};

__device__ __forceinline__ void copy16(void* smem, const void* gmem) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(smem)), "l"(gmem)
                 : "memory");
}
// Sends for the share's vectors; they have come when arrived() returns.
template <int TH, typename T>
__device__ __forceinline__ void fetch(uint4* buf, const Part<T>& p, int tid) {
    const T* src = p.x + p.first;
#pragma unroll 4
    for (int i = tid; i < p.nv; i += TH) copy16(buf + i, src + (size_t)i * Elem<T>::kPer);
}
// The next row's vectors, sent for as soon as this row's are no longer needed: one by one where
// the last pass has read a place, the rest when it is done.
template <typename T>
struct Next {
    uint4* buf;
    const T* src;
    int nv;
    __device__ __forceinline__ void refill(int i) const {
        if (i < nv) copy16(buf + i, src + (size_t)i * Elem<T>::kPer);
    }
    // places that this row's nv vectors did not reach
    template <int TH>
    __device__ __forceinline__ void rest(int old_nv, int tid) const {
        for (int i = old_nv + ((tid - old_nv) % TH + TH) % TH; i < nv; i += TH) refill(i);
    }
};
__device__ __forceinline__ void arrived() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void store16(void* p, const uint32_t (&w)[4]) {
    asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3])
                 : "memory");
}
// A vector's gradients, rounded once; element by element where the gradient's row is not aligned
// as the logits' is.
template <typename T>
__device__ __forceinline__ void store_vector(T* at, bool wide, const float (&y)[Elem<T>::kPer]) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 4) w[j] = __float_as_uint(y[j]);
        else w[j] = pack_bf16x2(y[2 * j], y[2 * j + 1]);
    }
    if (wide) {
        store16(at, w);
    } else {
#pragma unroll
        for (int j = 0; j < Elem<T>::kPer; ++j) narrow(element<T>(w, j), at + j);
    }
}

// f(i, vector i of the share) for this thread's vectors, one after another.
template <int TH, typename F>
__device__ __forceinline__ void each_in_turn(const uint4* buf, int nv, int tid, F&& f) {
#pragma unroll 1
    for (int i = tid; i < nv; i += TH) {
        const uint4 q = buf[i];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        f(i, w);
    }
}
// the same in groups of four
template <int TH, typename F>
__device__ __forceinline__ void each_vector(const uint4* buf, int nv, int tid, F&& f) {
    int i = tid;
    for (; i + 3 * TH < nv; i += 4 * TH) {
        uint4 q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = buf[i + u * TH];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
            f(i + u * TH, w);
        }
    }
#pragma unroll 1
    for (; i < nv; i += TH) {
        const uint4 q = buf[i];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        f(i, w);
    }
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

// A warp's statistics over its threads' vectors and edge values (-inf for none): m is the warp's,
// s and w the thread's own. top: the thread's own maximum. after(i): vector i has been read.
template <int TH, bool kW, typename T, typename After>
__device__ __forceinline__ Stats pass(const uint4* buf, int nv, int tid, float edge, float c2,
                                      float& top, After&& after) {
    if constexpr (sizeof(T) == 4) {
        top = edge;
        each_vector<TH>(buf, nv, tid, [&](int, const uint32_t (&w)[4]) {
            top = fmaxf(top, vector_max<T>(w));
        });
    } else {
        uint32_t a = Elem<T>::kFill;
        each_vector<TH>(buf, nv, tid, [&](int, const uint32_t (&w)[4]) {
            a = max_bf16x2(a, max_bf16x2(max_bf16x2(w[0], w[1]), max_bf16x2(w[2], w[3])));
        });
        top = fmaxf(edge, fmaxf(bf16_lo_to_f32(a), bf16_hi_to_f32(a)));
    }
    Stats st{lanes_max<TH>(top), 0.f, 0.f};
    const Scale k(c2, st.m);
    Pair s2 = 0, w2 = 0;  // (0, 0)
    auto add = [&](const Pair (&t)[Elem<T>::kPer / 2]) {
#pragma unroll
        for (int j = 0; j < Elem<T>::kPer / 2; ++j) {
            const Pair e = ex2_pair(t[j]);
            s2 = add2(s2, e);
            if constexpr (kW) w2 = fma2(e, t[j], w2);
        }
    };
    if (!k.far)
        each_vector<TH>(buf, nv, tid, [&](int i, const uint32_t (&w)[4]) {
            Pair t[Elem<T>::kPer / 2];
            exponents<T, kW, false>(w, k, t);
            add(t);
            after(i);
        });
    else
        each_in_turn<TH>(buf, nv, tid, [&](int i, const uint32_t (&w)[4]) {
            Pair t[Elem<T>::kPer / 2];
            exponents<T, kW, true>(w, k, t);
            add(t);
            after(i);
        });
    float s, s1, w = 0.f, w1 = 0.f;
    halves(s2, s, s1);
    s += s1;
    if constexpr (kW) {
        halves(w2, w, w1);
        w += w1;
    }
    const float back = ex2(-k.shift);
    const float te = exponent(edge, st.m, c2), e = ex2(te);
    st.s = fmaf(s, back, e);
    if constexpr (kW) st.w = fmaf(fmaf(-k.shift, s, w), back, e * te);
    return st;
}

// The triples of up to 32 lanes as one (the same in every lane).
template <bool kW>
__device__ __forceinline__ Stats join_lanes(float m, float s, float w, float c2) {
    const float M = lanes_max<32>(m);
    const float t = exponent(m, M, c2), f = ex2(t);
    Stats r{M, lanes_sum<32>(f * s), 0.f};
    if constexpr (kW) r.w = lanes_sum<32>(f * fmaf(s, t, w));
    return r;
}

// The barrier of N threads: those of a group, or of the whole CTA. Warps with different work may
// meet here from different places.
template <int N>
__device__ __forceinline__ void group_sync() {
    if constexpr (N <= 32) __syncwarp(lane_mask<N>());
    else asm volatile("barrier.sync 1, %0;" ::"n"(N) : "memory");
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

// Where a group's warps, and a cluster's CTAs, leave their triples. The places alternate between
// rows: a warp or CTA may leave its next row's triple while another still reads this row's.
template <int TH>
struct Joint {
    float warp[2][3][(TH + 31) / 32];
    float cta[2][3][kMaxCluster];
};

// The group's statistics in every thread of it, and of the N - TH threads beside it (which only
// read). Contains the barrier of all N (before it, threads may leave what the others need after it
// in shared memory).
template <int TH, bool kW, int N = TH>
__device__ __forceinline__ Stats join_group(Joint<TH>& j, Stats st, int tid, int parity, float c2) {
    st.s = lanes_sum<TH>(st.s);
    if constexpr (kW) st.w = lanes_sum<TH>(st.w);
    if constexpr (TH <= 32) {
        group_sync<TH>();
        return st;
    } else {
        static_assert(N % 32 == 0, "whole warps");
        const int lane = tid & 31;
        float(&at)[3][(TH + 31) / 32] = j.warp[parity];
        if (lane == 0 && tid < TH) {
            at[0][tid / 32] = st.m;
            at[1][tid / 32] = st.s;
            if constexpr (kW) at[2][tid / 32] = st.w;
        }
        group_sync<N>();
        const bool in = lane < TH / 32;
        return join_lanes<kW>(in ? at[0][lane] : -kInf, in ? at[1][lane] : 0.f,
                              kW && in ? at[2][lane] : 0.f, c2);
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
template <int TH, bool kW, int N = TH>
__device__ __forceinline__ Stats join_row(Joint<TH>& j, Stats st, int tid, int cluster, int rank,
                                          int parity, float c2) {
    st = join_group<TH, kW, N>(j, st, tid, parity, c2);
    if (cluster > 1) {
        if (tid < cluster) push_stats<TH, kW>(j, st, rank, tid, parity);
        cluster_sync();
        st = join_cluster<TH, kW>(j, tid, cluster, parity, c2);
    }
    return st;
}

// Threads of a CTA: groups of short rows share one.
template <int TH>
__host__ __device__ constexpr int block_of() { return TH > 128 ? TH : 128; }
// CTAs per SM that log probabilities of rows in shared memory and their gradient are compiled for:
// 64 registers a thread. (Those of longer rows and distillation have figures of their own.)
template <int TH>
__host__ __device__ constexpr int blocks_of() { return 1024 / block_of<TH>(); }
// A thread's number in its group, and its group's in the CTA.
template <int TH>
__device__ __forceinline__ int thread_in_group() { return TH < block_of<TH>() ? threadIdx.x % TH : threadIdx.x; }
template <int TH>
__device__ __forceinline__ int group_in_block() { return TH < block_of<TH>() ? threadIdx.x / TH : 0; }

// ------------------------------------------------------------------ host side

constexpr int kShortBytes = 8192;           // longest row of half a warp or a warp
constexpr int kPartBytes = 110 * 1024;      // a CTA's share that leaves room for two a SM
constexpr int kSmemBytes = 227 * 1024;

struct Shape {
    int threads, log_cluster;
};

// Threads and CTAs for a row of V elements: `few` threads up to 8 KB; else a CTA of 128 or 256.
// Rows over 110 KB that have to lie in shared memory whole, and rows of a batch that would leave
// SMs idle, are split over a cluster of up to 8 CTAs; rows that only pass through until there are
// 4 CTAs a SM, as each has 24 KB on its way (100 rows of 131072 float32 logits: 20.4 us unsplit, 9.8
// in fours; rows that lie whole gain nothing: 148 of 32000 take 8.4 us as pairs, 12.5 in fours).
// 110 KB: what a cluster's barriers cost is more than a third CTA a SM gains, and one CTA alone
// does not hide its own turns. 2000 rows of 100 KB, distillation and its gradient: 85 and 132 us
// as pairs, 50 and 93 in one CTA; 2000 of 120 KB, the gradient: 123 as pairs, 146 in one CTA.
inline Shape shape_of(int64_t rows, int V, int size, int few, bool whole) {
    const int64_t bytes = (int64_t)V * size;
    if (few && bytes <= kShortBytes) return {few, 0};
    int lc = 0;
    while (whole && lc < 3 && (bytes >> lc) > kPartBytes) ++lc;
    while (lc < 3 && (rows << (lc + 1)) <= 148 && (bytes >> (lc + 1)) >= 4096) ++lc;
    while (!whole && lc < 3 && (rows << (lc + 1)) <= 4 * 148 && (bytes >> (lc + 1)) >= 16384) ++lc;
    return {(bytes >> lc) <= 16384 ? 128 : 256, lc};
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
    // scales below 1e-30 would make ordinary exponents of differences past float32's range
    return scale >= 1.0e-30f && scale <= 1.0e30f;
}

// Rows of a gradient must not share memory: the smaller stride holds a row, the larger one all
// rows of the smaller.
inline bool rows_apart(int64_t S, int n, int V, int64_t ss, int64_t sn) {
    if (S <= 1) return n <= 1 || sn >= V;
    if (n <= 1) return ss >= V;
    if (sn <= ss) return sn >= V && ss >= sn * (n - 1) + V;
    return ss >= V && sn >= ss * (S - 1) + V;
}

// Whether a row at offset d from one of m rows of V elements, p >= V apart, and the m - 1 rows
// after it on the same stride share an element with them.
inline bool rows_meet(int64_t d, int64_t p, int64_t m, int64_t V) {
    const int64_t q = d / p - (d % p < 0), r = d - q * p;
    return (r < V && q < m && q > -m) || (r > p - V && q + 1 < m && q + 1 > -m);
}

// The gradient may take the logits' own place (same pointer and strides), or places between the
// logits' rows (same strides: two column ranges of one buffer, every other stream), but may not
// share elements with them in another way.
inline bool apart_or_same(const void* x, int64_t ss, int64_t sn, const void* d, int64_t dss,
                          int64_t dsn, int64_t S, int n, int V, int size) {
    const bool same = (S <= 1 || ss == dss) && (n <= 1 || sn == dsn);
    if (x == d) return same;
    const char* a = static_cast<const char*>(x);
    const char* b = static_cast<const char*>(d);
    const char* a1 = a + (ss * (S - 1) + sn * (n - 1) + V) * size;
    const char* b1 = b + (dss * (S - 1) + dsn * (n - 1) + V) * size;
    if (a1 <= b || b1 <= a) return true;
    if (!same) return false;
    // blocks of the smaller stride's rows, the larger stride apart (rows_apart holds for both)
    int64_t P = S > 1 ? ss : V, M = S, p = n > 1 ? sn : V, m = n;
    if (M == 1 || (m > 1 && p > P)) {
        int64_t t = P; P = p; p = t;
        t = M; M = m; m = t;
    }
    const int64_t off = (b - a) / size, q = off / P - (off % P < 0), r = off - q * P;
    return !(q < M && q > -M && rows_meet(r, p, m, V)) &&
           !(q + 1 < M && q + 1 > -M && rows_meet(r - P, p, m, V));
}

// One launch over all rows: as many groups as are resident, each with `slots` places of 16 bytes
// in dynamic shared memory, or one for each row if they are fewer (rows are dealt out to the whole
// grid from the start, so a CTA that has to wait for another's end would hold its rows back). Of
// clusters the device may run a few less than their shared memory allows (48 of 55 by eights):
// a grid of exactly those took the same time.
// kMore: threads of a CTA beside the row's TH; kPerSm: CTAs per SM the kernel is compiled for.
template <auto kernel, int TH, int kMore, int kPerSm, typename... Args>
cudaError_t launch_rows(const RowsIn& in, int static_smem, cudaStream_t stream, Args... args) {
    constexpr int block = block_of<TH>() + kMore, rows_per = block_of<TH>() / TH;
    const int smem = rows_per * in.slots * 16;
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // raise the kernel's shared-memory limit once per device
    static unsigned long long configured = 0;  // bit per device
    if (smem > 48 * 1024 - static_smem && (dev >= 64 || !(configured & (1ull << dev)))) {
        const cudaError_t e = cudaFuncSetAttribute(
            kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes - static_smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) __atomic_fetch_or(&configured, 1ull << dev, __ATOMIC_RELAXED);
    }
    int per_sm = (kSmemBytes + 1024) / (smem + static_smem + 1024);
    if (per_sm > kPerSm) per_sm = kPerSm;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    const int64_t groups = (in.rows + rows_per - 1) / rows_per;
    int64_t most = ((int64_t)sms * per_sm) >> in.log_cluster;
    if (most < 1) most = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((groups < most ? groups : most) << in.log_cluster));
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 1u << in.log_cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = in.log_cluster ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// 16-byte places a group needs for rows of V elements.
inline int slots_of(int V, int size, int log_cluster) {
    const int whole = V / (16 / size);
    return (whole + (1 << log_cluster) - 1) >> log_cluster;
}

}  // namespace logits
}  // namespace mimi
