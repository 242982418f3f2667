// logits.cu -- operators on the language model's logits over the packed token
// streams: log probabilities of given tokens with entropy, log-sum-exp and top
// alternatives, distillation from a teacher's top list, and the gradient of
// each. Declared in include/mimi_rvq_streams.h.
//
// A row is one position of one stream: V logits. Every statistic comes from
//     m = max x,  s = sum e^{c (x - m)},  w = sum e^{c (x - m)} (x - m)
// (c = scale), held in float32:
//     lse = c m + ln s,  ln p_i = c (x_i - m) - ln s,  entropy = ln s - c w / s.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/mimi_rvq.h"
#include "../../include/mimi_rvq_streams.h"

namespace mimi {
namespace {

constexpr int kMaxTop = MIMI_RVQ_MAX_TOP;
constexpr float kInf = INFINITY;
constexpr float kLog2e = 1.4426950408889634f;

// The rows of a logits tensor [S][n][V]; strides in elements.
struct RowsIn {
    const void* x;
    int64_t ss, sn;
    int64_t rows;  // S * n
    int n, V;
    float c;  // scale
};

struct TokensIn {
    const int32_t* tok;  // NULL: no targets
    int64_t ss, sn;
    int32_t pad;
    unsigned long long* n_bad;
};

struct ValuesOut {  // any may be NULL; [S][n], top [S][n][k]
    float* logprob;
    float* entropy;
    float* lse;
    int32_t* top_ids;
    float* top_logprob;
    int k;
};

struct GradIn {
    const float* g_logprob;
    const float* g_entropy;
    const float* g_lse;
    void* d;
    int64_t ss, sn;
};

struct TeacherIn {
    const int32_t* ids;  // [S][n][k]
    const void* t;
    int t_bf16;
    int k, tail;
    const float* g;  // NULL: 1
    float* loss;     // may be NULL with a gradient
    void* d;         // NULL: no gradient
    int64_t d_ss, d_sn;
    unsigned long long* n_bad;
};

__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void narrow(float v, float* p) { *p = v; }
__device__ __forceinline__ void narrow(float v, __nv_bfloat16* p) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Order of (value descending, index ascending) as one unsigned key: larger comes first. -0 and
// +0 are the same value (the sum makes both +0).
__device__ __forceinline__ unsigned long long order_key(float v, int index) {
    const uint32_t b = __float_as_uint(v + 0.f);
    const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
    return ((unsigned long long)o << 32) | (0xFFFFFFFFu - (uint32_t)index);
}
__device__ __forceinline__ float key_value(unsigned long long key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_index(unsigned long long key) {
    return (int)(0xFFFFFFFFu - (uint32_t)key);
}

constexpr int kT = 256;

template <typename V, typename Op>
__device__ V block_reduce(V v, Op op) {
    __shared__ V part[kT / 32];
    __shared__ V all;
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x == 0) {
        V a = part[0];
        for (int i = 1; i < kT / 32; ++i) a = op(a, part[i]);
        all = a;
    }
    __syncthreads();
    return all;
}
struct MaxOp {
    __device__ float operator()(float a, float b) const { return fmaxf(a, b); }
    __device__ unsigned long long operator()(unsigned long long a, unsigned long long b) const {
        return a > b ? a : b;
    }
};
struct AddOp {
    template <typename V>
    __device__ V operator()(V a, V b) const { return a + b; }
};

// A difference x - max below this has probability 0 in float32 (e^-200); clamping it there keeps
// 0 times -inf out of the products with a probability.
__device__ __forceinline__ float far_below(float c) { return fmaxf(-200.f / c, -3.0e38f); }

// max, sum and weighted sum of a row; the maximum of a row without a finite logit is taken as 0
// so that its sum is 0.
struct Stats {
    float m, s, w;
};
template <typename T>
__device__ Stats row_stats(const T* x, int V, float c) {
    float m = -kInf;
    for (int i = threadIdx.x; i < V; i += kT) m = fmaxf(m, widen(x[i]));
    m = block_reduce(m, MaxOp());
    if (m == -kInf) m = 0.f;
    const float c2 = c * kLog2e, low = far_below(c);
    float s = 0.f, w = 0.f;
    for (int i = threadIdx.x; i < V; i += kT) {
        const float d = widen(x[i]) - m, e = ex2(d * c2);
        s += e;
        w += e * fmaxf(d, low);
    }
    return Stats{m, block_reduce(s, AddOp()), block_reduce(w, AddOp())};
}

__device__ __forceinline__ int target_of(const TokensIn& tk, int64_t s, int j, int V) {
    if (tk.tok == nullptr) return -1;
    const int32_t t = tk.tok[s * tk.ss + j * tk.sn];
    if (t < 0 || t == tk.pad) return -1;
    if (t >= V) {
        if (threadIdx.x == 0 && tk.n_bad != nullptr) atomicAdd(tk.n_bad, 1ull);
        return -1;
    }
    return t;
}

// ln p of a logit of the row; the difference and product in float64, so that logits of opposite
// sign near float32's limits do not overflow (a few of these per row).
__device__ __forceinline__ float log_prob(float x, float c, float m, float ln_s) {
    return (float)((double)c * ((double)x - (double)m) - (double)ln_s);
}

__device__ __forceinline__ void put_values(const ValuesOut& o, int64_t r, int t, float xt, float c,
                                           const Stats& st) {
    const float ln_s = logf(st.s);
    const bool none = st.s == 0.f;
    if (o.logprob != nullptr)
        o.logprob[r] = t < 0 ? 0.f : none ? -kInf : log_prob(xt, c, st.m, ln_s);
    if (o.entropy != nullptr) o.entropy[r] = none ? 0.f : ln_s - c * (st.w / st.s);
    if (o.lse != nullptr) o.lse[r] = none ? -kInf : c * st.m + ln_s;
}

template <typename T>
__global__ void __launch_bounds__(kT) k_logprob(RowsIn in, TokensIn tk, ValuesOut o) {
    for (int64_t r = blockIdx.x; r < in.rows; r += gridDim.x) {
        const int64_t s = r / in.n;
        const int j = (int)(r - s * in.n);
        const T* x = static_cast<const T*>(in.x) + s * in.ss + j * in.sn;
        const Stats st = row_stats(x, in.V, in.c);
        const int t = target_of(tk, s, j, in.V);
        if (threadIdx.x == 0) put_values(o, r, t, t < 0 ? 0.f : widen(x[t]), in.c, st);
        unsigned long long last = ~0ull;
        const bool broken = !(st.s < kInf);
        for (int q = 0; q < o.k; ++q) {
            unsigned long long best = 0;
            if (!broken && last != 0)
                for (int i = threadIdx.x; i < in.V; i += kT) {
                    const float v = widen(x[i]);
                    const unsigned long long key = order_key(v, i);
                    if (v > -kInf && key < last && key > best) best = key;
                }
            best = block_reduce(best, MaxOp());
            if (threadIdx.x == 0) {
                if (o.top_ids != nullptr) o.top_ids[r * o.k + q] = best ? key_index(best) : -1;
                if (o.top_logprob != nullptr)
                    o.top_logprob[r * o.k + q] =
                        broken ? NAN : best ? log_prob(key_value(best), in.c, st.m, logf(st.s)) : -kInf;
            }
            last = best;
        }
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kT) k_logprob_grad(RowsIn in, TokensIn tk, GradIn g, ValuesOut o) {
    const bool values = o.logprob != nullptr || o.entropy != nullptr || o.lse != nullptr;
    for (int64_t r = blockIdx.x; r < in.rows; r += gridDim.x) {
        const int64_t s = r / in.n;
        const int j = (int)(r - s * in.n);
        const T* x = static_cast<const T*>(in.x) + s * in.ss + j * in.sn;
        T* d = static_cast<T*>(g.d) + s * g.ss + j * g.sn;
        const int t = target_of(tk, s, j, in.V);
        const float a = (t < 0 || g.g_logprob == nullptr) ? 0.f : g.g_logprob[r];
        const float b = g.g_entropy == nullptr ? 0.f : g.g_entropy[r];
        const float z = g.g_lse == nullptr ? 0.f : g.g_lse[r];
        const bool zero = a == 0.f && b == 0.f && z == 0.f;
        Stats st{0.f, 0.f, 0.f};
        if (!zero || values) {
            st = row_stats(x, in.V, in.c);
            if (threadIdx.x == 0) put_values(o, r, t, t < 0 ? 0.f : widen(x[t]), in.c, st);
        }
        __syncthreads();
        const bool none = zero || st.s == 0.f;
        const float inv = none ? 0.f : 1.f / st.s, ln_s = none ? 0.f : logf(st.s);
        const float h = ln_s - in.c * (st.w * inv);
        // c p_i [(z - a) - b (ln p_i + H)] + c a [i = t]
        const float c0 = in.c * inv * ((z - a) - b * (h - ln_s)), c1 = -in.c * inv * b * in.c;
        const float c2 = in.c * kLog2e, low = far_below(in.c);
        for (int i = threadIdx.x; i < in.V; i += kT) {
            float v = 0.f;
            if (!none) {
                const float df = widen(x[i]) - st.m;
                v = ex2(df * c2) * (c0 + c1 * fmaxf(df, low));
                if (i == t) v += in.c * a;
            }
            narrow(v, d + i);
        }
        __syncthreads();
    }
}

template <typename T>
__global__ void __launch_bounds__(kT) k_distill(RowsIn in, TeacherIn te) {
    extern __shared__ uint32_t listed[];  // bit i: token i is in the row's list
    __shared__ float sq[kMaxTop], sx[kMaxTop];
    __shared__ int sid[kMaxTop];
    const int words = (in.V + 31) / 32;
    for (int64_t r = blockIdx.x; r < in.rows; r += gridDim.x) {
        const int64_t s = r / in.n;
        const int j = (int)(r - s * in.n);
        const T* x = static_cast<const T*>(in.x) + s * in.ss + j * in.sn;
        T* d = te.d == nullptr ? nullptr : static_cast<T*>(te.d) + s * te.d_ss + j * te.d_sn;
        const float g = te.g == nullptr ? 1.f : te.g[r];
        for (int i = threadIdx.x; i < words; i += kT) listed[i] = 0;
        __syncthreads();
        float t = -kInf;
        bool first = false;
        int id = -1;
        if (threadIdx.x < te.k) {
            const int q = threadIdx.x;
            id = te.ids[r * te.k + q];
            if (id >= in.V) {
                if (te.n_bad != nullptr) atomicAdd(te.n_bad, 1ull);
                id = -1;
            }
            if (id >= 0) {
                t = te.t_bf16 ? widen(static_cast<const __nv_bfloat16*>(te.t)[r * te.k + q])
                              : static_cast<const float*>(te.t)[r * te.k + q];
                first = !((atomicOr(&listed[id / 32], 1u << (id % 32)) >> (id % 32)) & 1u);
                sx[q] = widen(x[id]);
            }
            sid[q] = id;
        }
        const int present = __syncthreads_count(id >= 0);
        const float tmax = block_reduce(t, MaxOp());
        double qs;  // sum of the weights (tail: their exact sum decides q_r)
        float q = 0.f, lq = -kInf;
        if (te.tail) {
            qs = block_reduce(id >= 0 ? exp((double)t) : 0.0, AddOp());
            lq = t;
        } else {
            const float tm = tmax == -kInf ? 0.f : tmax;
            qs = block_reduce(id >= 0 ? (double)expf(t - tm) : 0.0, AddOp());
            lq = t - tm - logf((float)qs);
        }
        if (id >= 0) q = expf(lq);
        if (threadIdx.x < te.k) sq[threadIdx.x] = q;
        const bool empty = present == 0 || (!te.tail && qs == 0.0);
        const bool want = te.loss != nullptr || g != 0.f;
        float loss = 0.f;
        Stats all{0.f, 0.f, 0.f}, rest{0.f, 0.f, 0.f};
        float qr = 0.f, Q = 1.f, ln_all = 0.f, ln_rest = 0.f;
        if (!empty && want) {
            all = row_stats(x, in.V, in.c);
            ln_all = logf(all.s);
            if (te.tail) {
                float m = -kInf, sum = 0.f;
                for (int i = threadIdx.x; i < in.V; i += kT)
                    if (!((listed[i / 32] >> (i % 32)) & 1u)) m = fmaxf(m, widen(x[i]));
                m = block_reduce(m, MaxOp());
                if (m == -kInf) m = 0.f;
                for (int i = threadIdx.x; i < in.V; i += kT)
                    if (!((listed[i / 32] >> (i % 32)) & 1u))
                        sum += ex2((widen(x[i]) - m) * (in.c * kLog2e));
                rest = Stats{m, block_reduce(sum, AddOp()), 0.f};
                ln_rest = logf(rest.s);
                qr = rest.s == 0.f ? 0.f : (float)fmax(0.0, 1.0 - qs);
                Q = (float)(qs + qr);
            } else if (!(qs < (double)kInf)) {
                Q = NAN;
            }
            float part = 0.f;
            if (id >= 0 && q != 0.f) {
                const float lp = log_prob(sx[threadIdx.x], in.c, all.m, ln_all);
                part = q * (lq - (all.s == 0.f ? -kInf : lp));
            }
            loss = block_reduce(part, AddOp());
            if (qr > 0.f)
                loss += qr * (logf(qr) - (in.c * (rest.m - all.m) + ln_rest - ln_all));
        }
        if (te.loss != nullptr && threadIdx.x == 0) te.loss[r] = loss;
        if (d != nullptr) {
            const bool none = empty || g == 0.f || all.s == 0.f;
            const float gc = g * in.c, c2 = in.c * kLog2e;
            const float ca = none ? 0.f : gc * Q / all.s, cr = qr > 0.f && !none ? gc * qr / rest.s : 0.f;
            __syncthreads();
            for (int i = threadIdx.x; i < in.V; i += kT) {
                float v = 0.f;
                if (!none) {
                    const float xi = widen(x[i]);
                    v = ca * ex2((xi - all.m) * c2);
                    if ((listed[i / 32] >> (i % 32)) & 1u) {
                        for (int l = 0; l < te.k; ++l)
                            if (sid[l] == i) v -= gc * sq[l];
                    } else if (cr != 0.f) {
                        v -= cr * ex2((xi - rest.m) * c2);
                    }
                }
                narrow(v, d + i);
            }
        }
        (void)first;
        __syncthreads();
    }
}

// ------------------------------------------------------------------ host side

bool on_device(const void* p, size_t align, int dev) {
    if (!p || (reinterpret_cast<uintptr_t>(p) % align) != 0) return false;
    cudaPointerAttributes a;
    if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return a.type == cudaMemoryTypeManaged || (a.type == cudaMemoryTypeDevice && a.device == dev);
}
bool maybe_on_device(const void* p, size_t align, int dev) {
    return p == nullptr || on_device(p, align, dev);
}

int status(cudaError_t e) {
    if (e == cudaSuccess) return MIMI_RVQ_OK;
    cudaGetLastError();
    return MIMI_RVQ_ECUDA;
}

bool rows_ok(int dtype, int64_t S, int n, int V, int64_t ss, int64_t sn, float scale) {
    if (dtype != MIMI_RVQ_F32 && dtype != MIMI_RVQ_BF16) return false;
    if (S < 0 || n < 0 || n > 65536 || S > (int64_t(1) << 40)) return false;
    if (V < 1 || V > MIMI_RVQ_MAX_VOCAB || ss < 0 || sn < 0) return false;
    if ((__int128)ss * S + (__int128)sn * n > ((__int128)1 << 58)) return false;  // no offset wraps
    return scale > 0.f && scale < kInf;
}

// Rows of a gradient must not share memory: the smaller stride holds a row, the larger one all
// rows of the smaller.
bool rows_apart(int64_t S, int n, int V, int64_t ss, int64_t sn) {
    if (S <= 1) return n <= 1 || sn >= V;
    if (n <= 1) return ss >= V;
    if (sn <= ss) return sn >= V && ss >= sn * (n - 1) + V;
    return ss >= V && sn >= ss * (S - 1) + V;
}

// The gradient may take the logits' own place (same pointer and strides) but may not overlap
// them in another way.
bool apart_or_same(const void* x, int64_t ss, int64_t sn, const void* d, int64_t dss, int64_t dsn,
                   int64_t S, int n, int V, int size) {
    if (x == d) return (S <= 1 || ss == dss) && (n <= 1 || sn == dsn);
    const char* a = static_cast<const char*>(x);
    const char* b = static_cast<const char*>(d);
    const char* a1 = a + (ss * (S - 1) + sn * (n - 1) + V) * size;
    const char* b1 = b + (dss * (S - 1) + dsn * (n - 1) + V) * size;
    return a1 <= b || b1 <= a;
}

int grid_of(int64_t rows) { return (int)(rows < (int64_t(1) << 30) ? rows : (int64_t(1) << 30)); }

}  // namespace
}  // namespace mimi

extern "C" int mimi_rvq_token_logprob(const void* logits, int dtype, int64_t S, int n, int V,
                                      int64_t stride_s, int64_t stride_n, const int32_t* tokens,
                                      int64_t tok_stride_s, int64_t tok_stride_n, int32_t pad,
                                      float scale, int top_k, float* logprob, float* entropy,
                                      float* lse, int32_t* top_ids, float* top_logprob,
                                      uint64_t* n_bad, struct CUstream_st* stream) {
    using namespace mimi;
    if (!rows_ok(dtype, S, n, V, stride_s, stride_n, scale) || top_k < 0 || top_k > kMaxTop ||
        (logprob != nullptr && tokens == nullptr))
        return MIMI_RVQ_EINVAL;
    if (S == 0 || n == 0) return MIMI_RVQ_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return status(cudaErrorInvalidDevice);
    const int size = dtype == MIMI_RVQ_BF16 ? 2 : 4;
    if (!on_device(logits, size, dev) || !maybe_on_device(tokens, 4, dev) ||
        !maybe_on_device(logprob, 4, dev) || !maybe_on_device(entropy, 4, dev) ||
        !maybe_on_device(lse, 4, dev) || !maybe_on_device(n_bad, 8, dev))
        return MIMI_RVQ_EINVAL;
    if (top_k > 0 && (!maybe_on_device(top_ids, 4, dev) || !maybe_on_device(top_logprob, 4, dev)))
        return MIMI_RVQ_EINVAL;
    const bool top = top_ids != nullptr || top_logprob != nullptr;
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale};
    const TokensIn tk{tokens, tok_stride_s, tok_stride_n, pad,
                      reinterpret_cast<unsigned long long*>(n_bad)};
    const ValuesOut o{logprob, entropy, lse, top_ids, top_logprob, top ? top_k : 0};
    if (dtype == MIMI_RVQ_BF16)
        k_logprob<__nv_bfloat16><<<grid_of(in.rows), kT, 0, stream>>>(in, tk, o);
    else
        k_logprob<float><<<grid_of(in.rows), kT, 0, stream>>>(in, tk, o);
    return status(cudaGetLastError());
}

extern "C" int mimi_rvq_token_logprob_grad(
    const void* logits, int dtype, int64_t S, int n, int V, int64_t stride_s, int64_t stride_n,
    const int32_t* tokens, int64_t tok_stride_s, int64_t tok_stride_n, int32_t pad, float scale,
    const float* g_logprob, const float* g_entropy, const float* g_lse, void* dlogits,
    int64_t d_stride_s, int64_t d_stride_n, float* logprob, float* entropy, float* lse,
    uint64_t* n_bad, struct CUstream_st* stream) {
    using namespace mimi;
    if (!rows_ok(dtype, S, n, V, stride_s, stride_n, scale) ||
        !rows_ok(dtype, S, n, V, d_stride_s, d_stride_n, scale) ||
        ((logprob != nullptr || g_logprob != nullptr) && tokens == nullptr))
        return MIMI_RVQ_EINVAL;
    if (!rows_apart(S, n, V, d_stride_s, d_stride_n)) return MIMI_RVQ_EINVAL;
    if (S == 0 || n == 0) return MIMI_RVQ_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return status(cudaErrorInvalidDevice);
    const int size = dtype == MIMI_RVQ_BF16 ? 2 : 4;
    if (!on_device(logits, size, dev) || !on_device(dlogits, size, dev) ||
        !apart_or_same(logits, stride_s, stride_n, dlogits, d_stride_s, d_stride_n, S, n, V, size) ||
        !maybe_on_device(tokens, 4, dev) || !maybe_on_device(g_logprob, 4, dev) ||
        !maybe_on_device(g_entropy, 4, dev) || !maybe_on_device(g_lse, 4, dev) ||
        !maybe_on_device(logprob, 4, dev) || !maybe_on_device(entropy, 4, dev) ||
        !maybe_on_device(lse, 4, dev) || !maybe_on_device(n_bad, 8, dev))
        return MIMI_RVQ_EINVAL;
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale};
    const TokensIn tk{tokens, tok_stride_s, tok_stride_n, pad,
                      reinterpret_cast<unsigned long long*>(n_bad)};
    const GradIn g{g_logprob, g_entropy, g_lse, dlogits, d_stride_s, d_stride_n};
    const ValuesOut o{logprob, entropy, lse, nullptr, nullptr, 0};
    if (dtype == MIMI_RVQ_BF16)
        k_logprob_grad<__nv_bfloat16><<<grid_of(in.rows), kT, 0, stream>>>(in, tk, g, o);
    else
        k_logprob_grad<float><<<grid_of(in.rows), kT, 0, stream>>>(in, tk, g, o);
    return status(cudaGetLastError());
}

namespace mimi {
namespace {

int distill(const void* logits, int dtype, int64_t S, int n, int V, int64_t stride_s,
            int64_t stride_n, const int32_t* ids, const void* teacher, int teacher_dtype, int k,
            int tail, float scale, const float* g, float* loss, bool grad, void* dlogits,
            int64_t d_stride_s, int64_t d_stride_n, uint64_t* n_bad, cudaStream_t stream) {
    if (!rows_ok(dtype, S, n, V, stride_s, stride_n, scale) || k < 1 || k > kMaxTop ||
        (tail != 0 && tail != 1) ||
        (teacher_dtype != MIMI_RVQ_F32 && teacher_dtype != MIMI_RVQ_BF16))
        return MIMI_RVQ_EINVAL;
    if (grad && (!rows_ok(dtype, S, n, V, d_stride_s, d_stride_n, scale) ||
                 !rows_apart(S, n, V, d_stride_s, d_stride_n)))
        return MIMI_RVQ_EINVAL;
    if (S == 0 || n == 0) return MIMI_RVQ_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return status(cudaErrorInvalidDevice);
    const int size = dtype == MIMI_RVQ_BF16 ? 2 : 4;
    if (!on_device(logits, size, dev) || !on_device(ids, 4, dev) ||
        !on_device(teacher, teacher_dtype == MIMI_RVQ_BF16 ? 2 : 4, dev) ||
        !maybe_on_device(g, 4, dev) || !maybe_on_device(loss, 4, dev) ||
        !maybe_on_device(n_bad, 8, dev))
        return MIMI_RVQ_EINVAL;
    if (!grad && loss == nullptr) return MIMI_RVQ_EINVAL;
    if (grad && (!on_device(dlogits, size, dev) ||
                 !apart_or_same(logits, stride_s, stride_n, dlogits, d_stride_s, d_stride_n, S, n,
                                V, size)))
        return MIMI_RVQ_EINVAL;
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale};
    const TeacherIn te{ids, teacher, teacher_dtype == MIMI_RVQ_BF16, k, tail, g, loss,
                       grad ? dlogits : nullptr, d_stride_s, d_stride_n,
                       reinterpret_cast<unsigned long long*>(n_bad)};
    const int smem = (V + 31) / 32 * 4;
    const void* f = dtype == MIMI_RVQ_BF16 ? (const void*)k_distill<__nv_bfloat16>
                                           : (const void*)k_distill<float>;
    const cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               MIMI_RVQ_MAX_VOCAB / 8);
    if (e != cudaSuccess) return status(e);
    if (dtype == MIMI_RVQ_BF16)
        k_distill<__nv_bfloat16><<<grid_of(in.rows), kT, smem, stream>>>(in, te);
    else
        k_distill<float><<<grid_of(in.rows), kT, smem, stream>>>(in, te);
    return status(cudaGetLastError());
}

}  // namespace
}  // namespace mimi

extern "C" int mimi_rvq_distill_topk(const void* logits, int dtype, int64_t S, int n, int V,
                                     int64_t stride_s, int64_t stride_n, const int32_t* ids,
                                     const void* teacher, int teacher_dtype, int k, int tail,
                                     float scale, float* loss, uint64_t* n_bad,
                                     struct CUstream_st* stream) {
    return mimi::distill(logits, dtype, S, n, V, stride_s, stride_n, ids, teacher, teacher_dtype, k,
                         tail, scale, nullptr, loss, false, nullptr, 0, 0, n_bad, stream);
}

extern "C" int mimi_rvq_distill_topk_grad(const void* logits, int dtype, int64_t S, int n, int V,
                                          int64_t stride_s, int64_t stride_n, const int32_t* ids,
                                          const void* teacher, int teacher_dtype, int k, int tail,
                                          float scale, const float* g, void* dlogits,
                                          int64_t d_stride_s, int64_t d_stride_n, float* loss,
                                          uint64_t* n_bad, struct CUstream_st* stream) {
    return mimi::distill(logits, dtype, S, n, V, stride_s, stride_n, ids, teacher, teacher_dtype, k,
                         tail, scale, g, loss, true, dlogits, d_stride_s, d_stride_n, n_bad, stream);
}
