// logits_logprob.cu -- log probabilities of the streams' tokens with entropy,
// log-sum-exp and top alternatives, and their gradient. Declared in
// include/mimi_rvq_streams.h; layout and statistics in logits.cuh.
//
// Forward: one pass over the row, bound by reading it (2 or 4 bytes a logit for
// one exponential, two sums and a maximum).
//
// Alternatives: the k largest by (logit descending, id ascending). A bound that
// at least k logits reach costs almost nothing on top of the pass: every
// thread has its share's maximum anyway, and the k-th largest of those maxima
// is such a bound (k threads hold a logit that reaches it). One warp finds it by
// bisecting the values' top 16 bits; only threads whose maximum reaches it look
// at their logits again and append those that do to a short list, which is
// ordered by counting. The order of appending has no influence. A list that
// overflows (rows of few distinct values) is replaced by k rounds that each
// take the largest key below the last.
//
// Gradient: d x_i = c p_i [(z - a) - b (ln p_i + H)] + c a [i = token] from the
// vectors in registers, so that the row is read once and written once.
#include "logits.cuh"

namespace mimi {
namespace {

using namespace logits;

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

using Key = unsigned long long;

// Order of a logit as an unsigned number; -0 and +0 are the same value (the sum makes both +0).
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t b = __float_as_uint(v + 0.f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
constexpr uint32_t kOrderNegInf = 0x007FFFFFu;  // order_of(-inf); NaN below it does not occur
// Larger comes first: (logit descending, id ascending).
__device__ __forceinline__ Key key_of(float v, int id) {
    return ((Key)order_of(v) << 32) | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float key_value(Key key) {
    const uint32_t o = (uint32_t)(key >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ int key_id(Key key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

// The row's target, -1 if it has none; count: add a token past V to n_bad.
__device__ __forceinline__ int target_of(const TokensIn& tk, int64_t s, int j, int V, bool count) {
    if (tk.tok == nullptr) return -1;
    const int32_t t = __ldg(tk.tok + s * tk.ss + j * tk.sn);
    if (t < 0 || t == tk.pad) return -1;
    if (t >= V) {
        if (count && tk.n_bad != nullptr) atomicAdd(tk.n_bad, 1ull);
        return -1;
    }
    return t;
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

// ------------------------------------------------------------------ alternatives

// Alternatives a warp's row may have: 32 maxima bound the list's length by about
// -32 ln(1 - k / 32) logits on rows in random order, 44 at k = 24.
constexpr int kWarpTop = 24;

template <int TH>
struct TopShared {
    static constexpr int kGroups = TH > 256 ? 256 : TH;  // maxima that bound the k-th logit
    static constexpr int kCap = TH == 32 ? 128 : 1024;
    uint32_t most[TH == 32 ? 1 : kGroups];
    uint32_t bound;
    int count;
    Key list[kCap];
    Key last[TH / 32];
};
template <int TH>
struct TopLists {  // the sorted lists of a cluster's CTAs, in the first one's memory
    Key of[TH == 32 ? 1 : kMaxCluster][TH == 32 ? 1 : kMaxTop];
};

// Sorted keys of this part's k largest logits: put(place, key) for places below the number of
// logits above -inf, put(place, 0) for the others. `v` holds the part where it is one chunk.
template <int TH, int NV, typename T, typename Put>
__device__ void part_top(TopShared<TH>& sh, const Part<T>& p, uint32_t (&v)[NV][4], float top,
                         int tid, int k, Put&& put) {
    constexpr int kG = TopShared<TH>::kGroups, kCap = TopShared<TH>::kCap;
    const int lane = tid & 31;
    const bool one = p.size() <= TH * NV;
    // the largest bound (in steps of 2^16) that k groups' maxima reach
    const uint32_t mine = order_of(top);
    uint32_t g = mine;
    if constexpr (TH == 32) {
        uint32_t b = 0;
        for (int bit = 31; bit >= 16; --bit) {
            const uint32_t t = b | (1u << bit);
            if (__popc(__ballot_sync(kFull, g >= t)) >= k) b = t;
        }
        if (lane == 0) {
            sh.bound = max(b, kOrderNegInf + 1);
            sh.count = 0;
        }
        __syncwarp();
    } else {
#pragma unroll
        for (int o = 1; o < TH / kG; o *= 2) g = max(g, __shfl_xor_sync(kFull, g, o));
        if (tid % (TH / kG) == 0) sh.most[tid / (TH / kG)] = g;
        __syncthreads();
        if (tid < 32) {
            uint32_t q[kG / 32];
#pragma unroll
            for (int i = 0; i < kG / 32; ++i) q[i] = sh.most[lane + 32 * i];
            uint32_t b = 0;
            for (int bit = 31; bit >= 16; --bit) {
                const uint32_t t = b | (1u << bit);
                unsigned n = 0;
#pragma unroll
                for (int i = 0; i < kG / 32; ++i) n += q[i] >= t;
                if ((int)__reduce_add_sync(kFull, n) >= k) b = t;
            }
            if (lane == 0) {
                sh.bound = max(b, kOrderNegInf + 1);
                sh.count = 0;
            }
        }
        __syncthreads();
    }
    const uint32_t bound = sh.bound;
    auto each_logit = [&](auto&& f) {  // this thread's logits, chunk by chunk
        for (int base = p.v0; base < p.v1; base += TH * NV) {
            if (!one) load_chunk<TH, NV>(p, base, tid, v);
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < Part<T>::kPer; ++j)
                    f(element<T>(v[i], j), p.first(base + i * TH + tid) + j);
        }
    };
    if (mine >= bound)
        each_logit([&](float x, int id) {
            if (order_of(x) >= bound) {
                const int at = atomicAdd(&sh.count, 1);
                if (at < kCap) sh.list[at] = key_of(x, id);
            }
        });
    group_sync<TH>();
    const int n = sh.count;
    if (n <= kCap) {
        for (int i = tid; i < n; i += TH) {
            const Key key = sh.list[i];
            int place = 0;
            for (int l = 0; l < n; ++l) place += sh.list[l] > key;
            if (place < k) put(place, key);
        }
        for (int i = n + tid; i < k; i += TH) put(i, Key(0));
    } else {
        Key last = ~Key(0);
        for (int q = 0; q < k; ++q) {
            Key best = 0;
            if (last != 0)
                each_logit([&](float x, int id) {
                    const Key key = key_of(x, id);
                    if (x > -kInf && key < last && key > best) best = key;
                });
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                const Key other = __shfl_xor_sync(kFull, best, o);
                best = other > best ? other : best;
            }
            if constexpr (TH > 32) {
                if (lane == 0) sh.last[tid / 32] = best;
                __syncthreads();
                for (int w = 0; w < TH / 32; ++w) best = sh.last[w] > best ? sh.last[w] : best;
                __syncthreads();
            }
            if (tid == 0) put(q, best);
            last = best;
        }
    }
}

// ------------------------------------------------------------------ forward

template <typename T, int TH, bool kTop>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<T, TH>()) k_logprob(RowsIn in, TokensIn tk, ValuesOut o) {
    constexpr int NV = vectors_of<T, TH>(), kRows = block_of<TH>() / TH;
    __shared__ Joint<TH> joint[kRows];
    __shared__ TopShared<kTop ? TH : 32> tops[kTop ? kRows : 1];
    __shared__ TopLists<kTop ? TH : 32> lists;
    const int tid = TH == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int group = TH == 32 ? threadIdx.x / 32 : 0;
    const int rank = in.cluster > 1 ? (int)cluster_ctarank() : 0;
    const float c2 = in.c * kLog2e, low = far_below(in.c);
    int parity = 0;
    if (in.cluster > 1) cluster_sync();  // every CTA runs before one writes to another
    for (int64_t r = (int64_t)(blockIdx.x / in.cluster) * kRows + group; r < in.rows;
         r += (int64_t)(gridDim.x / in.cluster) * kRows) {
        const int64_t s = r / in.n;
        const int j = (int)(r - s * in.n);
        const Part<T> p(static_cast<const T*>(in.x) + s * in.ss + j * in.sn, in.V, rank, in.cluster);
        uint32_t v[NV][4];
        load_chunk<TH, NV>(p, p.v0, tid, v);
        int t = -1;
        float xt = 0.f;
        if (tid == 0 && rank == 0) {
            t = target_of(tk, s, j, in.V, true);
            if (t >= 0) xt = widen(p.x[t]);
        }
        Stats st{-kInf, 0.f, 0.f};
        float top = -kInf;
        for (int base = p.v0; base < p.v1; base += TH * NV) {
            if (base != p.v0) load_chunk<TH, NV>(p, base, tid, v);
            add_chunk<TH, NV, true, T>(v, p.v1 - base, tid, c2, low, st, top);
        }
        st = join_row<TH, true>(joint[group], st, tid, in.cluster, rank, parity, c2, low);
        parity ^= 1;
        if (tid == 0 && rank == 0) put_values(o, r, t, xt, in.c, st);
        if constexpr (kTop) {
            const bool broken = !(st.s < kInf);
            const float ln_s = logf(st.s);
            auto out = [&](int place, Key key) {
                if (o.top_ids != nullptr) o.top_ids[r * o.k + place] = key ? key_id(key) : -1;
                if (o.top_logprob != nullptr)
                    o.top_logprob[r * o.k + place] =
                        broken ? NAN : key ? log_prob(key_value(key), in.c, st.m, ln_s) : -kInf;
            };
            if (broken) {
                if (rank == 0)
                    for (int i = tid; i < o.k; i += TH) out(i, Key(0));
            } else if (TH == 32 || in.cluster == 1) {
                part_top<TH, NV>(tops[group], p, v, top, tid, o.k, out);
            } else {
                const uint32_t to = cluster_map(smem_u32(&lists.of[rank][0]), 0);
                part_top<TH, NV>(tops[group], p, v, top, tid, o.k,
                                 [&](int place, Key key) { st_cluster_u64(to + 8 * place, key); });
                cluster_sync();
                // a key's place: its own list's, and what the other lists hold above it
                if (rank == 0)
                    for (int i = tid; i < in.cluster * o.k; i += TH) {
                        const int own = i / o.k;
                        const Key key = lists.of[own][i - own * o.k];
                        int place = i - own * o.k;
                        if (key == 0) {  // empty places: behind all keys, in their own order
                            for (int l = 0; l < in.cluster; ++l) {
                                if (l == own) continue;
                                for (int q = 0; q < o.k; ++q)
                                    place += lists.of[l][q] != 0 || l < own;
                            }
                        } else {
                            for (int l = 0; l < in.cluster; ++l) {
                                if (l == own) continue;
                                int a = 0, b = o.k;
                                while (a < b) {
                                    const int mid = (a + b) / 2;
                                    if (lists.of[l][mid] > key) a = mid + 1;
                                    else b = mid;
                                }
                                place += a;
                            }
                        }
                        if (place < o.k) out(place, key);
                    }
            }
        }
        group_sync<TH>();
    }
}

// ------------------------------------------------------------------ gradient

template <typename T, int TH>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<T, TH>()) k_logprob_grad(RowsIn in, TokensIn tk, GradIn g,
                                                               ValuesOut o) {
    constexpr int NV = vectors_of<T, TH>(), kRows = block_of<TH>() / TH, kPer = Part<T>::kPer;
    __shared__ Joint<TH> joint[kRows];
    const int tid = TH == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int group = TH == 32 ? threadIdx.x / 32 : 0;
    const int rank = in.cluster > 1 ? (int)cluster_ctarank() : 0;
    const float c2 = in.c * kLog2e, low = far_below(in.c);
    const bool values = o.logprob != nullptr || o.entropy != nullptr || o.lse != nullptr;
    int parity = 0;
    if (in.cluster > 1) cluster_sync();
    for (int64_t r = (int64_t)(blockIdx.x / in.cluster) * kRows + group; r < in.rows;
         r += (int64_t)(gridDim.x / in.cluster) * kRows) {
        const int64_t s = r / in.n;
        const int j = (int)(r - s * in.n);
        const Part<T> p(static_cast<const T*>(in.x) + s * in.ss + j * in.sn, in.V, rank, in.cluster);
        // the gradient's row has its own alignment
        T* d = static_cast<T*>(g.d) + s * g.ss + j * g.sn;
        const bool wide = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0;
        const int t = target_of(tk, s, j, in.V, tid == 0 && rank == 0);
        const float a = (t < 0 || g.g_logprob == nullptr) ? 0.f : __ldg(g.g_logprob + r);
        const float b = g.g_entropy == nullptr ? 0.f : __ldg(g.g_entropy + r);
        const float z = g.g_lse == nullptr ? 0.f : __ldg(g.g_lse + r);
        const bool zero = a == 0.f && b == 0.f && z == 0.f;
        uint32_t v[NV][4];
        Stats st{-kInf, 0.f, 0.f};
        const bool owner = t >= 0 && p.holds(p.vector_of(t)) && (p.vector_of(t) - p.v0) % TH == tid;
        float xt = 0.f;
        if (!zero || values) {
            load_chunk<TH, NV>(p, p.v0, tid, v);
            if (t >= 0 && (owner || (tid == 0 && rank == 0))) xt = widen(p.x[t]);
            float top = -kInf;
            for (int base = p.v0; base < p.v1; base += TH * NV) {
                if (base != p.v0) load_chunk<TH, NV>(p, base, tid, v);
                add_chunk<TH, NV, true, T>(v, p.v1 - base, tid, c2, low, st, top);
            }
            st = join_row<TH, true>(joint[group], st, tid, in.cluster, rank, parity, c2, low);
            parity ^= 1;
            if (tid == 0 && rank == 0) put_values(o, r, t, xt, in.c, st);
        }
        const bool none = zero || st.s == 0.f;
        const float m = none ? 0.f : st.m;
        const float inv = none ? 0.f : 1.f / st.s, ln_s = none ? 0.f : logf(st.s);
        const float h = ln_s - in.c * (st.w * inv);
        // c p_i [(z - a) - b (ln p_i + H)] = e^{c (x - m)} (c0 + c1 (x - m))
        const float c0 = in.c * inv * ((z - a) - b * (h - ln_s)), c1 = -in.c * inv * b * in.c;
        for (int base = p.v0; base < p.v1; base += TH * NV) {
            if (!none && p.size() > TH * NV) load_chunk<TH, NV>(p, base, tid, v);
            each_vector<TH, NV>(v, p.v1 - base, tid, [&](int i, uint32_t (&w)[4]) {
                const int vec = base + i * TH + tid, at = p.first(vec);
                float y[kPer];
                if (none) {
#pragma unroll
                    for (int e = 0; e < kPer; ++e) y[e] = 0.f;
                } else {
                    add_to(w, -m, y);
#pragma unroll
                    for (int e = 0; e < kPer; ++e)
                        y[e] = ex2(y[e] * c2) * fmaf(c1, fmaxf(y[e], low), c0);
                }
                store_vector<T>(d, at, y, wide && vec >= p.lo && vec < p.hi, vec < p.v1, in.V);
            });
        }
        if (owner && !none) {
            const float df = xt - m;
            narrow(ex2(df * c2) * fmaf(c1, fmaxf(df, low), c0) + in.c * a, d + t);
        }
        group_sync<TH>();
    }
}

template <typename T, bool kTop>
cudaError_t forward_of(const Shape& sh, const RowsIn& in, const TokensIn& tk, const ValuesOut& o,
                       cudaStream_t s) {
    switch (sh.threads) {
        case 32: return launch_rows(k_logprob<T, 32, kTop>, 32, in, 0, s, in, tk, o);
        case 128: return launch_rows(k_logprob<T, 128, kTop>, 128, in, 0, s, in, tk, o);
        case 256: return launch_rows(k_logprob<T, 256, kTop>, 256, in, 0, s, in, tk, o);
        default: return launch_rows(k_logprob<T, 512, kTop>, 512, in, 0, s, in, tk, o);
    }
}

template <typename T>
cudaError_t gradient_of(const Shape& sh, const RowsIn& in, const TokensIn& tk, const GradIn& g,
                        const ValuesOut& o, cudaStream_t s) {
    switch (sh.threads) {
        case 32: return launch_rows(k_logprob_grad<T, 32>, 32, in, 0, s, in, tk, g, o);
        case 128: return launch_rows(k_logprob_grad<T, 128>, 128, in, 0, s, in, tk, g, o);
        case 256: return launch_rows(k_logprob_grad<T, 256>, 256, in, 0, s, in, tk, g, o);
        default: return launch_rows(k_logprob_grad<T, 512>, 512, in, 0, s, in, tk, g, o);
    }
}

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
    if (cudaGetDevice(&dev) != cudaSuccess) return status_of(cudaErrorInvalidDevice);
    const int size = dtype == MIMI_RVQ_BF16 ? 2 : 4;
    if (!on_device(logits, size, dev) || !maybe_on_device(tokens, 4, dev) ||
        !maybe_on_device(logprob, 4, dev) || !maybe_on_device(entropy, 4, dev) ||
        !maybe_on_device(lse, 4, dev) || !maybe_on_device(n_bad, 8, dev))
        return MIMI_RVQ_EINVAL;
    if (top_k > 0 && (!maybe_on_device(top_ids, 4, dev) || !maybe_on_device(top_logprob, 4, dev)))
        return MIMI_RVQ_EINVAL;
    const int k = top_ids != nullptr || top_logprob != nullptr ? top_k : 0;
    const Shape sh = shape_of(S * n, V, size, k <= kWarpTop);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.cluster};
    const TokensIn tk{tokens, tok_stride_s, tok_stride_n, pad,
                      reinterpret_cast<unsigned long long*>(n_bad)};
    const ValuesOut o{logprob, entropy, lse, top_ids, top_logprob, k};
    if (dtype == MIMI_RVQ_BF16)
        return status_of(k ? forward_of<__nv_bfloat16, true>(sh, in, tk, o, stream)
                           : forward_of<__nv_bfloat16, false>(sh, in, tk, o, stream));
    return status_of(k ? forward_of<float, true>(sh, in, tk, o, stream)
                       : forward_of<float, false>(sh, in, tk, o, stream));
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
    if (S == 0 || n == 0) return MIMI_RVQ_OK;
    if (!rows_apart(S, n, V, d_stride_s, d_stride_n)) return MIMI_RVQ_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return status_of(cudaErrorInvalidDevice);
    const int size = dtype == MIMI_RVQ_BF16 ? 2 : 4;
    if (!on_device(logits, size, dev) || !on_device(dlogits, size, dev) ||
        !apart_or_same(logits, stride_s, stride_n, dlogits, d_stride_s, d_stride_n, S, n, V, size) ||
        !maybe_on_device(tokens, 4, dev) || !maybe_on_device(g_logprob, 4, dev) ||
        !maybe_on_device(g_entropy, 4, dev) || !maybe_on_device(g_lse, 4, dev) ||
        !maybe_on_device(logprob, 4, dev) || !maybe_on_device(entropy, 4, dev) ||
        !maybe_on_device(lse, 4, dev) || !maybe_on_device(n_bad, 8, dev))
        return MIMI_RVQ_EINVAL;
    const Shape sh = shape_of(S * n, V, size, true);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.cluster};
    const TokensIn tk{tokens, tok_stride_s, tok_stride_n, pad,
                      reinterpret_cast<unsigned long long*>(n_bad)};
    const GradIn g{g_logprob, g_entropy, g_lse, dlogits, d_stride_s, d_stride_n};
    const ValuesOut o{logprob, entropy, lse, nullptr, nullptr, 0};
    return status_of(dtype == MIMI_RVQ_BF16 ? gradient_of<__nv_bfloat16>(sh, in, tk, g, o, stream)
                                            : gradient_of<float>(sh, in, tk, g, o, stream));
}
