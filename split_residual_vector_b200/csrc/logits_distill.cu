// logits_distill.cu -- distillation from a teacher's top list and its gradient.
// Declared in include/mimi_rvq_streams.h; layout and statistics in logits.cuh.
//
// The row's listed tokens are taken out of the pass: the group's first warp
// reads the list, gathers the listed logits and marks their places (one byte
// per vector, a bit per element) while the row's loads are in flight, and
// marked elements enter the pass as -inf. The pass then gives the statistics of
// the rest, from which both the whole row's (joined with the listed logits) and
// the tail class's probability follow without cancellation, however certain
// the student is of the list. With (m_r, s_r) the rest's and ln s the row's:
//     ln p_i = c (x_i - m) - ln s,   ln p_rest = c (m_r - m) + ln s_r - ln s,
//     d x_i = g c (Q p_i - q_r e^{c (x_i - m_r)} / s_r)       unlisted
//           = e^{c (x_i - m_r)} (g c) (Q e^{c (m_r - m)} / s - q_r / s_r),
//     d x_i = g c (Q p_i - sum of the entries' q)             listed,
// so unlisted gradients need one exponential and the registers' vectors; the
// listed ones are written over them by the first warp.
#include "logits.cuh"

namespace mimi {
namespace {

using namespace logits;

struct TeacherIn {
    const int32_t* ids;  // [S][n][k]
    const void* t;
    int t_bf16;
    int k, tail;
    const float* g;  // NULL: 1
    float* loss;     // may be NULL with a gradient
    void* d;
    int64_t d_ss, d_sn;
    unsigned long long* n_bad;
};

constexpr int kLane = kMaxTop / 32;  // list entries of a lane

// The list, kept by the group's first warp, and what it leaves for the group before the row's
// barrier.
struct ListShared {
    int id[kMaxTop];      // -1: an empty place
    float q[kMaxTop], lq[kMaxTop], x[kMaxTop];  // weight, its logarithm, the student's logit
    float m, s;           // this part's listed logits
    float Q, tail_q;      // sum of the weights (renormalised: 1), 1 - it where the tail is a class
    int present;          // entries
};

// The listed logits of a row's parts, exchanged like the parts' own statistics.
struct ListJoint {
    float cta[2][2][kMaxCluster];
};

// Chunks of the longest part of a row of V: a row off a 16-byte boundary has one vector more.
template <typename T, int TH>
__host__ __device__ constexpr int most_chunks(int V, int cluster) {
    constexpr int kPer = Elem<T>::kPer, kChunk = TH * vectors_of<T, TH>();
    return (((V + kPer - 1) / kPer + 1 + cluster - 1) / cluster + kChunk - 1) / kChunk;
}

template <typename T, int TH, bool kGrad>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<T, TH>()) k_distill(RowsIn in, TeacherIn te) {
    constexpr int NV = vectors_of<T, TH>(), kRows = block_of<TH>() / TH, kPer = Part<T>::kPer;
    extern __shared__ __align__(16) uint8_t marks[];  // [groups][chunks][TH][NV]
    __shared__ Joint<TH> joint[kRows];
    __shared__ ListShared lists[kRows];
    __shared__ ListJoint listed_of;
    const int tid = TH == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int group = TH == 32 ? threadIdx.x / 32 : 0;
    const int rank = in.cluster > 1 ? (int)cluster_ctarank() : 0;
    const float c2 = in.c * kLog2e;
    ListShared& ls = lists[group];
    int parity = 0;
    if (in.cluster > 1) cluster_sync();
    RowWalk at_row((int64_t)(blockIdx.x / in.cluster) * kRows + group,
                   (int64_t)(gridDim.x / in.cluster) * kRows, in.n);
    for (; at_row.r < in.rows; at_row.next(in.n)) {
        const int64_t r = at_row.r, s = at_row.s;
        const int j = at_row.j;
        const Part<T> p(static_cast<const T*>(in.x) + s * in.ss + j * in.sn, in.V, rank, in.cluster);
        const int chunks = (p.size() + TH * NV - 1) / (TH * NV);
        uint8_t* mark = marks + (size_t)group * most_chunks<T, TH>(in.V, in.cluster) * TH * NV;
        const float g = kGrad && te.g != nullptr ? __ldg(te.g + r) : 1.f;
        const bool skip = kGrad && g == 0.f && te.loss == nullptr;  // its gradient is 0
        uint32_t v[NV][4];
        if (!skip) load_chunk<TH, NV>(p, p.v0, tid, v);
        for (int q = 0; q < chunks; ++q)
#pragma unroll
            for (int i = 0; i < NV; i += 8)
                *reinterpret_cast<uint2*>(mark + (q * TH + tid) * NV + i) = make_uint2(0, 0);

        // ---- the list (first warp; entries of lane l: l, l + 32, ...)
        if (tid < 32) {
            int id[kLane], n = 0, bad = 0;
            float tmax = -kInf;
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                const int e = tid + 32 * i;
                id[i] = e < te.k ? __ldg(te.ids + r * te.k + e) : -1;
            }
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                const int e = tid + 32 * i;
                if (id[i] >= in.V) {
                    ++bad;
                    id[i] = -1;
                }
                float t = -kInf, x = -kInf;
                if (id[i] >= 0) {
                    t = te.t_bf16 ? widen(static_cast<const __nv_bfloat16*>(te.t)[r * te.k + e])
                                  : static_cast<const float*>(te.t)[r * te.k + e];
                    x = widen(p.x[id[i]]);
                    tmax = fmaxf(tmax, t);
                    ++n;
                }
                if (e < te.k) {
                    ls.id[e] = id[i];
                    ls.lq[e] = t;
                    ls.x[e] = x;
                }
            }
            if (bad && rank == 0 && te.n_bad != nullptr)
                atomicAdd(te.n_bad, (unsigned long long)bad);
            n = (int)__reduce_add_sync(kFull, (unsigned)n);
            float Q = 1.f, tail_q = 0.f;
            if (te.tail) {
                // the tail's weight is what the list leaves of 1: in float64, or a tail of
                // 1e-6 would be rounding
                double sum = 0.0;
                for (int e = tid; e < te.k; e += 32) {
                    const bool in_list = ls.id[e] >= 0;
                    ls.q[e] = in_list ? expf(ls.lq[e]) : 0.f;
                    if (in_list) sum += exp((double)ls.lq[e]);
                }
                sum = warp_sum(sum);
                Q = (float)sum;
                tail_q = (float)fmax(0.0, 1.0 - sum);
            } else {
                tmax = warp_max(tmax);
                const float tm = tmax == -kInf ? 0.f : tmax;
                float sum = 0.f;
                for (int e = tid; e < te.k; e += 32)
                    if (ls.id[e] >= 0) sum += expf(ls.lq[e] - tm);
                sum = warp_sum(sum);
                if (sum == 0.f) n = 0;       // a list without weight
                if (!(sum < kInf)) Q = NAN;  // a broken entry
                const float ln = logf(sum);
                for (int e = tid; e < te.k; e += 32) {
                    const float lq = (ls.lq[e] - tm) - ln;
                    ls.lq[e] = lq;
                    ls.q[e] = ls.id[e] >= 0 ? expf(lq) : 0.f;
                }
            }
            if (tid == 0) {
                ls.present = n;
                ls.Q = Q;
                ls.tail_q = tail_q;
            }
        }
        group_sync<TH>();  // the marks are clear
        unsigned first = 0;  // bit i: entry tid + 32 i is this part's, the first of its id
        bool twice = false;  // some id is listed twice
        if (tid < 32) {
            float m = -kInf, sum = 0.f;
            for (int e = tid, i = 0; e < te.k; e += 32, ++i) {
                const int id = ls.id[e];
                const int vec = p.vector_of(id), at = vec - p.v0;
                if (id < 0 || !p.holds(vec)) continue;
                const int byte = ((at / (TH * NV)) * TH + at % TH) * NV + (at / TH) % NV;
                const uint32_t bit = 1u << ((byte & 3) * 8 + (id - p.first(vec)));
                const uint32_t old = atomicOr(reinterpret_cast<uint32_t*>(mark + (byte & ~3)), bit);
                if (old & bit) twice = true;
                first |= 1u << i;
                m = fmaxf(m, ls.x[e]);
            }
            twice = __any_sync(kFull, twice);
            if (twice)  // drop the later ones of equal ids
                for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                    for (int l = 0; l < e; ++l)
                        if (ls.id[l] == ls.id[e]) first &= ~(1u << i);
            m = warp_max(m);
            const float mu = m == -kInf ? 0.f : m;
            for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                if ((first >> i) & 1u) sum += ex2((ls.x[e] - mu) * c2);
            sum = warp_sum(sum);
            if (tid == 0) {
                ls.m = m;
                ls.s = sum;
            }
        }
        group_sync<TH>();  // the marks are set

        // ---- the rest
        Stats rest{-kInf, 0.f, 0.f}, all{-kInf, 0.f, 0.f};
        const bool empty = ls.present == 0;
        if (!skip && !empty) {
            for (int q2 = 0; q2 < chunks; ++q2) {
                const int base = p.v0 + q2 * TH * NV;
                if (q2) load_chunk<TH, NV>(p, base, tid, v);
                hide<NV, T>(mark + (q2 * TH + tid) * NV, v);
                add_chunk<TH, NV, false, T>(p, base, tid, v, c2, rest);
            }
            if (in.cluster > 1 && tid < in.cluster) {
                const uint32_t to = cluster_map(smem_u32(&listed_of.cta[parity][0][rank]), tid);
                st_cluster_f32(to, ls.m);
                st_cluster_f32(to + 4 * kMaxCluster, ls.s);
            }
            rest = join_row<TH, false>(joint[group], rest, tid, in.cluster, rank, parity, c2);
            float lm = ls.m, lsum = ls.s;
            parity ^= 1;
            if (in.cluster > 1) {
                const int lane = tid & 31;
                const bool in_c = lane < in.cluster;
                const Stats l = join_lanes<false>(in_c ? listed_of.cta[parity ^ 1][0][lane] : -kInf,
                                                  in_c ? listed_of.cta[parity ^ 1][1][lane] : 0.f, 0.f,
                                                  c2);
                lm = l.m;
                lsum = l.s;
            }
            all.m = fmaxf(rest.m, lm);
            const float mu = all.m == -kInf ? 0.f : all.m;
            all.s = rest.s * ex2((rest.m - mu) * c2) + lsum * ex2((lm - mu) * c2);
        }
        const bool none = g == 0.f || empty || all.s == 0.f;  // a gradient of zeros
        const float qr = rest.s == 0.f ? 0.f : ls.tail_q;
        const float Q = te.tail ? ls.Q + qr : ls.Q;
        if (te.loss != nullptr && rank == 0 && tid < 32) {
            const float ln_s = ln(all.s);
            float part = 0.f;
            if (!empty) {
                for (int e = tid; e < te.k; e += 32)
                    if (ls.q[e] != 0.f)
                        part += ls.q[e] * (ls.lq[e] - (all.s == 0.f ? -kInf : log_prob(ls.x[e], in.c, all.m, ln_s)));
                part = warp_sum(part);
                if (qr > 0.f)
                    part += qr * (logf(qr) - (in.c * (rest.m - all.m) + ln(rest.s) - ln_s));
            }
            if (tid == 0) te.loss[r] = part;
        }
        if constexpr (kGrad) {
            T* d = static_cast<T*>(te.d) + s * te.d_ss + j * te.d_sn;
            const bool wide =
                ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0;
            const float gc = g * in.c, inv = none ? 0.f : reciprocal(all.s);
            const Scale k(c2, rest.m);
            // a rest of -inf only has no gradient of its own: 2^t is 0 there
            const float f = none ? 0.f
                : gc * ex2(-k.shift) * (Q * inv * (rest.s == 0.f ? 1.f : ex2((rest.m - all.m) * c2))
                                        - (qr > 0.f ? qr / rest.s : 0.f));
            for (int q2 = 0; q2 < chunks; ++q2) {
                const int base = p.v0 + q2 * TH * NV;
                if (!none && chunks > 1) {
                    load_chunk<TH, NV>(p, base, tid, v);
                    hide<NV, T>(mark + (q2 * TH + tid) * NV, v);
                }
                store_chunk<TH, NV>(p, base, tid, d, wide, v, [&](const uint32_t (&w)[4], float (&y)[kPer]) {
                    if (none) {
#pragma unroll
                        for (int e = 0; e < kPer; ++e) y[e] = 0.f;
                    } else {
                        Pair t[kPer / 2];
                        exponents<T, false>(w, k, t);
#pragma unroll
                        for (int e = 0; e < kPer / 2; ++e)
                            halves(mul2(ex2_pair(t[e]), pair_of(f, f)), y[2 * e], y[2 * e + 1]);
                    }
                });
            }
            group_sync<TH>();  // the listed tokens' places hold the rest's gradient by now
            if (tid < 32 && !none) {
                for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                    if ((first >> i) & 1u) {
                        const int id = ls.id[e];
                        float w = ls.q[e];
                        if (twice) {
                            w = 0.f;
                            for (int l = 0; l < te.k; ++l)
                                if (ls.id[l] == id) w += ls.q[l];
                        }
                        const float pi = ex2((ls.x[e] - all.m) * c2) * inv;
                        narrow(gc * (Q * pi - w), d + id);
                    }
            }
        }
        group_sync<TH>();
    }
}

template <typename T, bool kGrad, int TH>
cudaError_t distill_with(const RowsIn& in, const TeacherIn& te, cudaStream_t s) {
    const int smem = block_of<TH>() * vectors_of<T, TH>() * most_chunks<T, TH>(in.V, in.cluster);
    return launch_rows(k_distill<T, TH, kGrad>, TH, in, smem, s, in, te);
}

template <typename T, bool kGrad>
cudaError_t distill_of(const Shape& sh, const RowsIn& in, const TeacherIn& te, cudaStream_t s) {
    switch (sh.threads) {
        case 32: return distill_with<T, kGrad, 32>(in, te, s);
        case 128: return distill_with<T, kGrad, 128>(in, te, s);
        case 256: return distill_with<T, kGrad, 256>(in, te, s);
        default: break;
    }
    // only a gradient holds rows that want 512 threads
    if constexpr (kGrad) return distill_with<T, kGrad, 512>(in, te, s);
    return cudaErrorInvalidConfiguration;
}

int distill(const void* logits, int dtype, int64_t S, int n, int V, int64_t stride_s,
            int64_t stride_n, const int32_t* ids, const void* teacher, int teacher_dtype, int k,
            int tail, float scale, const float* g, float* loss, bool grad, void* dlogits,
            int64_t d_stride_s, int64_t d_stride_n, uint64_t* n_bad, cudaStream_t stream) {
    if (!rows_ok(dtype, S, n, V, stride_s, stride_n, scale) || k < 1 || k > kMaxTop ||
        (tail != 0 && tail != 1) ||
        (teacher_dtype != MIMI_RVQ_F32 && teacher_dtype != MIMI_RVQ_BF16))
        return MIMI_RVQ_EINVAL;
    if (grad && !rows_ok(dtype, S, n, V, d_stride_s, d_stride_n, scale)) return MIMI_RVQ_EINVAL;
    if (S == 0 || n == 0) return MIMI_RVQ_OK;
    if (grad && !rows_apart(S, n, V, d_stride_s, d_stride_n)) return MIMI_RVQ_EINVAL;
    if (!grad && loss == nullptr) return MIMI_RVQ_EINVAL;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return status_of(cudaErrorInvalidDevice);
    const int size = dtype == MIMI_RVQ_BF16 ? 2 : 4;
    if (!on_device(logits, size, dev) || !on_device(ids, 4, dev) ||
        !on_device(teacher, teacher_dtype == MIMI_RVQ_BF16 ? 2 : 4, dev) ||
        !maybe_on_device(g, 4, dev) || !maybe_on_device(loss, 4, dev) ||
        !maybe_on_device(n_bad, 8, dev))
        return MIMI_RVQ_EINVAL;
    if (grad && (!on_device(dlogits, size, dev) ||
                 !apart_or_same(logits, stride_s, stride_n, dlogits, d_stride_s, d_stride_n, S, n,
                                V, size)))
        return MIMI_RVQ_EINVAL;
    const Shape sh = shape_of(S * n, V, size, true, grad);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.cluster};
    const TeacherIn te{ids, teacher, teacher_dtype == MIMI_RVQ_BF16, k, tail, g, loss, dlogits,
                       d_stride_s, d_stride_n, reinterpret_cast<unsigned long long*>(n_bad)};
    if (dtype == MIMI_RVQ_BF16)
        return status_of(grad ? distill_of<__nv_bfloat16, true>(sh, in, te, stream)
                              : distill_of<__nv_bfloat16, false>(sh, in, te, stream));
    return status_of(grad ? distill_of<float, true>(sh, in, te, stream)
                          : distill_of<float, false>(sh, in, te, stream));
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
