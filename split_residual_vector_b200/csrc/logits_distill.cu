// logits_distill.cu -- distillation from a teacher's top list and its gradient.
// Declared in include/mimi_rvq_streams.h; layout and statistics in logits.cuh.
//
// The row's listed tokens are taken out of the pass: once the row is in shared
// memory the group's first warp reads the listed logits there and puts -inf in
// their places (an id listed twice is seen by the entries' numbers that are
// written there in between). The pass then gives the statistics of the rest,
// from which both the whole row's (joined with the listed logits) and the tail
// class's probability follow without cancellation, however certain
// the student is of the list. With (m_r, s_r) the rest's and ln s the row's:
//     ln p_i = c (x_i - m) - ln s,   ln p_rest = c (m_r - m) + ln s_r - ln s,
//     d x_i = g c (Q p_i - q_r e^{c (x_i - m_r)} / s_r)       unlisted
//           = e^{c (x_i - m_r)} (g c) (Q e^{c (m_r - m)} / s - q_r / s_r),
//     d x_i = g c (Q p_i - sum of the entries' q)             listed,
// so unlisted gradients need one exponential; the listed ones are written over
// them by the first warp.
#include <type_traits>

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

// A place of the list: kept by the group's first lanes (16 or 32), lane l having places l,
// l + lanes, ...
struct alignas(16) Entry {
    int id;          // -1: an empty place
    float q, lq, x;  // weight, its logarithm, the student's logit
};

// What the list leaves for the group.
template <typename T>
struct ListShared {
    T edge[16];       // the elements beside the row's vectors
    float m, s;       // this share's listed logits
    float Q, tail_q;  // sum of the weights (renormalised: 1), 1 - it where the tail is a class
    int empty;        // no entry, or none with weight
};

// The listed logits of a row's shares, exchanged like the shares' own statistics.
struct ListJoint {
    float cta[2][2][kMaxCluster];
};

// The bits of an element in shared memory.
template <typename T>
using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;

template <typename T, int TH, bool kGrad>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<TH>()) k_distill(RowsIn in, TeacherIn te) {
    constexpr int kRows = block_of<TH>() / TH, kPer = Part<T>::kPer;
    extern __shared__ uint4 buffers[];  // [groups][slots]: the row's vectors, then the list
    __shared__ Joint<TH> joint[kRows];
    __shared__ ListShared<T> lists[kRows];
    __shared__ ListJoint listed_of;
    const int tid = thread_in_group<TH>();
    const int group = group_in_block<TH>();
    const int lc = TH <= 32 ? 0 : in.log_cluster, cluster = 1 << lc;
    const int rank = lc ? (int)cluster_ctarank() : 0;
    const bool first_lanes = rank == 0 && tid < lanes_of<TH>();  // have the row's edges
    uint4* buf = buffers + (size_t)group * in.slots;
    Entry* list = reinterpret_cast<Entry*>(buf + in.slots - te.k);
    const float c2 = in.c * kLog2e;
    ListShared<T>& ls = lists[group];
    constexpr int L = lanes_of<TH>(), kLane = kMaxTop / L;
    const unsigned mask = lane_mask<TH>();
    const bool lister = tid < L;
    if (lc) cluster_sync();  // every CTA runs before one writes to another
    RowWalk row((int64_t)(blockIdx.x >> lc) * kRows + group,
                (int64_t)(gridDim.x >> lc) * kRows, in.n);
    // the row's weight and list: loaded a row ahead
    float g_next = 1.f;
    int id_next[kLane];
    float t_next[kLane];
    auto list_at = [&]() {
        if (row.r >= in.rows) return;
        if (kGrad && te.g != nullptr) g_next = __ldg(te.g + row.r);
        if (lister) {
            const int64_t at = row.r * te.k;
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                if (i * L >= te.k) break;
                const int e = tid + L * i;
                id_next[i] = -1;
                if (e < te.k) {
                    id_next[i] = __ldg(te.ids + at + e);
                    t_next[i] = te.t_bf16 ? widen(__ldg(static_cast<const __nv_bfloat16*>(te.t) + at + e))
                                          : __ldg(static_cast<const float*>(te.t) + at + e);
                }
            }
        }
    };
    list_at();
    for (int parity = 0; row.r < in.rows;) {
        const int64_t r = row.r;
        const Part<T> p(static_cast<const T*>(in.x) + row.s * in.ss + row.j * in.sn, in.V, rank, lc);
        T* d = static_cast<T*>(te.d) + row.s * te.d_ss + row.j * te.d_sn;
        const bool wide = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0;
        T* out = d + p.first;
        const float g = kGrad ? g_next : 1.f;
        const bool skip = kGrad && g == 0.f && te.loss == nullptr;  // zeros, whatever the row is
        const int ie = first_lanes ? p.edge(tid) : -1;
        float edge = -kInf;
        if (!skip) {
            fetch<TH>(buf, p, tid);
            if (ie >= 0) edge = widen(p.x[ie]);
        }
        int n = 0, bad = 0;
        float tmax = -kInf;
        bool broken = false;  // NaN or +inf among the entries
        if (lister) {
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                if (i * L >= te.k) break;
                const int e = tid + L * i;
                if (e >= te.k) continue;
                int id = id_next[i];
                if (id >= in.V) ++bad;
                if (id < 0 || id >= in.V) id = -1;
                const float t = id >= 0 ? t_next[i] : -kInf;
                n += id >= 0;
                tmax = fmaxf(tmax, t);
                broken |= !(t < kInf);
                list[e].id = id;
                list[e].lq = t;
            }
            if (bad && rank == 0 && te.n_bad != nullptr)
                atomicAdd(te.n_bad, (unsigned long long)bad);
        }
        row.next(in.n);
        list_at();
        bool empty = true;
        unsigned first = 0;  // bit i: entry tid + L i is this share's, the first of its id
        bool twice = false;  // some id is listed twice
        if (!skip) {
            arrived();
            if (first_lanes && tid < 16 && ie >= 0) narrow(edge, &ls.edge[tid]);
            group_sync<TH>();  // the row is here
            if (lister) {
                using B = Bits<T>;
                // where a listed element of this share is
                auto cell = [&](int id) {
                    const int q = p.place(id);
                    return q >= 0 ? reinterpret_cast<B*>(buf) + q
                                  : reinterpret_cast<B*>(ls.edge) + p.edge_lane(id);
                };
                for (int e = tid, i = 0; e < te.k; e += L, ++i) {
                    const int id = list[e].id;
                    if (id < 0) continue;
                    if (p.place(id) >= 0 || (rank == 0 && p.in_edges(id))) {
                        first |= 1u << i;
                        list[e].x = widen(*reinterpret_cast<const T*>(cell(id)));
                    } else if (rank == 0) {
                        list[e].x = widen(p.x[id]);  // another CTA's; for the loss
                    }
                }
                __syncwarp(mask);
                auto each_first = [&](auto&& f) {
                    for (int e = tid, i = 0; e < te.k; e += L, ++i)
                        if ((first >> i) & 1u) f(e, i);
                    __syncwarp(mask);
                };
                each_first([&](int e, int) { *cell(list[e].id) = (B)e; });
                each_first([&](int e, int) { twice |= *cell(list[e].id) != (B)e; });
                each_first([&](int e, int) { *cell(list[e].id) = (B)Elem<T>::kFill; });
                twice = __any_sync(mask, twice);
                if (twice)  // the first of equal ids stands for all
                    each_first([&](int e, int i) {
                        for (int l = 0; l < e; ++l)
                            if (list[l].id == list[e].id) first &= ~(1u << i);
                    });
                const bool some = __any_sync(mask, n > 0);
                tmax = lanes_max<TH>(tmax);
                broken = __any_sync(mask, broken);
                if (tid == 0) ls.empty = !some || (!te.tail && tmax == -kInf && !broken);
                if (ie >= 0) edge = widen(ls.edge[tid]);
            }
            group_sync<TH>();  // the listed tokens are hidden
            empty = ls.empty != 0;
        }
        Stats rest{-kInf, 0.f, 0.f}, all{-kInf, 0.f, 0.f};
        if (!empty) {
            float top;
            rest = pass<TH, false, T>(buf, p.nv, tid, edge, c2, top);
            if (lister) {  // the weights and this share's listed logits
                float Q = 1.f, tail_q = 0.f;
                if (te.tail) {
                    // the tail's weight is what the list leaves of 1: in float64, or a tail of
                    // 1e-6 would be rounding
                    double sum = 0.0;
                    for (int e = tid; e < te.k; e += L) {
                        const bool in_list = list[e].id >= 0;
                        list[e].q = in_list ? expf(list[e].lq) : 0.f;
                        if (in_list) sum += exp((double)list[e].lq);
                    }
                    sum = lanes_sum<TH>(sum);
                    Q = broken ? NAN : (float)sum;
                    tail_q = (float)fmax(0.0, 1.0 - sum);
                } else {
                    const float tm = tmax == -kInf ? 0.f : tmax;
                    float sum = 0.f;
                    for (int e = tid; e < te.k; e += L)
                        if (list[e].id >= 0) sum += expf(list[e].lq - tm);
                    sum = lanes_sum<TH>(sum);
                    if (broken) Q = NAN;
                    const float ln_sum = logf(sum);
                    for (int e = tid; e < te.k; e += L) {
                        const float lq = (list[e].lq - tm) - ln_sum;
                        list[e].lq = lq;
                        list[e].q = list[e].id >= 0 ? expf(lq) : 0.f;
                    }
                }
                float m = -kInf, sum = 0.f;
                for (int e = tid, i = 0; e < te.k; e += L, ++i)
                    if ((first >> i) & 1u) m = fmaxf(m, list[e].x);
                m = lanes_max<TH>(m);
                for (int e = tid, i = 0; e < te.k; e += L, ++i)
                    if ((first >> i) & 1u) sum += ex2(exponent(list[e].x, m, c2));
                sum = lanes_sum<TH>(sum);
                if (tid == 0) {
                    ls.m = m;
                    ls.s = sum;
                    ls.Q = Q;
                    ls.tail_q = tail_q;
                }
                if (lc && tid < cluster) {
                    const uint32_t to = cluster_map(smem_u32(&listed_of.cta[parity][0][rank]), tid);
                    st_cluster_f32(to, m);
                    st_cluster_f32(to + 4 * kMaxCluster, sum);
                }
            }
            rest = join_row<TH, false>(joint[group], rest, tid, cluster, rank, parity, c2);
            float lm = ls.m, lsum = ls.s;
            if (lc) {
                const int lane = tid & 31;
                const bool in_c = lane < cluster;
                const Stats l = join_lanes<false>(in_c ? listed_of.cta[parity][0][lane] : -kInf,
                                                  in_c ? listed_of.cta[parity][1][lane] : 0.f, 0.f,
                                                  c2);
                lm = l.m;
                lsum = l.s;
            }
            parity ^= 1;
            all.m = fmaxf(rest.m, lm);
            const float mu = all.m == -kInf ? 0.f : all.m;
            all.s = rest.s * ex2((rest.m - mu) * c2) + lsum * ex2((lm - mu) * c2);
        }
        const bool none = g == 0.f || empty || all.s == 0.f;  // a gradient of zeros
        float qr = 0.f, Q = 0.f;
        if (!empty) {
            qr = rest.s == 0.f ? 0.f : ls.tail_q;
            Q = te.tail ? ls.Q + qr : ls.Q;
        }
        if (te.loss != nullptr && first_lanes) {
            const float ln_s = ln(all.s);
            float part = 0.f;
            if (!empty) {
                for (int e = tid; e < te.k; e += L)
                    if (list[e].id >= 0 && list[e].q != 0.f)
                        part += list[e].q * (list[e].lq - (all.s == 0.f ? -kInf : log_prob(list[e].x, in.c, all.m, ln_s)));
                part = lanes_sum<TH>(part);
                if (qr > 0.f)
                    part += qr * (logf(qr) - (in.c * (rest.m - all.m) + ln(rest.s) - ln_s));
            }
            if (tid == 0) te.loss[r] = Q != Q ? NAN : part;
        }
        if constexpr (kGrad) {
            if (none) {
                for (int i = tid; i < p.nv; i += TH) {
                    const float y[kPer] = {};
                    store_vector<T>(out + (size_t)i * kPer, wide, y);
                }
                if (ie >= 0) narrow(0.f, d + ie);
            } else {
                const float gc = g * in.c, inv = reciprocal(all.s);
                const Scale k(c2, rest.m);
                // a rest of -inf only has no gradient of its own: 2^t is 0 there
                const float f0 = gc * (Q * inv * (rest.s == 0.f ? 1.f : ex2((rest.m - all.m) * c2))
                                       - (qr > 0.f ? qr / rest.s : 0.f));
                const bool fast = !k.far && wide;
                const float f = fast ? f0 * ex2(-k.shift) : f0;
                auto put = [&](int i, const Pair (&t)[kPer / 2], bool whole) {
                    float y[kPer];
#pragma unroll
                    for (int e = 0; e < kPer / 2; ++e)
                        halves(mul2(ex2_pair(t[e]), pair_of(f, f)), y[2 * e], y[2 * e + 1]);
                    store_vector<T>(out + (size_t)i * kPer, whole, y);
                };
                if (fast)
                    each_vector<TH>(buf, p.nv, tid, [&](int i, const uint32_t (&w)[4]) {
                        Pair t[kPer / 2];
                        exponents<T, false, false>(w, k, t);
                        put(i, t, true);
                    });
                else
                    each_in_turn<TH>(buf, p.nv, tid, [&](int i, const uint32_t (&w)[4]) {
                        Pair t[kPer / 2];
                        exponents<T, false, true>(w, k, t);
                        put(i, t, wide);
                    });
                if (ie >= 0) narrow(ex2(exponent(edge, rest.m, c2)) * f0, d + ie);
                group_sync<TH>();  // the listed tokens' places hold the rest's gradient by now
                if (lister)
                    for (int e = tid, i = 0; e < te.k; e += L, ++i)
                        if ((first >> i) & 1u) {
                            const int id = list[e].id;
                            float w = list[e].q;
                            if (twice) {
                                w = 0.f;
                                for (int l = 0; l < te.k; ++l)
                                    if (list[l].id == id) w += list[l].q;
                            }
                            const float pi = ex2(exponent(list[e].x, all.m, c2)) * inv;
                            narrow(gc * (Q * pi - w), d + id);
                        }
            }
        }
        group_sync<TH>();  // the list and the row's place are free again
    }
}

template <typename T, bool kGrad>
cudaError_t distill_of(int threads, const RowsIn& in, const TeacherIn& te, cudaStream_t s) {
    switch (threads) {
        case 16: return launch_rows<&k_distill<T, 16, kGrad>, 16>(in, 1024, s, in, te);
        case 128: return launch_rows<&k_distill<T, 128, kGrad>, 128>(in, 1024, s, in, te);
        default: return launch_rows<&k_distill<T, 256, kGrad>, 256>(in, 1024, s, in, te);
    }
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
    const Shape sh = shape_of(S * n, V, size, 16, true);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.log_cluster,
                    slots_of(V, size, sh.log_cluster) + k};
    const TeacherIn te{ids, teacher, teacher_dtype == MIMI_RVQ_BF16, k, tail, g, loss, dlogits,
                       d_stride_s, d_stride_n, reinterpret_cast<unsigned long long*>(n_bad)};
    if (dtype == MIMI_RVQ_BF16)
        return status_of(grad ? distill_of<__nv_bfloat16, true>(sh.threads, in, te, stream)
                              : distill_of<__nv_bfloat16, false>(sh.threads, in, te, stream));
    return status_of(grad ? distill_of<float, true>(sh.threads, in, te, stream)
                          : distill_of<float, false>(sh.threads, in, te, stream));
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
