// logits_distill.cu -- distillation from a teacher's top list and its gradient.
// Declared in include/mimi_rvq_streams.h; layout and statistics in logits.cuh.
//
// The row's listed tokens are taken out of the pass: once the row is in shared
// memory its lister (a warp beside the row's threads; half a warp's row lists for
// itself) reads the listed logits there and puts -inf in their places. The pass
// then gives the statistics of the rest, from which both the whole row's (joined
// with the listed logits) and the tail class's probability follow without
// cancellation, however certain
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

// A place of the list: the lister's lane l has places l, l + lanes, ...
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

constexpr int kShortTop = 32;  // longest list of half a warp's row

// Threads beside a CTA's row: its lister.
template <int TH>
__host__ __device__ constexpr int lister_of() { return TH > 32 ? 32 : 0; }
template <int TH>
__host__ __device__ constexpr int distill_blocks() { return 1024 / (block_of<TH>() + lister_of<TH>()); }

template <typename T, int TH, bool kGrad>
__global__ void __launch_bounds__(block_of<TH>() + lister_of<TH>(), distill_blocks<TH>())
    k_distill(RowsIn in, TeacherIn te) {
    constexpr int kRows = block_of<TH>() / TH, kPer = Part<T>::kPer;
    constexpr int L = lanes_of<TH>(), kLane = (TH <= 32 ? kShortTop : kMaxTop) / L;
    using B = Bits<T>;
    extern __shared__ uint4 buffers[];  // [groups][slots]: the row's vectors, then the list
    __shared__ Joint<TH> joint[kRows];
    __shared__ ListShared<T> lists[kRows];
    __shared__ ListJoint listed_of;
    const int tid = TH > 32 ? threadIdx.x : thread_in_group<TH>();
    const int group = TH > 32 ? 0 : group_in_block<TH>();
    const int lc = TH <= 32 ? 0 : in.log_cluster, cluster = 1 << lc;
    const int rank = lc ? (int)cluster_ctarank() : 0;
    const bool worker = tid < TH, first_lanes = rank == 0 && tid < L;  // the latter have the edges
    const bool lister = TH <= 32 || !worker;
    const int me = TH <= 32 ? tid : tid - TH;  // the lister's lane
    const unsigned mask = lane_mask<TH>();
    uint4* buf = buffers + (size_t)group * in.slots;
    Entry* list = reinterpret_cast<Entry*>(buf + in.slots - te.k);
    const float c2 = in.c * kLog2e;
    ListShared<T>& ls = lists[group];
    if (lc) cluster_sync();  // every CTA runs before one writes to another
    RowWalk row((int64_t)(blockIdx.x >> lc) * kRows + group,
                (int64_t)(gridDim.x >> lc) * kRows, in.n);
    if (row.r >= in.rows) return;
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
                const int e = me + L * i;
                id_next[i] = -1;
                if (e < te.k) {
                    id_next[i] = __ldg(te.ids + at + e);
                    t_next[i] = te.t_bf16 ? widen(__ldg(static_cast<const __nv_bfloat16*>(te.t) + at + e))
                                          : __ldg(static_cast<const float*>(te.t) + at + e);
                }
            }
        }
    };
    // a row's part of what is read for it: its share of the vectors, and an element beside them
    struct At {
        Part<T> p;
        int64_t r, s;
        int j, ie;
        float g, edge;
        bool skip;  // a gradient of weight 0 alone: zeros, whatever the row is
    };
    auto at_row = [&]() {
        At at{Part<T>(static_cast<const T*>(in.x) + row.s * in.ss + row.j * in.sn, in.V, rank, lc),
              row.r, row.s, row.j, -1, kGrad ? g_next : 1.f, -kInf, false};
        at.skip = kGrad && at.g == 0.f && te.loss == nullptr;
        at.ie = first_lanes ? at.p.edge(tid) : -1;
        if (!at.skip && at.ie >= 0) at.edge = widen(at.p.x[at.ie]);
        return at;
    };
    list_at();
    At now = at_row();
    if (!now.skip && worker) fetch<TH>(buf, now.p, tid);
    for (int parity = 0;;) {
        const Part<T> p = now.p;
        const int64_t r = now.r;
        const int ie = now.ie;
        const float g = now.g;
        float edge = now.edge;
        const bool skip = now.skip;
        T* d = static_cast<T*>(te.d) + now.s * te.d_ss + now.j * te.d_sn;
        const bool wide = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0;
        T* out = d + p.first;
        int n = 0, bad = 0;
        float tmax = -kInf;
        bool broken = false;  // NaN or +inf among the entries
        unsigned first = 0;   // bit i: entry me + L i is this share's, the first of its id
        bool twice = false;   // some id is listed twice
        if (lister) {
            __syncwarp(mask);  // the last row's list has been read
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                if (i * L >= te.k) break;
                const int e = me + L * i;
                int id = -1 - e;  // empty places differ
                if (e < te.k) {
                    const int given = id_next[i];
                    bad += given >= in.V;
                    if (given >= 0 && given < in.V) id = given;
                    const float t = id >= 0 ? t_next[i] : -kInf;
                    n += id >= 0;
                    tmax = fmaxf(tmax, t);
                    broken |= !(t < kInf);
                    list[e].id = id < 0 ? -1 : id;
                    list[e].lq = t;
                }
                const unsigned same = __match_any_sync(mask, id);
                bool again = id >= 0 && (same & ((1u << (threadIdx.x & 31)) - 1u));
                __syncwarp(mask);
                for (int l = 0; l < i * L; ++l) again |= id >= 0 && list[l].id == id;
                twice |= again;
                if (id >= 0 && !again && (p.place(id) >= 0 || (rank == 0 && p.in_edges(id))))
                    first |= 1u << i;
            }
            twice = __any_sync(mask, twice);
            if (bad && rank == 0 && te.n_bad != nullptr)
                atomicAdd(te.n_bad, (unsigned long long)bad);
            tmax = lanes_max<TH>(tmax);
            broken = __any_sync(mask, broken);
            n = __any_sync(mask, n > 0);
        }
        row.next(in.n);
        const bool more = row.r < in.rows;
        list_at();
        bool empty = true;
        if (!skip) {
            arrived();
            if (first_lanes && tid < 16 && ie >= 0) narrow(edge, &ls.edge[tid]);
            group_sync<TH>();  // the row is here
            if (lister) {
                // the listed elements of this share: read, then hidden
                auto each = [&](auto&& f) {
                    for (int e = me, i = 0; e < te.k; e += L, ++i) {
                        const int id = list[e].id, q = p.place(id);
                        if (id < 0 || (q < 0 && (rank != 0 || !p.in_edges(id)))) continue;
                        f(e, q >= 0 ? reinterpret_cast<B*>(buf) + q
                                    : reinterpret_cast<B*>(ls.edge) + p.edge_lane(id));
                    }
                };
                auto read = [&](int e, B* at) { list[e].x = widen(*reinterpret_cast<const T*>(at)); };
                auto hide = [&](int, B* at) { *at = (B)Elem<T>::kFill; };
                if (!twice) {
                    each([&](int e, B* at) {
                        read(e, at);
                        hide(e, at);
                    });
                } else {
                    each(read);
                    __syncwarp(mask);
                    each(hide);
                }
                if (lc && rank == 0)  // other CTAs' elements; for the loss
                    for (int e = me; e < te.k; e += L) {
                        const int id = list[e].id;
                        if (id >= 0 && p.place(id) < 0 && !p.in_edges(id)) list[e].x = widen(p.x[id]);
                    }
                if (me == 0) ls.empty = !n || (!te.tail && tmax == -kInf && !broken);
            }
            group_sync<TH>();  // the listed tokens are hidden
            if (ie >= 0) edge = widen(ls.edge[tid]);
            empty = ls.empty != 0;
        }
        if (more) now = at_row();
        const Next<T> next{buf, now.p.x + now.p.first, more && !now.skip ? now.p.nv : 0};
        Stats rest{-kInf, 0.f, 0.f}, all{-kInf, 0.f, 0.f};
        if (!empty) {
            if (worker) {
                float top;
                rest = pass<TH, false, T>(buf, p.nv, tid, edge, c2, top, [&](int i) {
                    if (!kGrad) next.refill(i);
                });
            }
            if (lister) {  // the weights and this share's listed logits
                float Q = 1.f, tail_q = 0.f;
                if (te.tail) {
                    // the tail's weight is what the list leaves of 1: in float64, or a tail of
                    // 1e-6 would be rounding
                    double sum = 0.0;
                    for (int e = me; e < te.k; e += L) {
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
                    for (int e = me; e < te.k; e += L)
                        if (list[e].id >= 0) sum += expf(list[e].lq - tm);
                    sum = lanes_sum<TH>(sum);
                    if (broken) Q = NAN;
                    const float ln_sum = logf(sum);
                    for (int e = me; e < te.k; e += L) {
                        const float lq = (list[e].lq - tm) - ln_sum;
                        list[e].lq = lq;
                        list[e].q = list[e].id >= 0 ? expf(lq) : 0.f;
                    }
                }
                float m = -kInf, sum = 0.f;
                for (int e = me, i = 0; e < te.k; e += L, ++i)
                    if ((first >> i) & 1u) m = fmaxf(m, list[e].x);
                m = lanes_max<TH>(m);
                for (int e = me, i = 0; e < te.k; e += L, ++i)
                    if ((first >> i) & 1u) sum += ex2(exponent(list[e].x, m, c2));
                sum = lanes_sum<TH>(sum);
                if (me == 0) {
                    ls.m = m;
                    ls.s = sum;
                    ls.Q = Q;
                    ls.tail_q = tail_q;
                }
                if (lc && me < cluster) {
                    const uint32_t to = cluster_map(smem_u32(&listed_of.cta[parity][0][rank]), me);
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
        if (kGrad && worker) {
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
            }
        }
        if (more && worker) next.template rest<TH>(kGrad || empty ? 0 : p.nv, tid);
        if (te.loss != nullptr && lister && rank == 0) {
            const float ln_s = ln(all.s);
            float part = 0.f;
            if (!empty) {
                for (int e = me; e < te.k; e += L)
                    if (list[e].id >= 0 && list[e].q != 0.f)
                        part += list[e].q * (list[e].lq - (all.s == 0.f ? -kInf : log_prob(list[e].x, in.c, all.m, ln_s)));
                part = lanes_sum<TH>(part);
                if (qr > 0.f)
                    part += qr * (logf(qr) - (in.c * (rest.m - all.m) + ln(rest.s) - ln_s));
            }
            if (me == 0) te.loss[r] = Q != Q ? NAN : part;
        }
        if (kGrad && !none) {
            group_sync<TH>();  // the listed tokens' places hold the rest's gradient by now
            if (lister) {
                const float gc = g * in.c, inv = reciprocal(all.s);
                for (int e = me, i = 0; e < te.k; e += L, ++i)
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
        if (!more) break;
    }
}

template <typename T, bool kGrad>
cudaError_t distill_of(int threads, const RowsIn& in, const TeacherIn& te, cudaStream_t s) {
    switch (threads) {
        case 16: return launch_rows<&k_distill<T, 16, kGrad>, 16, lister_of<16>()>(in, 1024, s, in, te);
        case 128: return launch_rows<&k_distill<T, 128, kGrad>, 128, lister_of<128>()>(in, 1024, s, in, te);
        default: return launch_rows<&k_distill<T, 256, kGrad>, 256, lister_of<256>()>(in, 1024, s, in, te);
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
    const Shape sh = shape_of(S * n, V, size, k <= kShortTop ? 16 : 0, true);
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
