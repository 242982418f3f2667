// logits_distill.cu -- distillation from a teacher's top list and its gradient.
// Declared in include/mimi_rvq_streams.h; layout and statistics in logits.cuh.
//
// The row's listed tokens are taken out of the pass: once the row is in shared
// memory its lister (a warp beside the row's threads; half a warp's row lists for
// itself) reads the listed logits there and puts -inf in their places. The pass
// then gives the statistics of the rest, from which both the whole row's (joined
// with the listed logits) and the tail class's probability follow without
// cancellation, however certain the student is of the list. With (m_r, s_r) the
// rest's and ln s the row's:
//     ln p_i = c (x_i - m) - ln s,   ln p_rest = c (m_r - m) + ln s_r - ln s,
//     d x_i = g c (Q p_i - q_r e^{c (x_i - m_r)} / s_r)       unlisted
//           = e^{c (x_i - m_r)} (g c) (Q e^{c (m_r - m)} / s - q_r / s_r),
//     d x_i = g c (Q p_i - sum of the entries' q)             listed,
// so unlisted gradients need one exponential; the listed ones are written over
// them by the lister.
//
// Bound by reading the row, and for the gradient writing it. The lister has a loop
// of its own, so that the row's threads hold no registers for its list and weigh
// nothing while they could be adding: gradient of 3750 x 32000 bf16 rows with 64
// entries 97 to 102 us (in the first warp's share of the row's loop 120), of
// 16384 x 8 x 2048 bf16 rows with 16 entries 207 us at full clocks and 233 when the
// card has run warm (with one loop for both 264).
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

// A place of the list; the lister's lane l has places l, l + lanes, ... in registers, and what it
// looks up of others here.
struct Entry {
    int id;   // -1 - place: an empty place
    float q;  // weight (tail: first its logarithm)
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

// Longest list of half a warp's row: two places a lane. Longer ones take a CTA a row (16384 x 8 x
// 2048 bf16, losses and gradient: 148 and 217 us with 32 entries, 518 and 672 with 33).
constexpr int kShortTop = 32;

// Threads beside a CTA's row: its lister.
template <int TH>
__host__ __device__ constexpr int lister_of() { return TH > 32 ? 32 : 0; }
template <int TH>
__host__ __device__ constexpr int distill_blocks() { return 1024 / (block_of<TH>() + lister_of<TH>()); }

// A row's statistics when the rest's and the listed logits' are joined.
struct Whole {
    Stats rest, all;
    float Q, qr;  // sum of the weights, the tail's weight
    bool empty;
    __device__ __forceinline__ bool none(float g) const { return g == 0.f || empty || all.s == 0.f; }
};

// The list of a row, kept in registers by the lanes of its lister: lane l has places l, l + L, ...
template <typename T, int TH>
struct Lister {
    static constexpr int L = lanes_of<TH>(), kLane = (TH <= 32 ? kShortTop : kMaxTop) / L;
    using B = Bits<T>;
    int id[kLane];  // below 0: an empty place
    float q[kLane], lq[kLane], x[kLane];  // weight, its logarithm, the student's logit
    // bit i of `mine`: place me + L i is in this share, of `first`: and the first of its id
    unsigned mine, first;
    float tmax;
    bool broken, twice, some;  // NaN or +inf in an entry, an id listed twice, any entry
    int next_id[kLane];  // the next row's
    float next_t[kLane];

    template <typename F>
    __device__ __forceinline__ static void each(int k, F&& f) {
#pragma unroll
        for (int i = 0; i < kLane; ++i) {
            if (i * L >= k) break;
            f(i);
        }
    }
    // sends for a row's list
    __device__ __forceinline__ void load(const TeacherIn& te, int64_t r, int me) {
        const int64_t at = r * te.k;
        each(te.k, [&](int i) {
            const int e = me + L * i;
            next_id[i] = -1;
            next_t[i] = -kInf;
            if (e < te.k) {
                next_id[i] = __ldg(te.ids + at + e);
                next_t[i] = te.t_bf16 ? widen(__ldg(static_cast<const __nv_bfloat16*>(te.t) + at + e))
                                      : __ldg(static_cast<const float*>(te.t) + at + e);
            }
        });
    }
    // takes the list that was sent for; what can be known of it without the row
    __device__ __forceinline__ void take(const TeacherIn& te, const Part<T>& p, int rank, int me,
                                         Entry* list) {
        const unsigned mask = lane_mask<TH>();
        int n = 0, bad = 0;
        mine = 0;
        tmax = -kInf;
        broken = false;
        __syncwarp(mask);  // the last row's list has been read
        each(te.k, [&](int i) {
            const int e = me + L * i, given = next_id[i];
            bad += given >= p.V;
            id[i] = given >= 0 && given < p.V ? given : -1 - e;
            const bool there = id[i] >= 0;
            lq[i] = there ? next_t[i] : -kInf;
            q[i] = 0.f;
            x[i] = -kInf;
            n += there;
            tmax = fmaxf(tmax, lq[i]);
            broken |= !(lq[i] < kInf);
            if (e < te.k) list[e] = Entry{id[i], lq[i]};
            if (there && (p.place(id[i]) >= 0 || (rank == 0 && p.in_edges(id[i])))) mine |= 1u << i;
        });
        if (bad && rank == 0 && te.n_bad != nullptr)
            atomicAdd(te.n_bad, (unsigned long long)bad);
        tmax = lanes_max<TH>(tmax);
        broken = __any_sync(mask, broken);
        some = __any_sync(mask, n > 0);
    }
    __device__ __forceinline__ bool empty(const TeacherIn& te) const {
        return !some || (!te.tail && tmax == -kInf && !broken);
    }
    // Reads the listed elements of this share and hides them. In between the places' numbers stand
    // there, which shows an id that is listed twice (a warp's match instruction on the ids before
    // the row is here takes 600 cycles for each 32: 100 rows of 131072 with 128 entries 34 us, so 30).
    __device__ __forceinline__ void hide(const TeacherIn& te, const Part<T>& p, uint4* buf, T* edge,
                                         bool others, int me, const Entry* list) {
        const unsigned mask = lane_mask<TH>();
        auto each_mine = [&](auto&& f) {
            each(te.k, [&](int i) {
                if (!((mine >> i) & 1u)) return;
                const int at = p.place(id[i]);
                f(i, at >= 0 ? reinterpret_cast<B*>(buf) + at
                             : reinterpret_cast<B*>(edge) + p.edge_lane(id[i]));
            });
        };
        each_mine([&](int i, B* at) { x[i] = widen(*reinterpret_cast<const T*>(at)); });
        __syncwarp(mask);
        each_mine([&](int i, B* at) { *at = (B)(me + L * i); });
        __syncwarp(mask);
        bool lost = false;
        each_mine([&](int i, B* at) { lost |= *at != (B)(me + L * i); });
        twice = __any_sync(mask, lost);
        each_mine([&](int, B* at) { *at = (B)Elem<T>::kFill; });
        first = mine;
        if (twice)  // the first of equal ids stands for all (places in the share are below k)
            each(te.k, [&](int i) {
                if (!((mine >> i) & 1u)) return;
                for (int l = 0; l < me + L * i; ++l)
                    if (list[l].id == id[i]) first &= ~(1u << i);
            });
        if (others)  // other CTAs' elements, for the loss
            each(te.k, [&](int i) {
                if (!((mine >> i) & 1u) && id[i] >= 0) x[i] = widen(p.x[id[i]]);
            });
    }
    // the weights, and this share's listed logits, for the group
    __device__ __forceinline__ void weigh(const TeacherIn& te, int me, Entry* list,
                                          ListShared<T>& ls, float c2) {
        float Q = 1.f, tail_q = 0.f;
        if (te.tail) {
            // the tail's weight is what the list leaves of 1: in float64, or a tail of 1e-6 would
            // be rounding
            double sum = 0.0;
#pragma unroll 1
            for (int e = me; e < te.k; e += L)
                if (list[e].id >= 0) sum += exp((double)list[e].q);
            sum = lanes_sum<TH>(sum);
            Q = broken ? NAN : (float)sum;
            tail_q = (float)fmax(0.0, 1.0 - sum);
        } else {
            const float tm = tmax == -kInf ? 0.f : tmax;
            float sum = 0.f;
            each(te.k, [&](int i) {
                lq[i] -= tm;
                if (id[i] >= 0) sum += expf(lq[i]);
            });
            sum = lanes_sum<TH>(sum);
            if (broken) Q = NAN;
            const float ln_sum = logf(sum);
            each(te.k, [&](int i) { lq[i] -= ln_sum; });
        }
        float m = -kInf, sum = 0.f;
        each(te.k, [&](int i) {
            if (id[i] >= 0) q[i] = expf(lq[i]);
            if ((first >> i) & 1u) m = fmaxf(m, x[i]);
        });
        m = lanes_max<TH>(m);
        each(te.k, [&](int i) {
            if ((first >> i) & 1u) sum += ex2(exponent(x[i], m, c2));
        });
        sum = lanes_sum<TH>(sum);
        if (twice) {
            each(te.k, [&](int i) {
                if (me + L * i < te.k) list[me + L * i].q = q[i];
            });
            __syncwarp(lane_mask<TH>());
        }
        if (me == 0) {
            ls.m = m;
            ls.s = sum;
            ls.Q = Q;
            ls.tail_q = tail_q;
        }
    }
    __device__ __forceinline__ void put_loss(const TeacherIn& te, int64_t r, int me, const Whole& w,
                                             float c) const {
        const float ln_s = logf(w.all.s);
        float part = 0.f;
        if (!w.empty) {
            each(te.k, [&](int i) {
                if (id[i] >= 0 && q[i] != 0.f)
                    part += q[i] * (lq[i] - (w.all.s == 0.f ? -kInf : log_prob(x[i], c, w.all.m, ln_s)));
            });
            part = lanes_sum<TH>(part);
            if (w.qr > 0.f)
                part += w.qr * (logf(w.qr) - log_prob(w.rest.m, c, w.all.m, ln_s - logf(w.rest.s)));
        }
        if (me == 0) te.loss[r] = w.Q != w.Q ? NAN : part;
    }
    // the listed tokens' gradients, over the rest's
    __device__ __forceinline__ void put_listed(const TeacherIn& te, const Whole& w, float gc,
                                               float c2, const Entry* list, T* d) const {
        const float inv = reciprocal(w.all.s);
        each(te.k, [&](int i) {
            if (!((first >> i) & 1u)) return;
            float weight = q[i];
            if (twice) {
                weight = 0.f;
                for (int l = 0; l < te.k; ++l)
                    if (list[l].id == id[i]) weight += list[l].q;
            }
            const float pi = ex2(exponent(x[i], w.all.m, c2)) * inv;
            narrow(gc * (w.Q * pi - weight), d + id[i]);
        });
    }
};

// The unlisted tokens' gradients of a share.
template <int TH, typename T>
__device__ __forceinline__ void put_rest(const Part<T>& p, const uint4* buf, int tid, int ie,
                                         float edge, const Whole& w, bool none, float gc, float c2,
                                         T* d) {
    constexpr int kPer = Part<T>::kPer;
    const bool wide = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0;
    T* out = d + p.first;
    if (none) {
        for (int i = tid; i < p.nv; i += TH) {
            const float y[kPer] = {};
            store_vector<T>(out + (size_t)i * kPer, wide, y);
        }
        if (ie >= 0) narrow(0.f, d + ie);
        return;
    }
    const Scale k(c2, w.rest.m);
    // a rest of -inf only has no gradient of its own: 2^t is 0 there
    const float f0 = gc * (w.Q * reciprocal(w.all.s)
                               * (w.rest.s == 0.f ? 1.f : ex2((w.rest.m - w.all.m) * c2))
                           - (w.qr > 0.f ? w.qr / w.rest.s : 0.f));
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
        each_vector<TH>(buf, p.nv, tid, [&](int i, const uint32_t (&v)[4]) {
            Pair t[kPer / 2];
            exponents<T, false, false>(v, k, t);
            put(i, t, true);
        });
    else
        each_in_turn<TH>(buf, p.nv, tid, [&](int i, const uint32_t (&v)[4]) {
            Pair t[kPer / 2];
            exponents<T, false, true>(v, k, t);
            put(i, t, wide);
        });
    if (ie >= 0) narrow(ex2(exponent(edge, w.rest.m, c2)) * f0, d + ie);
}

// kGrad: the gradient, with the losses where they are wanted; else the losses.
template <typename T, int TH, bool kGrad>
__global__ void __launch_bounds__(block_of<TH>() + lister_of<TH>(), distill_blocks<TH>())
    k_distill(RowsIn in, TeacherIn te) {
    constexpr int kRows = block_of<TH>() / TH, N = TH + lister_of<TH>();
    extern __shared__ uint4 buffers[];  // [groups][slots]: the row's vectors, then the list
    __shared__ Joint<TH> joint[kRows];
    __shared__ ListShared<T> lists[kRows];
    __shared__ ListJoint listed_of;
    const int tid = TH > 32 ? threadIdx.x : thread_in_group<TH>();
    const int group = TH > 32 ? 0 : group_in_block<TH>();
    const int lc = TH <= 32 ? 0 : in.log_cluster, cluster = 1 << lc;
    const int rank = lc ? (int)cluster_ctarank() : 0;
    const bool first_lanes = rank == 0 && tid < lanes_of<TH>();  // have the row's edges
    uint4* buf = buffers + (size_t)group * in.slots;
    Entry* list = reinterpret_cast<Entry*>(buf + in.slots - (te.k + 1) / 2);
    const float c2 = in.c * kLog2e;
    ListShared<T>& ls = lists[group];
    Joint<TH>& jt = joint[group];
    if (lc) cluster_sync();  // every CTA runs before one writes to another
    RowWalk row((int64_t)(blockIdx.x >> lc) * kRows + group,
                (int64_t)(gridDim.x >> lc) * kRows, in.n);
    if (row.r >= in.rows) return;
    auto part_at = [&]() {
        return Part<T>(static_cast<const T*>(in.x) + row.s * in.ss + row.j * in.sn, in.V, rank, lc);
    };
    auto weight_at = [&]() {
        return kGrad && te.g != nullptr && row.r < in.rows ? __ldg(te.g + row.r) : 1.f;
    };
    // a gradient of weight 0 alone: zeros, whatever the row is
    auto skipped = [&](float g) { return kGrad && g == 0.f && te.loss == nullptr; };
    auto gradient_at = [&](const RowWalk& w) {
        return static_cast<T*>(te.d) + w.s * te.d_ss + w.j * te.d_sn;
    };
    int parity = 0;
    // the row's joined statistics, behind the barrier that the lister and the row's threads share
    auto join = [&](Stats rest) {
        Whole w;
        w.empty = false;
        w.rest = join_row<TH, false, N>(jt, rest, tid, cluster, rank, parity, c2);
        float lm = ls.m, lsum = ls.s;
        if (lc) {
            const int lane = tid & 31;
            const bool in_c = lane < cluster;
            const Stats l = join_lanes<false>(in_c ? listed_of.cta[parity][0][lane] : -kInf,
                                              in_c ? listed_of.cta[parity][1][lane] : 0.f, 0.f, c2);
            lm = l.m;
            lsum = l.s;
        }
        parity ^= 1;
        w.all = Stats{fmaxf(w.rest.m, lm), 0.f, 0.f};
        const float mu = w.all.m == -kInf ? 0.f : w.all.m;
        w.all.s = w.rest.s * ex2((w.rest.m - mu) * c2) + lsum * ex2((lm - mu) * c2);
        w.qr = w.rest.s == 0.f ? 0.f : ls.tail_q;
        w.Q = te.tail ? ls.Q + w.qr : ls.Q;
        return w;
    };
    const Whole nothing{{-kInf, 0.f, 0.f}, {-kInf, 0.f, 0.f}, 0.f, 0.f, true};
    const Stats no_rest{-kInf, 0.f, 0.f};

    if (TH > 32 && tid >= TH) {  // ---- the lister
        const int me = tid - TH;
        Lister<T, TH> lister;
        lister.load(te, row.r, me);
        float g_next = weight_at();
        while (true) {
            const Part<T> p = part_at();
            const int64_t r = row.r;
            T* d = gradient_at(row);
            const float g = g_next;
            lister.take(te, p, rank, me, list);
            row.next(in.n);
            const bool more = row.r < in.rows;
            if (more) lister.load(te, row.r, me);
            g_next = weight_at();
            Whole w = nothing;
            if (!skipped(g)) {
                group_sync<N>();  // the row is here
                lister.hide(te, p, buf, ls.edge, lc != 0 && rank == 0, me, list);
                const bool empty = lister.empty(te);
                if (me == 0) ls.empty = empty;
                group_sync<N>();  // the listed tokens are hidden
                if (!empty) {
                    lister.weigh(te, me, list, ls, c2);
                    __syncwarp();
                    if (lc && me < cluster) {
                        const uint32_t to = cluster_map(smem_u32(&listed_of.cta[parity][0][rank]), me);
                        st_cluster_f32(to, ls.m);
                        st_cluster_f32(to + 4 * kMaxCluster, ls.s);
                    }
                    w = join(no_rest);
                }
                if (te.loss != nullptr && rank == 0) lister.put_loss(te, r, me, w, in.c);
            }
            if (kGrad && !w.none(g)) {
                group_sync<N>();  // the listed tokens' places hold the rest's gradient by now
                lister.put_listed(te, w, g * in.c, c2, list, d);
            }
            if (!more) break;
        }
        return;
    }

    // ---- the row's threads; half a warp's row lists for itself
    Lister<T, 16> own;
    float g_next = weight_at();
    if constexpr (TH <= 32) own.load(te, row.r, tid);
    Part<T> p = part_at();
    float edge = -kInf;
    int ie = -1;
    auto send = [&]() {  // for the row's vectors, and the element beside them
        ie = first_lanes ? p.edge(tid) : -1;
        edge = -kInf;
        if (skipped(g_next)) return;
        fetch<TH>(buf, p, tid);
        if (ie >= 0) edge = widen(p.x[ie]);
    };
    send();
    while (true) {
        const int64_t r = row.r;
        T* d = gradient_at(row);
        const float g = g_next;
        if constexpr (TH <= 32) own.take(te, p, 0, tid, list);
        row.next(in.n);
        const bool more = row.r < in.rows;
        if constexpr (TH <= 32)
            if (more) own.load(te, row.r, tid);
        g_next = weight_at();
        Whole w = nothing;
        const int here = ie;
        float beside = edge;
        Next<T> next{buf, nullptr, 0};
        Part<T> coming = p;
        if (!kGrad && more) {  // losses read the row once: places are refilled as they are read
            coming = part_at();
            next = Next<T>{buf, coming.x + coming.first, coming.nv};
        }
        int refilled = 0;
        if (!skipped(g)) {
            arrived();
            if (here >= 0) narrow(beside, &ls.edge[tid]);
            group_sync<N>();  // the row is here
            bool empty;
            if constexpr (TH <= 32) {
                own.hide(te, p, buf, ls.edge, false, tid, list);
                empty = own.empty(te);
                group_sync<N>();
            } else {
                group_sync<N>();  // the listed tokens are hidden
                empty = ls.empty != 0;
            }
            if (here >= 0) beside = widen(ls.edge[tid]);
            if (!empty) {
                float top;
                const Stats rest = pass<TH, false, T>(buf, p.nv, tid, beside, c2, top, [&](int i) {
                    if (!kGrad) next.refill(i);
                });
                refilled = p.nv;
                if constexpr (TH <= 32) own.weigh(te, tid, list, ls, c2);
                w = join(rest);
            }
            if constexpr (TH <= 32)
                if (te.loss != nullptr) own.put_loss(te, r, tid, w, in.c);
        }
        if constexpr (kGrad) {
            const bool none = w.none(g);
            put_rest<TH>(p, buf, tid, here, beside, w, none, g * in.c, c2, d);
            if (more) {
                p = part_at();
                send();
            }
            if (!none) {
                group_sync<N>();  // the listed tokens' places hold the rest's gradient by now
                if constexpr (TH <= 32) own.put_listed(te, w, g * in.c, c2, list, d);
            }
        } else if (more) {
            next.template rest<TH>(refilled, tid);
            p = coming;
            ie = first_lanes ? p.edge(tid) : -1;
            edge = ie >= 0 ? widen(p.x[ie]) : -kInf;
        }
        if (!more) break;
    }
}

template <typename T, int TH, bool kGrad>
cudaError_t launch_distill(const RowsIn& in, const TeacherIn& te, cudaStream_t s) {
    return launch_rows<&k_distill<T, TH, kGrad>, TH, lister_of<TH>(), distill_blocks<TH>()>(
        in, 1024, s, in, te);
}

template <typename T, bool kGrad>
cudaError_t distill_of(int threads, const RowsIn& in, const TeacherIn& te, cudaStream_t s) {
    switch (threads) {
        case 16: return launch_distill<T, 16, kGrad>(in, te, s);
        case 128: return launch_distill<T, 128, kGrad>(in, te, s);
        default: return launch_distill<T, 256, kGrad>(in, te, s);
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
                    slots_of(V, size, sh.log_cluster) + (k + 1) / 2};
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
