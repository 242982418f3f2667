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

constexpr int kLane = kMaxTop / 32;  // list entries of a lane

// The list, kept by the group's first warp, and what it leaves for the group. Entries of lane l:
// l, l + 32, ...
struct ListShared {
    int id[kMaxTop];  // -1: an empty place
    float q[kMaxTop], lq[kMaxTop], x[kMaxTop];  // weight, its logarithm, the student's logit
    float edge[16];   // the elements beside the row's vectors
    float m, s;       // this share's listed logits
    float Q, tail_q;  // sum of the weights (renormalised: 1), 1 - it where the tail is a class
    int empty;        // no entry, or none with weight
};

// The listed logits of a row's shares, exchanged like the shares' own statistics.
struct ListJoint {
    float cta[2][2][kMaxCluster];
};

// An element's bits, in the buffer or (as float32) beside it.
template <typename T>
struct Cell {
    using Bits = typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type;
    Bits* in;
    float* beside;
    __device__ __forceinline__ Cell(uint4* buf, float* edge, const Part<T>& p, int id)
        : in(reinterpret_cast<Bits*>(buf) + p.place(id)),
          beside(p.in_edges(id) ? edge + p.edge_lane(id) : nullptr) {}
    __device__ __forceinline__ float value() const {
        if (beside) return *beside;
        if constexpr (sizeof(T) == 4) return __uint_as_float(*in);
        else return __uint_as_float((uint32_t)*in << 16);
    }
    __device__ __forceinline__ void mark(int e) const {
        if (beside) *beside = (float)e;
        else *in = (Bits)e;
    }
    __device__ __forceinline__ bool marked(int e) const {
        return beside ? *beside == (float)e : *in == (Bits)e;
    }
    __device__ __forceinline__ void hide() const {
        if (beside) *beside = -kInf;
        else *in = (Bits)Elem<T>::kFill;
    }
};

template <typename T, int TH, bool kGrad>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<TH>()) k_distill(RowsIn in, TeacherIn te) {
    constexpr int kRows = block_of<TH>() / TH, kPer = Part<T>::kPer;
    extern __shared__ uint4 buffers[];  // [groups][slots]
    __shared__ Joint<TH> joint[kRows];
    __shared__ ListShared lists[kRows];
    __shared__ ListJoint listed_of;
    const int tid = TH == 32 ? threadIdx.x & 31 : threadIdx.x;
    const int group = TH == 32 ? threadIdx.x / 32 : 0;
    const int lc = TH == 32 ? 0 : in.log_cluster, cluster = 1 << lc;
    const int rank = lc ? (int)cluster_ctarank() : 0;
    const bool first_warp = rank == 0 && tid < 32;  // has the row's edges
    uint4* buf = buffers + (size_t)group * in.slots;
    const float c2 = in.c * kLog2e;
    ListShared& ls = lists[group];
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
        if (tid < 32) {
            const int64_t at = row.r * te.k;
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                const int e = tid + 32 * i;
                id_next[i] = -1;
                t_next[i] = -kInf;
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
        const int ie = first_warp ? p.edge(tid) : -1;
        float edge = -kInf;
        if (!skip) {
            fetch<TH>(buf, p, tid);
            if (ie >= 0) edge = widen(p.x[ie]);
        }
        int n = 0, bad = 0;
        float tmax = -kInf;
        bool broken = false;  // NaN or +inf among the entries
        if (tid < 32) {
#pragma unroll
            for (int i = 0; i < kLane; ++i) {
                const int e = tid + 32 * i;
                int id = id_next[i];
                if (id >= in.V) {
                    ++bad;
                    id = -1;
                }
                const float t = id >= 0 ? t_next[i] : -kInf;
                n += id >= 0;
                tmax = fmaxf(tmax, t);
                broken |= !(t < kInf);
                if (e < te.k) {
                    ls.id[e] = id < 0 ? -1 : id;
                    ls.lq[e] = t;
                }
            }
            if (bad && rank == 0 && te.n_bad != nullptr)
                atomicAdd(te.n_bad, (unsigned long long)bad);
        }
        row.next(in.n);
        list_at();
        bool empty = true;
        unsigned first = 0;  // bit i: entry tid + 32 i is this share's, the first of its id
        bool twice = false;  // some id is listed twice
        if (!skip) {
            arrived();
            if (tid < 16) ls.edge[tid] = edge;
            group_sync<TH>();  // the row is here
            if (tid < 32) {
                n = (int)__reduce_add_sync(kFull, (unsigned)n);
                tmax = warp_max(tmax);
                broken = __any_sync(kFull, broken);
                for (int e = tid, i = 0; e < te.k; e += 32, ++i) {
                    const int id = ls.id[e];
                    if (id < 0) continue;
                    if (p.place(id) >= 0 || (rank == 0 && p.in_edges(id))) {
                        first |= 1u << i;
                        ls.x[e] = Cell<T>(buf, ls.edge, p, id).value();
                    } else if (rank == 0) {
                        ls.x[e] = widen(p.x[id]);  // another CTA's; for the loss
                    }
                }
                __syncwarp();
                auto each_first = [&](auto&& f) {
                    for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                        if ((first >> i) & 1u) f(e, i);
                    __syncwarp();
                };
                each_first([&](int e, int) { Cell<T>(buf, ls.edge, p, ls.id[e]).mark(e); });
                each_first([&](int e, int) { twice |= !Cell<T>(buf, ls.edge, p, ls.id[e]).marked(e); });
                each_first([&](int e, int) { Cell<T>(buf, ls.edge, p, ls.id[e]).hide(); });
                twice = __any_sync(kFull, twice);
                if (twice)  // the first of equal ids stands for all
                    each_first([&](int e, int i) {
                        for (int l = 0; l < e; ++l)
                            if (ls.id[l] == ls.id[e]) first &= ~(1u << i);
                    });
                if (tid == 0) ls.empty = n == 0 || (!te.tail && tmax == -kInf && !broken);
                if (tid < 16) edge = ls.edge[tid];
            }
            group_sync<TH>();  // the listed tokens are hidden
            empty = ls.empty != 0;
        }
        Stats rest{-kInf, 0.f, 0.f}, all{-kInf, 0.f, 0.f};
        if (!empty) {
            float top;
            rest = pass<TH, false, T>(buf, p.nv, tid, edge, c2, top);
            if (tid < 32) {  // the weights and this share's listed logits
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
                    Q = broken ? NAN : (float)sum;
                    tail_q = (float)fmax(0.0, 1.0 - sum);
                } else {
                    const float tm = tmax == -kInf ? 0.f : tmax;
                    float sum = 0.f;
                    for (int e = tid; e < te.k; e += 32)
                        if (ls.id[e] >= 0) sum += expf(ls.lq[e] - tm);
                    sum = warp_sum(sum);
                    if (broken) Q = NAN;
                    const float ln_sum = logf(sum);
                    for (int e = tid; e < te.k; e += 32) {
                        const float lq = (ls.lq[e] - tm) - ln_sum;
                        ls.lq[e] = lq;
                        ls.q[e] = ls.id[e] >= 0 ? expf(lq) : 0.f;
                    }
                }
                float m = -kInf, sum = 0.f;
                for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                    if ((first >> i) & 1u) m = fmaxf(m, ls.x[e]);
                m = warp_max(m);
                for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                    if ((first >> i) & 1u) sum += ex2(exponent(ls.x[e], m, c2));
                sum = warp_sum(sum);
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
        if (te.loss != nullptr && first_warp) {
            const float ln_s = ln(all.s);
            float part = 0.f;
            if (!empty) {
                for (int e = tid; e < te.k; e += 32)
                    if (ls.id[e] >= 0 && ls.q[e] != 0.f)
                        part += ls.q[e] * (ls.lq[e] - (all.s == 0.f ? -kInf : log_prob(ls.x[e], in.c, all.m, ln_s)));
                part = warp_sum(part);
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
                if (tid < 32)
                    for (int e = tid, i = 0; e < te.k; e += 32, ++i)
                        if ((first >> i) & 1u) {
                            const int id = ls.id[e];
                            float w = ls.q[e];
                            if (twice) {
                                w = 0.f;
                                for (int l = 0; l < te.k; ++l)
                                    if (ls.id[l] == id) w += ls.q[l];
                            }
                            const float pi = ex2(exponent(ls.x[e], all.m, c2)) * inv;
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
        case 32: return launch_rows<&k_distill<T, 32, kGrad>, 32>(in, 18 * 1024, s, in, te);
        case 128: return launch_rows<&k_distill<T, 128, kGrad>, 128>(in, 4096, s, in, te);
        default: return launch_rows<&k_distill<T, 256, kGrad>, 256>(in, 4096, s, in, te);
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
    const Shape sh = shape_of(S * n, V, size, true);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.log_cluster,
                    slots_of(V, size, sh.log_cluster)};
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
