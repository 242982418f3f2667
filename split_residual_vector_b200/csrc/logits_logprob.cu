// logits_logprob.cu -- log probabilities of the streams' tokens with entropy,
// log-sum-exp and top alternatives, and their gradient. Declared in
// include/mimi_rvq_streams.h; layout and statistics in logits.cuh.
//
// Forward: one pass, bound by reading the row (2 or 4 bytes a logit for one
// exponential, two sums and a maximum). Rows of up to 8 KB lie in shared memory
// whole, half a warp each (16384 x 16 x 2048 bf16: 221 us, 4.9 TB/s; a whole warp a
// row spent half its instructions on what is done once a row: 247 us). A longer row
// passes through a ring of chunks with a running maximum a warp; the ring runs on into
// the CTA's next row while this one's sums are joined and its alternatives ordered
// (3750 x 32000 float32: 82 us, 5.9 TB/s; with the row held in registers and 5
// alternatives 256 us, through the ring 95 to 102).
//
// Alternatives: the k largest by (logit descending, id ascending). A bound that
// at least k logits reach comes with the pass: every thread has its share's
// maximum anyway, and the k-th largest of those maxima is such a bound (k threads
// hold a logit that reaches it). On long rows the list adds a fifth (82 us, so 102);
// on short ones it is most of the work (16384 x 16 x 2048 bf16 at full clocks: 195
// us, with 8 alternatives 451). One warp finds the bound by bisecting the values'
// top 16 bits; only warps with a maximum that reaches it look at their logits again
// and append those that do to a short list, which is ordered by counting. The order
// of appending has no influence. Where the list overflows (rows of few distinct
// values), the bound is bisected over the keys themselves, which all differ, until
// between k and the list's length reach it (128 alternatives of 65536 x 2048 rows:
// 17.6 ms by k rounds of taking the next largest, 1.2 so).
//
// Gradient: d x_i = c p_i [(z - a) - b (ln p_i + H)] + c a [i = token] from the
// row in shared memory, so that it is read once from global memory and written
// once. What decides whether a row is needed at all (its token and upstream
// gradients) is loaded a row ahead of its logits. Bound by that traffic: 3750 x
// 32000 bf16 94 to 101 us (a copy of the tensor takes 80), 3750 x 16 x 2048 float32
// 176 to 180 (a copy 154).
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
constexpr uint32_t kOrderNegInf = 0x007FFFFFu;  // order_of(-inf)
// Larger comes first: (logit descending, id ascending).
__device__ __forceinline__ Key key_of(float v, int id) {
    return ((Key)order_of(v) << 32) | (0xFFFFFFFFu - (uint32_t)id);
}
__device__ __forceinline__ float order_value(uint32_t o) {
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ float key_value(Key key) { return order_value((uint32_t)(key >> 32)); }
__device__ __forceinline__ int key_id(Key key) { return (int)(0xFFFFFFFFu - (uint32_t)key); }

__device__ __forceinline__ int32_t token_at(const TokensIn& tk, const RowWalk& row, int64_t rows) {
    return tk.tok == nullptr || row.r >= rows ? -1 : __ldg(tk.tok + row.s * tk.ss + row.j * tk.sn);
}
// A row's target by its token, -1 if it has none; count: add a token past V to n_bad.
__device__ __forceinline__ int target_of(const TokensIn& tk, int32_t t, int V, bool count) {
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
    if (o.entropy != nullptr) o.entropy[r] = none ? 0.f : ln_s - kLn2 * (st.w * reciprocal(st.s));
    if (o.lse != nullptr) o.lse[r] = none ? -kInf : c * st.m + ln_s;
}

// ------------------------------------------------------------------ alternatives

// g maxima bound the list's length by about -g ln(1 - k / g) logits on rows in random order. So
// lists of up to kFewTop take 32 maxima (44 logits at k = 24), up to kWarpTop 128 (89 at k = 64),
// longer ones 256 (177 at k = 128).
constexpr int kFewTop = 24, kWarpTop = 64;

template <int TH>
struct TopShared {
    static constexpr int kCap = TH == 32 ? 256 : 512;
    uint32_t most[2][TH == 32 ? 1 : TH];  // the threads' maxima of two halves of their logits
    float bound;
    int count;
    alignas(16) Key list[kCap + 8];
    Key last[TH == 32 ? kCap / 4 : TH / 32];  // a warp: the vectors that have a listed logit
    int counts[2][TH / 32];
};
// The keys that a cluster's CTAs give its first one.
struct TopLists {
    Key of[kMaxCluster][kMaxTop];
    alignas(16) Key all[kMaxCluster * kMaxTop + 8];  // together
    int count[kMaxCluster];
};

// f(value, id) for this thread's logits of the share, which are in `buf` (any memory).
template <int TH, typename T, typename F>
__device__ __forceinline__ void each_logit(const uint4* buf, const Part<T>& p, int tid, float edge,
                                           F&& f) {
#pragma unroll 2
    for (int i = tid; i < p.nv; i += TH) {
        const uint4 q = buf[i];
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < Part<T>::kPer; ++j)
            f(element<T>(w, j), p.first + i * Part<T>::kPer + j);
    }
    if (edge > -kInf) f(edge, p.edge(tid));
}

// The largest bound (in steps of 2^16 of the values' order) that k of a warp's values reach, each
// lane having kN of them; the lowest finite value where fewer are above it.
template <int kN>
__device__ __forceinline__ float bound_of(const uint32_t (&q)[kN], int k) {
    uint32_t hi = q[0], lo = q[0];
#pragma unroll
    for (int i = 1; i < kN; ++i) {
        hi = max(hi, q[i]);
        lo = min(lo, q[i]);
    }
    hi = __reduce_max_sync(kFull, hi);
    lo = __reduce_min_sync(kFull, lo);
    // bits that all values share are the bound's, and k values exactly is as good as it gets
    uint32_t b = 0;
    if (k <= 32 * kN) {
        const int top_bit = 31 - __clz(lo ^ hi);  // -1: all are equal
        b = lo == hi ? lo : lo & ~((2u << top_bit) - 1u);
        for (int bit = top_bit; bit >= 16; --bit) {
            const uint32_t t = b | (1u << bit);
            int n = 0;
#pragma unroll
            for (int i = 0; i < kN; ++i) n += __popc(__ballot_sync(kFull, q[i] >= t));
            if (n >= k) b = t;
            if (n == k) break;
        }
    }
    return order_value(max(b, kOrderNegInf + 1));
}

// Leaves a CTA's bound for its k largest logits in sh.bound; called by its first warp when the
// threads' maxima are there; short lists take the maxima of 4 threads as one value.
template <int TH>
__device__ __forceinline__ void find_bound(TopShared<TH>& sh, int tid, int k) {
    static_assert(TH == 128, "eight maxima a lane");
    uint32_t q[8], half[4], all[1];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = sh.most[i / 4][tid + 32 * (i % 4)];
#pragma unroll
    for (int i = 0; i < 4; ++i) half[i] = max(q[i], q[i + 4]);
    all[0] = max(max(half[0], half[1]), max(half[2], half[3]));
    const float bound = k <= kFewTop ? bound_of(all, k) : k <= kWarpTop ? bound_of(half, k) : bound_of(q, k);
    if (tid == 0) {
        sh.bound = bound;
        sh.count = 0;
    }
}

// The list of a share whose logits above sh's bound were more than it holds: bisects a bound over
// their keys; returns the number of keys, between min(k, logits above -inf) and kCap.
template <int TH, typename T>
__device__ __noinline__ int refine(TopShared<TH>& sh, const Part<T> p, const uint4* buf, float edge,
                                   float bound, int tid, int k) {
    constexpr int kCap = TopShared<TH>::kCap, kWarps = TH / 32;
    Key top = 0;
    each_logit<TH>(buf, p, tid, edge, [&](float x, int id) {
        const Key key = key_of(x, id);
        if (x >= bound && key > top) top = key;
    });
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const Key other = __shfl_xor_sync(kFull, top, o);
        top = other > top ? other : top;
    }
    if constexpr (TH > 32) {
        if ((tid & 31) == 0) sh.last[tid / 32] = top;
        group_sync<TH>();
        for (int w = 0; w < kWarps; ++w) top = sh.last[w] > top ? sh.last[w] : top;
    }
    // more than kCap keys are at least lo, none is above hi
    Key lo = (Key)order_of(bound) << 32, hi = top, at = lo;
    for (int parity = 0;; parity ^= 1) {
        at = lo + (hi - lo + 1) / 2;
        unsigned n = 0;
        each_logit<TH>(buf, p, tid, edge, [&](float x, int id) { n += x >= bound && key_of(x, id) >= at; });
        n = __reduce_add_sync(kFull, n);
        if constexpr (TH > 32) {
            if ((tid & 31) == 0) sh.counts[parity][tid / 32] = (int)n;
            group_sync<TH>();
            n = 0;
            for (int w = 0; w < kWarps; ++w) n += sh.counts[parity][w];
        }
        if ((int)n > kCap) lo = at;
        else if ((int)n < k) hi = at - 1;
        else break;
        if (lo >= hi) break;  // cannot be: keys differ, so some bound has between k and kCap
    }
    if (tid == 0) sh.count = 0;
    group_sync<TH>();
    each_logit<TH>(buf, p, tid, edge, [&](float x, int id) {
        const Key key = key_of(x, id);
        if (x >= bound && key >= at) {
            const int place = atomicAdd(&sh.count, 1);
            if (place < kCap) sh.list[place] = key;
        }
    });
    group_sync<TH>();
    return min(sh.count, kCap);
}

// A warp's row: the logits that reach the bound, as unordered keys in sh.list; returns their
// number, at least min(k, the logits above -inf). Vectors with such a logit are listed first, then
// their elements are spread over the lanes.
template <typename T>
__device__ __forceinline__ int collect(TopShared<32>& sh, const Part<T>& p, const uint4* buf,
                                       float edge, float top, int lane, int k) {
    constexpr int kCap = TopShared<32>::kCap, kPer = Elem<T>::kPer;
    float bound;
    if (k <= kFewTop) {
        const uint32_t q[1] = {order_of(top)};
        bound = bound_of(q, k);
    } else {  // a lane's vectors in four parts
        float m[4] = {edge, -kInf, -kInf, -kInf};
        for (int base = lane; base < p.nv; base += 128)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (base + 32 * u < p.nv) {
                    const uint4 v = buf[base + 32 * u];
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    m[u] = fmaxf(m[u], vector_max<T>(w));
                }
        const uint32_t q[4] = {order_of(m[0]), order_of(m[1]), order_of(m[2]), order_of(m[3])};
        bound = bound_of(q, k);
    }
    const unsigned below = (1u << lane) - 1u;
    uint16_t* vectors = reinterpret_cast<uint16_t*>(sh.last);  // kCap of them
    int nv = 0;
    for (int base = 0; base < p.nv; base += 32) {
        const int i = base + lane;
        bool hit = false;
        if (i < p.nv) {
            const uint4 v = buf[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
            hit = vector_max<T>(w) >= bound;
        }
        const unsigned hits = __ballot_sync(kFull, hit);
        if (hit && nv + __popc(hits & below) < kCap) vectors[nv + __popc(hits & below)] = (uint16_t)i;
        nv += __popc(hits);
    }
    if (nv > kCap) return refine<32>(sh, p, buf, edge, bound, lane, k);
    __syncwarp();
    int n = 0;
    auto keep = [&](float x, int id, bool any) {
        const bool hit = any && x >= bound;
        const unsigned hits = __ballot_sync(kFull, hit);
        const int at = n + __popc(hits & below);
        if (hit && at < kCap) sh.list[at] = key_of(x, id);
        n += __popc(hits);
    };
    const T* logits = reinterpret_cast<const T*>(buf);
    for (int base = 0; base < nv * kPer; base += 32) {
        const int e = base + lane;
        const bool any = e < nv * kPer;
        const int at = any ? vectors[e / kPer] * kPer + e % kPer : 0;
        keep(any ? widen(logits[at]) : 0.f, p.first + at, any);
    }
    const int ie = p.edge(lane);
    keep(edge, ie, ie >= 0);
    __syncwarp();
    return n > kCap ? refine<32>(sh, p, buf, edge, bound, lane, k) : n;
}

// put(place, key) for the k largest of a list's n keys, and nothing for places past n; by G
// threads together (a warp or the group). The list has room for 8 more.
template <int G, typename Put>
__device__ __forceinline__ void order_list(Key* list, int n, int tid, int k, Put&& put) {
    if (tid < 8) list[n + tid] = 0;  // a round number to count
    group_sync<G>();
    for (int i = tid; i < n; i += G) {
        const Key key = list[i];
        int place = 0;
        for (int l = 0; l < n; l += 8) {
            ulonglong2 q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) q[u] = *reinterpret_cast<const ulonglong2*>(list + l + 2 * u);
#pragma unroll
            for (int u = 0; u < 4; ++u) place += (q[u].x > key) + (q[u].y > key);
        }
        if (place < k) put(place, key);
    }
}

// ------------------------------------------------------------------ forward

// A row's alternatives from the n keys of a list, by G threads.
template <int G>
__device__ __forceinline__ void put_top(Key* list, const ValuesOut& o, int64_t r, int n,
                                        const Stats& st, float c, int tid) {
    const bool broken = !(st.s < kInf);
    const float ln_s = logf(st.s), m = st.m;
    int32_t* const ids = o.top_ids == nullptr ? nullptr : o.top_ids + r * o.k;
    float* const lps = o.top_logprob == nullptr ? nullptr : o.top_logprob + r * o.k;
    auto out = [=](int place, Key key) {
        if (ids != nullptr) ids[place] = key ? key_id(key) : -1;
        if (lps != nullptr)
            lps[place] = broken ? NAN : key ? log_prob(key_value(key), c, m, ln_s) : -kInf;
    };
    if (broken) n = 0;
    else order_list<G>(list, n, tid, o.k, out);
    for (int i = n + tid; i < o.k; i += G) out(i, Key(0));
}

// Rows of up to 8 KB, each in its group's shared memory: half a warp a row, or a warp where
// alternatives are wanted.
template <typename T, int TH, bool kTop>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<TH>())
    k_logprob(RowsIn in, TokensIn tk, ValuesOut o) {
    static_assert(TH == 16 || TH == 32, "half a warp or a warp");
    constexpr int kRows = block_of<TH>() / TH;
    extern __shared__ uint4 buffers[];  // [groups][slots]
    __shared__ Joint<TH> joint[kRows];
    __shared__ TopShared<32> tops[kTop ? kRows : 1];
    const int tid = thread_in_group<TH>();
    const int group = group_in_block<TH>();
    uint4* buf = buffers + (size_t)group * in.slots;
    const float c2 = in.c * kLog2e;
    RowWalk row((int64_t)blockIdx.x * kRows + group, (int64_t)gridDim.x * kRows, in.n);
    if (row.r >= in.rows) return;
    auto part_at = [&]() {
        return Part<T>(static_cast<const T*>(in.x) + row.s * in.ss + row.j * in.sn, in.V, 0, 0);
    };
    auto edge_of = [&](const Part<T>& p) {
        const int i = p.edge(tid);
        return i < 0 ? -kInf : widen(p.x[i]);
    };
    Part<T> p = part_at();
    fetch<TH>(buf, p, tid);
    float edge = edge_of(p);
    int32_t token = token_at(tk, row, in.rows);
    while (true) {
        const int64_t r = row.r;
        const int t = target_of(tk, token, in.V, tid == 0);
        const float xt = t >= 0 ? widen(p.x[t]) : 0.f;
        arrived();
        float top;
        Stats st = pass<TH, true, T>(buf, p.nv, tid, edge, c2, top, [](int) {});
        row.next(in.n);
        const bool more = row.r < in.rows;
        auto send_next = [&]() {
            if (!more) return;
            p = part_at();
            fetch<TH>(buf, p, tid);
            edge = edge_of(p);
            token = token_at(tk, row, in.rows);
        };
        if constexpr (kTop) {
            st = join_group<TH, true>(joint[group], st, tid, 0, c2);
            const int n = collect(tops[group], p, buf, edge, top, tid, o.k);
            if (tid == 0) put_values(o, r, t, xt, in.c, st);
            send_next();
            put_top<TH>(tops[group].list, o, r, n, st, in.c, tid);
        } else {
            send_next();
            st = join_group<TH, true>(joint[group], st, tid, 0, c2);
            if (tid == 0) put_values(o, r, t, xt, in.c, st);
        }
        if (!more) break;
    }
}

// Longer rows: 128 threads a row, or the CTAs of a cluster where rows are few. A thread copies
// and reads its own places of a ring of kStages chunks of kU vectors a thread; copies run
// kStages - 1 chunks ahead, across rows.
constexpr int kLong = 128, kU = 4, kStages = 3, kChunk = kU * kLong, kRemember = 8;
__host__ __device__ constexpr int long_blocks(bool top) { return top ? 6 : blocks_of<kLong>(); }

template <typename T, bool kTop>
__global__ void __launch_bounds__(kLong, long_blocks(kTop))
    k_logprob_long(RowsIn in, TokensIn tk, ValuesOut o) {
    constexpr int TH = kLong, kPer = Elem<T>::kPer, kPairs = kPer / 2;
    extern __shared__ uint4 ring[];  // [kStages][kU][TH], then TopLists in a cluster
    __shared__ Joint<TH> joint;
    __shared__ TopShared<kTop ? TH : 32> tops;
    __shared__ float of_chunk[kTop ? kRemember : 1][TH];  // threads' maxima of chunks c, c + 8, ...
    TopLists& lists = *reinterpret_cast<TopLists*>(ring + kStages * kChunk);
    const int tid = threadIdx.x;
    const int lc = in.log_cluster, cluster = 1 << lc;
    const int rank = lc ? (int)cluster_ctarank() : 0;
    const bool first_warp = rank == 0 && tid < 32;  // has the row's edges
    const float c2 = in.c * kLog2e;
    if (lc) cluster_arrive();  // every CTA runs before one writes to another
    bool started = lc == 0;
    RowWalk row(blockIdx.x >> lc, gridDim.x >> lc, in.n);
    auto part_at = [&](const RowWalk& w) {
        return Part<T>(static_cast<const T*>(in.x) + w.s * in.ss + w.j * in.sn, in.V, rank, lc);
    };
    // chunks begin on 128-byte lines: the first one's first `skip` places stay empty (rows of odd
    // lengths would touch five lines with each warp's copy instead of four: 3750 x 32001 float32 93
    // us, so 87; with alternatives it gains nothing, 103 against 108)
    auto skip_of = [](const Part<T>& p) {
        return kTop ? 0 : (int)((reinterpret_cast<uintptr_t>(p.x + p.first) >> 4) & 7u);
    };
    auto chunks_of = [&](const Part<T>& p) {
        return max(1, (p.nv + skip_of(p) + kChunk - 1) / kChunk);
    };
    // copies, ahead of the chunk that is read; one group of copies per call
    RowWalk ahead = row;
    Part<T> to_come = part_at(ahead);
    int next_chunk = 0, left_to_come = chunks_of(to_come), stage_in = 0, stage_out = 0;
    auto send = [&]() {
        if (ahead.r < in.rows) {
            const int base = next_chunk * kChunk + tid - skip_of(to_come);
            const T* src = to_come.x + to_come.first + (int64_t)base * kPer;
            uint4* dst = ring + stage_in * kChunk + tid;
#pragma unroll
            for (int u = 0; u < kU; ++u)
                if (base + u * TH < to_come.nv && (u > 0 || base >= 0))
                    copy16(dst + u * TH, src + (size_t)u * TH * kPer);
            ++next_chunk;
            if (--left_to_come == 0) {
                ahead.next(in.n);
                if (ahead.r < in.rows) {
                    to_come = part_at(ahead);
                    left_to_come = chunks_of(to_come);
                    next_chunk = 0;
                }
            }
        }
        stage_in = stage_in == kStages - 1 ? 0 : stage_in + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) send();
    int32_t token = first_warp ? token_at(tk, row, in.rows) : -1;
    for (int parity = 0; row.r < in.rows; parity ^= 1) {
        const int64_t r = row.r;
        const Part<T> p = part_at(row);
        const int chunks = chunks_of(p), skip = skip_of(p);
        const int ie = first_warp ? p.edge(tid) : -1;
        const float edge = ie < 0 ? -kInf : widen(p.x[ie]);
        const int t = first_warp ? target_of(tk, token, in.V, tid == 0) : -1;
        const float xt = t >= 0 ? widen(p.x[t]) : 0.f;
        row.next(in.n);
        token = first_warp ? token_at(tk, row, in.rows) : -1;
        float m = -kInf;  // the warp's maximum
        float halves_top[2] = {edge, -kInf};  // the thread's, of two halves of its logits
        Scale k(c2, m);
        Pair s2 = 0, w2 = 0;  // (0, 0)
        for (int c = 0; c < chunks; ++c) {
            send();
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            const uint4* at = ring + stage_out * kChunk + tid;
            stage_out = stage_out == kStages - 1 ? 0 : stage_out + 1;
            const int left = p.nv + skip - c * kChunk;
            uint32_t w[kU][4];
            if (left >= kChunk && (c > 0 || skip == 0)) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    const uint4 q = at[u * TH];
                    w[u][0] = q.x, w[u][1] = q.y, w[u][2] = q.z, w[u][3] = q.w;
                }
            } else {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    uint4 q = make_uint4(Elem<T>::kFill, Elem<T>::kFill, Elem<T>::kFill, Elem<T>::kFill);
                    if (u * TH + tid < left && (u > 0 || c > 0 || tid >= skip)) q = at[u * TH];
                    w[u][0] = q.x, w[u][1] = q.y, w[u][2] = q.z, w[u][3] = q.w;
                }
            }
            float mx;
            if constexpr (sizeof(T) == 4) {
                float a = -kInf, b = -kInf;
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    a = fmaxf(a, fmaxf(__uint_as_float(w[u][0]), __uint_as_float(w[u][1])));
                    b = fmaxf(b, fmaxf(__uint_as_float(w[u][2]), __uint_as_float(w[u][3])));
                }
                halves_top[0] = fmaxf(halves_top[0], a);
                halves_top[1] = fmaxf(halves_top[1], b);
                mx = fmaxf(a, b);
            } else {
                uint32_t a = Elem<T>::kFill;
#pragma unroll
                for (int u = 0; u < kU; ++u)
                    a = max_bf16x2(a, max_bf16x2(max_bf16x2(w[u][0], w[u][1]), max_bf16x2(w[u][2], w[u][3])));
                halves_top[0] = fmaxf(halves_top[0], bf16_lo_to_f32(a));
                halves_top[1] = fmaxf(halves_top[1], bf16_hi_to_f32(a));
                mx = fmaxf(bf16_lo_to_f32(a), bf16_hi_to_f32(a));
            }
            if constexpr (kTop) {
                float& of = of_chunk[c % kRemember][tid];
                of = c < kRemember ? mx : fmaxf(of, mx);
            }
            if (c == chunks - 1) mx = fmaxf(mx, edge);
            if (__any_sync(kFull, mx > m)) {  // a new maximum: the sums so far move to it
                const float m_new = fmaxf(m, lanes_max<32>(mx));
                const Scale k_new(c2, m_new);
                float s, s1, w0, w1;
                halves(s2, s, s1);
                halves(w2, w0, w1);
                s += s1;
                const float back = ex2(-k.shift);
                w0 = fmaf(-k.shift, s, w0 + w1) * back;
                s *= back;
                const float d = m == -kInf ? 0.f : exponent(m, m_new, c2) + k_new.shift;
                const float f = ex2(d);
                s2 = pair_of(s * f, 0.f);
                w2 = pair_of(f * fmaf(s, d, w0), 0.f);
                m = m_new;
                k = k_new;
            }
            auto add = [&](const Pair (&q)[kPairs]) {
#pragma unroll
                for (int j = 0; j < kPairs; ++j) {
                    const Pair e = ex2_pair(q[j]);
                    s2 = add2(s2, e);
                    w2 = fma2(e, q[j], w2);
                }
            };
            if (!k.far) {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    Pair q[kPairs];
                    exponents<T, true, false>(w[u], k, q);
                    add(q);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kU; ++u) {
                    Pair q[kPairs];
                    exponents<T, true, true>(w[u], k, q);
                    add(q);
                }
            }
        }
        Stats st{m, 0.f, 0.f};
        {
            float s, s1, w0, w1;
            halves(s2, s, s1);
            halves(w2, w0, w1);
            s += s1;
            const float back = ex2(-k.shift), te = exponent(edge, m, c2), e = ex2(te);
            st.s = fmaf(s, back, e);
            st.w = fmaf(fmaf(-k.shift, s, w0 + w1), back, e * te);
        }
        const float top = fmaxf(halves_top[0], halves_top[1]);
        if constexpr (kTop) {
            tops.most[0][tid] = order_of(halves_top[0]);
            tops.most[1][tid] = order_of(halves_top[1]);
        }
        st = join_group<TH, true>(joint, st, tid, parity, c2);
        int n = 0;
        const uint4* vectors = reinterpret_cast<const uint4*>(p.x + p.first);
        if constexpr (kTop) {
            if (tid < 32) find_bound(tops, tid, o.k);
            group_sync<TH>();
            const float bound = tops.bound;
            if (__any_sync(kFull, top >= bound)) {
                // the logits that reach it, from the chunks whose maximum does: each lane goes
                // through its own, so that the lanes' loads travel together
                auto keep = [&](float x, int id) {
                    if (x < bound) return;
                    const int at = atomicAdd(&tops.count, 1);
                    if (at < TopShared<TH>::kCap) tops.list[at] = key_of(x, id);
                };
                for (int c = top >= bound ? 0 : chunks;; ++c) {
                    while (c < chunks && of_chunk[c % kRemember][tid] < bound) ++c;
                    if (!__any_sync(kFull, c < chunks)) break;
                    const int first = c * kChunk + tid - skip;
                    uint4 q[kU];
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        q[u] = make_uint4(Elem<T>::kFill, Elem<T>::kFill, Elem<T>::kFill, Elem<T>::kFill);
                        if (c < chunks && first + u * TH < p.nv && (u > 0 || first >= 0))
                            q[u] = vectors[first + u * TH];
                    }
#pragma unroll
                    for (int u = 0; u < kU; ++u) {
                        const uint32_t w[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
                        if (vector_max<T>(w) < bound) continue;
                        const int id = p.first + (first + u * TH) * kPer;
#pragma unroll
                        for (int j = 0; j < kPer; ++j) keep(element<T>(w, j), id + j);
                    }
                }
                if (ie >= 0) keep(edge, ie);
            }
            group_sync<TH>();
            n = tops.count;
            if (n > TopShared<TH>::kCap) n = refine<TH>(tops, p, vectors, edge, bound, tid, o.k);
        }
        if (lc) {  // the first CTA gets the others' triples and keys
            if (!started) cluster_wait();
            started = true;
            if (tid == 0) push_stats<TH, true>(joint, st, rank, 0, 0);
            if constexpr (kTop) {
                const uint32_t to = cluster_map(smem_u32(&lists.of[rank][0]), 0);
                auto give = [to](int place, Key key) { st_cluster_u64(to + 8 * place, key); };
                if (n > o.k) {
                    order_list<TH>(tops.list, n, tid, o.k, give);
                    n = o.k;
                } else {
                    for (int i = tid; i < n; i += TH) give(i, tops.list[i]);
                }
                if (tid == 0) st_cluster_u32(cluster_map(smem_u32(&lists.count[rank]), 0), n);
            }
            cluster_sync();
            if (rank == 0) st = join_cluster<TH, true>(joint, tid, cluster, 0, c2);
        }
        if (rank == 0) {
            if (tid == 0) put_values(o, r, t, xt, in.c, st);
            if constexpr (kTop) {
                if (lc) {
                    n = 0;
                    for (int l = 0; l < cluster; ++l) {
                        const int more = lists.count[l];
                        for (int e = tid; e < more; e += TH) lists.all[n + e] = lists.of[l][e];
                        n += more;
                    }
                    put_top<TH>(lists.all, o, r, n, st, in.c, tid);
                } else if (tid < 32) {  // the other warps go on
                    put_top<32>(tops.list, o, r, n, st, in.c, tid);
                }
            }
        }
        if (lc && row.r < in.rows) cluster_sync();  // the first CTA has read what it was given
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!started) cluster_wait();
}

// ------------------------------------------------------------------ gradient

template <typename T, int TH>
__global__ void __launch_bounds__(block_of<TH>(), blocks_of<TH>())
    k_logprob_grad(RowsIn in, TokensIn tk, GradIn g, ValuesOut o) {
    constexpr int kRows = block_of<TH>() / TH, kPer = Part<T>::kPer;
    extern __shared__ uint4 buffers[];  // [groups][slots]
    __shared__ Joint<TH> joint[kRows];
    const int tid = thread_in_group<TH>();
    const int group = group_in_block<TH>();
    const int lc = TH <= 32 ? 0 : in.log_cluster, cluster = 1 << lc;
    const int rank = lc ? (int)cluster_ctarank() : 0;
    const bool first_warp = rank == 0 && tid < 32;
    uint4* buf = buffers + (size_t)group * in.slots;
    const float c2 = in.c * kLog2e;
    const bool values = o.logprob != nullptr || o.entropy != nullptr || o.lse != nullptr;
    if (lc) cluster_sync();  // every CTA runs before one writes to another
    RowWalk row((int64_t)(blockIdx.x >> lc) * kRows + group,
                (int64_t)(gridDim.x >> lc) * kRows, in.n);
    // what the row's gradient comes from: loaded a row ahead
    struct Up {
        int32_t token;
        float a, b, z;
    };
    auto up_at = [&]() {
        Up u{token_at(tk, row, in.rows), 0.f, 0.f, 0.f};
        if (row.r < in.rows) {
            if (g.g_logprob != nullptr) u.a = __ldg(g.g_logprob + row.r);
            if (g.g_entropy != nullptr) u.b = __ldg(g.g_entropy + row.r);
            if (g.g_lse != nullptr) u.z = __ldg(g.g_lse + row.r);
        }
        return u;
    };
    auto part_at = [&]() {
        return Part<T>(static_cast<const T*>(in.x) + row.s * in.ss + row.j * in.sn, in.V, rank, lc);
    };
    Up up = up_at();
    for (int parity = 0; row.r < in.rows;) {
        const int64_t r = row.r;
        const Part<T> p = part_at();
        // the gradient's row has its own alignment
        T* d = static_cast<T*>(g.d) + row.s * g.ss + row.j * g.sn;
        const bool wide = ((reinterpret_cast<uintptr_t>(d) ^ reinterpret_cast<uintptr_t>(p.x)) & 15u) == 0;
        const int t = target_of(tk, up.token, in.V, first_warp && tid == 0);
        const float a = t < 0 ? 0.f : up.a, b = up.b, z = up.z;
        const bool zero = a == 0.f && b == 0.f && z == 0.f;
        row.next(in.n);
        const int ie = first_warp ? p.edge(tid) : -1;
        float edge = -kInf, xt = 0.f;
        if (!zero || values) {
            fetch<TH>(buf, p, tid);
            if (ie >= 0) edge = widen(p.x[ie]);
            if (t >= 0) xt = widen(p.x[t]);
        }
        up = up_at();
        Stats st{-kInf, 0.f, 0.f};
        if (!zero || values) {
            arrived();
            float top;
            st = pass<TH, true, T>(buf, p.nv, tid, edge, c2, top, [](int) {});
            st = join_row<TH, true>(joint[group], st, tid, cluster, rank, parity, c2);
            parity ^= 1;
            if (first_warp && tid == 0) put_values(o, r, t, xt, in.c, st);
        }
        T* out = d + p.first;
        if (zero || st.s == 0.f) {
            for (int i = tid; i < p.nv; i += TH) {
                const float y[kPer] = {};
                store_vector<T>(out + (size_t)i * kPer, wide, y);
            }
            if (ie >= 0) narrow(0.f, d + ie);
            continue;
        }
        const float inv = reciprocal(st.s), ln_s = ln(st.s), h = ln_s - kLn2 * (st.w * inv);
        // c p_i [(z - a) - b (ln p_i + H)] = 2^t (c0 + c1 t), t = log2(e) c (x - m)
        const float c0 = in.c * inv * ((z - a) - b * (h - ln_s)), c1 = -in.c * inv * b * kLn2;
        const Scale k(c2, st.m);
        const bool fast = !k.far && wide;
        const float shift = fast ? k.shift : 0.f, back = ex2(-shift);
        const float k0 = back * fmaf(-shift, c1, c0), k1 = back * c1;  // for t off by the shift
        auto put = [&](int i, const Pair (&q)[kPer / 2], bool whole) {
            float y[kPer];
#pragma unroll
            for (int e = 0; e < kPer / 2; ++e)
                halves(mul2(ex2_pair(q[e]), fma2(pair_of(k1, k1), q[e], pair_of(k0, k0))),
                       y[2 * e], y[2 * e + 1]);
            store_vector<T>(out + (size_t)i * kPer, whole, y);
        };
        if (fast)
            each_vector<TH>(buf, p.nv, tid, [&](int i, const uint32_t (&w)[4]) {
                Pair q[kPer / 2];
                exponents<T, true, false>(w, k, q);
                put(i, q, true);
            });
        else
            each_in_turn<TH>(buf, p.nv, tid, [&](int i, const uint32_t (&w)[4]) {
                Pair q[kPer / 2];
                exponents<T, true, true>(w, k, q);
                put(i, q, wide);
            });
        auto one = [&](float x) {
            const float e = exponent(x, st.m, c2);
            return ex2(e) * fmaf(c1, e, c0);
        };
        if (ie >= 0) narrow(one(edge) + (ie == t ? in.c * a : 0.f), d + ie);
        // the target's own term, by the thread that stored its vector
        const int at = t >= 0 ? p.place(t) : -1;
        if (at >= 0 && at / kPer % TH == tid) narrow(one(xt) + in.c * a, d + t);
    }
}

template <typename T, bool kTop>
cudaError_t forward_of(int threads, const RowsIn& in, const TokensIn& tk, const ValuesOut& o,
                       cudaStream_t s) {
    constexpr int kShort = kTop ? 32 : 16;
    if (threads == kShort)  // the last figures: static shared memory, rounded up
        return launch_rows<&k_logprob<T, kShort, kTop>, kShort, 0, blocks_of<kShort>()>(
            in, kTop ? 12 * 1024 : 512, s, in, tk, o);
    RowsIn with_ring = in;
    with_ring.slots = kStages * kChunk + (kTop && in.log_cluster ? (int)sizeof(TopLists) / 16 + 1 : 0);
    return launch_rows<&k_logprob_long<T, kTop>, kLong, 0, long_blocks(kTop)>(
        with_ring, kTop ? 11 * 1024 : 1024, s, with_ring, tk, o);
}

template <typename T>
cudaError_t gradient_of(int threads, const RowsIn& in, const TokensIn& tk, const GradIn& g,
                        const ValuesOut& o, cudaStream_t s) {
    switch (threads) {
        case 16: return launch_rows<&k_logprob_grad<T, 16>, 16, 0, blocks_of<16>()>(
            in, 1024, s, in, tk, g, o);
        case 128: return launch_rows<&k_logprob_grad<T, 128>, 128, 0, blocks_of<128>()>(
            in, 1024, s, in, tk, g, o);
        default: return launch_rows<&k_logprob_grad<T, 256>, 256, 0, blocks_of<256>()>(
            in, 1024, s, in, tk, g, o);
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
    const Shape sh = shape_of(S * n, V, size, k == 0 ? 16 : k <= kWarpTop ? 32 : 0, false);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.log_cluster,
                    slots_of(V, size, sh.log_cluster)};
    const TokensIn tk{tokens, tok_stride_s, tok_stride_n, pad,
                      reinterpret_cast<unsigned long long*>(n_bad)};
    const ValuesOut o{logprob, entropy, lse, top_ids, top_logprob, k};
    if (dtype == MIMI_RVQ_BF16)
        return status_of(k ? forward_of<__nv_bfloat16, true>(sh.threads, in, tk, o, stream)
                           : forward_of<__nv_bfloat16, false>(sh.threads, in, tk, o, stream));
    return status_of(k ? forward_of<float, true>(sh.threads, in, tk, o, stream)
                       : forward_of<float, false>(sh.threads, in, tk, o, stream));
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
    const Shape sh = shape_of(S * n, V, size, 16, true);
    const RowsIn in{logits, stride_s, stride_n, S * n, n, V, scale, sh.log_cluster,
                    slots_of(V, size, sh.log_cluster)};
    const TokensIn tk{tokens, tok_stride_s, tok_stride_n, pad,
                      reinterpret_cast<unsigned long long*>(n_bad)};
    const GradIn g{g_logprob, g_entropy, g_lse, dlogits, d_stride_s, d_stride_n};
    const ValuesOut o{logprob, entropy, lse, nullptr, nullptr, 0};
    return status_of(dtype == MIMI_RVQ_BF16 ? gradient_of<__nv_bfloat16>(sh.threads, in, tk, g, o, stream)
                                            : gradient_of<float>(sh.threads, in, tk, g, o, stream));
}
